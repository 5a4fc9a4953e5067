// kv16_cache.cu — rotation by position, and rows into the paged 16-bit cache.
//
// Pair i of a row at position p is turned by the angle a = p * f_i, f_i = inv_freq[i] in radians.  Only a modulo
// a turn counts, and fp32 loses it at far positions (p * f near 10^6 has steps of 2^-4), so it is kept as a 64-bit
// fraction of a turn: F_i = 2^64 (f_i / 2 pi mod 1) once in fp64, then p * F_i in integers, which wrap where turns
// do.  F_i is off by about (f_i / 2 pi) 2^-53 + 2^-65 turns, its product by |p| times that.  The fraction's upper
// 32 bits go to fp32 (2^-25 of a half turn at most) and through sincospif; the pair is turned in fp32 and rounded
// once.  fp64 runs at a 64th of the fp32 rate here: F is formed once a pair and block, which is once for all heads of
// a token in rotate, and for all rows that a block takes in append.
//
// Rotation of many heads and append are bound by HBM: 2048 tokens of 64 heads rotated in 41.5 us (6.5 TB/s, 95 % of a plain
// copy; heads of 128 elements 16 us, 4.2 TB/s), 50001 rows appended in 19.1 us (5.3 TB/s, 79 %; 120000 in 42.4, 5.8 TB/s),
// of which some 4 us are the start: slots, then rows.  A few rows cost a launch (61 rows 2.4 us, 48 tokens rotated 3.3).
// Rotation of one head a token is not: a token is a block whatever its heads are, so that its time is that of the blocks,
// each with its own F and two loads that wait for each other (2048 rows 8.7 us, 50001 rows of 512 or of 128 elements 197 us,
// 13 times what the former's bytes take; with 256 pairs 254 us).  Rows on their way into the cache take append.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ds4x_internal.h"
#include "ds4x_ptx.cuh"

namespace ds4x {
namespace {

constexpr int kThreads = 256;
constexpr int kRowDim = 512;             // elements of a cached row
constexpr int kRowPieces = kRowDim / 8;  // of 16 bytes

__device__ __forceinline__ uint64_t turns_of(double f) {
  const double u = f * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((u - floor(u)) * 18446744073709551616.0);
}
// cos and sin of p * F turns
__device__ __forceinline__ float2 unit_at(int p, uint64_t F) {
  const uint64_t phase = (uint64_t)(int64_t)p * F + 0x80000000ull;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t turn(uint32_t pair, float2 cs) {
  if constexpr (kBf16) {
    const float x0 = __uint_as_float(pair << 16), x1 = __uint_as_float(pair & 0xffff0000u);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0 * cs.x - x1 * cs.y, x1 * cs.x + x0 * cs.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pair));
    const __half2 h = __floats2half2_rn(x.x * cs.x - x.y * cs.y, x.y * cs.x + x.x * cs.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// The 16-byte piece whose first pair is pair i of the rotation (i < 0: pairs before it stay as they are).
template <bool kBf16, typename Unit>
__device__ __forceinline__ uint4 turn_piece(uint4 v, int i, Unit unit) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + k >= 0) w[k] = turn<kBf16>(w[k], unit(i + k));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of many heads share their token's angles: a block takes kPieces pieces of one token, and forms the
// token's units in shared memory while they are on their way.
constexpr int kBatch = 8;                       // pieces a thread
constexpr int kPieces = kBatch * kThreads;
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const uint4* x, const int32_t* __restrict__ positions,
                                                          const double* __restrict__ inv_freq, int heads, int row_pieces,
                                                          int first, int head_pairs, int pairs, float sign, uint4* out) {
  // per token: `heads` rows of row_pieces pieces, of which those from `first` on are taken; pair 0 of the rotation
  // lies head_pairs pairs behind a row's beginning
  extern __shared__ float2 unit_s[];
  pdl_wait();
  pdl_trigger();
  const int per_row = row_pieces - first, n = heads * per_row;
  const int64_t base = (int64_t)blockIdx.y * heads * row_pieces;
  const int k0 = blockIdx.x * kPieces + threadIdx.x;
  uint4 v[kBatch];
  int at[kBatch], pair[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int k = k0 + i * kThreads, row = k / per_row, piece = first + k - row * per_row;
    at[i] = row * row_pieces + piece;
    pair[i] = 4 * piece - head_pairs;
    if (k < n) v[i] = x[base + at[i]];
  }
  const int p = positions[blockIdx.y];
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const float2 cs = unit_at(p, turns_of(inv_freq[i]));
    unit_s[i] = make_float2(cs.x, cs.y * sign);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (k0 + i * kThreads < n)
      out[base + at[i]] = pair[i] > -4 ? turn_piece<kBf16>(v[i], pair[i], [&](int j) { return unit_s[j]; }) : v[i];
}

// One block takes `group` rows at a time: first what is rotated, so that all of a warp's lanes form angles, then
// what is only copied.
constexpr int kGroupMax = 32, kPerSm = 8;  // blocks an SM
template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
    kv16_append_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ slots,
                       const int32_t* __restrict__ positions, const double* __restrict__ inv_freq, int n, int pairs,
                       int group, uint4* __restrict__ pool, int n_slots) {
  __shared__ uint64_t turns_s[kRowDim / 2];
  __shared__ int slot_s[kGroupMax], pos_s[kGroupMax];
  pdl_wait();
  pdl_trigger();
  const int head_pairs = kRowDim / 2 - pairs;
  const int first = head_pairs / 4, turned = pairs > 0 ? kRowPieces - first : 0, plain = kRowPieces - turned;
  for (int i = threadIdx.x; i < pairs; i += kThreads) turns_s[i] = turns_of(inv_freq[i]);
  for (int64_t r0 = (int64_t)blockIdx.x * group; r0 < n; r0 += (int64_t)gridDim.x * group) {
    __syncthreads();  // the slots of the group before are read, the turns written
    const int m = (int)min((int64_t)group, n - r0);
    if (threadIdx.x < m) {
      const int s = slots[r0 + threadIdx.x];
      slot_s[threadIdx.x] = s >= 0 && s < n_slots ? s : -1;
      pos_s[threadIdx.x] = pairs > 0 ? positions[r0 + threadIdx.x] : 0;
    }
    __syncthreads();
    const uint4* src = rows + r0 * kRowPieces;
    for (int k = threadIdx.x; k < m * turned; k += kThreads) {
      const int r = k / turned, piece = first + k - r * turned;
      const int s = slot_s[r], p = pos_s[r];
      if (s < 0) continue;
      pool[(int64_t)s * kRowPieces + piece] =
          turn_piece<kBf16>(src[r * kRowPieces + piece], 4 * piece - head_pairs,
                            [&](int j) { return unit_at(p, turns_s[j]); });
    }
#pragma unroll 4
    for (int k = threadIdx.x; k < m * plain; k += kThreads) {
      const int r = k / plain, piece = k - r * plain;
      const int s = slot_s[r];
      if (s >= 0) pool[(int64_t)s * kRowPieces + piece] = src[r * kRowPieces + piece];
    }
  }
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

}  // namespace
}  // namespace ds4x

using namespace ds4x;

extern "C" {

int ds4x_rotate(const void* x, ds4x_dtype dtype, const int32_t* positions, const double* inv_freq, int32_t T, int32_t H,
                int32_t D, int32_t rot, int32_t inverse, void* out, void* stream) {
  call_begin();
  if (T < 0 || H < 0 || D <= 0 || rot < 2 || rot > D || (rot & 1) || (dtype != DS4X_F16 && dtype != DS4X_BF16))
    return DS4X_ERR_INVALID;
  if ((D & 7) || rot > DS4X_MAX_ROT || (int64_t)H * D > INT32_MAX) return DS4X_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return call_end(DS4X_OK);
  if (!x || !out || !positions || !inv_freq || !aligned16(x) || !aligned16(out) || !aligned4(positions) ||
      !aligned8(inv_freq))
    return DS4X_ERR_INVALID;
  const int head_pairs = (D - rot) / 2;
  const int first = x == out ? head_pairs / 4 : 0;  // in place: only what changes
  const int pieces = H * (D / 8 - first);
  const size_t smem = (size_t)rot / 2 * sizeof(float2);
  const size_t row = (size_t)H * D * 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int64_t t0 = 0; t0 < T; t0 += 65535) {  // the grid's second axis; t0 may step over INT32_MAX
    const int32_t m = T - t0 < 65535 ? (int32_t)(T - t0) : 65535;
    const cudaError_t e = launch_pdl(
        dtype == DS4X_BF16 ? rotate_kernel<true> : rotate_kernel<false>, dim3((pieces + kPieces - 1) / kPieces, m),
        dim3(kThreads), smem, st, reinterpret_cast<const uint4*>(static_cast<const char*>(x) + t0 * row),
        positions + t0, inv_freq, H, D / 8, first, head_pairs, rot / 2, inverse ? -1.f : 1.f,
        reinterpret_cast<uint4*>(static_cast<char*>(out) + t0 * row));
    if (e != cudaSuccess) return DS4X_ERR_CUDA;
    count_launch();
  }
  return call_end(DS4X_OK);
}

int ds4x_kv16_append(const void* rows, ds4x_dtype dtype, const int32_t* slots, const int32_t* positions,
                     const double* inv_freq, int32_t n, int32_t Dkv, int32_t rot, void* pool, int32_t n_slots,
                     void* stream) {
  call_begin();
  if (n < 0 || Dkv <= 0 || n_slots < 0 || rot < 0 || rot > Dkv || (rot & 1) ||
      (dtype != DS4X_F16 && dtype != DS4X_BF16))
    return DS4X_ERR_INVALID;
  if (Dkv != kRowDim) return DS4X_ERR_UNSUPPORTED;
  if (n == 0) return call_end(DS4X_OK);
  if (!rows || !slots || !aligned16(rows) || !aligned4(slots) || (n_slots > 0 && (!pool || !aligned16(pool))) ||
      (rot > 0 && (!positions || !inv_freq || !aligned4(positions) || !aligned8(inv_freq))))
    return DS4X_ERR_INVALID;
  // Two blocks an SM for few rows, else eight, and groups of one size that every block takes the same number of:
  // groups of 32 with a few blocks taking one more are slower (5000 rows 4.3 us instead of 3.4, 50001 21.9 instead of
  // 19.5), and so are groups of up to 64 (20.4) or four blocks an SM (23.3).
  const int64_t sms = device_sm_count();
  const int64_t most = sms * (n >= sms * kPerSm * 8 ? kPerSm : 2), rounds = (n - 1) / (most * kGroupMax) + 1;
  const int group = (int)((n - 1) / (most * rounds) + 1);
  const int64_t want = ((int64_t)n + group - 1) / group;
  const cudaError_t e = launch_pdl(
      dtype == DS4X_BF16 ? kv16_append_kernel<true> : kv16_append_kernel<false>, dim3((int)(want < most ? want : most)),
      dim3(kThreads), 0, static_cast<cudaStream_t>(stream), static_cast<const uint4*>(rows), slots, positions, inv_freq,
      n, rot / 2, group, static_cast<uint4*>(pool), n_slots);
  if (e != cudaSuccess) return DS4X_ERR_CUDA;
  count_launch();
  return call_end(DS4X_OK);
}

}  // extern "C"
