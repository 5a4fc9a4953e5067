// kv16_attn.cu — multi-query attention of 64 heads over the rows of the paged 16-bit cache that a token sees.
//
//   x_r = scale * q[t,h,:] . kv_r,  cap tanh(x / cap),  - slopes[h] |e - 1 - r|
//   out[t,h,:] = (sum_r 2^(x_r - m) kv_r + 2^(o - m) other_out[t,h,:]) / (sum_r 2^(x_r - m) + 2^(s - m) + 2^(o - m))
//
// with s the head's sink, o the other attention's log-sum-exp, all in log2 units.
//
// One warp a token and head: a lane holds 16 dims of q and of the running sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "ds4x_internal.h"
#include "ds4x_ptx.cuh"

namespace ds4x {
namespace {

constexpr int kHq = 64;
constexpr int kDim = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct Params {
  const uint16_t *q, *pool;
  const int32_t *tables, *rows, *req, *positions, *first, *prefix;
  const float *slopes, *sinks, *other_lse;
  const uint16_t* other;
  uint16_t* out;
  float* lse;
  int n_slots, n_req, max_pages, log_page, ratio, window, T;
  float scale, cap;
};

// Rows [lo, hi) of its request that token t sees, and the row e it stands before.
struct Span {
  int b, lo, hi, e;
};
__device__ __forceinline__ Span span_of(const Params& p, int t) {
  Span s{p.req ? __ldg(p.req + t) : t, 0, 0, 0};
  if (s.b < 0 || s.b >= p.n_req) return s;
  const int held = min(max(__ldg(p.rows + s.b), 0), p.max_pages << p.log_page);
  s.e = held;
  if (p.positions) {
    const int pos = __ldg(p.positions + t);
    if (pos < 0) return s;
    s.e = (int)min(((uint32_t)pos + 1u) / (uint32_t)p.ratio, 0x7fffffffu);
  }
  s.hi = min(held, p.prefix ? max(s.e, __ldg(p.prefix + s.b)) : s.e);
  s.lo = p.window > 0 ? max(s.e - p.window, 0) : 0;
  if (p.first) s.lo = max(s.lo, __ldg(p.first + t));
  s.hi = max(s.hi, s.lo);
  return s;
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack(uint32_t u) {
  if constexpr (kBf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool kBf16>
__device__ __forceinline__ void load16(const uint16_t* src, int lane, float (&v)[16]) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  const uint4 a = __ldg(s + lane), b = __ldg(s + lane + 32);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack<kBf16>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(256) kv16_attn_kernel(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const Span s = span_of(p, t);
    const int64_t at = ((int64_t)t * kHq + h);
    float q[16], o[16];
    load16<kBf16>(p.q + at * kDim, lane, q);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float slope = p.slopes ? p.slopes[h] * kLog2e : 0.f;
    for (int r = s.lo; r < s.hi; ++r) {
      const int page = __ldg(p.tables + (int64_t)s.b * p.max_pages + (r >> p.log_page));
      const int64_t slot = ((int64_t)page << p.log_page) + (r & ((1 << p.log_page) - 1));
      if (page < 0 || slot >= p.n_slots) continue;
      float k[16];
      load16<kBf16>(p.pool + slot * kDim, lane, k);
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= p.scale;
      if (p.cap > 0.f) x = p.cap * tanhf(x / p.cap);
      x *= kLog2e;
      if (p.slopes) x -= slope * fabsf((float)(s.e - 1 - r));
      const float mn = fmaxf(m, x);
      const float f = mn == -INFINITY ? 0.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(x - mn);
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = o[i] * f + w * k[i];
    }
    const float snk = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
    const float oth = p.other ? p.other_lse[at] * kLog2e : -INFINITY;
    const float M = fmaxf(m, fmaxf(snk, oth)), M0 = M == -INFINITY ? 0.f : M;
    const float f = exp2f(m - M0), fo = exp2f(oth - M0);
    l = l * f + exp2f(snk - M0) + fo;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= f;
    if (fo != 0.f) {
      float k[16];
      load16<kBf16>(p.other + at * kDim, lane, k);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] += fo * k[i];
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack<kBf16>(o[2 * i] * inv, o[2 * i + 1] * inv);
    uint4* dst = reinterpret_cast<uint4*>(p.out + at * kDim);
    dst[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[lane + 32] = make_uint4(w[4], w[5], w[6], w[7]);
    if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (M0 + log2f(l)) * kLn2;
  }
}

}  // namespace

size_t kv16_attn_workspace_bytes(int T, int max_rows) { return 0; }

int launch_kv16_attn(const Kv16AttnArgs& a, cudaStream_t stream) {
  Params p;
  p.q = static_cast<const uint16_t*>(a.q_attn);
  p.pool = static_cast<const uint16_t*>(a.pool);
  p.tables = a.tables;
  p.rows = a.rows;
  p.req = a.req;
  p.positions = a.positions;
  p.first = a.first;
  p.prefix = a.prefix;
  p.slopes = a.slopes;
  p.sinks = a.sinks;
  p.other = static_cast<const uint16_t*>(a.other_out);
  p.other_lse = a.other_lse;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.n_slots = a.n_slots;
  p.n_req = a.n_req;
  p.max_pages = a.max_pages;
  p.log_page = a.log_page;
  p.ratio = a.ratio;
  p.window = a.window;
  p.T = a.T;
  p.scale = a.scale;
  p.cap = a.cap;
  const int blocks = a.T < 65536 ? a.T : 65536;
  if (launch_pdl(a.bf16 ? kv16_attn_kernel<true> : kv16_attn_kernel<false>, dim3(blocks, kHq / 8), dim3(256), 0, stream,
                 p) != cudaSuccess)
    return DS4X_ERR_CUDA;
  count_launch();
  return DS4X_OK;
}

}  // namespace ds4x

using namespace ds4x;

extern "C" {

size_t ds4x_kv16_attn_workspace_bytes(int32_t T, int32_t max_rows) {
  return T > 0 && max_rows > 0 ? kv16_attn_workspace_bytes(T, max_rows) : 0;
}

int ds4x_kv16_attn(const void* q_attn, ds4x_dtype dtype, const void* pool, int32_t n_slots, const int32_t* tables,
                   const int32_t* rows, int32_t n_req, int32_t max_pages, int32_t page_rows, const int32_t* req,
                   const int32_t* positions, int32_t ratio, int32_t window, const int32_t* first, const int32_t* prefix,
                   int32_t T, int32_t Hq, int32_t Dkv, float scale, float cap, const float* slopes, const float* sinks,
                   const void* other_out, const float* other_lse, void* out, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream) {
  call_begin();
  if (T < 0 || Hq <= 0 || Dkv <= 0 || n_slots < 0 || n_req < 0 || max_pages < 0 || page_rows < 1 || ratio < 1 ||
      window < 0 || !(cap >= 0.f) || isinf(cap) || (dtype != DS4X_F16 && dtype != DS4X_BF16))
    return DS4X_ERR_INVALID;
  if (Hq != kHq || Dkv != kDim) return DS4X_ERR_UNSUPPORTED;
  if ((page_rows & (page_rows - 1)) != 0 || page_rows > DS4X_MAX_PAGE_ROWS) return DS4X_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_rows > INT32_MAX) return DS4X_ERR_UNSUPPORTED;
  if (T == 0) return call_end(DS4X_OK);
  if (!q_attn || !out || !aligned16(q_attn) || !aligned16(out) || (lse && !aligned16(lse)) || !aligned16(other_out) ||
      (other_out == nullptr) != (other_lse == nullptr))
    return DS4X_ERR_INVALID;
  if (!req && T > n_req) return DS4X_ERR_INVALID;
  if (n_req > 0 && (!rows || (max_pages > 0 && !tables))) return DS4X_ERR_INVALID;
  if (n_slots > 0 && (!pool || !aligned16(pool))) return DS4X_ERR_INVALID;
  const void* words[] = {tables, rows, req, positions, first, prefix, slopes, sinks, other_lse};
  for (const void* w : words)
    if (!aligned4(w)) return DS4X_ERR_INVALID;
  int max_rows = max_pages * page_rows;
  if (!prefix && window > 0 && window < max_rows) max_rows = window;
  const size_t need = ds4x_kv16_attn_workspace_bytes(T, max_rows);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DS4X_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return DS4X_ERR_INVALID;
  int log_page = 0;
  while ((1 << log_page) < page_rows) ++log_page;
  const Kv16AttnArgs a{q_attn, dtype == DS4X_BF16 ? 1 : 0, pool, n_slots, tables, rows, n_req, max_pages, log_page, req,
                       positions, ratio, window, first, prefix, T, scale, cap, slopes, sinks, other_out, other_lse, out,
                       lse, need > 0 ? workspace : nullptr, max_rows};
  return call_end(launch_kv16_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
