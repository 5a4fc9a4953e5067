// kv4_cache.cu — the paged 4-bit cache of pooled rows: rows in (quantised), rows out, and the block
// tables and slots of a step, built on the GPU from request lengths.  The row format is described in
// kv4_common.cuh.
//
// Rows in and out are bound by HBM: a row is 1024 bytes of 16-bit values against 272 bytes of cache.
// One warp takes a row, 16 values a lane: two 16-byte loads a lane make 1 KB a warp in whole sectors,
// and a group of 32 values is two lanes, so its largest magnitude is one shuffle away.
//
// The step plan is bound by latency at a decode step's sizes (a few hundred bytes) and by its writes at
// a large step's (8 bytes a token).  Every block computes the prefix sums over all requests for itself
// (at most 4096 of them: cheaper than handing them over through memory) and then fills its share of the
// outputs: a warp takes a run of neighbouring elements, finds the request of the first by a search in which
// each lane looks at one place (three steps for 4096), and from there on the requests of 128 elements at a
// time, between which a lane searches.  Where the state is updated in place the blocks are one cluster,
// whose barrier separates its reads from the update (17.4 us for 1500 requests with 96000 tokens on eight
// blocks); otherwise there are as many as have something to fill (7.3 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds4x_internal.h"
#include "ds4x_ptx.cuh"
#include "kv4_common.cuh"

namespace ds4x {
namespace {

constexpr int kWarpsPerBlock = 8;

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (kBf16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2_rn(float a, float b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Eight values to a word of codes (v[0].x in the lowest nibble): nearest, ties to the even code,
// saturating.
__device__ __forceinline__ uint32_t encode8(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

template <bool kBf16>
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    kv4_append_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ slots, int n, int n_slots,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5); r < n; r += gridDim.x * kWarpsPerBlock) {
    const int slot = __ldg(slots + r);
    if (slot < 0 || slot >= n_slots) continue;  // the same for the whole warp
    const uint4* src = rows + (int64_t)r * (kKv4Dim / 8) + lane * 2;
    const uint4 u0 = __ldg(src), u1 = __ldg(src + 1);
    const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    float2 v[2][4];
    // the largest magnitude, compared as bits: a NaN is above infinity and is seen
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<kBf16>(u[i]);
      v[i >> 2][i & 3] = f;
      top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    // the least e with top <= 6 * 2^e = 1.5 * 2^(e + 2)
    int e = (int)(top >> 23) - 129 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);
    e = min(max(e, kKv4ExpMin), kKv4ExpMax);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // a power of two: the products are exact
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i >> 2][i & 3].x *= inv;
      v[i >> 2][i & 3].y *= inv;
    }
    *reinterpret_cast<uint2*>(codes + (int64_t)slot * kKv4CodeBytes + lane * 8) =
        make_uint2(encode8(v[0]), encode8(v[1]));
    if ((lane & 1) == 0)
      scales[(int64_t)slot * kKv4ScaleBytes + (lane >> 1)] = (uint8_t)(top > 0x7f800000u ? 255 : e + 127);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    kv4_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int n_slots,
                    const int32_t* __restrict__ slots, int n, uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5); r < n; r += gridDim.x * kWarpsPerBlock) {
    const int slot = __ldg(slots + r);
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0 && slot < n_slots) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + (int64_t)slot * kKv4CodeBytes) + lane);
      const float s = kv4_scale(__ldg(scales + (int64_t)slot * kKv4ScaleBytes + (lane >> 1)));
      uint32_t h[8];
      kv4_decode8(w.x, *reinterpret_cast<uint32_t(*)[4]>(&h[0]));
      kv4_decode8(w.y, *reinterpret_cast<uint32_t(*)[4]>(&h[4]));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        o[i] = pack2_rn<kBf16>(f.x * s, f.y * s);
      }
    }
    uint4* dst = out + (int64_t)r * (kKv4Dim / 8) + lane * 2;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ------------------------------------------------------------------------------------ step plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = DS4X_MAX_REQ / kPlanThreads;  // requests a thread sums up
constexpr int kPlanCluster = 8, kPlanBlocks = 64;
constexpr uint32_t kSat = 0x7fffffffu;

struct PlanParams {
  const int32_t *seen, *n_new, *rows, *free_pages, *n_free;
  int32_t *tables, *positions, *req, *slots, *seen_out, *rows_out, *n_free_out, *totals;
  int n_req, ratio, log_page, max_pages, free_cap, T_cap, R_cap;
  int in_place;  // an output is its input: with more than one block they are a cluster
};

// Sums of counts stay at kSat once they reach it (associative, so a scan may use it).
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// First request in [lo, hi) whose inclusive sum is above x; hi if there is none.
__device__ __forceinline__ int find_above(const uint32_t* ends, int lo, int hi, uint32_t x) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}
// The same by a whole warp: each lane looks at the last place of its part.
__device__ __forceinline__ int warp_find_above(const uint32_t* ends, int lo, int hi, uint32_t x) {
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + (lane + 1) * step - 1;
    const uint32_t above = __ballot_sync(0xffffffffu, at >= hi || ends[at] > x);
    if (above == 0) return hi;  // 32 whole parts, and none of them ends above x
    const int f = __ffs(above) - 1;
    if (step == 1) return min(lo + f, hi);
    hi = min(hi, lo + (f + 1) * step - 1);  // that place is above x already
    lo += f * step;
  }
  return lo;
}
// f(element, request) for elements [0, n) of lists packed by request, `ends` their inclusive sums; request
// n_req for what lies behind the last list.  Each warp takes a run of whole 32s; `shift` moves the runs on
// by as many warps, so that short lists are filled by warps of their own.  Returns the shift for the next.
template <typename F>
__device__ __forceinline__ uint32_t for_packed(const uint32_t* ends, int n_req, uint32_t n, uint32_t shift, F f) {
  const uint32_t warps = gridDim.x * (kPlanThreads / 32), lane = threadIdx.x & 31;
  const uint32_t run = ((n + 31) / 32 + warps - 1) / warps * 32, runs = run ? (n + run - 1) / run : 0;
  const uint32_t mine = (blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5) + warps - shift % warps) % warps;
  if (mine < runs) {
    const uint32_t begin = mine * run, end = min(begin + run, n);
    int b0 = warp_find_above(ends, 0, n_req, begin);
    for (uint32_t x0 = begin; x0 < end; x0 += 128) {
      const uint32_t x1 = min(x0 + 127, end - 1);
      const int at = b0 + (int)lane;
      const uint32_t above = __ballot_sync(0xffffffffu, at >= n_req || ends[at] > x1);
      const int b1 = above ? min(b0 + __ffs(above) - 1, n_req) : warp_find_above(ends, b0 + 32, n_req, x1);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t x = x0 + 32 * i + lane;
        if (x < end) f(x, find_above(ends, b0, b1, x));
      }
      b0 = b1;
    }
  }
  return shift + runs;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
  extern __shared__ uint32_t sm[];
  const int B = p.n_req;
  uint32_t* tok_end = sm;              // inclusive sums over requests: tokens,
  uint32_t* row_end = sm + B;          // completed rows,
  uint32_t* page_end = sm + 2 * B;     // pages wanted
  int32_t* seen_s = reinterpret_cast<int32_t*>(sm + 3 * B);
  int32_t* rows_s = reinterpret_cast<int32_t*>(sm + 4 * B);
  uint32_t* new_s = sm + 5 * B;        // tokens of each request (a saturated sum does not give them back)
  int32_t* fits_s = reinterpret_cast<int32_t*>(sm + 6 * B);  // completed rows that its table has room for
  __shared__ uint32_t part[96];        // [3][32] the warps' sums
  __shared__ unsigned long long placed_s[32];  // placed rows, by warp of block 0
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ps = 1 << p.log_page;
  const int cap = p.max_pages << p.log_page;
  pdl_wait();
  pdl_trigger();

  uint32_t n[kPlanPer], c[kPlanPer], g[kPlanPer], sn = 0, sc = 0, sg = 0;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = tid * per;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    n[i] = c[i] = g[i] = 0;
    const int b = b0 + i;
    if (i < per && b < B) {
      const int s = max(p.seen[b], 0);
      const int after = (int)min((uint32_t)s + (uint32_t)max(p.n_new[b], 0), kSat);
      const int r0 = min(max(p.rows[b], 0), cap);
      n[i] = after - s;
      c[i] = after / p.ratio - s / p.ratio;
      // row r of a request is its r-th pooled row: one that ran short earlier takes no more rows
      const int fits = r0 < s / p.ratio ? 0 : min((int)c[i], cap - r0);
      const int held = (r0 >> p.log_page) + ((r0 & (ps - 1)) != 0);
      const int end = r0 + fits;
      g[i] = (end >> p.log_page) + ((end & (ps - 1)) != 0) - held;
      seen_s[b] = s;
      rows_s[b] = r0;
      new_s[b] = n[i];
      fits_s[b] = fits;
    }
    sn = sat_add(sn, n[i]);
    sc = sat_add(sc, c[i]);
    sg = sat_add(sg, g[i]);
  }
  const int F = min(max(p.n_free[0], 0), p.free_cap);
  // inclusive scan of the threads' sums
  uint32_t in = sn, ic = sc, ig = sg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, in, d), b = __shfl_up_sync(0xffffffffu, ic, d),
                   e = __shfl_up_sync(0xffffffffu, ig, d);
    if (lane >= d) {
      in = sat_add(in, a);
      ic = sat_add(ic, b);
      ig = sat_add(ig, e);
    }
  }
  if (lane == 31) {
    part[warp] = in;
    part[32 + warp] = ic;
    part[64 + warp] = ig;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t a = part[lane], b = part[32 + lane], e = part[64 + lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d),
                     z = __shfl_up_sync(0xffffffffu, e, d);
      if (lane >= d) {
        a = sat_add(a, x);
        b = sat_add(b, y);
        e = sat_add(e, z);
      }
    }
    part[lane] = a;
    part[32 + lane] = b;
    part[64 + lane] = e;
  }
  __syncthreads();
  {
    // exclusive sums before this thread, then the inclusive ones of its requests
    uint32_t a = __shfl_up_sync(0xffffffffu, in, 1), b = __shfl_up_sync(0xffffffffu, ic, 1),
             e = __shfl_up_sync(0xffffffffu, ig, 1);
    if (lane == 0) a = b = e = 0;
    if (warp > 0) {
      a = sat_add(a, part[warp - 1]);
      b = sat_add(b, part[32 + warp - 1]);
      e = sat_add(e, part[64 + warp - 1]);
    }
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      a = sat_add(a, n[i]);
      b = sat_add(b, c[i]);
      e = sat_add(e, g[i]);
      if (i < per && b0 + i < B) {
        tok_end[b0 + i] = a;
        row_end[b0 + i] = b;
        page_end[b0 + i] = e;
      }
    }
  }
  // updated in place, the request state has been read by every block before any block writes it
  if (p.in_place && gridDim.x > 1) cluster_sync(); else __syncthreads();

  auto pages_got = [&](int b, int& first) {
    first = (int)min(b > 0 ? page_end[b - 1] : 0u, (uint32_t)F);
    return (int)min(page_end[b], (uint32_t)F) - first;
  };
  auto rows_placed = [&](int b, int held, int got) {
    const int64_t room = ((int64_t)(held + got) << p.log_page) - rows_s[b];
    return (int)min((int64_t)fits_s[b], room);
  };
  auto held_pages = [&](int b) { return (rows_s[b] >> p.log_page) + ((rows_s[b] & (ps - 1)) != 0); };

  uint32_t shift = for_packed(tok_end, B, (uint32_t)p.T_cap, 0, [&](uint32_t t, int b) {
    p.req[t] = b < B ? b : -1;
    p.positions[t] = b < B ? seen_s[b] + (int)(t - (b > 0 ? tok_end[b - 1] : 0u)) : -1;
  });
  shift = for_packed(row_end, B, (uint32_t)p.R_cap, shift, [&](uint32_t j, int b) {
    int slot = -1;
    if (b < B) {
      const int i = (int)(j - (b > 0 ? row_end[b - 1] : 0u));
      const int held = held_pages(b);
      int first;
      const int got = pages_got(b, first);
      if (i < rows_placed(b, held, got)) {
        const int row = rows_s[b] + i, pg = row >> p.log_page;
        const int page = pg < held ? p.tables[(int64_t)b * p.max_pages + pg]
                                   : p.free_pages[F - 1 - (first + pg - held)];
        const int64_t at = ((int64_t)page << p.log_page) + (row & (ps - 1));
        if (page >= 0 && at <= (int64_t)kSat) slot = (int)at;
      }
    }
    p.slots[j] = slot;
  });
  const int taken = B > 0 ? (int)min(page_end[B - 1], (uint32_t)F) : 0;
  for_packed(page_end, B, (uint32_t)taken, shift, [&](uint32_t k, int b) {
    const int first = (int)(b > 0 ? page_end[b - 1] : 0u);
    p.tables[(int64_t)b * p.max_pages + held_pages(b) + ((int)k - first)] = p.free_pages[F - 1 - (int)k];
  });
  if (blockIdx.x == 0) {
    unsigned long long mine = 0;
    for (int b = tid; b < B; b += kPlanThreads) {
      int first;
      const int held = held_pages(b), got = pages_got(b, first);
      const int pl = rows_placed(b, held, got);
      mine += (unsigned)pl;
      if (p.rows_out) p.rows_out[b] = rows_s[b] + pl;
      if (p.seen_out) p.seen_out[b] = seen_s[b] + (int)new_s[b];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if (lane == 0) placed_s[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < 32; ++i) mine += placed_s[i];
      if (p.n_free_out) *p.n_free_out = F - taken;
      if (p.totals) {
        p.totals[0] = B > 0 ? (int)tok_end[B - 1] : 0;
        p.totals[1] = B > 0 ? (int)row_end[B - 1] : 0;
        p.totals[2] = (int)min(mine, (unsigned long long)kSat);
        p.totals[3] = taken;
      }
    }
  }
}

// Blocks of 8 rows: every row its own warp while that fits the GPU eight times over, then strided.
int row_blocks(int n) {
  const int64_t want = ((int64_t)n + kWarpsPerBlock - 1) / kWarpsPerBlock;
  const int64_t most = (int64_t)device_sm_count() * 8 * 8;
  return (int)(want < most ? want : most);
}

}  // namespace
}  // namespace ds4x

using namespace ds4x;

extern "C" {

int ds4x_kv4_append(const void* rows, ds4x_dtype dtype, const int32_t* slots, int32_t n, int32_t Dkv, uint8_t* codes,
                    uint8_t* scales, int32_t n_slots, void* stream) {
  call_begin();
  if (n < 0 || Dkv <= 0 || n_slots < 0 || (dtype != DS4X_F16 && dtype != DS4X_BF16)) return DS4X_ERR_INVALID;
  if (Dkv != kKv4Dim) return DS4X_ERR_UNSUPPORTED;
  if (n == 0) return call_end(DS4X_OK);
  if (!rows || !slots || !aligned16(rows) || !aligned4(slots) ||
      (n_slots > 0 && (!codes || !scales || !aligned16(codes) || !aligned16(scales))))
    return DS4X_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_pdl(dtype == DS4X_BF16 ? kv4_append_kernel<true> : kv4_append_kernel<false>,
                                   dim3(row_blocks(n)), dim3(32 * kWarpsPerBlock), 0, st,
                                   static_cast<const uint4*>(rows), slots, n, n_slots, codes, scales);
  if (e != cudaSuccess) return DS4X_ERR_CUDA;
  count_launch();
  return call_end(DS4X_OK);
}

int ds4x_kv4_read(const uint8_t* codes, const uint8_t* scales, int32_t n_slots, const int32_t* slots, int32_t n,
                  int32_t Dkv, void* out, ds4x_dtype dtype, void* stream) {
  call_begin();
  if (n < 0 || Dkv <= 0 || n_slots < 0 || (dtype != DS4X_F16 && dtype != DS4X_BF16)) return DS4X_ERR_INVALID;
  if (Dkv != kKv4Dim) return DS4X_ERR_UNSUPPORTED;
  if (n == 0) return call_end(DS4X_OK);
  if (!out || !slots || !aligned16(out) || !aligned4(slots) ||
      (n_slots > 0 && (!codes || !scales || !aligned16(codes) || !aligned16(scales))))
    return DS4X_ERR_INVALID;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_pdl(dtype == DS4X_BF16 ? kv4_read_kernel<true> : kv4_read_kernel<false>,
                                   dim3(row_blocks(n)), dim3(32 * kWarpsPerBlock), 0, st, codes, scales, n_slots,
                                   slots, n, static_cast<uint4*>(out));
  if (e != cudaSuccess) return DS4X_ERR_CUDA;
  count_launch();
  return call_end(DS4X_OK);
}

int ds4x_page_plan(const int32_t* seen, const int32_t* n_new, const int32_t* rows, int32_t* tables,
                   const int32_t* free_pages, int32_t free_capacity, const int32_t* n_free, int32_t n_req,
                   int32_t max_pages, int32_t page_rows, int32_t ratio, int32_t T_cap, int32_t R_cap,
                   int32_t* positions, int32_t* req, int32_t* slots, int32_t* seen_out, int32_t* rows_out,
                   int32_t* n_free_out, int32_t* totals, void* stream) {
  call_begin();
  if (n_req < 0 || max_pages < 0 || free_capacity < 0 || T_cap < 0 || R_cap < 0 || ratio < 1 || page_rows < 1)
    return DS4X_ERR_INVALID;
  if ((page_rows & (page_rows - 1)) != 0 || page_rows > DS4X_MAX_PAGE_ROWS || n_req > DS4X_MAX_REQ)
    return DS4X_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_rows > INT32_MAX) return DS4X_ERR_UNSUPPORTED;
  if (n_req == 0 && (T_cap > 0 || R_cap > 0)) return DS4X_ERR_INVALID;  // nothing to fill the outputs from
  if (n_req == 0 && !n_free_out && !totals) return call_end(DS4X_OK);
  if ((n_req > 0 && (!seen || !n_new || !rows || (max_pages > 0 && !tables))) || !n_free ||
      (free_capacity > 0 && !free_pages) || (T_cap > 0 && (!positions || !req)) || (R_cap > 0 && !slots))
    return DS4X_ERR_INVALID;
  const void* all[] = {seen, n_new, rows, tables, free_pages, n_free, positions, req, slots,
                       seen_out, rows_out, n_free_out, totals};
  for (const void* q : all)
    if (!aligned4(q)) return DS4X_ERR_INVALID;
  int log_page = 0;
  while ((1 << log_page) < page_rows) ++log_page;
  const PlanParams p{seen,     n_new,    rows,       free_pages, n_free,  tables, positions, req,       slots,
                     seen_out, rows_out, n_free_out, totals,     n_req,   ratio,  log_page,  max_pages, free_capacity,
                     T_cap,    R_cap,    seen == seen_out || rows == rows_out || n_free == n_free_out};
  // four elements a thread to fill, if the blocks need not wait for one another
  const int64_t want = ((int64_t)T_cap + R_cap + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  const int most = p.in_place ? kPlanCluster : kPlanBlocks;
  const int blocks = want <= 1 ? 1 : p.in_place || want > most ? most : (int)want;
  const size_t smem = (size_t)7 * n_req * sizeof(uint32_t);
  // a launch has 48 KB without asking, the kernel's static arrays among them
  if (smem > 40 * 1024 && ensure_dynamic_smem(page_plan_kernel, 7 * DS4X_MAX_REQ * 4) != cudaSuccess)
    return DS4X_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.in_place && blocks > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, page_plan_kernel, p) != cudaSuccess) return DS4X_ERR_CUDA;
  count_launch();
  return call_end(DS4X_OK);
}

}  // extern "C"
