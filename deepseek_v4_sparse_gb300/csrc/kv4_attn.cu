// kv4_attn.cu — multi-query attention of 64 heads over rows of the paged 4-bit cache.
//
//   out[t,h,:] = sum_j softmax_j( scale * q[t,h,:] . kv_j ) * kv_j
//
// over the rows j that a token selected (indices) or over every row of its request that it can see,
// each row decoded from its codes and scales (kv4_common.cuh) on the way in.
//
// One warp a head, eight heads a block: every lane holds 16 of the 512 dims of q and of the output, a
// row's product is one warp reduction, and the softmax is the running one (maximum and sum of what has
// been seen, the output rescaled when the maximum moves).  All statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "ds4x_internal.h"
#include "ds4x_ptx.cuh"
#include "kv4_common.cuh"

namespace ds4x {
namespace {

constexpr int kHq = 64;

struct Params {
  const uint16_t* q;
  const uint8_t *codes, *scales;
  const int32_t *tables, *rows, *req, *positions, *indices, *counts;
  uint16_t* out;
  float* lse;
  int n_slots, n_req, max_pages, log_page, ratio, T, k_top;
  float scale;
};

// Request of token t and how many rows its list has (selected: list entries; else visible rows);
// `held` bounds the row numbers.
__device__ __forceinline__ int token_rows(const Params& p, int t, int& b, int& held) {
  b = p.req ? __ldg(p.req + t) : t;
  if (b < 0 || b >= p.n_req) return 0;
  held = min(max(__ldg(p.rows + b), 0), p.max_pages << p.log_page);
  if (p.indices) return p.counts ? min(max(__ldg(p.counts + t), 0), p.k_top) : p.k_top;
  if (!p.positions) return held;
  const int pos = __ldg(p.positions + t);
  return pos < 0 ? 0 : (int)min((int64_t)held, ((int64_t)pos + 1) / p.ratio);
}

// Slot of row `row` of request b, -1 if there is none.
__device__ __forceinline__ int row_slot(const Params& p, int b, int row, int held) {
  if (row < 0 || row >= held) return -1;
  const int page = __ldg(p.tables + (int64_t)b * p.max_pages + (row >> p.log_page));
  const int64_t slot = ((int64_t)page << p.log_page) + (row & ((1 << p.log_page) - 1));
  return page >= 0 && slot < p.n_slots ? (int)slot : -1;
}

template <bool kBf16>
__global__ void __launch_bounds__(256) kv4_attn_kernel(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x >> 3, h = (blockIdx.x & 7) * 8 + (threadIdx.x >> 5);
  int b, held = 0;
  const int n = token_rows(p, t, b, held);
  const int64_t at = ((int64_t)t * kHq + h) * kKv4Dim + lane * 16;
  float q[16], o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (kBf16) q[i] = __uint_as_float((uint32_t)p.q[at + i] << 16);
    else q[i] = __half2float(__ushort_as_half(p.q[at + i]));
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const int slot = row_slot(p, b, p.indices ? __ldg(p.indices + (int64_t)t * p.k_top + j) : j, held);
    if (slot < 0) continue;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes + (int64_t)slot * kKv4CodeBytes) + lane);
    const float s = kv4_scale(__ldg(p.scales + (int64_t)slot * kKv4ScaleBytes + (lane >> 1)));
    uint32_t c[8];
    kv4_decode8(w.x, *reinterpret_cast<uint32_t(*)[4]>(&c[0]));
    kv4_decode8(w.y, *reinterpret_cast<uint32_t(*)[4]>(&c[4]));
    float v[16], dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
      v[2 * i] = f.x * s;
      v[2 * i + 1] = f.y * s;
      dot += q[2 * i] * v[2 * i] + q[2 * i + 1] * v[2 * i + 1];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    const float x = dot * p.scale;
    if (x > m) {
      const float a = expf(m - x);  // 0 at the first row
      l *= a;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] *= a;
      m = x;
    }
    const float e = m == -INFINITY ? 0.f : expf(x - m);
    l += e;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] += e * v[i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (kBf16) {
      const __nv_bfloat16 r = __float2bfloat16_rn(o[i] * inv);
      p.out[at + i] = *reinterpret_cast<const uint16_t*>(&r);
    } else {
      p.out[at + i] = __half_as_ushort(__float2half_rn(o[i] * inv));
    }
  }
  if (p.lse && lane == 0) p.lse[(int64_t)t * kHq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv4_attn_workspace_bytes(int, int) { return 0; }

int launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  Params p;
  p.q = static_cast<const uint16_t*>(a.q_attn);
  p.codes = a.codes;
  p.scales = a.scales;
  p.tables = a.tables;
  p.rows = a.rows;
  p.req = a.req;
  p.positions = a.positions;
  p.indices = a.indices;
  p.counts = a.counts;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.n_slots = a.n_slots;
  p.n_req = a.n_req;
  p.max_pages = a.max_pages;
  p.log_page = a.log_page;
  p.ratio = a.ratio;
  p.T = a.T;
  p.k_top = a.k_top;
  p.scale = a.scale;
  if (launch_pdl(a.bf16 ? kv4_attn_kernel<true> : kv4_attn_kernel<false>, dim3((unsigned)a.T * 8u), dim3(256), 0,
                 stream, p) != cudaSuccess)
    return DS4X_ERR_CUDA;
  count_launch();
  return DS4X_OK;
}

}  // namespace ds4x

using namespace ds4x;

namespace {
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
}  // namespace

extern "C" {

size_t ds4x_kv4_attn_workspace_bytes(int32_t T, int32_t max_rows) {
  return T > 0 && max_rows > 0 ? kv4_attn_workspace_bytes(T, max_rows) : 0;
}

int ds4x_kv4_attn(const void* q_attn, ds4x_dtype dtype, const uint8_t* codes, const uint8_t* scales, int32_t n_slots,
                  const int32_t* tables, const int32_t* rows, int32_t n_req, int32_t max_pages, int32_t page_rows,
                  const int32_t* req, const int32_t* positions, int32_t ratio, const int32_t* indices,
                  const int32_t* counts, int32_t T, int32_t Hq, int32_t Dkv, int32_t k_top, float scale, void* out,
                  float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  call_begin();
  if (T < 0 || Hq <= 0 || Dkv <= 0 || n_slots < 0 || n_req < 0 || max_pages < 0 || page_rows < 1 || ratio < 1 ||
      (indices && k_top < 1) || (dtype != DS4X_F16 && dtype != DS4X_BF16))
    return DS4X_ERR_INVALID;
  if (Hq != 64 || Dkv != kKv4Dim || (indices && k_top > DS4X_MAX_KTOP)) return DS4X_ERR_UNSUPPORTED;
  if ((page_rows & (page_rows - 1)) != 0 || page_rows > DS4X_MAX_PAGE_ROWS) return DS4X_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_rows > INT32_MAX) return DS4X_ERR_UNSUPPORTED;
  if (T == 0) return call_end(DS4X_OK);
  if (!q_attn || !out || !aligned16(q_attn) || !aligned16(out) || (lse && !aligned16(lse)))
    return DS4X_ERR_INVALID;
  if (!req && T > n_req) return DS4X_ERR_INVALID;
  if (n_req > 0 && (!rows || (max_pages > 0 && !tables))) return DS4X_ERR_INVALID;
  if (n_slots > 0 && (!codes || !scales || !aligned16(codes) || !aligned16(scales))) return DS4X_ERR_INVALID;
  const void* ints[] = {tables, rows, req, positions, indices, counts};
  for (const void* i : ints)
    if (!aligned4(i)) return DS4X_ERR_INVALID;
  const int max_rows = indices ? k_top : max_pages * page_rows;
  const size_t need = ds4x_kv4_attn_workspace_bytes(T, max_rows);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DS4X_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return DS4X_ERR_INVALID;
  int log_page = 0;
  while ((1 << log_page) < page_rows) ++log_page;
  const Kv4AttnArgs a{q_attn, dtype == DS4X_BF16 ? 1 : 0, codes,     scales,    n_slots, tables,
                      rows,   n_req,                      max_pages, log_page,  req,     positions,
                      ratio,  indices,                    counts,    T,         k_top,   scale,
                      out,    lse,                        workspace};
  return call_end(launch_kv4_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
