// kv4_attn.cu — multi-query attention of 64 heads over rows of the paged 4-bit cache.
//
//   out[t,h,:] = sum_j softmax_j( scale * q[t,h,:] . kv_j ) * kv_j
//
// over the rows j that a token selected (indices) or over every row of its request that it can see.
//
// The products run on the tensor cores in fp16, whatever the type of q: a row's values (code times a
// power of two, kv4_common.cuh) are exact in fp16, q is made so by a power of two a head (which moves its
// largest magnitude to [2^14, 2^15); what falls below fp16's range then is under 2^-39 of the largest),
// and the softmax weights keep eleven bits instead of bf16's eight.
//
// One block an SM.  The tokens' rows are cut into chunks of 64; all chunks of all tokens form one
// sequence, and each block takes an equal, contiguous part of it.  A token whose chunks lie in several
// blocks leaves its unnormalised sums there in fp32 and kv4_combine_kernel joins them, so a long row list
// of one token, a ragged batch and a full prefill chunk are all spread evenly.  Per chunk:
//   S   [64 heads x 64 rows] = Q . K^T       tcgen05, M = 64 (heads on TMEM lanes), K-major
//   O^T [512 x 64 heads]    += V^T . P^T     tcgen05, M = 128 (dims), A MN-major, B K-major
// with K = V = the chunk, decoded once into 128B-swizzled shared memory (8 slots of 64 dims, two buffers).
//
// Warps: 0-7 fetch and decode rows, 8-11 softmax (heads 16*(warp-8) .. +15, 4 threads a head), 12-15
// convert q and write the output (O^T lanes by quadrant), 16 issues the S products, 17 the O^T products.
// A fetching thread owns 32 values (one scale group) of a row in each quarter of the dims: the codes of
// the next chunk are in its registers while it decodes this one, the table entries of the one after and
// the indices of the third are on their way.  Buffers are released in quarters, O^T rotates over six
// 64-column TMEM slots (a token uses four), so neighbouring tokens overlap.
//
// The running maximum of a head moves only when a logit exceeds it by more than 2^8 (O^T's column and
// the sums are rescaled then); weights are 2^7 times 2^(x - m), which keeps them below fp16's largest
// value and small ones away from its least.  Statistics and sums are fp32.
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
constexpr int kRows = 64;                        // rows per chunk
constexpr int kSlots = kKv4Dim / 64;             // 8 slots of 64 dims
constexpr int kPairs = kSlots / 2;               // quarters of 128 dims
constexpr int kSlotBytes = kRows * 128;          // 8 KB
constexpr int kBufBytes = kSlots * kSlotBytes;   // 64 KB a chunk
constexpr int kQBlockBytes = kHq * 128;          // 8 KB (64 heads x 64 dims)
constexpr int kQBytes = kSlots * kQBlockBytes;   // 64 KB
constexpr int kPBytes = kHq * 128;               // 8 KB: P[h][j]
constexpr int kTokens = 2048;                    // tokens a launch plans for
constexpr int kDecWarps = 8, kSoftWarp = 8, kOutWarp = 12, kSWarp = 16, kOWarp = 17;
constexpr int kWarps = 18, kThreads = 32 * kWarps;
constexpr int kOSlots = 6;                       // O^T slots of 64 TMEM columns
constexpr int kOffKV = kQBytes;
constexpr int kOffP = kOffKV + 2 * kBufBytes;
constexpr int kOffAlpha = kOffP + 2 * kPBytes;   // float[64]: rescale factors of one chunk
constexpr int kOffLM = kOffAlpha + kHq * 4;      // float[2 items][4][64]: sum of rounded weights, sum, m, 1 / first
constexpr int kOffCq = kOffLM + 2 * 4 * kHq * 4; // float[2 items][2][64]: logit factor, q factor of a head
constexpr int kOffRows = kOffCq + 2 * 2 * kHq * 4;  // int[kTokens]: rows of each token's list
constexpr int kOffMask = kOffRows + kTokens * 4; // uint16[2 buffers][4]: rows of the chunk that count
constexpr int kOffScan = kOffMask + 16;          // int64[18] warp sums, then int[4]: the block's part
constexpr int kOffBars = kOffScan + 18 * 8 + 16;
constexpr int kNumBars = 2 * kPairs + 2 * 2 * kPairs + 4 * 2 + 2 * kOSlots + 2 * 2;
constexpr int kOffTmemSlot = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmemSlot + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kColO = 128;  // S in columns [0, 128), O^T from 128
constexpr float kRescaleLog2 = 8.0f, kWeightLog2 = 7.0f;
constexpr int kSoftBar = 1, kEpiBar = 2, kGroupThreads = 128;
constexpr int kPartFloats = kHq * kKv4Dim;        // unnormalised sums of a part, then its statistics
constexpr int kStatFloats = 3 * kHq;              // sum of rounded weights, sum, m

struct Params {
  const uint16_t* q;
  const uint8_t *codes, *scales;
  const int32_t *tables, *rows, *req, *positions, *indices, *counts;
  uint16_t* out;
  float* lse;
  int* status;
  int4* parts_of;  // [grid]: the token a block starts in, chunks of it before the block, chunks it has, quota
  float* part;     // [2 grid][kPartFloats]
  float* stat;     // [2 grid][kStatFloats]
  int n_slots, n_req, max_pages, log_page, ratio, t0, T, k_top;
  float scale;
};

__device__ __forceinline__ int request_of(const Params& p, int t) { return p.req ? __ldg(p.req + t) : p.t0 + t; }

// Rows in the list of token t (selected: list entries; else visible rows).
__device__ __forceinline__ int token_rows(const Params& p, int t) {
  const int b = request_of(p, t);
  if (b < 0 || b >= p.n_req) return 0;
  if (p.indices) return p.counts ? min(max(__ldg(p.counts + t), 0), p.k_top) : p.k_top;
  const int held = min(max(__ldg(p.rows + b), 0), p.max_pages << p.log_page);
  if (!p.positions) return held;
  const int pos = __ldg(p.positions + t);
  return pos < 0 ? 0 : (int)min((int64_t)held, ((int64_t)pos + 1) / p.ratio);
}
__device__ __forceinline__ int chunks_of(int rows) { return rows > kRows ? (rows - 1) / kRows + 1 : 1; }

// A block's part of the chunk sequence, walked token by token: chunks [c0, c1) of token t.
struct Walk {
  int t, c0, c1, left;
  const int* rows;
  __device__ __forceinline__ Walk(const int* rows_s, const int* start) : t(start[0]), c0(start[1]), left(start[2]), rows(rows_s) {
    c1 = left > 0 ? min(chunks_of(rows[t]), c0 + left) : c0;
  }
  __device__ __forceinline__ void next() {
    left -= c1 - c0;
    ++t;
    c0 = 0;
    c1 = left > 0 ? min(chunks_of(rows[t]), left) : 0;
  }
};

template <bool kBf16>
__device__ __forceinline__ uint16_t to16(float x) {
  if constexpr (kBf16) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
  } else {
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
  }
}
// Two 16-bit values as fp32, times f, as fp16.
template <bool kBf16>
__device__ __forceinline__ uint32_t scaled2(uint32_t u, float f) {
  float2 v;
  if constexpr (kBf16) v = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else v = __half22float2(*reinterpret_cast<const __half2*>(&u));
  const __half2 h = __floats2half2_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_kernel(const Params p) {
  constexpr uint32_t kIdescS = idesc_f16(64, kHq, 0, 0, 0);
  constexpr uint32_t kIdescO = idesc_f16(128, kHq, 0, 1, 0);
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) report_timeout(p.status, 0x7d);
    return;
  }
  uint8_t* sq = smem;
  uint8_t* skv = smem + kOffKV;
  uint8_t* sp = smem + kOffP;
  float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);
  float* lm = reinterpret_cast<float*>(smem + kOffLM);
  float* cq = reinterpret_cast<float*>(smem + kOffCq);
  int* rows_s = reinterpret_cast<int*>(smem + kOffRows);
  uint16_t* mask_s = reinterpret_cast<uint16_t*>(smem + kOffMask);
  long long* scan = reinterpret_cast<long long*>(smem + kOffScan);
  int* start = reinterpret_cast<int*>(smem + kOffScan + 18 * 8);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + kOffBars);  // [quarter]
  uint64_t* qempty = qfull + kPairs;        // [quarter]
  uint64_t* kvfull = qempty + kPairs;       // [buffer][quarter]
  uint64_t* kvempty = kvfull + 2 * kPairs;  // [buffer][quarter]
  uint64_t* sfull = kvempty + 2 * kPairs;
  uint64_t* sempty = sfull + 2;
  uint64_t* pfull = sempty + 2;
  uint64_t* pempty = pfull + 2;
  uint64_t* ofull = pempty + 2;             // [O^T slot]
  uint64_t* oempty = ofull + kOSlots;       // [O^T slot]
  uint64_t* lready = oempty + kOSlots;      // [item parity] statistics written
  uint64_t* lfree = lready + 2;             // [item parity] ... and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmemSlot);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto oslot = [](uint32_t item, int db) { return (int)((4u * (item % 3u) + (uint32_t)db) % kOSlots); };

  if (tid == 0) {
    for (int i = 0; i < kPairs; ++i) {
      mbar_init(&qfull[i], 4);
      mbar_init(&qempty[i], 1);
    }
    for (int i = 0; i < 2 * kPairs; ++i) {
      mbar_init(&kvfull[i], kDecWarps);
      mbar_init(&kvempty[i], 1);
    }
    for (int i = 0; i < kOSlots; ++i) {
      mbar_init(&ofull[i], 1);
      mbar_init(&oempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 2);  // the products' completion and the issuing warp itself
      mbar_init(&sempty[i], 4);
      mbar_init(&pfull[i], 4);
      mbar_init(&pempty[i], 1);
      mbar_init(&lready[i], 4);
      mbar_init(&lfree[i], 4);
    }
    fence_mbarrier_init();
  }
  if (warp == kSWarp) tmem_alloc(tmem_slot, kTmemCols);
  pdl_wait();  // everything above touched only this block's own resources
  pdl_trigger();

  // --------------------------------------------------- every token's rows; this block's part
  {
    constexpr int kPer = (kTokens + kThreads - 1) / kThreads;
    const int per = (p.T + kThreads - 1) / kThreads;
    int n[kPer];
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tid * per + i;
      n[i] = (i < per && t < p.T) ? token_rows(p, t) : -1;
      if (n[i] >= 0) {
        rows_s[t] = n[i];
        sum += chunks_of(n[i]);
      }
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) start[2] = 0;
    __syncthreads();
    long long before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long v = scan[w];
      if (w < warp) before += v;
      total += v;
    }
    const long long quota = (total + gridDim.x - 1) / gridDim.x;
    const long long g0 = quota * blockIdx.x, g1 = min(total, g0 + quota);
    if (g0 < total) {
      long long at = before;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (n[i] < 0) continue;
        const int nch = chunks_of(n[i]);
        if (at <= g0 && g0 < at + nch) {
          start[0] = tid * per + i;
          start[1] = (int)(g0 - at);
          start[2] = (int)(g1 - g0);
          p.parts_of[blockIdx.x] = make_int4(tid * per + i, (int)(g0 - at), nch, (int)quota);
        }
        at += nch;
      }
    } else if (tid == 0) {
      p.parts_of[blockIdx.x] = make_int4(-1, 0, 0, (int)quota);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kDecWarps) {
    // --------------------------------------------------------------------- fetch and decode
    // row 16 (warp % 4) + lane % 16 of the chunk; in each quarter of the dims the 32 values of slot
    // warp / 4, half lane / 16.  Eight neighbouring lanes store to eight rows of one 16-byte column:
    // the swizzle puts them in different banks; the two halves of a row share its 32-byte sectors.
    const int r = 16 * (warp & 3) + (lane & 15);
    const int sub = 2 * (warp >> 2) + (lane >> 4);  // group within a quarter
    uint32_t st_off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      st_off[k] = (uint32_t)((warp >> 2) * kSlotBytes + r * 128 + ((((lane >> 4) * 4 + k) ^ (r & 7)) << 4));
    const bool listed = p.indices != nullptr;
    // cursor: the next chunk whose row number is to be fetched
    int t = start[0], c = start[1], left = start[2];
    int row_a = -1, b_a = 0;                       // stage a: row number and request on their way
    int row_b = -1, page_b = -1, held_b = 0;       // stage b: table entry (and rows held) on their way
    auto fetch_row = [&]() {
      row_a = -1;
      if (left > 0) {
        const int j = c * kRows + r, n = rows_s[t];
        b_a = request_of(p, t);
        if (j < n) row_a = listed ? __ldg(p.indices + (int64_t)t * p.k_top + j) : j;
        --left;
        if (++c >= chunks_of(n)) {
          c = 0;
          ++t;
        }
      }
    };
    auto fetch_page = [&]() {
      row_b = row_a;
      page_b = -1;
      if (row_a >= 0 && (row_a >> p.log_page) < p.max_pages) {
        page_b = __ldg(p.tables + (int64_t)b_a * p.max_pages + (row_a >> p.log_page));
        held_b = listed ? __ldg(p.rows + b_a) : 0x7fffffff;
      }
    };
    const uint8_t* src = nullptr;   // codes of the chunk to load next; nullptr: the row does not count
    uint4 d[kPairs], sc = make_uint4(0, 0, 0, 0);
    auto resolve = [&]() {
      const int64_t slot = ((int64_t)page_b << p.log_page) + (row_b & ((1 << p.log_page) - 1));
      const bool ok = page_b >= 0 && slot < p.n_slots && row_b < held_b;
      src = ok ? p.codes + slot * kKv4CodeBytes + sub * 16 : nullptr;
      return ok ? p.scales + slot * kKv4ScaleBytes : nullptr;
    };
    auto load_quarter = [&](int pr) {
      d[pr] = src ? __ldg(reinterpret_cast<const uint4*>(src + pr * 64)) : make_uint4(0, 0, 0, 0);
    };
    const int chunks = left;
    fetch_row();
    fetch_page();
    fetch_row();
    {
      const uint8_t* s = resolve();
      sc = s ? __ldg(reinterpret_cast<const uint4*>(s)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int pr = 0; pr < kPairs; ++pr) load_quarter(pr);
    }
    bool live = src != nullptr;
    fetch_page();
    fetch_row();
    bool ok = true;
    for (int g = 0; g < chunks && ok; ++g) {
      const int b = g & 1;
      const uint32_t ph = ((g >> 1) & 1) ^ 1;
      const uint8_t* s_next = resolve();  // of chunk g + 1
      const bool live_next = src != nullptr;
      const uint4 sc_now = sc;
      sc = s_next ? __ldg(reinterpret_cast<const uint4*>(s_next)) : make_uint4(0, 0, 0, 0);
      fetch_page();  // of g + 2
      fetch_row();   // of g + 3
      const uint32_t live_bits = __ballot_sync(0xffffffffu, live);
      const uint32_t base = smem_u32(skv) + b * kBufBytes;
#pragma unroll
      for (int pr = 0; pr < kPairs; ++pr) {
        const uint4 now = d[pr];
        load_quarter(pr);
        const uint32_t word = pr == 0 ? sc_now.x : pr == 1 ? sc_now.y : pr == 2 ? sc_now.z : sc_now.w;
        const __half2 s2 = __float2half2_rn(kv4_scale((word >> (8 * sub)) & 255u));
        if (!mbar_wait(&kvempty[b * kPairs + pr], ph, p.status, 61)) {
          ok = false;
          break;
        }
        if (pr == 0 && warp < 4 && lane == 0) mask_s[b * 4 + warp] = (uint16_t)live_bits;
        const uint32_t w4[4] = {now.x, now.y, now.z, now.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h[4];
          kv4_decode8(w4[k], h);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + 2 * pr * kSlotBytes + st_off[k]),
                       "r"(mul2(h[0], s2)), "r"(mul2(h[1], s2)), "r"(mul2(h[2], s2)), "r"(mul2(h[3], s2))
                       : "memory");
        }
        fence_proxy_async();  // decoded rows -> visible to the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&kvfull[b * kPairs + pr]);
      }
      live = live_next;
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------------------ S = Q K^T
    uint32_t gc = 0, item = 0;
    bool ok = true;
    const uint32_t q_addr = smem_u32(sq), kv_addr = smem_u32(skv);
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next(), ++item) {
      for (int c = w.c0; c < w.c1; ++c, ++gc) {
        const int b = gc & 1;
        if (!mbar_wait_warp(&sempty[b], ((gc >> 1) & 1) ^ 1, p.status, 62)) { ok = false; break; }
        for (int pr = 0; pr < kPairs; ++pr) {
          if (c == w.c0 && !mbar_wait_warp(&qfull[pr], item & 1, p.status, 63)) { ok = false; break; }
          if (!mbar_wait_warp(&kvfull[b * kPairs + pr], (gc >> 1) & 1, p.status, 64)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const int kb = 2 * pr + h2;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t a = desc_sw128(q_addr + kb * kQBlockBytes + kk * 32, 16, 1024);
              const uint64_t bd = desc_sw128(kv_addr + b * kBufBytes + kb * kSlotBytes + kk * 32, 16, 1024);
              tc_mma_f16_elect(tmem + b * kHq, a, bd, kIdescS, (kb | kk) != 0);
            }
          }
          if (c == w.c1 - 1) tc_commit_elect(&qempty[pr]);  // the next item's q may replace this quarter
        }
        if (!ok) break;
        // the arrival of this warp hands on what it waited for (the chunk's mask, the item's factors)
        if (lane == 0) mbar_arrive(&sfull[b]);
        tc_commit_elect(&sfull[b]);
      }
    }
  } else if (warp == kOWarp) {
    // --------------------------------------------------------------------- O^T += V^T P^T
    uint32_t gc = 0, item = 0;
    uint32_t o_ph = 0;  // bit s: phase of O^T slot s's empty barrier
    bool ok = true;
    const uint32_t kv_addr = smem_u32(skv), p_addr = smem_u32(sp);
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next(), ++item) {
      for (int c = w.c0; c < w.c1; ++c, ++gc) {
        const int b = gc & 1;
        if (!mbar_wait_warp(&pfull[b], (gc >> 1) & 1, p.status, 65)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int db = 0; db < kPairs; ++db) {
          const int os = oslot(item, db);
          // an item's first product overwrites its slot: the output that last read it is done
          if (c == w.c0) {
            if (!mbar_wait_warp(&oempty[os], ((o_ph >> os) & 1u) ^ 1u, p.status, 66)) { ok = false; break; }
            o_ph ^= 1u << os;
            tc_fence_after();
          }
#pragma unroll
          for (int ks = 0; ks < kRows / 16; ++ks) {
            const uint64_t a = desc_sw128(kv_addr + b * kBufBytes + (2 * db) * kSlotBytes + ks * 2048, kSlotBytes, 1024);
            const uint64_t bd = desc_sw128(p_addr + b * kPBytes + ks * 32, 16, 1024);
            tc_mma_f16_elect(tmem + kColO + os * kHq, a, bd, kIdescO, (c > w.c0 || ks > 0));
          }
          tc_commit_elect(&kvempty[b * kPairs + db]);  // this quarter of the chunk is free
          if (c == w.c1 - 1) tc_commit_elect(&ofull[os]);
        }
        if (!ok) break;
        tc_commit_elect(&pempty[b]);
      }
    }
  } else if (warp < kOutWarp) {
    // ---------------------------------------------------------------------------- softmax
    // S holds head 16 quad + i on TMEM lane 32 quad + i (i < 16).  The 16x256b load gives thread
    // (g = lane / 4, e = lane % 4) the heads hA = 16 quad + g and hB = hA + 8 and, of each, the
    // columns 8 r + 2 e + {0, 1}, r = 0..7: a head's 64 logits are spread over 4 threads.
    const int quad = warp - kSoftWarp;
    const int g = lane >> 2, e = lane & 3;
    const int hA = 16 * quad + g, hB = hA + 8;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t gc = 0, item = 0;
    bool ok = true;
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next(), ++item) {
      float mA = -INFINITY, mB = -INFINITY;          // running maximum (log2 units)
      float lA = 0.f, lB = 0.f, rA = 0.f, rB = 0.f;  // sums of the weights, and of the rounded ones
      for (int ci = w.c0; ci < w.c1; ++ci, ++gc) {
        const int b = gc & 1;
        ok = named_and(kSoftBar, kGroupThreads, mbar_wait(&sfull[b], (gc >> 1) & 1, p.status, 67));
        if (!ok) break;
        tc_fence_after();
        float x[32];
        tmem_ld_16x256b_x8(tmem + t_lane + b * kHq, x);
        const uint2 live = *reinterpret_cast<const uint2*>(mask_s + b * 4);
        const float cA = cq[(item & 1) * 2 * kHq + hA], cB = cq[(item & 1) * 2 * kHq + hB];
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[b]);
        const uint32_t v0 = live.x >> (2 * e), v1 = live.y >> (2 * e);
        float mxA = -INFINITY, mxB = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t bits = (r < 4 ? v0 : v1) >> (8 * (r & 3));
          const bool ok0 = (bits & 1u) != 0, ok1 = (bits & 2u) != 0;
          x[4 * r] = ok0 ? x[4 * r] * cA : -INFINITY;
          x[4 * r + 2] = ok0 ? x[4 * r + 2] * cB : -INFINITY;
          x[4 * r + 1] = ok1 ? x[4 * r + 1] * cA : -INFINITY;
          x[4 * r + 3] = ok1 ? x[4 * r + 3] * cB : -INFINITY;
          mxA = fmaxf(mxA, fmaxf(x[4 * r], x[4 * r + 1]));
          mxB = fmaxf(mxB, fmaxf(x[4 * r + 2], x[4 * r + 3]));
        }
        mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 1));
        mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 1));
        mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, 2));
        mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, 2));
        float aA = 1.f, aB = 1.f;
        bool needA = false, needB = false;
        if (mxA > mA + kRescaleLog2) {
          needA = mA != -INFINITY;  // nothing has been accumulated before a head's first row
          aA = needA ? ex2_approx(mA - mxA) : 0.f;
          mA = mxA;
        }
        if (mxB > mB + kRescaleLog2) {
          needB = mB != -INFINITY;
          aB = needB ? ex2_approx(mB - mxB) : 0.f;
          mB = mxB;
        }
        if (named_or(kSoftBar, kGroupThreads, needA || needB)) {
          if (e == 0) {
            alpha_s[hA] = needA ? aA : 1.f;
            alpha_s[hB] = needB ? aB : 1.f;
          }
          named_sync(kSoftBar, kGroupThreads);
          // O^T must hold all of the previous chunk before its columns are rescaled
          const uint32_t prev = gc - 1;
          ok = named_and(kSoftBar, kGroupThreads, mbar_wait(&pempty[prev & 1], (prev >> 1) & 1, p.status, 68));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int q2 = 0; q2 < 2 * kPairs; ++q2) {  // 4 quarters x 2 halves of 32 heads
            float v[32];
            const uint32_t ta = tmem + t_lane + kColO + oslot(item, q2 >> 1) * kHq + (q2 & 1) * 32;
            tmem_ld32(ta, v);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= alpha_s[(q2 & 1) * 32 + i];
            tmem_st32(ta, v);
          }
          tc_wait_st();
          named_sync(kSoftBar, kGroupThreads);
        }
        lA *= aA;
        rA *= aA;
        lB *= aB;
        rB *= aB;
        // weights 2^(x - m + 7), rounded to fp16 for the product
        const float nA = kWeightLog2 - (mA == -INFINITY ? 0.f : mA);
        const float nB = kWeightLog2 - (mB == -INFINITY ? 0.f : mB);
        uint32_t pkA[8], pkB[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float a0 = ex2_approx(x[4 * r] + nA), a1 = ex2_approx(x[4 * r + 1] + nA);
          const float b0 = ex2_approx(x[4 * r + 2] + nB), b1 = ex2_approx(x[4 * r + 3] + nB);
          const __half2 hp = __floats2half2_rn(a0, a1), hq = __floats2half2_rn(b0, b1);
          lA += a0 + a1;
          lB += b0 + b1;
          const float2 fp = __half22float2(hp), fq = __half22float2(hq);
          rA += fp.x + fp.y;
          rB += fq.x + fq.y;
          pkA[r] = *reinterpret_cast<const uint32_t*>(&hp);
          pkB[r] = *reinterpret_cast<const uint32_t*>(&hq);
        }
        ok = named_and(kSoftBar, kGroupThreads, mbar_wait(&pempty[b], ((gc >> 1) & 1) ^ 1, p.status, 69));
        if (!ok) break;
        {
          // P[h][j], K-major with the 128-byte swizzle: 16-byte chunk r of line h at (r ^ (h & 7))
          uint8_t* lineA = sp + b * kPBytes + hA * 128 + 4 * e;
          uint8_t* lineB = sp + b * kPBytes + hB * 128 + 4 * e;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            *reinterpret_cast<uint32_t*>(lineA + ((r ^ (hA & 7)) << 4)) = pkA[r];
            *reinterpret_cast<uint32_t*>(lineB + ((r ^ (hB & 7)) << 4)) = pkB[r];
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[b]);
      }
      if (!ok) break;
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        lA += __shfl_xor_sync(0xffffffffu, lA, d);
        lB += __shfl_xor_sync(0xffffffffu, lB, d);
        rA += __shfl_xor_sync(0xffffffffu, rA, d);
        rB += __shfl_xor_sync(0xffffffffu, rB, d);
      }
      // the slot of this item's parity was last read by the output of item - 2
      ok = named_and(kSoftBar, kGroupThreads, mbar_wait(&lfree[item & 1], ((item >> 1) & 1) ^ 1, p.status, 70));
      if (!ok) break;
      if (e == 0) {
        float* row = lm + (item & 1) * 4 * kHq;
        row[hA] = rA;
        row[kHq + hA] = lA;
        row[2 * kHq + hA] = mA;
        row[3 * kHq + hA] = rA == 0.f ? 0.f : 1.f / rA;
        row[hB] = rB;
        row[kHq + hB] = lB;
        row[2 * kHq + hB] = mB;
        row[3 * kHq + hB] = rB == 0.f ? 0.f : 1.f / rB;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&lready[item & 1]);
    }
  } else {
    // ------------------------------------------------------------- q in, output out
    const int quad = warp - kOutWarp, tid4 = tid - kOutWarp * 32;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    const bool odd = lane & 1;
    // a head's factors: q is multiplied by +-2^s, s from its largest magnitude (compared as bits); a
    // logit in log2 units is then |scale| log2(e) 2^-s times the product
    auto head_factors = [&](int t, uint32_t item) {
      float* f = cq + (item & 1) * 2 * kHq;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((int64_t)t * kHq + quad * 16) * kKv4Dim) + lane * 2;
#pragma unroll
      for (int h0 = 0; h0 < 16; h0 += 4) {
        uint4 u[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i][0] = __ldg(src + (h0 + i) * (kKv4Dim / 8));
          u[i][1] = __ldg(src + (h0 + i) * (kKv4Dim / 8) + 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top = __vmaxu2(top, u[i][k].x & 0x7fff7fffu);
            top = __vmaxu2(top, u[i][k].y & 0x7fff7fffu);
            top = __vmaxu2(top, u[i][k].z & 0x7fff7fffu);
            top = __vmaxu2(top, u[i][k].w & 0x7fff7fffu);
          }
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, d));
          top = max(top & 0xffffu, top >> 16);
          if (lane == 0) {
            const float a = kBf16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((uint16_t)top));
            int s = 0;
            if (a > 0.f && a < INFINITY) s = min(14 + 127 - (int)(__float_as_uint(a) >> 23), 126);
            const int h = quad * 16 + h0 + i;
            f[h] = fabsf(p.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - s) << 23);
            const float up = __uint_as_float((uint32_t)(127 + s) << 23);
            f[kHq + h] = p.scale < 0.f ? -up : up;
          }
        }
      }
    };
    // q of token t as fp16 into the operand's layout, quarter by quarter as the quarters become free
    auto convert_q = [&](int t, uint32_t item) {
      const float* f = cq + (item & 1) * 2 * kHq + kHq;
      const int h0 = tid4 >> 4, ch = tid4 & 15;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((int64_t)t * kHq + h0) * kKv4Dim) + ch;
      bool got = true;
      for (int pr = 0; pr < kPairs; ++pr) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __ldg(src + 8 * i * (kKv4Dim / 8) + pr * 16);
        got = got && mbar_wait_warp(&qempty[pr], (item & 1) ^ 1, p.status, 71);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int h = h0 + 8 * i;
          const float m = f[h];
          uint4 o;
          o.x = scaled2<kBf16>(u[i].x, m);
          o.y = scaled2<kBf16>(u[i].y, m);
          o.z = scaled2<kBf16>(u[i].z, m);
          o.w = scaled2<kBf16>(u[i].w, m);
          *reinterpret_cast<uint4*>(sq + (2 * pr + (ch >> 3)) * kQBlockBytes + h * 128 + (((ch & 7) ^ (h & 7)) << 4)) = o;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[pr]);
      }
      return got;
    };
    uint32_t item = 0;
    uint32_t f_ph = 0;  // bit s: phase of O^T slot s's full barrier
    bool ok = true;
    Walk w(rows_s, start);
    if (w.left > 0) {
      head_factors(w.t, 0);
      named_sync(kEpiBar, kGroupThreads);
      ok = named_and(kEpiBar, kGroupThreads, convert_q(w.t, 0));
    }
    // a wait that gave up is acted on where the four warps meet, so that they leave together
    for (; w.left > 0; w.next(), ++item) {
      if (w.left > w.c1 - w.c0) {  // the next item's q, while this item is worked on
        head_factors(w.t + 1, item + 1);
        named_sync(kEpiBar, kGroupThreads);
        const bool got = convert_q(w.t + 1, item + 1);
        ok = named_and(kEpiBar, kGroupThreads, ok && got);
        if (!ok) break;
      }
      const int par = item & 1;
      ok = named_and(kEpiBar, kGroupThreads, ok && mbar_wait(&lready[par], (item >> 1) & 1, p.status, 72));
      if (!ok) break;
      const float* lrow = lm + par * 4 * kHq;
      // chunks before the block, or behind it: the sums go to the block's first or second part
      const bool whole = w.c0 == 0 && w.c1 == chunks_of(rows_s[w.t]);
      const int64_t part = 2 * (int64_t)blockIdx.x + (w.c0 == 0);
      if (quad == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int hh = lane + 32 * k;
          const float l = lrow[kHq + hh], m = lrow[2 * kHq + hh];
          if (!whole) {
            float* st = p.stat + part * kStatFloats;
            st[hh] = lrow[hh];
            st[kHq + hh] = l;
            st[2 * kHq + hh] = m;
          } else if (p.lse) {
            p.lse[(int64_t)w.t * kHq + hh] = l == 0.f ? -INFINITY : (m + (log2f(l) - kWeightLog2)) * 0.69314718055994531f;
          }
        }
      }
#pragma unroll 1
      for (int db = 0; db < kPairs; ++db) {
        const int os = oslot(item, db);
        ok = ok && mbar_wait_warp(&ofull[os], (f_ph >> os) & 1u, p.status, 73);
        f_ph ^= 1u << os;
        tc_fence_after();
        float va[32], vb[32];
        tmem_ld32(tmem + t_lane + kColO + os * kHq, va);
        tmem_ld32(tmem + t_lane + kColO + os * kHq + 32, vb);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&oempty[os]);
        if (whole) {
          uint32_t* orow = reinterpret_cast<uint32_t*>(p.out + (int64_t)w.t * kHq * kKv4Dim);
          const int d_even = db * 128 + quad * 32 + (lane & ~1);
#pragma unroll
          for (int h0 = 0; h0 < kHq; h0 += 2) {
            const float a0 = (h0 < 32 ? va[h0 & 31] : vb[h0 & 31]) * lrow[3 * kHq + h0];
            const float a1 = (h0 < 32 ? va[(h0 + 1) & 31] : vb[(h0 + 1) & 31]) * lrow[3 * kHq + h0 + 1];
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
            const int hw = h0 + (odd ? 1 : 0);
            orow[((int64_t)hw * kKv4Dim + d_even) >> 1] =
                odd ? (uint32_t)to16<kBf16>(got) | ((uint32_t)to16<kBf16>(a1) << 16)
                    : (uint32_t)to16<kBf16>(a0) | ((uint32_t)to16<kBf16>(got) << 16);
          }
        } else {
          float* dst = p.part + part * kPartFloats + db * 128 + quad * 32 + lane;
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            dst[h * kKv4Dim] = va[h];
            dst[(h + 32) * kKv4Dim] = vb[h];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&lfree[par]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of a token that several blocks worked on (one block per boundary between two of them
// and head, 4 dims a thread): part i holds O_i = sum_j 2^(x_j - m_i) kv_j and the sums r_i of its rounded
// weights and l_i of the exact ones, so with M = max_i m_i
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) r_i,   lse = ln 2 (M + log2 sum_i 2^(m_i - M) l_i).
// The parts are added in the order of the blocks: the same bits on every run.
template <bool kBf16>
__global__ void __launch_bounds__(kKv4Dim / 4) kv4_combine_kernel(const int4* __restrict__ parts_of,
                                                                  const float* __restrict__ part,
                                                                  const float* __restrict__ stat, uint16_t* out,
                                                                  float* lse) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x + 1, h = blockIdx.y;
  const int4 at = parts_of[i];  // token, its chunks before block i, its chunks, a block's chunks
  // the boundary before block i joins a token only if it is the first that the token crosses
  if (at.x < 0 || at.y == 0 || at.y > at.w) return;
  const int n = 1 + (at.z - at.y + at.w - 1) / at.w;  // parts: block i - 1's second, then the first ones
  auto part_no = [&](int k) { return k == 0 ? 2 * (int64_t)(i - 1) + 1 : 2 * (int64_t)(i - 1 + k); };
  float mx = -INFINITY;
  for (int k = 0; k < n; ++k) mx = fmaxf(mx, stat[part_no(k) * kStatFloats + 2 * kHq + h]);
  float r = 0.f, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float* st = stat + part_no(k) * kStatFloats;
    const float4 o = *reinterpret_cast<const float4*>(part + part_no(k) * kPartFloats + h * kKv4Dim + 4 * threadIdx.x);
    const float m = st[2 * kHq + h];
    const float f = mx == -INFINITY ? 1.f : exp2f(m - mx);  // without a maximum all is 0 (or NaN)
    r += f * st[h];
    l += f * st[kHq + h];
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
  }
  const float inv = r == 0.f ? 0.f : 1.f / r;
  const uint32_t lo = (uint32_t)to16<kBf16>(acc.x * inv) | ((uint32_t)to16<kBf16>(acc.y * inv) << 16);
  const uint32_t hi = (uint32_t)to16<kBf16>(acc.z * inv) | ((uint32_t)to16<kBf16>(acc.w * inv) << 16);
  *reinterpret_cast<uint2*>(out + ((int64_t)at.x * kHq + h) * kKv4Dim + 4 * threadIdx.x) = make_uint2(lo, hi);
  if (threadIdx.x == 0 && lse)
    lse[(int64_t)at.x * kHq + h] =
        l == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx) + (log2f(l) - kWeightLog2)) * 0.69314718055994531f;
}

// Blocks for T tokens of up to max_rows rows: one an SM, at most one a chunk.
int grid_of(int T, int max_rows) {
  const int64_t chunks = (int64_t)T * (max_rows > kRows ? (max_rows - 1) / kRows + 1 : 1);
  const int sms = device_sm_count();
  return (int)(chunks < sms ? chunks : sms);
}
constexpr size_t kHeadBytes = 4096;  // the int4 of every block
static_assert(kHeadBytes / 16 >= 256, "blocks a launch may have");

}  // namespace

size_t kv4_attn_workspace_bytes(int T, int max_rows) {
  const int grid = grid_of(T < kTokens ? T : kTokens, max_rows);
  return kHeadBytes + (size_t)2 * grid * (kPartFloats + kStatFloats) * sizeof(float);
}

template <bool kBf16>
static int launch_typed(const Kv4AttnArgs& a, int max_rows, cudaStream_t stream) {
  if (ensure_dynamic_smem(kv4_attn_kernel<kBf16>, kSmem) != cudaSuccess) return DS4X_ERR_CUDA;
  Params p;
  p.codes = a.codes;
  p.scales = a.scales;
  p.tables = a.tables;
  p.rows = a.rows;
  p.status = device_status_ptr();
  p.n_slots = a.n_slots;
  p.n_req = a.n_req;
  p.max_pages = a.max_pages;
  p.log_page = a.log_page;
  p.ratio = a.ratio;
  p.k_top = a.k_top;
  p.scale = a.scale;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.parts_of = reinterpret_cast<int4*>(ws);
  for (int t0 = 0; t0 < a.T; t0 += kTokens) {  // launches on one stream: they may share the workspace
    p.t0 = t0;
    p.T = a.T - t0 < kTokens ? a.T - t0 : kTokens;
    const int grid = grid_of(p.T, max_rows);
    p.part = reinterpret_cast<float*>(ws + kHeadBytes);
    p.stat = p.part + (size_t)2 * grid * kPartFloats;
    p.q = static_cast<const uint16_t*>(a.q_attn) + (int64_t)t0 * kHq * kKv4Dim;
    p.out = static_cast<uint16_t*>(a.out) + (int64_t)t0 * kHq * kKv4Dim;
    p.lse = a.lse ? a.lse + (int64_t)t0 * kHq : nullptr;
    p.req = a.req ? a.req + t0 : nullptr;
    p.positions = a.positions ? a.positions + t0 : nullptr;
    p.indices = a.indices ? a.indices + (int64_t)t0 * a.k_top : nullptr;
    p.counts = a.counts ? a.counts + t0 : nullptr;
    if (launch_pdl(kv4_attn_kernel<kBf16>, dim3(grid), dim3(kThreads), (size_t)kSmem, stream, p) != cudaSuccess)
      return DS4X_ERR_CUDA;
    count_launch();
    if (grid > 1 && max_rows > kRows) {  // a token of one chunk is never split
      if (launch_pdl(kv4_combine_kernel<kBf16>, dim3(grid - 1, kHq), dim3(kKv4Dim / 4), 0, stream,
                     (const int4*)p.parts_of, (const float*)p.part, (const float*)p.stat, p.out, p.lse) != cudaSuccess)
        return DS4X_ERR_CUDA;
      count_launch();
    }
  }
  return DS4X_OK;
}

int launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int max_rows = a.indices ? a.k_top : a.max_pages << a.log_page;
  return a.bf16 ? launch_typed<true>(a, max_rows, stream) : launch_typed<false>(a, max_rows, stream);
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
