// kv16_attn.cu — multi-query attention of 64 heads over the rows of the paged 16-bit cache that a token sees.
//
//   x_r = scale q[t,h,:] . kv_r,  cap tanh(x_r / cap),  - slopes[h] |e - 1 - r|          (all in log2 units)
//   out[t,h,:] = (sum_r 2^(x_r - m) kv_r + 2^(o - m) other_out[t,h,:]) / (sum_r 2^(x_r - m) + 2^(s - m) + 2^(o - m))
//
// with s the head's sink and o the other attention's log-sum-exp.  What a token sees is a run of rows [lo, hi); its
// list runs backwards from hi - 1, so that with a bias that grows with the distance the largest logits come first
// and the running maximum seldom moves.
//
// One block an SM.  The tokens' lists are cut into chunks of 128 rows; all chunks of all tokens form one sequence,
// and each block takes an equal, contiguous part of it.  A token whose chunks lie in several blocks leaves its
// unnormalised sums there in fp32 and kv16_combine_kernel joins them, so one long cache, a ragged batch and a
// prefill chunk are all spread evenly.  A token's chunks in a block are an item (several, if they are many:
// kItemChunks).  Per chunk:
//   S^T [128 rows x 64 heads] = K . Q^T       tcgen05, M = 128 (rows on TMEM lanes), both K-major
//   O^T [512 x 64 heads]     += V^T . P       tcgen05, M = 128 (dims), both MN-major
// with K = V = the chunk in 128B-swizzled shared memory (8 slots of 64 dims, 128 KB).  With the rows on the lanes of
// S^T a product of 16 dims serves 128 rows at the price of 64 (the matrix unit takes about 64 clocks for any
// product of up to 64 columns), a row's mask and distance belong to a thread, and P goes back to shared memory in
// whole 16-byte pieces: 32 heads of a row.
//
// Warps: 0-7 copy rows (16-byte cp.async, 16 rows of a chunk each: one step of the O^T products), 8-15 softmax
// (rows by quadrant, 32 heads each), 16-19 write the output (O^T lanes by quadrant), 20 issues the S^T products,
// 21 the O^T products, 22 looks up the rows' slots a few chunks ahead and brings the rows to L2, 23 loads q.
// There is room for one chunk: it is copied and released in quarters of the dims, so that the next chunk comes in
// while the O^T products go through this one.  O^T rotates over seven 64-column TMEM slots (a token uses four).
// A chunk that is not full costs its O^T products and copies by 16 rows.
//
// The running maximum of a head moves only when a logit exceeds it by more than 2^11 (O^T and the sums are
// rescaled then, which stalls the products); weights are 2^4 times 2^(x - m), which keeps them below fp16's
// largest value and small ones away from its least.  Statistics and sums are fp32.  Weights are rounded to the rows'
// type, which the matrix unit asks for (8 bits in bf16); out is normalised by the sum of the rounded weights, so that
// what a weight's rounding does to a row it does to the normaliser too; lse takes the exact ones.
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
constexpr int kRows = 128;                       // rows per chunk
constexpr int kSlots = kDim / 64;                // 8 slots of 64 dims
constexpr int kPairs = kSlots / 2;               // quarters of 128 dims: what is copied and released together
constexpr int kSlotBytes = kRows * 128;          // 16 KB
constexpr int kKvBytes = kSlots * kSlotBytes;    // 128 KB
constexpr int kQBlockBytes = kHq * 128;          // 8 KB (64 heads x 64 dims)
constexpr int kQBytes = kSlots * kQBlockBytes;   // 64 KB
constexpr int kPBytes = kRows * 128;             // 16 KB: P[row][head]
constexpr int kTokens = 2048;                    // tokens a launch plans for
constexpr int kSoftWarp = 8, kOutWarp = 16, kSWarp = 20, kOWarp = 21, kSlotWarp = 22, kQWarp = 23;
constexpr int kCopyWarps = 8, kSoftWarps = 8, kOutWarps = 4;
constexpr int kWarps = 24, kThreads = 32 * kWarps;
// registers a thread: 80 at launch; the sum over the six warpgroups stays what it was
constexpr int kLaunchRegs = 80, kCopyRegs = 56, kMiscRegs = 40, kSoftRegs = 120, kOutRegs = 88;
static_assert(kThreads * kLaunchRegs <= 65536 && 2 * kCopyRegs + 2 * kSoftRegs + kOutRegs + kMiscRegs <= 6 * kLaunchRegs, "registers");
constexpr int kRing = 4;                         // chunks whose slots are looked up ahead
// Chunks of a token that are added up in one go: the matrix unit truncates its fp32 sums, over 16384 rows without
// a trace, over 262144 of one sign by 0.14 %.  Longer lists are joined with rounded sums.
constexpr int kItemChunks = 128;
constexpr int kOSlots = 7;                       // O^T slots of 64 TMEM columns
constexpr int kOffKV = kQBytes;
constexpr int kOffP = kOffKV + kKvBytes;
constexpr int kOffRows = kOffP + kPBytes;        // int[kTokens]: rows of each token's list
constexpr int kOffSlots = kOffRows + kTokens * 4;      // int[kRing][kRows]: slot of each row of the chunk, -1 for none
constexpr int kOffAhead = kOffSlots + kRing * kRows * 4;  // int[kRing]: e - hi of the chunk's token
constexpr int kOffStat = kOffAhead + kRing * 4;        // float[2 items][4 quadrants][sum of rounded weights, sum][64]
constexpr int kOffM = kOffStat + 2 * 4 * 2 * kHq * 4;  // float[2 items][64]: offsets
constexpr int kOffMax = kOffM + 2 * kHq * 4;     // float[4 quadrants][64]: maxima of one chunk
constexpr int kOffAlpha = kOffMax + 4 * kHq * 4; // float[64]: rescale factors of one chunk
constexpr int kOffSlope = kOffAlpha + kHq * 4;   // float[64]: slopes in log2 units
constexpr int kOffJoin = kOffSlope + kHq * 4;    // float[5][64]: a token's offset, sum of rounded weights and sum so far; factors
                                                 // of the sums so far (or of the other attention) and of the item's
constexpr int kOffScan = kOffJoin + 5 * kHq * 4; // int64[kWarps] warp sums, then int[4]: the block's part
constexpr int kOffBars = kOffScan + kWarps * 8 + 16;
constexpr int kNumBars = 2 + 2 * kRing + 2 * kPairs + 4 + 2 * kOSlots + 4;
constexpr int kOffTmemSlot = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmemSlot + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kColO = 64;  // S^T in columns [0, 64), O^T from 64
constexpr float kRescaleLog2 = 11.0f, kWeightLog2 = 4.0f;
// A head's offset is its maximum less kWeightLog2, kNone before its first row: finite, so that differences with it are
// numbers or infinities, and 2^(x - kNone) is 0 for the -infinity of a masked row.
constexpr float kNone = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr int kSoftBar = 1, kOutBar = 2;
constexpr int kPartFloats = kHq * kDim;          // unnormalised sums of a part, then its statistics
constexpr int kStatFloats = 3 * kHq;             // sum of rounded weights, sum, offset

struct Params {
  const uint16_t *q, *pool;
  const int32_t *tables, *rows, *req, *positions, *first, *prefix;
  const float *slopes, *sinks, *other_lse;
  const uint16_t* other;
  uint16_t* out;
  float* lse;
  int* status;
  int4* parts_of;  // [grid]: the token a block starts in, chunks of it before the block, chunks it has, quota;
                   // NULL without a workspace, when there can be no rows at all
  float* part;     // [2 grid][kPartFloats]
  float* stat;     // [2 grid][kStatFloats]
  int n_slots, n_req, max_pages, log_page, ratio, window, t0, T;
  float scale, cap;
};

// Bounded waits.  A try suspends the thread for up to a microsecond, so the limit lies between a tenth of
// a second and a few seconds.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* status, int site) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  report_timeout(status, site);
  return false;
}
// The same outcome in every lane of the (converged) warp.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, int* status, int site) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, status, site));
}

// D (+)= A B by an elected lane of a converged warp; descriptors by their low words (the addresses): the high
// words are the same for all operands here.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_elect(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(add)
      : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Rows [lo, hi) of its request that token t sees, and the row e that it stands before.
struct Span {
  int b, lo, hi, e;
};
__device__ __forceinline__ Span span_of(const Params& p, int t) {
  Span s{p.req ? __ldg(p.req + t) : p.t0 + t, 0, 0, 0};
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
__device__ __forceinline__ int chunks_of(int rows) { return rows > kRows ? (rows - 1) / kRows + 1 : 1; }

// A block's part of the chunk sequence, walked item by item: chunks [c0, c1) of token t, of which the block
// has the chunks up to `end`.  What is read from shared memory goes through a warp reduction, whose result is a
// uniform register: the loops over it are then known to be the same in every lane, and the issuing warps'
// operands stay in such registers.
struct Walk {
  int t, c0, c1, end, left;
  const int* rows;
  __device__ __forceinline__ static int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
  __device__ __forceinline__ Walk(const int* rows_s, const int* start)
      : t(uniform(start[0])), c0(uniform(start[1])), left(uniform(start[2])), rows(rows_s) {
    cut();
  }
  __device__ __forceinline__ void cut() {
    end = left > 0 ? min(chunks_of(uniform(rows[t])), c0 + left) : c0;
    c1 = min(end, c0 + kItemChunks);
  }
  __device__ __forceinline__ void next() {
    const int over = c1 == end;
    left -= c1 - c0;
    t += over;
    c0 = over ? 0 : c1;
    cut();
  }
  // steps of 16 rows in chunk c: one at least, whose rows are all masked where the list is empty
  __device__ __forceinline__ int steps(int c) const {
    const int n = min(uniform(rows[t]) - c * kRows, kRows);
    return n > 16 ? (n + 15) >> 4 : 1;
  }
};

template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
  if constexpr (kBf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// Column sums over the warp by transposing: v[c] of every lane -> lane c holds the sum over all lanes of column c.
__device__ __forceinline__ float columns_sum(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 16; step >= 1; step >>= 1) {
    const bool upper = (lane & step) != 0;
#pragma unroll
    for (int i = 0; i < step; ++i) {
      const float send = upper ? v[i] : v[i + step];
      const float keep = upper ? v[i + step] : v[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, step);
      v[i] = keep + recv;
    }
  }
  return v[0];
}
// The largest x of the warp (NaN do not count), in every lane.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
// What joins a head's own rows (offset m in log2 units, sums r of the rounded and l of the exact weights 2^(x - m)) to
// its sink and to the other attention: factors of the unnormalised sums and of other's output, and lse.
struct Joined {
  float own, other, lse;
};
__device__ __forceinline__ Joined join_head(float m, float r, float l, float sink2, float other2) {
  const float M = fmaxf(m, fmaxf(sink2, other2));
  const float a = exp2f(m - M), s = exp2f(sink2 - M), o = exp2f(other2 - M);
  const float d = fmaf(a, r, s + o), e = fmaf(a, l, s + o);
  const float inv = d == 0.f ? 0.f : 1.f / d;
  return Joined{a * inv, o * inv, e == 0.f ? -INFINITY : (M + log2f(e)) * kLn2};
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    kv16_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const Params p) {
  constexpr uint32_t kIdescS = idesc_f16(128, kHq, kBf16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescO = idesc_f16(128, kHq, kBf16 ? 1 : 0, 1, 1);
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) report_timeout(p.status, 0x7b);
    return;
  }
  uint8_t* sq = smem;
  uint8_t* skv = smem + kOffKV;
  uint8_t* sp = smem + kOffP;
  int* rows_s = reinterpret_cast<int*>(smem + kOffRows);
  int* slot_s = reinterpret_cast<int*>(smem + kOffSlots);
  int* ahead_s = reinterpret_cast<int*>(smem + kOffAhead);
  float* stat_s = reinterpret_cast<float*>(smem + kOffStat);
  float* m_s = reinterpret_cast<float*>(smem + kOffM);
  float* max_s = reinterpret_cast<float*>(smem + kOffMax);
  float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);
  float* slope_s = reinterpret_cast<float*>(smem + kOffSlope);
  float* join_s = reinterpret_cast<float*>(smem + kOffJoin);
  long long* scan = reinterpret_cast<long long*>(smem + kOffScan);
  int* start = reinterpret_cast<int*>(smem + kOffScan + kWarps * 8);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* qempty = qfull + 1;
  uint64_t* slfull = qempty + 1;         // [ring] slots of a chunk
  uint64_t* slempty = slfull + kRing;    // by the copying and the softmax warps
  uint64_t* kvfull = slempty + kRing;    // [quarter], by every copying thread
  uint64_t* kvempty = kvfull + kPairs;   // [quarter]
  uint64_t* sfull = kvempty + kPairs;
  uint64_t* sempty = sfull + 1;
  uint64_t* pfull = sempty + 1;
  uint64_t* pempty = pfull + 1;
  uint64_t* ofull = pempty + 1;          // [O^T slot]
  uint64_t* oempty = ofull + kOSlots;    // [O^T slot]
  uint64_t* lready = oempty + kOSlots;   // [item parity] statistics written
  uint64_t* lfree = lready + 2;          // [item parity] ... and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmemSlot);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto oslot = [](uint32_t item, int db) { return (int)((4u * (item % 7u) + (uint32_t)db) % kOSlots); };

  if (tid < kNumBars) {  // one barrier a thread
    uint64_t* bar = qfull + tid;
    mbar_init(bar, bar >= slempty && bar < kvfull ? kCopyWarps + kSoftWarps
                   : bar >= kvfull && bar < kvempty ? 32 * kCopyWarps
                   : bar == sempty || bar == pfull || (bar >= lready && bar < lfree) ? kSoftWarps
                   : bar >= oempty ? kOutWarps : 1);
    fence_mbarrier_init();
  }
  if (warp == kSWarp) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == kQWarp && lane == 0) tma_prefetch_desc(&tm_q);
  pdl_wait();  // everything above touched only this block's own resources
  pdl_trigger();

  // --------------------------------------------------- every token's rows; this block's part
  {
    if (tid < kHq) slope_s[tid] = p.slopes ? p.slopes[tid] * kLog2e : 0.f;
    const int per = (p.T + kThreads - 1) / kThreads;
    const int first = tid * per, last = min(first + per, p.T);
    long long sum = 0;
#pragma unroll 1
    for (int t = first; t < last; ++t) {
      const Span s = span_of(p, t);
      const int n = s.hi - s.lo;
      rows_s[t] = n;
      sum += chunks_of(n);
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) start[0] = start[1] = start[2] = 0;
    __syncthreads();
    long long before = lane < kWarps ? scan[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    const long long total = __shfl_sync(0xffffffffu, before, 31);
    before = __shfl_sync(0xffffffffu, before, (warp + 31) & 31);
    before = (warp > 0 ? before : 0) + incl - sum;
    const long long quota = total >> 31 ? (total + gridDim.x - 1) / gridDim.x
                                        : (long long)(((uint32_t)total + gridDim.x - 1u) / gridDim.x);
    const long long g0 = quota * blockIdx.x, g1 = min(total, g0 + quota);
    if (g0 < total) {
      long long at = before;
#pragma unroll 1
      for (int t = first; t < last; ++t) {
        const int nch = chunks_of(rows_s[t]);
        if (at <= g0 && g0 < at + nch) {
          start[0] = t;
          start[1] = (int)(g0 - at);
          start[2] = (int)(g1 - g0);
          if (p.parts_of) p.parts_of[blockIdx.x] = make_int4(t, (int)(g0 - at), nch, (int)quota);
        }
        at += nch;
      }
    } else if (tid == 0 && p.parts_of) {
      p.parts_of[blockIdx.x] = make_int4(-1, 0, 0, (int)quota);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kCopyWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    // ------------------------------------------------------------------------------- copies
    // rows 16 warp .. + 15 of the chunk, two at a time: lane / 16 the row, lane % 16 the 16-byte piece of the
    // quarter's 256 bytes.  Rows 8 apart lie 1024 bytes apart with the same swizzle.
    const int hi = lane >> 4, piece = lane & 15;
    uint32_t dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * i + hi;
      dst[i] = smem_u32(skv) + (piece >> 3) * kSlotBytes + (16 * warp + r) * 128 + (((piece & 7) ^ r) << 4);
    }
    const char* pool = reinterpret_cast<const char*>(p.pool) + piece * 16;
    uint32_t g = 0;
    bool ok = true;
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next()) {
#pragma unroll 1
      for (int c = w.c0; c < w.c1 && ok; ++c, ++g) {
        const bool mine = warp < w.steps(c);
        ok = wait_bar_warp(&slfull[g % kRing], (g / kRing) & 1, p.status, 100);
        const int* sl = slot_s + (g % kRing) * kRows + 16 * warp + hi;
        int at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = sl[2 * i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&slempty[g % kRing]);
#pragma unroll 1
        for (int pr = 0; pr < kPairs && ok; ++pr) {
          ok = wait_bar_warp(&kvempty[pr], (g & 1) ^ 1, p.status, 101);
          if (mine && ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // a row without a slot is filled with zeros
              const char* src = at[i] < 0 ? reinterpret_cast<const char*>(p.q) : pool + ((int64_t)at[i] << 10) + pr * 256;
              cp_async16(dst[i & 3] + (i >> 2) * 1024 + pr * 2 * kSlotBytes, src, at[i] < 0 ? 0u : 16u);
            }
          }
          cp_async_arrive(&kvfull[pr]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kSWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMiscRegs));
    if (warp == kSWarp) {
      // -------------------------------------------------------------------- S^T = K Q^T
      uint32_t g = 0, item = 0;
      bool ok = true;
      const uint32_t q_lo = (uint32_t)desc_sw128(smem_u32(sq), 16, 1024), k_lo = (uint32_t)desc_sw128(smem_u32(skv), 16, 1024);
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++g) {
          if (!wait_bar_warp(sempty, (g & 1) ^ 1, p.status, 102)) { ok = false; break; }
          if (c == w.c0 && !wait_bar_warp(qfull, item & 1, p.status, 103)) { ok = false; break; }
#pragma unroll 1
          for (int pr = 0; pr < kPairs; ++pr) {
            if (!wait_bar_warp(&kvfull[pr], g & 1, p.status, 104)) { ok = false; break; }
            fence_proxy_async();  // copied rows -> visible to the tensor core
            tc_fence_after();
            const uint32_t a = k_lo + (pr * 2 * kSlotBytes >> 4), b = q_lo + (pr * 2 * kQBlockBytes >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_elect(tmem, a + ((i >> 2) * kSlotBytes + (i & 3) * 32 >> 4), b + ((i >> 2) * kQBlockBytes + (i & 3) * 32 >> 4),
                        kIdescS, (uint32_t)(pr | i));
          }
          if (!ok) break;
          if (c == w.c1 - 1) tc_commit_elect(qempty);  // the next item's q may replace this one's
          tc_commit_elect(sfull);
        }
      }
    } else if (warp == kOWarp) {
      // ------------------------------------------------------------------- O^T += V^T P
      uint32_t g = 0, item = 0;
      uint32_t o_ph = 0;  // bit s: phase of O^T slot s's empty barrier
      bool ok = true;
      const uint32_t v_lo = (uint32_t)desc_sw128(smem_u32(skv), kSlotBytes, 1024), p_lo = (uint32_t)desc_sw128(smem_u32(sp), 16, 1024);
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++g) {
          const int steps = w.steps(c);
          if (!wait_bar_warp(pfull, g & 1, p.status, 105)) { ok = false; break; }
          fence_proxy_async();
          tc_fence_after();
#pragma unroll 1
          for (int db = 0; db < kPairs; ++db) {
            const int os = oslot(item, db);
            // an item's first product overwrites its slot: the output that last read it is done
            if (c == w.c0) {
              if (!wait_bar_warp(&oempty[os], ((o_ph >> os) & 1u) ^ 1u, p.status, 106)) { ok = false; break; }
              o_ph ^= 1u << os;
              tc_fence_after();
            }
            const uint32_t a = v_lo + (db * 2 * kSlotBytes >> 4);
            const uint32_t d = tmem + kColO + os * kHq;
            if (steps == kRows / 16) {
#pragma unroll
              for (int ks = 0; ks < kRows / 16; ++ks)
                mma_elect(d, a + (ks * 2048 >> 4), p_lo + (ks * 2048 >> 4), kIdescO, (uint32_t)((c > w.c0) | ks));
            } else {
#pragma unroll 1
              for (int ks = 0; __all_sync(0xffffffffu, ks < steps); ++ks)
                mma_elect(d, a + (ks * 2048 >> 4), p_lo + (ks * 2048 >> 4), kIdescO, (uint32_t)((c > w.c0) | ks));
            }
            tc_commit_elect(&kvempty[db]);  // this quarter of the chunk is free
            if (c == w.c1 - 1) tc_commit_elect(&ofull[os]);
          }
          if (!ok) break;
          tc_commit_elect(pempty);
        }
      }
    } else if (warp == kSlotWarp) {
      // --------------------------------------------------------- slots of the rows, a few chunks ahead
      uint32_t g = 0;
      bool ok = true;
      for (Walk w(rows_s, start); w.left > 0 && ok; w.next()) {
        const Span s = span_of(p, w.t);
        const int n = s.hi - s.lo;
        const int32_t* table = p.tables + (int64_t)(n > 0 ? s.b : 0) * p.max_pages;
        for (int c = w.c0; c < w.c1; ++c, ++g) {
          int slot[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = c * kRows + lane + 32 * i;
            slot[i] = -1;
            if (j < n) {
              const int row = s.hi - 1 - j;
              const int page = __ldg(table + (row >> p.log_page));
              const int64_t at = ((int64_t)page << p.log_page) + (row & ((1 << p.log_page) - 1));
              if (page >= 0 && at < p.n_slots) slot[i] = (int)at;
            }
          }
          ok = wait_bar_warp(&slempty[g % kRing], ((g / kRing) & 1) ^ 1, p.status, 107);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            slot_s[(g % kRing) * kRows + lane + 32 * i] = slot[i];
            if (slot[i] >= 0) prefetch_l2(p.pool + (int64_t)slot[i] * kDim, kDim * 2);
          }
          if (lane == 0) ahead_s[g % kRing] = s.e - s.hi;
          __syncwarp();
          if (lane == 0) mbar_arrive(&slfull[g % kRing]);
        }
      }
    } else {
      // ------------------------------------------------------------------------------ q
      uint32_t item = 0;
      bool ok = true;
      for (Walk w(rows_s, start); w.left > 0 && ok; w.next(), ++item) {
        ok = wait_bar_warp(qempty, (item & 1) ^ 1, p.status, 108);
        if (!ok) break;
        mbar_arrive_expect_tx_elect(qfull, kQBytes);
#pragma unroll 1
        for (int i = 0; i < kSlots; ++i) tma_load_2d_elect(sq + i * kQBlockBytes, &tm_q, qfull, i * 64, w.t * kHq);
        if (lane == 0) {  // what the item's output and the next item will ask for
          if (p.other && w.c0 == 0) prefetch_l2(p.other + (int64_t)w.t * kHq * kDim, kHq * kDim * 2);
          if (w.c1 == w.end && w.left > w.c1 - w.c0) prefetch_l2(p.q + (int64_t)(w.t + 1) * kHq * kDim, kHq * kDim * 2);
        }
        __syncwarp();
      }
    }
  } else if (warp < kOutWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------------------- softmax
    // thread: row 32 quad + lane of the chunk, heads 32 half .. + 31
    const int quad = warp & 3, half = (warp - kSoftWarp) >> 2;
    const int row = 32 * quad + lane, h0 = 32 * half;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    const float scale2 = p.scale * kLog2e;
    const float cap2 = p.cap * kLog2e, in_cap = p.cap > 0.f ? 2.f * kLog2e * (p.scale / p.cap) : 0.f;
    const bool capped = p.cap > 0.f, sloped = p.slopes != nullptr;
    uint8_t* line = sp + row * 128;
    uint32_t g = 0, item = 0;
    // a wait that gave up is acted on where the eight warps meet, so that they leave together
    bool ok = true, leave = false;
    for (Walk w(rows_s, start); w.left > 0 && !leave; w.next(), ++item) {
      float* m_row = m_s + (item & 1) * kHq;
      float l = 0.f, r = 0.f;  // of head h0 + lane over the quadrant's rows: sums of the weights, and of the rounded ones
      // the slot of this item's parity was last read by the output of item - 2
      ok = ok && wait_bar_warp(&lfree[item & 1], ((item >> 1) & 1) ^ 1, p.status, 109);
#pragma unroll 1
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        ok = ok && wait_bar_warp(&slfull[g % kRing], (g / kRing) & 1, p.status, 110);
        const bool live = slot_s[(g % kRing) * kRows + row] >= 0;
        const int ahead = ahead_s[g % kRing];
        __syncwarp();
        if (lane == 0) mbar_arrive(&slempty[g % kRing]);
        ok = ok && wait_bar_warp(sfull, g & 1, p.status, 111);
        tc_fence_after();
        float x[32];
        tmem_ld32(tmem + t_lane + h0, x);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty);
        if (capped) {  // tanh y = 1 - 2 / (e^2y + 1)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = fmaf(-2.f * cap2, __frcp_rn(ex2_approx(x[i] * in_cap) + 1.f), cap2);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] *= scale2;
        }
        if (sloped) {
          const float dist = fabsf((float)(ahead + c * kRows + row));  // e - 1 - r, r = hi - 1 - list index
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 s = *reinterpret_cast<const float4*>(slope_s + h0 + i);
            x[i] = fmaf(-s.x, dist, x[i]);
            x[i + 1] = fmaf(-s.y, dist, x[i + 1]);
            x[i + 2] = fmaf(-s.z, dist, x[i + 2]);
            x[i + 3] = fmaf(-s.w, dist, x[i + 3]);
          }
        }
        if (!live) {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = -INFINITY;
        }
        bool moved = c == w.c0 || !ok;
        if (c > w.c0) {
          float over = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(m_row + h0 + i);
            over = fmaxf(over, fmaxf(fmaxf(x[i] - m.x, x[i + 1] - m.y), fmaxf(x[i + 2] - m.z, x[i + 3] - m.w)));
          }
          moved = moved || over > kRescaleLog2 + kWeightLog2;
        }
        if (named_or(kSoftBar, 32 * kSoftWarps, moved)) {
          leave = named_or(kSoftBar, 32 * kSoftWarps, !ok);
          if (leave) break;
          float mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float mx = warp_max(x[i]);
            if (lane == i) mine = mx;
          }
          max_s[quad * kHq + h0 + lane] = mine;
          named_sync(kSoftBar, 32 * kSoftWarps);
          const int th = tid - 32 * kSoftWarp;
          if (th < kHq) {
            const float mx = fmaxf(fmaxf(max_s[th], max_s[kHq + th]), fmaxf(max_s[2 * kHq + th], max_s[3 * kHq + th]));
            const float m = c == w.c0 ? kNone : m_row[th];
            const bool up = mx - m > kRescaleLog2 + kWeightLog2;
            alpha_s[th] = up ? ex2_approx(m - (mx - kWeightLog2)) : 1.f;
            m_row[th] = up ? mx - kWeightLog2 : m;
          }
          named_sync(kSoftBar, 32 * kSoftWarps);
          if (c > w.c0) {
            l *= alpha_s[h0 + lane];
            r *= alpha_s[h0 + lane];
            // O^T must hold all of the previous chunk before its columns are rescaled
            ok = wait_bar_warp(pempty, (g - 1) & 1, p.status, 112);
            tc_fence_after();
#pragma unroll 1
            for (int db = 0; db < kPairs; ++db) {
              float v[32];
              const uint32_t ta = tmem + t_lane + kColO + oslot(item, db) * kHq + h0;
              tmem_ld32(ta, v);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= alpha_s[h0 + i];
              tmem_st32(ta, v);
            }
            tc_wait_st();
          }
        }
        // weights 2^(x - offset), rounded for the product
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(m_row + h0 + i);
          x[i] = ex2_approx(x[i] - m.x);
          x[i + 1] = ex2_approx(x[i + 1] - m.y);
          x[i + 2] = ex2_approx(x[i + 2] - m.z);
          x[i + 3] = ex2_approx(x[i + 3] - m.w);
          pk[i / 2] = pack16<kBf16>(x[i], x[i + 1]);
          pk[i / 2 + 1] = pack16<kBf16>(x[i + 2], x[i + 3]);
        }
        ok = ok && wait_bar_warp(pempty, (g & 1) ^ 1, p.status, 113);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(line + (((4 * half + k) ^ (row & 7)) << 4)) =
              make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
        // the sums over the rows, while the products run
        l += columns_sum(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 u = unpack16<kBf16>(pk[i]);
          x[2 * i] = u.x;
          x[2 * i + 1] = u.y;
        }
        r += columns_sum(x);
      }
      if (leave) break;
      float* st = stat_s + ((item & 1) * 4 + quad) * 2 * kHq + h0 + lane;
      st[0] = r;
      st[kHq] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&lready[item & 1]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    // --------------------------------------------------------------------------- output
    const int quad = warp & 3, to = tid - 32 * kOutWarp;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    const bool odd = lane & 1;
    float *so_far = join_s, *f_first = join_s + 3 * kHq, *f_item = join_s + 4 * kHq;
    uint32_t item = 0;
    uint32_t f_ph = 0;  // bit s: phase of O^T slot s's full barrier
    bool ok = true;
    int from = 0;       // the block's first chunk of the token
    for (Walk w(rows_s, start); w.left > 0; w.next(), ++item) {
      const int par = item & 1;
      ok = ok && wait_bar_warp(&lready[par], (item >> 1) & 1, p.status, 114);
      // chunks before the block, or behind it: the sums go to the block's first or second part
      if (w.c0 == 0 || item == 0) from = w.c0;
      const bool begins = w.c0 == from, ends = w.c1 == w.end;
      const bool whole = ends && from == 0 && w.c1 == chunks_of(rows_s[w.t]);
      const bool joins = !(begins && ends);  // one of several items: joined to those so far
      const int64_t part = 2 * (int64_t)blockIdx.x + (from == 0);
      // the factors of the item before are read by all
      if (!named_and(kOutBar, 32 * kOutWarps, ok)) break;
      if (to < kHq) {
        const float* st = stat_s + par * 8 * kHq + to;
        float r = (st[0] + st[2 * kHq]) + (st[4 * kHq] + st[6 * kHq]);
        float l = (st[kHq] + st[3 * kHq]) + (st[5 * kHq] + st[7 * kHq]);
        float m = m_s[par * kHq + to];
        float f0 = 0.f, fi = 1.f;
        if (joins) {
          const float m0 = begins ? kNone : so_far[to], mi = m;
          m = fmaxf(m0, mi);
          f0 = begins ? 0.f : ex2_approx(m0 - m);
          fi = ex2_approx(mi - m);
          r = r * fi + (begins ? 0.f : so_far[kHq + to] * f0);
          l = l * fi + (begins ? 0.f : so_far[2 * kHq + to] * f0);
          so_far[to] = m;
          so_far[kHq + to] = r;
          so_far[2 * kHq + to] = l;
        }
        if (whole) {
          const float sink2 = p.sinks ? p.sinks[to] * kLog2e : -INFINITY;
          const float other2 = p.other ? p.other_lse[(int64_t)w.t * kHq + to] * kLog2e : -INFINITY;
          const Joined j = join_head(m, r, l, sink2, other2);
          if (p.lse) p.lse[(int64_t)w.t * kHq + to] = j.lse;
          f0 = joins ? f0 * j.own : j.other;
          fi *= j.own;
          if (joins) so_far[to] = j.other;  // a token's last item: nothing is joined to it any more
        } else if (ends) {
          float* ps = p.stat + part * kStatFloats;
          ps[to] = r;
          ps[kHq + to] = l;
          ps[2 * kHq + to] = m;
        }
        f_first[to] = f0;
        f_item[to] = fi;
      }
      named_sync(kOutBar, 32 * kOutWarps);
      if (lane == 0) mbar_arrive(&lfree[par]);
#pragma unroll 1
      for (int step = 0; step < 2 * kPairs; ++step) {  // quarters of the dims by halves of the heads
        const int db = step >> 1, hb = (step & 1) * 32;
        const int os = oslot(item, db);
        const int d = db * 128 + quad * 32 + lane;
        // neighbouring lanes exchange, so that each reads and writes two dims of one head: of an even lane the
        // even head of a pair, of an odd one the odd head
        const int64_t at = (((int64_t)w.t * kHq + hb + (odd ? 1 : 0)) * kDim + d) >> 1;
        uint32_t o2[16];
        const float* f_other = joins ? so_far : f_first;
        if (whole && p.other) {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(p.other) + at;
#pragma unroll
          for (int i = 0; i < 16; ++i) o2[i] = f_other[hb + 2 * i + odd] == 0.f ? 0u : __ldg(src + i * kDim);
        }
        if (hb == 0) {
          ok = wait_bar_warp(&ofull[os], (f_ph >> os) & 1u, p.status, 115);
          if (!ok) break;
          f_ph ^= 1u << os;
          tc_fence_after();
        }
        float v[32];
        tmem_ld32(tmem + t_lane + kColO + os * kHq + hb, v);
        tc_wait_ld();
        if (hb) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&oempty[os]);
        }
        if (joins || !whole) {
          // Sums so far lie where the part's go: the second part's own token is the block's last, behind all that
          // lie whole in the block.  A thread reads back only what it wrote.
          float* sums = p.part + part * kPartFloats + hb * kDim + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] *= f_item[hb + i];
            if (!begins) v[i] = fmaf(f_first[hb + i], sums[i * kDim], v[i]);
          }
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sums[i * kDim] = v[i];
            continue;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= f_item[hb + i];
        }
        if (p.other) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t theirs = __shfl_xor_sync(0xffffffffu, o2[i], 1);
            // heads 2 i and 2 i + 1 at this lane's dim
            const float2 a = unpack16<kBf16>(__byte_perm(o2[i], theirs, odd ? 0x3276u : 0x5410u));
            v[2 * i] = fmaf(f_other[hb + 2 * i], a.x, v[2 * i]);
            v[2 * i + 1] = fmaf(f_other[hb + 2 * i + 1], a.y, v[2 * i + 1]);
          }
        }
        uint32_t* orow = reinterpret_cast<uint32_t*>(p.out) + at;
        const uint32_t sel = odd ? 0x3276u : 0x5410u;  // even: both first heads; odd: both second ones
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t mine = pack16<kBf16>(v[2 * i], v[2 * i + 1]);
          orow[i * kDim] = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), sel);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of a token that several blocks worked on: part k holds O_k = sum_j 2^(x_j - m_k) kv_j and
// the sums r_k of its rounded weights and l_k of the exact ones, so with M = max_k m_k the token's are
//   O = sum_k 2^(m_k - M) O_k, r and l alike,
// and the sink and the other attention join them as they do in the kernel above.  A thread holds 4 dims; kGroups
// groups of threads take the parts in turn and are added up at the end, in an order that depends on the parts'
// number alone: the same bits on every run.
//   Many tokens (two or three parts each): a block per boundary between two blocks and four heads, one group
//   of 128 threads a head.
//   Few tokens (under a quarter of the blocks; one may have a part of every block): a block per token and head,
//   four groups.  Under 8 tokens four blocks a head, each a quarter of the dims, eight groups.
constexpr int kMaxParts = 256;
template <bool kBf16, bool kByToken, int kGroups, int kHeads, int kDimBlocks>
__global__ void __launch_bounds__(kGroups * kHeads * kDim / 4 / kDimBlocks)
    kv16_combine_kernel(const int4* __restrict__ parts_of, int blocks, const float* __restrict__ part,
                        const float* __restrict__ stat, const float* __restrict__ sinks,
                        const uint16_t* __restrict__ other, const float* __restrict__ other_lse, uint16_t* out,
                        float* lse) {
  constexpr int kLane4 = kDim / 4 / kDimBlocks, kTeam = kGroups * kLane4;
  static_assert(kTeam >= 32 && (kHeads == 1 || kGroups == 1), "a team's first warp takes its statistics");
  __shared__ float weight[kHeads][kMaxParts], own_s[kHeads], other_s[kHeads];
  __shared__ float4 acc_s[kGroups > 1 ? kGroups - 1 : 1][kLane4];
  __shared__ int found;
  pdl_wait();
  pdl_trigger();
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, h = blockIdx.y * kHeads + team;
  // block i's entry: the token it starts in, its chunks before the block, its chunks, a block's chunks.  The
  // first block that a token reaches into tells all about it.
  int i = blockIdx.x + 1;
  auto joins_at = [](int4 at) { return at.x >= 0 && at.y > 0 && at.y <= at.w; };
  if constexpr (kByToken) {
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    for (int k = 1 + threadIdx.x; k < blocks; k += blockDim.x) {
      const int4 at = parts_of[k];
      if (at.x == (int)blockIdx.x && joins_at(at)) found = k;  // there is one at most
    }
    __syncthreads();
    i = found;
    if (i == 0) return;
  }
  const int4 at = parts_of[i];
  if (!joins_at(at)) return;
  const int n = 1 + (at.z - at.y + at.w - 1) / at.w;  // parts: block i - 1's second, then the first ones
  auto part_no = [&](int k) { return k == 0 ? 2 * (int64_t)(i - 1) + 1 : 2 * (int64_t)(i - 1 + k); };
  const int64_t row = (int64_t)at.x * kHq + h;
  if (tid < 32) {
    float mx = kNone, r = 0.f, l = 0.f;
    for (int k = tid; k < n; k += 32) mx = fmaxf(mx, stat[part_no(k) * kStatFloats + 2 * kHq + h]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    for (int k = tid; k < n; k += 32) {
      const float* st = stat + part_no(k) * kStatFloats + h;
      const float f = exp2f(st[2 * kHq] - mx);
      weight[team][k] = f;
      r += f * st[0];
      l += f * st[kHq];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      r += __shfl_xor_sync(0xffffffffu, r, d);
      l += __shfl_xor_sync(0xffffffffu, l, d);
    }
    if (tid == 0) {
      const Joined j = join_head(mx, r, l, sinks ? sinks[h] * kLog2e : -INFINITY,
                                 other ? other_lse[row] * kLog2e : -INFINITY);
      own_s[team] = j.own;
      other_s[team] = j.other;
      if (lse && blockIdx.z == 0) lse[row] = j.lse;
    }
  }
  __syncthreads();
  const int group = tid / kLane4, lane4 = tid % kLane4, x = blockIdx.z * kLane4 + lane4;
  const float4* src = reinterpret_cast<const float4*>(part + h * kDim) + x;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = group; k < n; k += kGroups) {
    const float4 o = src[part_no(k) * (kPartFloats / 4)];
    const float f = weight[team][k];
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
  }
  if constexpr (kGroups > 1) {
    if (group > 0) acc_s[group - 1][lane4] = acc;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 o = acc_s[k][lane4];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
  }
  const float own = own_s[team], fo = other_s[team];
  acc.x *= own;
  acc.y *= own;
  acc.z *= own;
  acc.w *= own;
  if (other && fo != 0.f) {
    const uint2 u = *reinterpret_cast<const uint2*>(other + row * kDim + 4 * x);
    const float2 a = unpack16<kBf16>(u.x), b = unpack16<kBf16>(u.y);
    acc.x = fmaf(fo, a.x, acc.x);
    acc.y = fmaf(fo, a.y, acc.y);
    acc.z = fmaf(fo, b.x, acc.z);
    acc.w = fmaf(fo, b.y, acc.w);
  }
  *reinterpret_cast<uint2*>(out + row * kDim + 4 * x) = make_uint2(pack16<kBf16>(acc.x, acc.y), pack16<kBf16>(acc.z, acc.w));
}

// Blocks for T tokens of up to max_rows rows: one an SM, at most one a chunk.
int grid_of(int T, int max_rows) {
  const int64_t chunks = (int64_t)T * (max_rows > kRows ? (max_rows - 1) / kRows + 1 : 1);
  const int sms = device_sm_count();
  const int64_t most = sms < kMaxParts ? sms : kMaxParts;  // a token has at most a part of every block
  return (int)(chunks < most ? chunks : most);
}
constexpr size_t kHeadBytes = 16 * kMaxParts;  // the int4 of every block

}  // namespace

// A token of one chunk is never split: the head alone then, which the launch writes all the same.
size_t kv16_attn_workspace_bytes(int T, int max_rows) {
  if (max_rows <= kRows) return kHeadBytes;
  const int grid = grid_of(T < kTokens ? T : kTokens, max_rows);
  return kHeadBytes + (size_t)2 * grid * (kPartFloats + kStatFloats) * sizeof(float);
}

template <bool kBf16>
static int launch_typed(const Kv16AttnArgs& a, cudaStream_t stream) {
  if (ensure_dynamic_smem(kv16_attn_kernel<kBf16>, kSmem) != cudaSuccess) return DS4X_ERR_CUDA;
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return DS4X_ERR_CUDA;
  Params p;
  p.pool = static_cast<const uint16_t*>(a.pool);
  p.tables = a.tables;
  p.rows = a.rows;
  p.prefix = a.prefix;
  p.slopes = a.slopes;
  p.sinks = a.sinks;
  p.status = device_status_ptr();
  p.n_slots = a.n_slots;
  p.n_req = a.n_req;
  p.max_pages = a.max_pages;
  p.log_page = a.log_page;
  p.ratio = a.ratio;
  p.window = a.window;
  p.scale = a.scale;
  p.cap = a.cap;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.parts_of = reinterpret_cast<int4*>(ws);
  for (int t0 = 0; t0 < a.T; t0 += kTokens) {  // launches on one stream: they may share the workspace
    p.t0 = t0;
    p.T = a.T - t0 < kTokens ? a.T - t0 : kTokens;
    const int grid = grid_of(p.T, a.max_rows);
    const int64_t row0 = (int64_t)t0 * kHq;
    p.part = reinterpret_cast<float*>(ws + kHeadBytes);
    p.stat = p.part + (size_t)2 * grid * kPartFloats;
    p.q = static_cast<const uint16_t*>(a.q_attn) + row0 * kDim;
    p.out = static_cast<uint16_t*>(a.out) + row0 * kDim;
    p.lse = a.lse ? a.lse + row0 : nullptr;
    p.other = a.other_out ? static_cast<const uint16_t*>(a.other_out) + row0 * kDim : nullptr;
    p.other_lse = a.other_lse ? a.other_lse + row0 : nullptr;
    p.req = a.req ? a.req + t0 : nullptr;
    p.positions = a.positions ? a.positions + t0 : nullptr;
    p.first = a.first ? a.first + t0 : nullptr;
    CUtensorMap tq;
    const cuuint64_t dims[2] = {(cuuint64_t)kDim, (cuuint64_t)p.T * kHq}, strides[1] = {(cuuint64_t)kDim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)kHq}, estr[2] = {1, 1};
    if (fn(&tq, kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
           const_cast<uint16_t*>(p.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return DS4X_ERR_CUDA;
    if (launch_pdl(kv16_attn_kernel<kBf16>, dim3(grid), dim3(kThreads), (size_t)kSmem, stream, tq, p) != cudaSuccess)
      return DS4X_ERR_CUDA;
    count_launch();
    if (grid > 1 && a.max_rows > kRows) {  // a token of one chunk is never split
      auto join = [&](auto kernel, dim3 blocks, int threads) {
        return launch_pdl(kernel, blocks, dim3(threads), 0, stream, (const int4*)p.parts_of, grid, (const float*)p.part,
                          (const float*)p.stat, p.sinks, p.other, p.other_lse, p.out, p.lse);
      };
      cudaError_t e;
      if (4 * p.T < grid && p.T < 8)  // few tokens: four blocks a head fill more of the GPU
        e = join(kv16_combine_kernel<kBf16, true, 8, 1, 4>, dim3(p.T, kHq, 4), 256);
      else if (4 * p.T < grid)
        e = join(kv16_combine_kernel<kBf16, true, 4, 1, 1>, dim3(p.T, kHq), 512);
      else
        e = join(kv16_combine_kernel<kBf16, false, 1, 4, 1>, dim3(grid - 1, kHq / 4), 512);
      if (e != cudaSuccess) return DS4X_ERR_CUDA;
      count_launch();
    }
  }
  return DS4X_OK;
}

int launch_kv16_attn(const Kv16AttnArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
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
