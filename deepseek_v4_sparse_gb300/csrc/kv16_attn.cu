// kv16_attn.cu — multi-query attention of 64 heads over the rows of the paged 16-bit cache that a token sees.
//
//   x_r = scale q[t,h,:] . kv_r,  cap tanh(x_r / cap),  - slopes[h] |e - 1 - r|          (all in log2 units)
//   out[t,h,:] = (sum_r 2^(x_r - m) kv_r + 2^(o - m) other_out[t,h,:]) / (sum_r 2^(x_r - m) + 2^(s - m) + 2^(o - m))
//
// with s the head's sink and o the other attention's log-sum-exp.  What a token sees is a run of rows [lo, hi); its
// list runs backwards from hi - 1, so that with a bias that grows with the distance the largest logits come first
// and the running maximum seldom moves.
//
// One block an SM.  The tokens' lists are cut into chunks of 64 rows; all chunks of all tokens form one sequence,
// and each block takes an equal, contiguous part of it.  A token whose chunks lie in several blocks leaves its
// unnormalised sums there in fp32 and another kernel joins them, so one long cache, a ragged batch and a
// prefill chunk are all spread evenly.  A token's chunks in a block are an item (several, if they are many:
// kItemChunks).  Per chunk:
//   S   [64 heads x 64 rows] = Q . K^T       tcgen05, M = 64 (heads on TMEM lanes), K-major
//   O^T [512 x 64 heads]    += V^T . P^T     tcgen05, M = 128 (dims), A MN-major, B K-major
// with K = V = the chunk in 128B-swizzled shared memory (8 slots of 64 dims, two buffers).
//
// Warps: 0-3 copy rows (16-byte cp.async; 16 rows each, one step of the O^T products), 4-11 softmax (16 heads by
// quadrant and half of the rows each, 4 threads a head), 12-27 write the output (O^T lanes by quadrant, a quarter
// of the dims each), 28 issues the S products, 29 the O^T products, 30 looks up the rows' slots a few chunks ahead, 31
// loads q and works out what the heads' output needs.
// Buffers are copied and released in quarters of the dims, O^T rotates over six 64-column TMEM
// slots (a token uses four), so neighbouring tokens overlap.  A chunk that is not full costs its O^T products and
// copies by 16 rows.  The other attention's output is where a token's sums begin: the output warps put it, times
// 2^(o - m), into the O^T slots that they have emptied.
//
// The running maximum of a head moves only when a logit exceeds it by more than 2^11 in fp16, 2^32 in bf16 (O^T and
// the sums are rescaled then, which stalls the products); weights are 2^4 times 2^(x - m), which keeps them below
// fp16's largest value and small ones away from its least.  Statistics and sums are fp32.  Weights are rounded to the
// rows' type, which the matrix unit asks for (8 bits in bf16); out is normalised by the sum of the rounded weights, so
// that what a weight's rounding does to a row it does to the normaliser too; lse takes the exact ones.
//
// What bounds it.  A chunk's products read q, K, V and (four times) P from shared memory at 128 bytes a clock: 1792
// clocks for 8.4 MFLOP, the accesses of the warps 430 more, of 2330 a chunk (512 tokens over 8192 rows, 530 us: 1005
// TFLOP/s, that path busy in 93 % of the cycles, the tensor pipe in 65 %).  M = 64 is why, twice: a product of 64 heads
// reads as many bytes for q as for K, and takes as long as one of 128 rows (64 x 256 x 16: 133 clocks, 128 x 256 x 16: 134),
// so S is 1024 clocks of the tensor pipe and O^T 512, 1536 where full rate is 1024.  Without the limit of shared memory the
// chunk would be at two thirds of the peak.  Two tokens at once (M = 128) would need 128 KB for q and all 512 TMEM columns
// for O^T in one block; a pair of blocks that share K and V was not built.
// Decode tokens are bound by HBM in the long run (152 over 4096 rows each 113 us, 5.8 TB/s; 6.4 TB/s from 2048 to
// 4096 rows), which takes 64 KB chunks in two buffers; about 16 us are not: the plan 2, slots and first rows 4 to 6, the
// last chunk's way through the roles 3, parts and their joining 6 to 10.
// Rows come by cp.async, not by TMA boxes of whole chunks: a quarter's copy is on the way product -> free -> copy ->
// product, and boxes take twice as long to land (750 us).  One buffer of 128 rows: 750 us too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "ds4x_internal.h"
#include "ds4x_ptx.cuh"

namespace ds4x {
namespace {

constexpr int kHq = 64;
constexpr int kDim = 512;
constexpr int kRows = 64;                        // rows per chunk
constexpr int kSlots = kDim / 64;                // 8 slots of 64 dims
constexpr int kPairs = kSlots / 2;               // quarters of 128 dims: what is copied and released together
constexpr int kSlotBytes = kRows * 128;          // 8 KB
constexpr int kBufBytes = kSlots * kSlotBytes;   // 64 KB a chunk
constexpr int kQBlockBytes = kHq * 128;          // 8 KB (64 heads x 64 dims)
constexpr int kQBytes = kSlots * kQBlockBytes;   // 64 KB
constexpr int kPBytes = kHq * 128;               // 8 KB: P[h][j]
constexpr int kTokens = 2048;                    // tokens a launch plans for
constexpr int kSoftWarp = 4, kOutWarp = 12, kSWarp = 28, kOWarp = 29, kSlotWarp = 30, kQWarp = 31;
constexpr int kCopyWarps = 4, kSoftWarps = 8, kOutWarps = 16;
constexpr int kWarps = 32, kThreads = 32 * kWarps;
// registers a thread: 64 at launch; the sum over the eight warpgroups stays within that
constexpr int kLaunchRegs = 64, kCopyRegs = 56, kMiscRegs = 40, kSoftRegs = 80;  // and 64 for the output
static_assert(kCopyRegs < kLaunchRegs && kMiscRegs < kLaunchRegs && kSoftRegs > kLaunchRegs, "dec, dec and inc below");
static_assert(kThreads * kLaunchRegs <= 65536, "registers");
static_assert(kCopyRegs + 2 * kSoftRegs + 4 * kLaunchRegs + kMiscRegs <= 8 * kLaunchRegs, "registers of the warpgroups");
constexpr int kRing = 4, kMaskRing = 8;          // chunks whose slots, and masks, are looked up ahead
// Chunks of a token that are added up in one go: the matrix unit truncates its fp32 sums, over 16384 rows without
// a trace, over 262144 of one sign by 0.14 %.  Longer lists are joined with rounded sums.
constexpr int kItemChunks = 256;
// What a token costs beside its chunks, in chunks (61 tokens of 5 to 32768 rows: none 68.7 us, 2 and 3 64.8, 4 65.9; 400
// of 20 to 4000: 2 86.7, 3 89, 4 92).
constexpr int kTokenUnits = 2;
// Chunks of a token that no boundary divides: parts cost two more trips through L2 and a launch (256 tokens of two
// chunks over 152 blocks: 17 us, and 22 with boundaries that divide them).
constexpr int kWholeChunks = 4;
constexpr int kOSlots = 6;                       // O^T slots of 64 TMEM columns
constexpr int kOffKV = kQBytes;
constexpr int kOffP = kOffKV + 2 * kBufBytes;
constexpr int kOffRows = kOffP + 2 * kPBytes;    // int[kTokens]: rows of each token's list
constexpr int kOffSlots = kOffRows + kTokens * 4;      // int[kRing][kRows]: slot of each row of the chunk, -1 for none
constexpr int kOffMask = kOffSlots + kRing * kRows * 4;  // uint32[kMaskRing][2]: rows of the chunk that count
constexpr int kOffAhead = kOffMask + kMaskRing * 8;    // int[kMaskRing]: e - hi of the chunk's token
// float[2 items][2 halves of the rows' sums of rounded weights, 2 halves' sums, offset][64]
constexpr int kOffStat = kOffAhead + kMaskRing * 4;
constexpr int kOffMax = kOffStat + 2 * 5 * kHq * 4;    // float[2 halves of the rows][64]: maxima of one chunk
// float[2 items][2][64]: factors of a token's sums so far, of an item's sums; [3 items][64]: of the other output that
// the sums begin with
constexpr int kOffJoin = kOffMax + 2 * kHq * 4;
// int64[kWarps] warp sums and [2] chunks before the block and to its end, then int[4]: the block's part, and the last
// chunk (+ 1) in which a maximum moved
constexpr int kOffScan = kOffJoin + 7 * kHq * 4;
constexpr int kOffBars = kOffScan + (kWarps + 2) * 8 + 16;
constexpr int kNumBars = 2 + 2 * kRing + 2 * 2 * kPairs + 5 * 2 + 3 * kOSlots + 4 * 2;
constexpr int kOffTmemSlot = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmemSlot + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kColO = 128;  // S in columns [0, 128), O^T from 128
constexpr float kWeightLog2 = 4.0f;
// A head's offset is its maximum less kWeightLog2, kNone before its first row: finite, so that differences with it are
// numbers or infinities, and 2^(x - kNone) is 0 for the -infinity of a masked row.
constexpr float kNone = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kMaxScale = 1.7014118346046923e38f;  // 2^127: log2 e times it is in fp32's range
constexpr int kSoftBar = 1;
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
                   // NULL without a workspace, where no token can be split
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

// D (+)= A B^T by an elected lane of a converged warp; descriptors by their low words (the addresses): the high
// words are the same for all operands here.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool kAdd>
__device__ __forceinline__ void mma_elect(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  if constexpr (kAdd)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(add)
        : "memory");
}
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kDst), "n"(kSrc)
               : "memory");
}
template <int kDst>
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes), "n"(kDst)
               : "memory");
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
  const int pos = p.positions ? __ldg(p.positions + t) : 0;
  const int first = p.first ? __ldg(p.first + t) : 0;
  if (s.b < 0 || s.b >= p.n_req || pos < 0) return s;
  const int held = min(max(__ldg(p.rows + s.b), 0), p.max_pages << p.log_page);
  s.e = p.positions ? (int)min(((uint32_t)pos + 1u) / (uint32_t)p.ratio, 0x7fffffffu) : held;
  s.hi = min(held, p.prefix ? max(s.e, __ldg(p.prefix + s.b)) : s.e);
  s.lo = max(p.window > 0 ? max(s.e - p.window, 0) : 0, first);
  s.hi = max(s.hi, s.lo);
  return s;
}
__device__ __forceinline__ int chunks_of(int rows) { return rows > kRows ? (rows - 1) / kRows + 1 : 1; }

// A block's part of the chunk sequence, walked item by item: chunks [c0, c1) of token t, of which the block
// has the chunks up to `end`.  What is read from shared memory goes through a warp reduction, whose result is a
// uniform register: the loops over it are then known to be the same in every lane, and the issuing warps'
// operands stay in such registers.
struct Walk {
  int t, c0, c1, end, left, n;
  const int* rows;
  __device__ __forceinline__ static int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
  __device__ __forceinline__ Walk(const int* rows_s, const int* start)
      : t(uniform(start[0])), c0(uniform(start[1])), left(uniform(start[2])), rows(rows_s) {
    cut();
  }
  __device__ __forceinline__ void cut() {
    n = left > 0 ? uniform(rows[t]) : 0;
    end = left > 0 ? min(chunks_of(n), c0 + left) : c0;
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
    const int m = min(n - c * kRows, kRows);
    return m > 16 ? (m + 15) >> 4 : 1;
  }
};

// An item among its token's: the block's first of the token (`from` its first chunk), the block's last, all of it.
struct ItemPart {
  bool begins, ends, whole, joins;  // joins: one of several, whose sums are added to those so far
  int64_t part;  // chunks before the block, or behind it: the sums go to the block's first or second part
  __device__ __forceinline__ ItemPart(const Walk& w, uint32_t item, int& from) {
    if (w.c0 == 0 || item == 0) from = w.c0;
    begins = w.c0 == from;
    ends = w.c1 == w.end;
    whole = ends && from == 0 && w.c1 == chunks_of(w.n);
    joins = !(begins && ends);
    part = 2 * (int64_t)blockIdx.x + (from == 0);
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
__device__ __forceinline__ float from16(uint16_t u) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)u << 16);
  else return __half2float(*reinterpret_cast<const __half*>(&u));
}
// a plus both halves of the pair u, in fp32.
template <bool kBf16>
__device__ __forceinline__ void add_pair(float& a, uint32_t u) {
  if constexpr (kBf16)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.f32.bf16 %0, lo, %0;\n\tadd.f32.bf16 %0, hi, %0;\n\t}"
        : "+f"(a)
        : "r"(u));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.f32.f16 %0, lo, %0;\n\tadd.f32.f16 %0, hi, %0;\n\t}"
        : "+f"(a)
        : "r"(u));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap tanh y from v = 2 y log2 e: tanh y = 1 - 2 / (e^2y + 1), off by some 2^-21 of the cap, which is less than 2^-13
// up to kNearCap.  Above, where |y| < 1/4, the logit x times the series of tanh y / y: 1 - y^2 / 3 +
// 2 y^4 / 15 - 17 y^6 / 315, off by 62 / 2835 y^8 < 2^-21 of x itself.
constexpr float kNearCap = 256.f;
__device__ __forceinline__ float cap_near(float v, float cap) {
  return fmaf(-2.f * cap, rcp_approx(ex2_approx(v) + 1.f), cap);
}
__device__ __forceinline__ float cap_wide(float x, float v, float cap) {
  constexpr float kY = 0.5f / kLog2e;  // y = v kY
  const float z = (v * kY) * (v * kY);
  const float s = fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f);
  return fabsf(v) < 0.25f / kY ? fmaf(x * z, s, x) : cap_near(v, cap);
}
// A head's rows (offset m in log2 units, sums r of the rounded and l of the exact weights 2^(x - m)) and its sink:
// the factor of the unnormalised sums, and lse.  A sink may be as large or as low as fp32 goes, and log2 e times that
// is beyond it.  So where either is large, or no row was seen, both are halved (exactly) until they are subtracted; no rows
// are -infinity, below any sink.  The same of the other attention's lse (at *other, if there is one): where the offset is
// fp32's lowest or largest number it stands for that lse, beside which no row counts.  That way for all heads gives the
// same bits for ordinary ones, but costs time behind every token (2048 windows 98 us instead of 94, documents 114 and 108).
struct Joined {
  float own, lse;
};
__device__ __forceinline__ const float* other_at(const float* lse, int t, int h) {
  return lse ? lse + (int64_t)t * kHq + h : nullptr;
}
__device__ __forceinline__ Joined join_head(float m, float r, float l, float sink, const float* other) {
  if (fabsf(m) < 1e38f && (fabsf(sink) < 1e38f || sink == -INFINITY)) {  // log2 e times these is in range
    const float sink2 = sink * kLog2e, M = fmaxf(m, sink2);
    const float a = exp2f(m - M), s = exp2f(sink2 - M);
    const float d = fmaf(a, r, s), e = fmaf(a, l, s);
    return Joined{d == 0.f ? 0.f : a / d, e == 0.f ? -INFINITY : (M + log2f(e)) * kLn2};
  }
  float mh = l == 0.f ? -INFINITY : 0.5f * m;
  if (other && fabsf(m) == -kNone && l != 0.f && *other > -INFINITY) mh = *other * (0.5f * kLog2e);
  const float sh = sink * (0.5f * kLog2e);
  const float M = fmaxf(mh, sh);
  if (l == 0.f && sink == -INFINITY) return Joined{0.f, -INFINITY};
  const float a = exp2f(2.f * (mh - M)), s = exp2f(2.f * (sh - M));
  const float d = fmaf(a, r, s), e = fmaf(a, l, s);
  const float lse = (M + 0.5f * log2f(e)) * (2.f * kLn2);  // what rounds beyond fp32 is its last number
  return Joined{d == 0.f ? 0.f : a / d, isinf(lse) && e < INFINITY ? copysignf(-kNone, lse) : lse};
}
// Where a token's sums begin with another attention to join: its offset, and the weight of that attention's output: 1
// where the offset is fp32's lowest or largest number and lse finite, so that a type's lowest value counts where nothing
// else does, and one whose log2 is beyond fp32 alone.
__device__ __forceinline__ float log2_of(float x) { return fminf(fmaxf(x * kLog2e, kNone), -kNone); }
__device__ __forceinline__ float first_offset(float lse) { return fminf(fmaxf(lse * kLog2e - kWeightLog2, kNone), -kNone); }
__device__ __forceinline__ float first_weight(float lse) {
  if (!(fabsf(lse * kLog2e) <= -kNone)) return lse < kNone ? 0.f : lse == lse ? 1.f : lse;
  return ex2_approx(lse * kLog2e - first_offset(lse));
}

// What becomes of a product: scaled only; capped (up to kNearCap), with a slope, or both; or with a larger cap.  A kernel
// each, since one for all waits for instructions (512 tokens over 8192 rows 540 instead of 531 us, and
// with the series of large caps documents of 1021 tokens 129 instead of 110).  What each costs (us, without a cap / a cap
// of 30 / of 1000): 512 tokens over 8192 rows 527 / 558 / 681, documents 108 / 121 / 159, 61 decode tokens 64 / 66 / 71.
enum Logits { kPlain, kBiased, kWide };
template <bool kBf16, Logits kLogits>
__global__ void __launch_bounds__(kThreads, 1)
    kv16_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const Params p) {
  constexpr float kRescale = kBf16 ? 32.f : 11.f;  // log2 of what a logit may exceed its head's maximum by
  constexpr uint32_t kIdescS = idesc_f16(64, kHq, kBf16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescO = idesc_f16(128, kHq, kBf16 ? 1 : 0, 1, 0);
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
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + kOffMask);
  int* ahead_s = reinterpret_cast<int*>(smem + kOffAhead);
  float* stat_s = reinterpret_cast<float*>(smem + kOffStat);
  float* max_s = reinterpret_cast<float*>(smem + kOffMax);
  float* join_s = reinterpret_cast<float*>(smem + kOffJoin);
  long long* scan = reinterpret_cast<long long*>(smem + kOffScan);
  int* start = reinterpret_cast<int*>(smem + kOffScan + (kWarps + 2) * 8);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* qempty = qfull + 1;
  uint64_t* slfull = qempty + 1;            // [ring] slots of a chunk
  uint64_t* slempty = slfull + kRing;
  uint64_t* kvfull = slempty + kRing;       // [buffer][quarter], by every copying thread
  uint64_t* kvempty = kvfull + 2 * kPairs;  // [buffer][quarter]
  uint64_t* sfull = kvempty + 2 * kPairs;
  uint64_t* sempty = sfull + 2;
  uint64_t* pfull = sempty + 2;
  uint64_t* pempty = pfull + 2;
  uint64_t* looked = pempty + 2;            // every softmax warp has seen whether its maxima move
  uint64_t* ofull = looked + 2;             // [O^T slot]
  uint64_t* oempty = ofull + kOSlots;       // [O^T slot] read out
  uint64_t* oready = oempty + kOSlots;      // [O^T slot] with another attention to join: holds what the sums begin with
  uint64_t* lready = oready + kOSlots;      // [item parity] statistics written
  uint64_t* lfree = lready + 2;             // [item parity] ... and read
  uint64_t* fready = lfree + 2;             // [item parity] the output's factors written
  uint64_t* ffree = fready + 2;             // [item parity] ... and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmemSlot);

  // the warp's number through a warp reduction: a branch on it is then known not to divide a warp, and the issuing warps'
  // operands stay uniform (512 tokens over 8192 rows 640 us without it, 543 with)
  const int tid = threadIdx.x, warp = Walk::uniform(tid >> 5), lane = tid & 31;
  // use u = 4 item + quarter of an O^T slot: the slot is u % 6, and this is the slot's (u / 6)-th use
  auto oslot = [](uint32_t item, int db) { return (int)((4u * item + (uint32_t)db) % kOSlots); };
  auto ophase = [](uint32_t item, int db) { return ((4u * item + (uint32_t)db) / kOSlots) & 1u; };

  if (tid < kNumBars) {  // one barrier a thread
    uint64_t* bar = qfull + tid;
    mbar_init(bar, bar >= slempty && bar < kvfull ? kCopyWarps
                   : bar >= kvfull && bar < kvempty ? 32 * kCopyWarps
                   : bar >= sfull && bar < sempty ? 2  // the products' completion and the issuing warp itself
                   : (bar >= sempty && bar < pempty) || (bar >= looked && bar < ofull) || (bar >= lready && bar < lfree)
                       ? kSoftWarps
                   : bar >= ffree ? kOutWarps : bar >= oempty && bar < lready ? kOutWarps / kPairs : 1);
    fence_mbarrier_init();
  }
  if (warp == kSWarp) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == kQWarp && lane == 0) tma_prefetch_desc(&tm_q);
  pdl_wait();  // everything above touched only this block's own resources
  pdl_trigger();

  // --------------------------------------------------- every token's rows; this block's part
  {
    // A token costs its chunks and about two chunks' time to begin and end: each counts as that many units, the token's
    // own first, and the blocks take equal numbers of units.
    const int own = p.T > 1 ? kTokenUnits : 0;
    const int per = (p.T + kThreads - 1) / kThreads;
    const int first = tid * per, last = min(first + per, p.T);
    long long sum = 0;
#pragma unroll 1
    for (int t = first; t < last; ++t) {
      const Span s = span_of(p, t);
      const int n = s.hi - s.lo;
      rows_s[t] = n;
      sum += chunks_of(n) + own;
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) start[0] = start[1] = start[2] = start[3] = 0;
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
    // The block's first chunk, and how many chunks lie before its first and its last unit.  A boundary that falls into
    // a short token (a few chunks, or an eighth of a block's) moves to the token's nearer end: to join parts costs more.
    long long at = before, chunks = before - (long long)min(first, p.T) * own;
#pragma unroll 1
    for (int t = first; t < last; ++t) {
      const int nch = chunks_of(rows_s[t]), units = own + nch;
      auto chunk_at = [&](long long unit) {  // of this token's, at a unit of its
        if (nch <= kWholeChunks || (2 * (long long)nch <= quota && (nch <= 8 || 8 * (long long)nch <= quota)))
          return 2 * unit > units ? nch : 0;
        return (int)max(unit - own, 0ll);
      };
      if (at <= g0 && g0 < at + units) {
        const int c0 = chunk_at(g0 - at);
        const bool over = c0 == nch;
        scan[kWarps] = chunks + c0;
        start[0] = t + over;
        start[1] = over ? 0 : c0;
        if (p.parts_of) p.parts_of[blockIdx.x] = make_int4(t + over, over ? 0 : c0, nch, (int)quota);
      }
      if (g0 < total && at < g1 && g1 <= at + units) scan[kWarps + 1] = chunks + (g1 == at + units ? nch : chunk_at(g1 - at));
      at += units;
      chunks += nch;
    }
    if (g0 >= total && tid == 0) {
      scan[kWarps] = scan[kWarps + 1] = 0;
      if (p.parts_of) p.parts_of[blockIdx.x] = make_int4(-1, 0, 0, (int)quota);
    }
    __syncthreads();
    if (tid == 0) start[2] = (int)(scan[kWarps + 1] - scan[kWarps]);
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
#pragma unroll 1
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next()) {
#pragma unroll 1
      for (int c = w.c0; c < w.c1 && ok; ++c, ++g) {
        const uint32_t b = g & 1;
        const bool mine = warp < w.steps(c);
        ok = wait_bar_warp(&slfull[g % kRing], (g / kRing) & 1, p.status, 100);
        const int* sl = slot_s + (g % kRing) * kRows + 16 * warp + hi;
        const char* src[8];
        uint32_t there = 0;  // bit i: row i has a slot (else it is filled with zeros)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = sl[2 * i];
          src[i] = at < 0 ? reinterpret_cast<const char*>(p.q) : pool + ((int64_t)at << 10);
          there |= at < 0 ? 0u : 1u << i;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&slempty[g % kRing]);
        const uint32_t par = ((g >> 1) & 1) ^ 1;
        uint64_t *full = kvfull + b * kPairs, *empty = kvempty + b * kPairs;
        if (__all_sync(0xffffffffu, mine && there == 0xffu)) {
          uint32_t to[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i] = dst[i] + b * kBufBytes;
          auto quarter = [&](auto n) {
            constexpr int kN = decltype(n)::value, kTo = kN * 2 * kSlotBytes;
            ok = ok && wait_bar_warp(&empty[kN], par, p.status, 101);
            if (ok) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                cp_async16<kTo, kN * 256>(to[i], src[i]);
                cp_async16<kTo + 1024, kN * 256>(to[i], src[i + 4]);
              }
            }
            cp_async_arrive(&full[kN]);
          };
          quarter(std::integral_constant<int, 0>());
          quarter(std::integral_constant<int, 1>());
          quarter(std::integral_constant<int, 2>());
          quarter(std::integral_constant<int, 3>());
        } else {
#pragma unroll 1
          for (int pr = 0; pr < kPairs; ++pr) {
            ok = ok && wait_bar_warp(&empty[pr], par, p.status, 119);
            if (mine && ok) {
              const uint32_t to = b * kBufBytes + pr * 2 * kSlotBytes;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                cp_async16_or_zero<0>(dst[i] + to, src[i] + pr * 256, (there >> i & 1u) << 4);
                cp_async16_or_zero<1024>(dst[i] + to, src[i + 4] + pr * 256, (there >> (i + 4) & 1u) << 4);
              }
            }
            cp_async_arrive(&full[pr]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kSWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMiscRegs));
    if (warp == kSWarp) {
      // ------------------------------------------------------------------------ S = Q K^T
      uint32_t g = 0, item = 0;
      bool ok = true;
      const uint32_t q_lo = (uint32_t)desc_sw128(smem_u32(sq), 16, 1024), k_lo = (uint32_t)desc_sw128(smem_u32(skv), 16, 1024);
#pragma unroll 1
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
#pragma unroll 1
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++g) {
          const int b = g & 1;
          if (!wait_bar_warp(&sempty[b], ((g >> 1) & 1) ^ 1, p.status, 102)) { ok = false; break; }
          if (c == w.c0 && !wait_bar_warp(qfull, item & 1, p.status, 103)) { ok = false; break; }
          const uint32_t k = k_lo + (b * kBufBytes >> 4), d = tmem + b * kHq;
#pragma unroll
          for (int pr = 0; pr < kPairs; ++pr) {
            ok = ok && wait_bar_warp(&kvfull[b * kPairs + pr], (g >> 1) & 1, p.status, 104);
            fence_proxy_async();  // copied rows -> visible to the tensor core
            tc_fence_after();
            // the arrival of this warp hands on what it waited for (the chunk's mask)
            if (pr == kPairs - 1 && lane == 0) mbar_arrive(&sfull[b]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t qa = q_lo + ((2 * pr + (i >> 2)) * kQBlockBytes + (i & 3) * 32 >> 4);
              const uint32_t ka = k + ((2 * pr + (i >> 2)) * kSlotBytes + (i & 3) * 32 >> 4);
              if (pr + i == 0) mma_elect<false>(d, qa, ka, kIdescS, 0);
              else mma_elect<true>(d, qa, ka, kIdescS, 1);
            }
          }
          if (!ok) break;
          tc_commit_elect(&sfull[b]);
          if (c == w.c1 - 1) tc_commit_elect(qempty);  // the next item's q may replace this one's
        }
      }
    } else if (warp == kOWarp) {
      // --------------------------------------------------------------------- O^T += V^T P^T
      uint32_t g = 0, item = 0;
      bool ok = true;
      const uint32_t v_lo = (uint32_t)desc_sw128(smem_u32(skv), kSlotBytes, 1024), p_lo = (uint32_t)desc_sw128(smem_u32(sp), 16, 1024);
#pragma unroll 1
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
        const int begun = p.other != nullptr && w.c0 == 0;  // the slots hold what the sums begin with
        uint32_t d[kPairs];
#pragma unroll
        for (int db = 0; db < kPairs; ++db) d[db] = Walk::uniform(tmem + kColO + oslot(item, db) * kHq);
#pragma unroll 1
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++g) {
          const int b = g & 1, steps = w.steps(c);
          const uint32_t v = v_lo + (b * kBufBytes >> 4), k = p_lo + (b * kPBytes >> 4);
          const bool plain = __all_sync(0xffffffffu, c > w.c0 && c < w.c1 - 1 && steps == kRows / 16);
          if (!wait_bar_warp(&pfull[b], (g >> 1) & 1, p.status, 105)) { ok = false; break; }
          tc_fence_after();
          if (plain) {  // neither an item's first chunk nor its last, and full: straight through
#pragma unroll
            for (int db = 0; db < kPairs; ++db) {
#pragma unroll
              for (int ks = 0; ks < kRows / 16; ++ks)
                mma_elect<true>(d[db], v + (2 * db * kSlotBytes + ks * 2048 >> 4), k + 2 * ks, kIdescO, 1);
              tc_commit_elect(&kvempty[b * kPairs + db]);  // this quarter of the chunk is free
            }
            tc_commit_elect(&pempty[b]);
            continue;
          }
#pragma unroll 1
          for (int db = 0; db < kPairs; ++db) {
            const int os = oslot(item, db);
            if (c == w.c0) {
              uint64_t* bar = p.other ? &oready[os] : &oempty[os];
              if (!wait_bar_warp(bar, ophase(item, db) ^ (p.other ? 0u : 1u), p.status, 106)) { ok = false; break; }
              tc_fence_after();
            }
            const uint32_t a = v + (2 * db * kSlotBytes >> 4), to = tmem + kColO + os * kHq;
            mma_elect<false>(to, a, k, kIdescO, (uint32_t)((c > w.c0) | begun));
            if (__all_sync(0xffffffffu, steps == kRows / 16)) {
#pragma unroll
              for (int ks = 1; ks < kRows / 16; ++ks) mma_elect<true>(to, a + (ks * 2048 >> 4), k + 2 * ks, kIdescO, 1);
            } else {
#pragma unroll 1
              for (int ks = 1; __all_sync(0xffffffffu, ks < steps); ++ks)
                mma_elect<true>(to, a + (ks * 2048 >> 4), k + 2 * ks, kIdescO, 1);
            }
            tc_commit_elect(&kvempty[b * kPairs + db]);
            if (c == w.c1 - 1) tc_commit_elect(&ofull[os]);
          }
          if (!ok) break;
          tc_commit_elect(&pempty[b]);
        }
      }
    } else if (warp == kSlotWarp) {
      // --------------------------------------------------------- slots of the rows, a few chunks ahead
      uint32_t g = 0;
      bool ok = true;
#pragma unroll 1
      for (Walk w(rows_s, start); w.left > 0 && ok; w.next()) {
        const Span s = span_of(p, w.t);
        const int32_t* table = p.tables + (int64_t)(w.n > 0 ? s.b : 0) * p.max_pages;
#pragma unroll 1
        for (int c = w.c0; c < w.c1; ++c, ++g) {
          int slot[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = c * kRows + lane + 32 * i;
            slot[i] = -1;
            if (j < w.n) {
              const int row = s.hi - 1 - j;
              const int page = __ldg(table + (row >> p.log_page));
              const int64_t at = ((int64_t)page << p.log_page) + (row & ((1 << p.log_page) - 1));
              if (page >= 0 && at < p.n_slots) slot[i] = (int)at;
            }
          }
          const uint32_t m0 = __ballot_sync(0xffffffffu, slot[0] >= 0), m1 = __ballot_sync(0xffffffffu, slot[1] >= 0);
          ok = wait_bar_warp(&slempty[g % kRing], ((g / kRing) & 1) ^ 1, p.status, 107);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) slot_s[(g % kRing) * kRows + lane + 32 * i] = slot[i];
          // a mask is overwritten eight chunks later: its slots were read then four chunks ago, by warps that
          // are at most two chunks ahead of the softmax
          if (lane == 0) {
            *reinterpret_cast<uint2*>(mask_s + (g % kMaskRing) * 2) = make_uint2(m0, m1);
            ahead_s[g % kMaskRing] = s.e - s.hi;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&slfull[g % kRing]);
        }
      }
    } else {
      // -------------------------------------------------------------- q, and the arithmetic of the heads
      // q of an item goes in when the products of the one before are done with theirs.  Then, when that one's statistics
      // are there, what its output needs: two heads a lane.
      auto load_q = [&](int t) {
        mbar_arrive_expect_tx_elect(qfull, kQBytes);
#pragma unroll 1
        for (int i = 0; i < kSlots; ++i) tma_load_2d_elect(sq + i * kQBlockBytes, &tm_q, qfull, i * 64, t * kHq);
      };
      float m_far[2], r_far[2], l_far[2];  // a token's offsets and sums so far
      uint32_t item = 0;
      int from = 0;       // the block's first chunk of the token
      bool ok = true;
      Walk w(rows_s, start);
      if (w.left > 0) load_q(w.t);
#pragma unroll 1
      while (w.left > 0) {
        const int par = item & 1;
        const ItemPart it(w, item, from);
        const int t = w.t;
        if (lane == 0 && w.c1 == w.end && w.left > w.c1 - w.c0) {  // what the next token will ask for
          prefetch_l2(p.q + (int64_t)(w.t + 1) * kHq * kDim, kHq * kDim * 2);
          if (p.other) prefetch_l2(p.other + (int64_t)(w.t + 1) * kHq * kDim, kHq * kDim * 2);
        }
        __syncwarp();
        w.next();
        const bool begun = w.left > 0 && p.other && w.c0 == 0;  // the next item
        float sink[2], next[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sink[i] = it.whole && p.sinks ? __ldg(p.sinks + lane + 32 * i) : -INFINITY;
          next[i] = begun ? __ldg(p.other_lse + (int64_t)w.t * kHq + lane + 32 * i) : 0.f;
        }
        if (w.left > 0) {
          ok = wait_bar_warp(qempty, item & 1, p.status, 108);
          if (!ok) break;
          load_q(w.t);
        }
        next[0] = first_weight(next[0]);
        next[1] = first_weight(next[1]);
        // these factors' place was last read two items ago, that of the next item's other weights before
        ok = wait_bar_warp(&ffree[par], ((item >> 1) & 1) ^ 1, p.status, 118);
        ok = ok && wait_bar_warp(&lready[par], (item >> 1) & 1, p.status, 114);
        if (!ok) break;
        float rr[2], ll[2], mm[2], f0s[2], fis[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = lane + 32 * i;
          const float* st = stat_s + par * 5 * kHq + h;
          float &r = rr[i], &l = ll[i], &m = mm[i], &f0 = f0s[i], &fi = fis[i];
          r = st[0] + st[kHq], l = st[2 * kHq] + st[3 * kHq], m = st[4 * kHq];
          f0 = 0.f, fi = 1.f;
          if (it.joins) {
            const float m0 = it.begins ? kNone : m_far[i], mi = m;
            m = fmaxf(m0, mi);
            f0 = it.begins ? 0.f : ex2_approx(m0 - m);
            fi = ex2_approx(mi - m);
            r_far[i] = r = r * fi + (it.begins ? 0.f : r_far[i] * f0);
            l_far[i] = l = l * fi + (it.begins ? 0.f : l_far[i] * f0);
            m_far[i] = m;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = lane + 32 * i;
          const float r = rr[i], l = ll[i], m = mm[i];
          float f0 = f0s[i], fi = fis[i];
          if (it.whole) {
            const Joined j = join_head(m, r, l, sink[i], other_at(p.other_lse, t, h));
            if (p.lse) p.lse[(int64_t)t * kHq + h] = j.lse;
            f0 *= j.own;
            fi *= j.own;
          } else if (it.ends) {
            float* ps = p.stat + it.part * kStatFloats + h;
            ps[0] = r;
            ps[kHq] = l;
            ps[2 * kHq] = m;
          }
          float* f = join_s + par * 2 * kHq + h;
          f[0] = f0;
          f[kHq] = fi;
          if (begun) join_s[(4 + (item + 1) % 3) * kHq + h] = next[i];
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&lfree[par]);
          mbar_arrive(&fready[par]);
        }
        ++item;
      }
    }
  } else if (warp < kOutWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------------------- softmax
    // S holds head 16 quad + i on TMEM lane 32 quad + i (i < 16).  A warp takes half of the chunk's rows; the 16x256b
    // load gives thread (g8 = lane / 4, e = lane % 4) the heads hA = 16 quad + g8 and hB = hA + 8 and, of each, the
    // columns r0 + 8 k + 2 e + {0, 1}, k = 0..3: a head's 64 logits are spread over 4 threads of two warps.
    const int quad = warp & 3, half = (warp - kSoftWarp) >> 2, r0 = 32 * half;
    const int g8 = lane >> 2, e = lane & 3;
    const int hA = 16 * quad + g8, hB = hA + 8;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    const bool capped = kLogits != kPlain && p.cap > 0.f, sloped = kLogits != kPlain && p.slopes != nullptr;
    const float scale2 = p.scale * kLog2e;
    // the cap in log2 units, and what takes a product to log2 of e^2y, y = x / cap: finite for any cap
    const float cap2 = fminf(p.cap * kLog2e, -0.25f * kNone);
    const float in_cap = capped ? fminf(fmaxf(2.f * kLog2e * (p.scale / p.cap), kNone), -kNone) : 0.f;
    // slopes are finite in log2 units too, so that a distance of 0 leaves a logit as it is
    const float slopeA = sloped ? log2_of(p.slopes[hA]) : 0.f, slopeB = sloped ? log2_of(p.slopes[hB]) : 0.f;
    uint32_t g = 0, item = 0;
    // a wait that gave up is acted on where the eight warps meet, so that they leave together
    bool ok = true, leave = false;
#pragma unroll 1
    for (Walk w(rows_s, start); w.left > 0 && !leave; w.next(), ++item) {
      float oA = kNone, oB = kNone;                  // offsets, the same in both warps of a head
      float lA = 0.f, lB = 0.f, rA = 0.f, rB = 0.f;  // sums of this thread's weights, and of the rounded ones
      const bool begun = p.other != nullptr && w.c0 == 0;
      if (begun) {
        const float a = __ldg(p.other_lse + (int64_t)w.t * kHq + hA), b = __ldg(p.other_lse + (int64_t)w.t * kHq + hB);
        oA = first_offset(a);
        oB = first_offset(b);
        if (e == 0 && half == 0) {
          lA = rA = first_weight(a);
          lB = rB = first_weight(b);
        }
      }
#pragma unroll 1
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        const int b = g & 1;
        ok = ok && wait_bar_warp(&sfull[b], (g >> 1) & 1, p.status, 111);
        tc_fence_after();
        float x[16];
        tmem_ld_16x256b_x4(tmem + t_lane + b * kHq + r0, x);
        const uint32_t live = mask_s[(g % kMaskRing) * 2 + half] >> (2 * e);
        const int ahead = ahead_s[g % kMaskRing];
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[b]);
        // logits in log2 units
        if (capped) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (kLogits == kWide) x[i] = cap_wide(x[i] * scale2, x[i] * in_cap, cap2);
            else x[i] = cap_near(x[i] * in_cap, cap2);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= scale2;
        }
        if (sloped) {  // e - 1 - r of row r = hi - 1 - list index
          const int d0 = ahead + c * kRows + r0 + 2 * e;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float near = fabsf((float)(d0 + 8 * k)), far = fabsf((float)(d0 + 8 * k + 1));
            x[4 * k] = fmaf(-slopeA, near, x[4 * k]);
            x[4 * k + 1] = fmaf(-slopeA, far, x[4 * k + 1]);
            x[4 * k + 2] = fmaf(-slopeB, near, x[4 * k + 2]);
            x[4 * k + 3] = fmaf(-slopeB, far, x[4 * k + 3]);
          }
        }
        if ((live & 0x03030303u) != 0x03030303u) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (!(live >> (8 * k) & 1u)) x[4 * k] = x[4 * k + 2] = -INFINITY;
            if (!(live >> (8 * k) & 2u)) x[4 * k + 1] = x[4 * k + 3] = -INFINITY;
          }
        }
        float mxA = fmaxf(x[0], x[1]), mxB = fmaxf(x[2], x[3]);
#pragma unroll
        for (int k = 1; k < 4; ++k) {
          mxA = fmaxf(mxA, fmaxf(x[4 * k], x[4 * k + 1]));
          mxB = fmaxf(mxB, fmaxf(x[4 * k + 2], x[4 * k + 3]));
        }
        // Whether any head's maximum moves is said now and asked for when the weights are ready (the same answer in
        // all eight warps: a later chunk's word is written after all have read this one's).  An item's first chunk
        // asks at once: without sums that have begun there is no offset yet.
        const bool moved = __any_sync(0xffffffffu, mxA - oA > kRescale + kWeightLog2 || mxB - oB > kRescale + kWeightLog2 || !ok);
        if (lane == 0) {
          if (moved) *const_cast<volatile int*>(start + 3) = (int)(g + 1);
          mbar_arrive(&looked[b]);
        }
        uint32_t pkA[4], pkB[4];
        float sA, sB;
        // weights 2^(x - offset), rounded for the product
        auto weigh = [&]() {
          sA = sB = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a0 = ex2_approx(x[4 * k] - oA), a1 = ex2_approx(x[4 * k + 1] - oA);
            const float b0 = ex2_approx(x[4 * k + 2] - oB), b1 = ex2_approx(x[4 * k + 3] - oB);
            sA += a0 + a1;
            sB += b0 + b1;
            pkA[k] = pack16<kBf16>(a0, a1);
            pkB[k] = pack16<kBf16>(b0, b1);
          }
        };
        const bool fresh = c == w.c0 && !begun;
        if (!fresh) weigh();
        ok = ok && wait_bar_warp(&looked[b], (g >> 1) & 1, p.status, 110);
        if (*const_cast<volatile int*>(start + 3) == (int)(g + 1)) {
          leave = named_or(kSoftBar, 32 * kSoftWarps, !ok);
          if (leave) break;
#pragma unroll
          for (int d = 1; d <= 2; d <<= 1) {
            mxA = fmaxf(mxA, __shfl_xor_sync(0xffffffffu, mxA, d));
            mxB = fmaxf(mxB, __shfl_xor_sync(0xffffffffu, mxB, d));
          }
          if (e == 0) {
            max_s[half * kHq + hA] = mxA;
            max_s[half * kHq + hB] = mxB;
          }
          named_sync(kSoftBar, 32 * kSoftWarps);
          // the factor of what head h has so far, from the offset it had, and its new offset
          auto raise = [&](int h, float& o) {
            const float mx = fmaxf(max_s[h], max_s[kHq + h]);
            const bool up = mx - o > kRescale + kWeightLog2;
            const float f = up ? ex2_approx(o - (mx - kWeightLog2)) : 1.f;
            if (up) o = mx - kWeightLog2;
            return f;
          };
          const float aA = raise(hA, oA), aB = raise(hB, oB);
          lA *= aA;
          rA *= aA;
          lB *= aB;
          rB *= aB;
          if (!fresh) {
            named_sync(kSoftBar, 32 * kSoftWarps);  // the maxima are read: their place takes the factors
            if (e == 0 && half == 0) {
              max_s[hA] = aA;
              max_s[hB] = aB;
            }
            named_sync(kSoftBar, 32 * kSoftWarps);
            // O^T must hold all of the previous chunk, or what the sums begin with, before its columns are rescaled
            if (c > w.c0) {
              const uint32_t prev = g - 1;
              ok = wait_bar_warp(&pempty[prev & 1], (prev >> 1) & 1, p.status, 112);
            } else {
              for (int db = 0; db < kPairs; ++db)
                ok = ok && wait_bar_warp(&oready[oslot(item, db)], ophase(item, db), p.status, 116);
            }
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 2 * kPairs; ++q) {  // the quarters of this half of the heads, 16 at a time
              float v[16];
              const int h0 = r0 + 16 * (q & 1);
              const uint32_t ta = tmem + t_lane + kColO + oslot(item, q >> 1) * kHq + h0;
              tmem_ld16(ta, v);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= max_s[h0 + i];
              tmem_st16(ta, v);
            }
            tc_wait_st();
          }
          named_sync(kSoftBar, 32 * kSoftWarps);
          weigh();
        } else if (fresh) {
          weigh();  // no row at all
        }
        lA += sA;
        lB += sB;
        {
          // P's buffer is free: S of this chunk needed rows that were copied over those of two chunks ago, when O^T had
          // taken all of them and their weights.  P[h][j], K-major with the 128-byte swizzle: 16-byte piece k of line h
          // at k ^ (h & 7), the same for hA and hB.
          uint8_t* line = sp + b * kPBytes + hA * 128 + 4 * e;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint8_t* to = line + (((4 * half + k) ^ g8) << 4);
            *reinterpret_cast<uint32_t*>(to) = pkA[k];
            *reinterpret_cast<uint32_t*>(to + 1024) = pkB[k];
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[b]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          add_pair<kBf16>(rA, pkA[k]);
          add_pair<kBf16>(rB, pkB[k]);
        }
      }
      if (leave) break;
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        lA += __shfl_xor_sync(0xffffffffu, lA, d);
        lB += __shfl_xor_sync(0xffffffffu, lB, d);
        rA += __shfl_xor_sync(0xffffffffu, rA, d);
        rB += __shfl_xor_sync(0xffffffffu, rB, d);
      }
      // the statistics of this item's parity were last read by the output of item - 2
      ok = ok && wait_bar_warp(&lfree[item & 1], ((item >> 1) & 1) ^ 1, p.status, 109);
      if (e == 0) {
        float* st = stat_s + (item & 1) * 5 * kHq + half * kHq;
        st[hA] = rA;
        st[2 * kHq + hA] = lA;
        st[hB] = rB;
        st[2 * kHq + hB] = lB;
        if (half == 0) {
          st[4 * kHq + hA] = oA;
          st[4 * kHq + hB] = oB;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&lready[item & 1]);
    }
  } else {
    // --------------------------------------------------------------------------- output
    // A warp takes a quarter db of the dims, of which its quadrant of O^T's lanes are 32, and all heads, 16 at a time.
    const int quad = warp & 3, db = (warp - kOutWarp) >> 2;
    const bool odd = lane & 1;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kColO;
    const int d = db * 128 + quad * 32 + lane;       // this thread's dim
    uint32_t item = 0;
    int from = 0;       // the block's first chunk of the token
    bool ok = true;
    uint32_t even[8], uneven[8];
    // The other attention's output of token t, heads 16 n .. + 15: an even lane the even heads at its dim and the next, an
    // odd one the odd heads at the dim before and its own; neighbours exchange.
    auto load_other = [&](int t, int n, uint32_t (&u)[8]) {
      const uint32_t* src =
          reinterpret_cast<const uint32_t*>(p.other + ((int64_t)t * kHq + 16 * n + (odd ? 1 : 0)) * kDim + (d & ~1));
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __ldg(src + i * kDim);
    };
    // The slot of item n's quarter, once it is empty, is ready for its products: with weights of the other attention token
    // t's sums begin there with its output, whose first 32 heads are on their way.
    auto begin = [&](uint32_t n, int t, const float* f_other) {
      const int os = oslot(n, db);
      const bool got = wait_bar_warp(&oempty[os], ophase(n, db) ^ 1u, p.status, 117);
      tc_fence_after();
      auto fill = [&](int h, uint32_t (&u)[8]) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t pair = __byte_perm(u[i], __shfl_xor_sync(0xffffffffu, u[i], 1), odd ? 0x3276u : 0x5410u);
          const float2 f = *reinterpret_cast<const float2*>(f_other + 16 * h + 2 * i);
          v[2 * i] = f.x == 0.f ? 0.f : f.x * from16<kBf16>((uint16_t)pair);
          v[2 * i + 1] = f.y == 0.f ? 0.f : f.y * from16<kBf16>((uint16_t)(pair >> 16));
        }
        if (h + 2 < kHq / 16) load_other(t, h + 2, u);
        tmem_st16(t_lane + os * kHq + 16 * h, v);
      };
      if (f_other) {
#pragma unroll 1
        for (int h = 0; h < kHq / 16; h += 2) {
          fill(h, even);
          fill(h + 1, uneven);
        }
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&oready[os]);
      return got;
    };
    Walk w(rows_s, start);
    if (w.left > 0 && p.other) {
      const float* f_other = nullptr;
      if (w.c0 == 0) {
        load_other(w.t, 0, even);
        load_other(w.t, 1, uneven);
        float* f = join_s + 4 * kHq;  // every warp writes the same values
        const float* lse = p.other_lse + (int64_t)w.t * kHq + lane;
        f[lane] = first_weight(__ldg(lse));
        f[lane + 32] = first_weight(__ldg(lse + 32));
        __syncwarp();
        f_other = f;
      }
      ok = begin(0, w.t, f_other);
    }
#pragma unroll 1
    while (w.left > 0) {
      const int par = item & 1;
      const ItemPart it(w, item, from);
      const int t = w.t;
      w.next();
      const bool begun = w.left > 0 && p.other && w.c0 == 0;  // the next item
      if (begun) {
        load_other(w.t, 0, even);
        load_other(w.t, 1, uneven);
      }
      ok = ok && wait_bar_warp(&fready[par], (item >> 1) & 1, p.status, 113);
      if (!ok) break;
      const float *f_first = join_s + par * 2 * kHq, *f_item = f_first + kHq;
      const float* f_other = begun ? join_s + (4 + (item + 1) % 3) * kHq : nullptr;
      const int os = oslot(item, db);
      ok = wait_bar_warp(&ofull[os], ophase(item, db), p.status, 115);
      if (!ok) break;
      tc_fence_after();
      float v[16];
      tmem_ld16(t_lane + os * kHq, v);
#pragma unroll 1
      for (int h = 0; h < kHq; h += 16) {
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(f_item + h + i);
          v[i] *= f.x;
          v[i + 1] *= f.y;
          v[i + 2] *= f.z;
          v[i + 3] *= f.w;
        }
        if (!it.whole || it.joins) {
          // Sums so far lie where the part's go: the second part's own token is the block's last, behind all that
          // lie whole in the block.  A thread reads back only what it wrote.
          float* sums = p.part + it.part * kPartFloats + h * kDim + d;
          if (!it.begins) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(f_first[h + i], sums[i * kDim], v[i]);
          }
          if (!it.whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[i * kDim] = v[i];
          }
        }
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = pack16<kBf16>(v[2 * i], v[2 * i + 1]);
        if (h + 16 < kHq) {  // on their way while these are stored
          tmem_ld16(t_lane + os * kHq + h + 16, v);
        } else {  // the slot and the factors are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&oempty[os]);
            mbar_arrive(&ffree[par]);
          }
        }
        if (it.whole) {
          uint16_t* to_out = p.out + ((int64_t)t * kHq + h) * kDim + d;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            to_out[2 * i * kDim] = (uint16_t)u[i];
            to_out[(2 * i + 1) * kDim] = (uint16_t)(u[i] >> 16);
          }
        }
      }
      ++item;
      if (p.other && w.left > 0) ok = begin(item, w.t, f_other);
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
// and the sink joins them as it does in the kernel above.  Sums run in an order that depends on the parts' number
// alone: the same bits on every run.  A thread holds 4 dims; its first parts are on their way while the weights are worked
// out.
constexpr int kMaxParts = 256;
static_assert(2 * kMaxParts * kPartFloats < 1 << 30, "32-bit indexes");
struct Parts {
  int token, first, n;  // n parts: block first - 1's second, then the first ones of those from `first` on
  __device__ __forceinline__ int no(int k) const { return 2 * (first - 1 + k) + (k == 0); }
};
// Block i's entry: the token it starts in, its chunks before the block, its chunks, a block's chunks.  The first block
// that a token reaches into tells all about it.
__device__ __forceinline__ bool reached(int4 at) { return at.x >= 0 && at.y > 0 && at.y <= at.w; }
__device__ __forceinline__ Parts parts_at(int4 at, int i) { return Parts{at.x, i, 1 + (at.z - at.y + at.w - 1) / at.w}; }

struct Sum4 {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float f, const float4& o) {
    v.x += f * o.x;
    v.y += f * o.y;
    v.z += f * o.z;
    v.w += f * o.w;
  }
  template <bool kBf16>
  __device__ __forceinline__ void store(float own, uint16_t* to) const {
    *reinterpret_cast<uint2*>(to) = make_uint2(pack16<kBf16>(v.x * own, v.y * own), pack16<kBf16>(v.z * own, v.w * own));
  }
};

// Three ways of joining, by the number of tokens (us of the whole call, bf16):
//   1 token over 9728 / 120001 rows: few 15.6 / 38.6, some 32 / 42
//   4 tokens of 3000, 12 of 700, 37 of 3000: some 16.4, 15.8, 39.8, few 19.6, 20.7, 60 (blocks a token and head)
//   404 capped tokens, 400 of 20 to 4000 rows: many 79.8, 85.7, some 82.8, 87.3
// Under 4 tokens (one may have a part of every block): a block per token, head and quarter of the dims, eight groups of
// 32 threads that take the parts in turn.
constexpr int kFewTokens = 4, kFewGroups = 8, kFewBlocks = 4, kFewThreads = kFewGroups * kDim / 4 / kFewBlocks;
template <bool kBf16>
__global__ void __launch_bounds__(kFewThreads, 2)
    kv16_join_few_kernel(const int4* __restrict__ parts_of, int blocks, const float* __restrict__ part,
                         const float* __restrict__ stat, const float* __restrict__ sinks,
                         const float* __restrict__ other, uint16_t* out, float* lse) {
  constexpr int kLane4 = kDim / 4 / kFewBlocks, kGroups = kFewGroups;
  constexpr int kEarly = 20;  // parts that a thread loads before their weights are there
  __shared__ float weight[kMaxParts], own_s;
  __shared__ float4 acc_s[kGroups - 1][kLane4];
  __shared__ int found;
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  for (int k = 1 + threadIdx.x; k < blocks; k += blockDim.x) {
    const int4 at = parts_of[k];
    if (at.x == (int)blockIdx.x && reached(at)) found = k;  // there is one at most
  }
  __syncthreads();
  if (found == 0) return;
  const Parts ps = parts_at(parts_of[found], found);
  const int group = threadIdx.x / kLane4, lane4 = threadIdx.x % kLane4, x = blockIdx.z * kLane4 + lane4;
  const float4* src = reinterpret_cast<const float4*>(part + h * kDim) + x;
  float4 early[kEarly];
#pragma unroll
  for (int j = 0; j < kEarly; ++j)
    if (group + j * kGroups < ps.n) early[j] = src[ps.no(group + j * kGroups) * (kPartFloats / 4)];
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    float m[kMaxParts / 32], r[kMaxParts / 32], l[kMaxParts / 32], mx = kNone, rs = 0.f, ls = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxParts / 32; ++j) {
      const int k = lane + 32 * j;
      const float* st = stat + (k < ps.n ? ps.no(k) : 0) * kStatFloats + h;
      r[j] = k < ps.n ? st[0] : 0.f;
      l[j] = k < ps.n ? st[kHq] : 0.f;
      m[j] = k < ps.n ? st[2 * kHq] : kNone;
    }
#pragma unroll
    for (int j = 0; j < kMaxParts / 32; ++j) mx = fmaxf(mx, m[j]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
#pragma unroll
    for (int j = 0; j < kMaxParts / 32; ++j) {
      const float f = exp2f(m[j] - mx);
      weight[lane + 32 * j] = f;
      rs += f * r[j];
      ls += f * l[j];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      rs += __shfl_xor_sync(0xffffffffu, rs, d);
      ls += __shfl_xor_sync(0xffffffffu, ls, d);
    }
    if (lane == 0) {
      const Joined j = join_head(mx, rs, ls, sinks ? sinks[h] : -INFINITY, other_at(other, ps.token, h));
      own_s = j.own;
      if (lse && blockIdx.z == 0) lse[(int64_t)ps.token * kHq + h] = j.lse;
    }
  }
  __syncthreads();
  Sum4 acc;
#pragma unroll
  for (int j = 0; j < kEarly; ++j)
    if (group + j * kGroups < ps.n) acc.add(weight[group + j * kGroups], early[j]);
#pragma unroll 8
  for (int k = group + kEarly * kGroups; k < ps.n; k += kGroups) acc.add(weight[k], src[ps.no(k) * (kPartFloats / 4)]);
  if (group > 0) acc_s[group - 1][lane4] = acc.v;
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int k = 0; k < kGroups - 1; ++k) acc.add(1.f, acc_s[k][lane4]);
  acc.store<kBf16>(own_s, out + ((int64_t)ps.token * kHq + h) * kDim + 4 * x);
}

// Fewer tokens than blocks: two blocks an SM list the tokens that have parts, and their teams of 128 threads take a head
// of a token each in turn.  Where a token has more than kLongParts and that leaves half of the teams without work, the
// four teams of a block share a head's parts (12 tokens of 50 to 30000 rows 33.5 us, apart 38.6; but 8 of 8192, of
// 20 parts each, 31.0 and 30.3).
constexpr int kJoinTeams = 4, kJoinThreads = kJoinTeams * kDim / 4, kLongParts = 20;
template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads, 2)
    kv16_join_some_kernel(const int4* __restrict__ parts_of, int blocks, const float* __restrict__ part,
                          const float* __restrict__ stat, const float* __restrict__ sinks,
                          const float* __restrict__ other, uint16_t* out, float* lse) {
  constexpr int kBatch = 4;  // parts that a thread has on their way
  static_assert(kMaxParts <= kJoinThreads && 32 % (kJoinTeams * kBatch) == 0, "a thread an entry, whole batches a warp's weights");
  __shared__ Parts list[kMaxParts];
  __shared__ int count[kMaxParts / 32];
  __shared__ float4 acc_s[kJoinTeams - 1][kDim / 4];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int4 at = tid > 0 && tid < blocks ? parts_of[tid] : make_int4(-1, 0, 0, 0);
  const uint32_t has = __ballot_sync(0xffffffffu, reached(at));
  if (lane == 0 && warp < kMaxParts / 32) count[warp] = __popc(has);
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int k = 0; k < kMaxParts / 32; ++k) {
    before += k < warp ? count[k] : 0;
    total += count[k];
  }
  bool is_long = false;
  if (reached(at)) {
    const Parts ps = parts_at(at, tid);
    is_long = ps.n > kLongParts;
    list[before + __popc(has & ((1u << lane) - 1u))] = ps;
  }
  const int units = total * kHq, team = tid / (kDim / 4), lane4 = tid % (kDim / 4);
  const bool share = __syncthreads_or(is_long) && 2 * units <= (int)gridDim.x * kJoinTeams;
  const int step = share ? kJoinTeams : 1, first = share ? team : 0;  // a thread's parts are first + step * j
#pragma unroll 1
  for (int u = share ? blockIdx.x : blockIdx.x * kJoinTeams + team; u < units; u += gridDim.x * (kJoinTeams / step)) {
    const Parts ps = list[u / kHq];
    const int h = u % kHq;
    const float4* src = reinterpret_cast<const float4*>(part + h * kDim) + lane4;
    const float* st = stat + h;
    float4 o[kBatch];
    auto load = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = first + step * (j0 + i);
        if (k < ps.n) o[i] = src[ps.no(k) * (kPartFloats / 4)];
      }
    };
    load(0);
    // every warp of the team works out the statistics, a lane a part
    const float sink = sinks ? sinks[h] : -INFINITY;
    float m0 = kNone, r = 0.f, l = 0.f;
    if (lane < ps.n) {
      const float* s0 = st + ps.no(lane) * kStatFloats;
      r = s0[0];
      l = s0[kHq];
      m0 = s0[2 * kHq];
    }
    float mx = m0;
    for (int k = lane + 32; k < ps.n; k += 32) mx = fmaxf(mx, st[ps.no(k) * kStatFloats + 2 * kHq]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float f = exp2f(m0 - mx);
    r *= f;
    l *= f;
    for (int k = lane + 32; k < ps.n; k += 32) {
      const float* sk = st + ps.no(k) * kStatFloats;
      const float fk = exp2f(sk[2 * kHq] - mx);
      r += fk * sk[0];
      l += fk * sk[kHq];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      r += __shfl_xor_sync(0xffffffffu, r, d);
      l += __shfl_xor_sync(0xffffffffu, l, d);
    }
    const Joined j = join_head(mx, r, l, sink, other_at(other, ps.token, h));
    if (lse && lane4 == 0 && first == 0) lse[(int64_t)ps.token * kHq + h] = j.lse;
    Sum4 acc;
#pragma unroll 1
    for (int j0 = 0; step * j0 < ps.n; j0 += kBatch) {  // as often for all teams of a block that share a head
      const int base = step * j0;
      if (j0 > 0) load(j0);
      if (j0 > 0 && base % 32 == 0)  // the weights of the next 32 parts
        f = base + lane < ps.n ? exp2f(st[ps.no(base + lane) * kStatFloats + 2 * kHq] - mx) : 0.f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = first + base + step * i;
        const float w = __shfl_sync(0xffffffffu, f, k % 32);
        if (k < ps.n) acc.add(w, o[i]);
      }
    }
    if (share) {
      if (team > 0) acc_s[team - 1][lane4] = acc.v;
      __syncthreads();
      if (team == 0) {
#pragma unroll
        for (int k = 0; k < kJoinTeams - 1; ++k) acc.add(1.f, acc_s[k][lane4]);
      }
      __syncthreads();  // read: the next head's may go there
      if (team > 0) continue;
    }
    acc.store<kBf16>(j.own, out + ((int64_t)ps.token * kHq + h) * kDim + 4 * lane4);
  }
}

// More tokens (two or three parts each): a block per boundary between two blocks and eight heads, whose teams of 128
// threads take two heads each.
constexpr int kManyHeads = 2 * kJoinTeams;
template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads)
    kv16_join_many_kernel(const int4* __restrict__ parts_of, const float* __restrict__ part, const float* __restrict__ stat,
                          const float* __restrict__ sinks, const float* __restrict__ other, uint16_t* out, float* lse) {
  constexpr int kEarly = 2;  // parts of a head that a thread loads before their weights are there
  __shared__ float weight[kManyHeads][kMaxParts], own_s[kManyHeads];
  pdl_wait();
  pdl_trigger();
  const int4 at = parts_of[blockIdx.x + 1];
  if (!reached(at)) return;
  const Parts ps = parts_at(at, blockIdx.x + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h0 = blockIdx.y * kManyHeads;
  const int team = threadIdx.x / (kDim / 4), lane4 = threadIdx.x % (kDim / 4);
  const float4* src = reinterpret_cast<const float4*>(part + (h0 + team) * kDim) + lane4;  // of the first head
  float4 early[2][kEarly];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (k < ps.n) early[q][k] = src[ps.no(k) * (kPartFloats / 4) + q * kJoinTeams * (kDim / 4)];
  if (warp < kManyHeads) {
    const int h = h0 + warp;
    float mx = kNone, r = 0.f, l = 0.f;
    for (int k = lane; k < ps.n; k += 32) mx = fmaxf(mx, stat[ps.no(k) * kStatFloats + 2 * kHq + h]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    for (int k = lane; k < ps.n; k += 32) {
      const float* st = stat + ps.no(k) * kStatFloats + h;
      const float f = exp2f(st[2 * kHq] - mx);
      weight[warp][k] = f;
      r += f * st[0];
      l += f * st[kHq];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      r += __shfl_xor_sync(0xffffffffu, r, d);
      l += __shfl_xor_sync(0xffffffffu, l, d);
    }
    if (lane == 0) {
      const Joined j = join_head(mx, r, l, sinks ? sinks[h] : -INFINITY, other_at(other, ps.token, h));
      own_s[warp] = j.own;
      if (lse) lse[(int64_t)ps.token * kHq + h] = j.lse;
    }
  }
  __syncthreads();
  Sum4 acc[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (k < ps.n) acc[q].add(weight[q * kJoinTeams + team][k], early[q][k]);
#pragma unroll 4
  for (int k = kEarly; k < ps.n; ++k) {
    float4 o[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) o[q] = src[ps.no(k) * (kPartFloats / 4) + q * kJoinTeams * (kDim / 4)];
#pragma unroll
    for (int q = 0; q < 2; ++q) acc[q].add(weight[q * kJoinTeams + team][k], o[q]);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int hs = q * kJoinTeams + team;  // the head among the block's
    acc[q].store<kBf16>(own_s[hs], out + ((int64_t)ps.token * kHq + h0 + hs) * kDim + 4 * lane4);
  }
}

// Tokens of up to kWholeChunks chunks are never split (which takes a quarter of the time of joining parts, a launch at
// least): a call that can have no others has no parts, and a block a token at most.
constexpr int kUnsplitRows = kWholeChunks * kRows;
// Blocks for T tokens of up to max_rows rows: one an SM, at most one a chunk.
int grid_of(int T, int max_rows) {
  const int64_t chunks = (int64_t)T * (max_rows > kUnsplitRows ? (max_rows - 1) / kRows + 1 : 1);
  const int sms = device_sm_count();
  const int64_t most = sms < kMaxParts ? sms : kMaxParts;  // a token has at most a part of every block
  return (int)(chunks < most ? chunks : most);
}
constexpr size_t kHeadBytes = 16 * kMaxParts;  // the int4 of every block

}  // namespace

// Nothing without parts: an allocation less in a call whose cost is its launch.
size_t kv16_attn_workspace_bytes(int T, int max_rows) {
  if (max_rows <= kUnsplitRows) return 0;
  const int grid = grid_of(T < kTokens ? T : kTokens, max_rows);
  return kHeadBytes + (size_t)2 * grid * (kPartFloats + kStatFloats) * sizeof(float);
}

template <bool kBf16, Logits kLogits>
static int launch_typed(const Kv16AttnArgs& a, cudaStream_t stream) {
  const auto kernel = kv16_attn_kernel<kBf16, kLogits>;
  if (ensure_dynamic_smem(kernel, kSmem) != cudaSuccess) return DS4X_ERR_CUDA;
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
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);  // NULL: no parts
  p.parts_of = reinterpret_cast<int4*>(ws);
  for (int t0 = 0; t0 < a.T; t0 += kTokens) {  // launches on one stream: they may share the workspace
    p.t0 = t0;
    p.T = a.T - t0 < kTokens ? a.T - t0 : kTokens;
    const int grid = grid_of(p.T, a.max_rows);
    const int64_t row0 = (int64_t)t0 * kHq;
    p.part = ws ? reinterpret_cast<float*>(ws + kHeadBytes) : nullptr;
    p.stat = ws ? p.part + (size_t)2 * grid * kPartFloats : nullptr;
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
    if (launch_pdl(kernel, dim3(grid), dim3(kThreads), (size_t)kSmem, stream, tq, p) != cudaSuccess)
      return DS4X_ERR_CUDA;
    count_launch();
    if (grid > 1 && a.max_rows > kUnsplitRows) {
      const int4* of = p.parts_of;
      const float *part = p.part, *stat = p.stat;
      cudaError_t e;
      if (p.T < kFewTokens)
        e = launch_pdl(kv16_join_few_kernel<kBf16>, dim3(p.T, kHq, kFewBlocks), dim3(kFewThreads), 0, stream, of, grid, part,
                       stat, p.sinks, p.other_lse, p.out, p.lse);
      else if (p.T < grid)
        e = launch_pdl(kv16_join_some_kernel<kBf16>, dim3(2 * device_sm_count()), dim3(kJoinThreads), 0, stream, of, grid,
                       part, stat, p.sinks, p.other_lse, p.out, p.lse);
      else
        e = launch_pdl(kv16_join_many_kernel<kBf16>, dim3(grid - 1, kHq / kManyHeads), dim3(kJoinThreads), 0, stream, of,
                       part, stat, p.sinks, p.other_lse, p.out, p.lse);
      if (e != cudaSuccess) return DS4X_ERR_CUDA;
      count_launch();
    }
  }
  return DS4X_OK;
}

int launch_kv16_attn(const Kv16AttnArgs& a, cudaStream_t stream) {
  if (a.cap > kNearCap) return a.bf16 ? launch_typed<true, kWide>(a, stream) : launch_typed<false, kWide>(a, stream);
  if (a.cap > 0.f || a.slopes) return a.bf16 ? launch_typed<true, kBiased>(a, stream) : launch_typed<false, kBiased>(a, stream);
  return a.bf16 ? launch_typed<true, kPlain>(a, stream) : launch_typed<false, kPlain>(a, stream);
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
      window < 0 || !(cap >= 0.f) || isinf(cap) || !(fabsf(scale) <= kMaxScale) ||
      (dtype != DS4X_F16 && dtype != DS4X_BF16))
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
