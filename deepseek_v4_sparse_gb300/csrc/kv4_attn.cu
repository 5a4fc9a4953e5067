// kv4_attn.cu — multi-query attention of 64 heads over rows of the paged 4-bit cache.
//
//   out[t,h,:] = sum_j softmax_j( scale * q[t,h,:] . kv_j ) * kv_j
//
// over the rows j that a token selected (indices) or over every row of its request that it can see.
//
// The products run on the tensor cores in fp16, whatever the type of q: a row's values (code times a
// power of two, kv4_common.cuh) are exact in fp16, a bf16 q is made so by a power of two a head (which
// moves its largest magnitude to [2^14, 2^15); what comes to lie under 2^-14 is off by at most 2^-15, 2^-29 of
// the head's largest), and the softmax weights keep eleven bits instead of bf16's eight.
//
// One block an SM.  The tokens' rows are cut into chunks of 64; all chunks of all tokens form one
// sequence, and each block takes an equal, contiguous part of it.  A token whose chunks lie in several
// blocks leaves its unnormalised sums there in fp32 and kv4_combine_kernel joins them, so a long row list
// of one token, a ragged batch and a full prefill chunk are all spread evenly.  A token's chunks in a block
// are an item (several, if they are many: kItemChunks).  Per chunk:
//   S   [64 heads x 64 rows] = Q . K^T       tcgen05, M = 64 (heads on TMEM lanes), K-major
//   O^T [512 x 64 heads]    += V^T . P^T     tcgen05, M = 128 (dims), A MN-major, B K-major
// with K = V = the chunk, decoded once into 128B-swizzled shared memory (8 slots of 64 dims, two buffers).
//
// Warps: 0-15 fetch and decode rows and convert q, 16-19 softmax (heads 16*(warp-16) .. +15, 4 threads a
// head), 20-23 write the output (O^T lanes by quadrant), 24 issues the S products, 25 the O^T products,
// 26 looks up the rows' slots a few chunks ahead.  A fetching thread owns 32 values (one scale group) of
// two rows: it decodes the chunk into registers, has the codes of the next one on their way and then waits
// for the buffer.  Buffers are released in halves of the dims, O^T rotates over six 64-column TMEM slots
// (a token uses four), so neighbouring tokens overlap.  q of a token goes in before its first chunk is
// decoded: the fetching warps wait for a buffer then, and have it converted when the products of the token
// before are done with theirs.  It is brought to L2 an item ahead.
//
// What bounds it: a chunk's way through the roles (fetch, S, softmax, O^T, release), two chunks at a time, in
// about 3950 clocks a chunk.  221 us for 2048 tokens of 512 rows: 622 TFLOP/s, 33 % of the measured peak.  With
// three quarters of the products left out it took 189 us, without fetches and stores 200 us, with neither and
// without 2^x 168 us: no one resource, most is the hand-overs.  (The data path of L1 and shared memory has
// something to do in 93 % of its cycles, 1790 accesses a chunk of the products and 1880 of the warps, but 37 %
// fewer accesses saved 14 % of the time: it is not what bounds.)  Slower: three buffers of 48 rows (272 us: S
// products cost nearly the same at 48 rows as at 64), rows in 16 lines a load and slots looked up in every
// warp (247 us), rows by bulk copies into a stage of their own (345 us).
//
// The running maximum of a head moves only when a logit exceeds it by more than 2^11 (O^T's column and
// the sums are rescaled then, which stalls the products); weights are 2^4 times 2^(x - m), which keeps them
// below fp16's largest value and small ones away from its least.  Statistics and sums are fp32.
//
// The roles share the SM's instruction caches: every loop that need not be unrolled for its registers is
// kept rolled, and the waits' failure path is short.  (Unrolled throughout, the kernel was 152 KB of code
// and a 2048-token chunk took 377 us, a third of the warps' time waiting for instructions.)
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
constexpr int kHalves = 2;                       // of the dims: what is fetched and released together
constexpr int kSlotBytes = kRows * 128;          // 8 KB
constexpr int kBufBytes = kSlots * kSlotBytes;   // 64 KB a chunk
constexpr int kQBlockBytes = kHq * 128;          // 8 KB (64 heads x 64 dims)
constexpr int kQBytes = kSlots * kQBlockBytes;   // 64 KB
constexpr int kPBytes = kHq * 128;               // 8 KB: P[h][j]
constexpr int kTokens = 2048;                    // tokens a launch plans for
constexpr int kDecWarps = 16, kSoftWarp = 16, kOutWarp = 20, kSWarp = 24, kOWarp = 25, kSlotWarp = 26;
constexpr int kWarps = 28, kThreads = 32 * kWarps;  // whole warpgroups; the last warp only takes part in the scan
// registers a thread: 72 at launch; the sum over the seven warpgroups stays what it was
constexpr int kLaunchRegs = 72, kDecRegs = 72, kMmaRegs = 40, kSoftRegs = 88, kOutRegs = 80;
static_assert(kThreads * kLaunchRegs <= 65536 && 4 * kDecRegs + kMmaRegs + kSoftRegs + kOutRegs <= 7 * kLaunchRegs, "registers");
constexpr int kRing = 4, kMaskRing = 8;          // chunks whose slots, and masks, are looked up ahead
constexpr int kItems = 4;                        // items whose logit factors are kept
// Chunks of a token that are added up in one go.  The matrix unit truncates its fp32 sums: over one token's
// 262144 rows of one sign they came out 0.14 % low, over 4194304 rows 2.6 %; items of 16384 rows, joined with
// rounded sums, show nothing of it.  An item's end costs the output warps a read and a write of 128 KB.
constexpr int kItemChunks = 256;
constexpr int kOSlots = 6;                       // O^T slots of 64 TMEM columns
constexpr int kOffKV = kQBytes;
constexpr int kOffP = kOffKV + 2 * kBufBytes;
constexpr int kOffAlpha = kOffP + 2 * kPBytes;   // float[64]: rescale factors of one chunk
constexpr int kOffLM = kOffAlpha + kHq * 4;      // float[2 items][4][64]: sum of rounded weights, sum, m, 1 / first
constexpr int kOffCq = kOffLM + 2 * 4 * kHq * 4; // float[kItems][64]: logit factor of a head
constexpr int kOffRows = kOffCq + kItems * kHq * 4;  // int[kTokens]: rows of each token's list
constexpr int kOffJoin = kOffRows + kTokens * 4; // float[4][5][64], a copy for each output warp: a token's m, sum of rounded
                                                 // weights and sum so far; factors of the sums so far and of the item's
constexpr int kOffMask = kOffJoin + 4 * 5 * kHq * 4; // uint32[kMaskRing][2]: rows of the chunk that count
constexpr int kOffSlots = kOffMask + kMaskRing * 8;  // int[kRing][64]: slot of each row of the chunk, -1 for none
constexpr int kOffScan = kOffSlots + kRing * kRows * 4;         // int64[kWarps] warp sums, then int[4]: the block's part, and
                                                 // the last chunk (+ 1) in which a maximum moved
constexpr int kOffBars = kOffScan + kWarps * 8 + 16;
constexpr int kNumBars = 2 + 2 * kRing + 2 * 2 * kHalves + 5 * 2 + 2 * kOSlots + 2 * 2;
constexpr int kOffTmemSlot = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmemSlot + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kColO = 128;  // S in columns [0, 128), O^T from 128
constexpr float kRescaleLog2 = 11.0f, kWeightLog2 = 4.0f;
constexpr int kSoftBar = 1, kGroupThreads = 128;
constexpr int kPartFloats = kHq * kKv4Dim;        // unnormalised sums of a part, then its statistics
constexpr int kStatFloats = 3 * kHq;              // sum of rounded weights, sum, m

struct Params {
  const uint16_t* q;
  const uint8_t *codes, *scales;
  const int32_t *tables, *rows, *req, *positions, *indices, *counts;
  uint16_t* out;
  float* lse;
  int* status;
  int4* parts_of;  // [grid]: the token a block starts in, chunks of it before the block, chunks it has, quota;
                   // NULL without a workspace, when there can be no rows at all
  float* part;     // [2 grid][kPartFloats]
  float* stat;     // [2 grid][kStatFloats]
  int n_slots, n_req, max_pages, log_page, ratio, t0, T, k_top;
  float scale;
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

// D (+)= A B^T by an elected lane of a converged warp; descriptors by their low words (the addresses): the
// high words are the same for all operands here.
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

__device__ __forceinline__ int request_of(const Params& p, int t) { return p.req ? __ldg(p.req + t) : p.t0 + t; }

// Rows in the list of token t (selected: list entries; else visible rows).
__device__ __forceinline__ int token_rows(const Params& p, int t) {
  const int b = request_of(p, t);
  if (b < 0 || b >= p.n_req) return 0;
  if (p.indices) return p.counts ? min(max(__ldg(p.counts + t), 0), p.k_top) : p.k_top;
  const int held = min(max(__ldg(p.rows + b), 0), p.max_pages << p.log_page);
  if (!p.positions) return held;
  const int pos = __ldg(p.positions + t);
  return pos < 0 ? 0 : (int)min((uint32_t)held, ((uint32_t)pos + 1u) / (uint32_t)p.ratio);
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
// Two bf16 values as fp16, their exponents lowered by the head's offset (twice in `bias`, in place).  Exact from
// 2^-14 on (and so from 2^-28 of the head's largest magnitude on); what falls one exponent below reads as the
// subnormal of its mantissa, the rest as 0: off by at most 2^-15.
__device__ __forceinline__ uint32_t bf16_to_fp16(uint32_t u, uint32_t bias) {
  const uint32_t a = __vmaxu2(u & 0x7fff7fffu, bias);
  return (a * 8u - bias * 8u) | (u & 0x80008000u);
}
// r + the two halves of v
__device__ __forceinline__ void add_halves(float& r, __half2 v) {
  const __half_raw lo = __low2half(v), hi = __high2half(v);
  asm("add.f32.f16 %0, %1, %0;" : "+f"(r) : "h"(lo.x));
  asm("add.f32.f16 %0, %1, %0;" : "+f"(r) : "h"(hi.x));
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
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + kOffMask);
  int* slot_s = reinterpret_cast<int*>(smem + kOffSlots);
  long long* scan = reinterpret_cast<long long*>(smem + kOffScan);
  int* start = reinterpret_cast<int*>(smem + kOffScan + kWarps * 8);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* qempty = qfull + 1;
  uint64_t* slfull = qempty + 1;            // [ring] slots of a chunk
  uint64_t* slempty = slfull + kRing;
  uint64_t* kvfull = slempty + kRing;       // [buffer][half]
  uint64_t* kvempty = kvfull + 2 * kHalves; // [buffer][half]
  uint64_t* sfull = kvempty + 2 * kHalves;
  uint64_t* sempty = sfull + 2;
  uint64_t* pfull = sempty + 2;
  uint64_t* pempty = pfull + 2;
  uint64_t* looked = pempty + 2;            // every softmax warp has seen whether its maxima move
  uint64_t* ofull = looked + 2;             // [O^T slot]
  uint64_t* oempty = ofull + kOSlots;       // [O^T slot]
  uint64_t* lready = oempty + kOSlots;      // [item parity] statistics written
  uint64_t* lfree = lready + 2;             // [item parity] ... and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmemSlot);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto oslot = [](uint32_t item, int db) { return (int)((4u * (item % 3u) + (uint32_t)db) % kOSlots); };

  if (tid < kNumBars) {  // one barrier a thread
    uint64_t* bar = qfull + tid;
    const bool four = (bar >= sempty && bar < pempty) || (bar >= looked && bar < ofull) || bar >= oempty;  // by the softmax or the output warps
    mbar_init(bar, bar == qfull ? kDecWarps
                   : bar >= slempty && bar < kvfull ? kDecWarps
                   : bar >= kvfull && bar < kvempty ? kDecWarps / kHalves
                   : bar >= sfull && bar < sempty ? 2  // the products' completion and the issuing warp itself
                   : four ? 4 : 1);
    fence_mbarrier_init();
  }
  if (warp == kSWarp) tmem_alloc(tmem_slot, kTmemCols);
  pdl_wait();  // everything above touched only this block's own resources
  pdl_trigger();

  // --------------------------------------------------- every token's rows; this block's part
  {
    const int per = (p.T + kThreads - 1) / kThreads;
    const int first = tid * per, last = min(first + per, p.T);
    long long sum = 0;
#pragma unroll 1
    for (int t = first; t < last; ++t) {
      const int n = token_rows(p, t);
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
    if (tid == 0) start[2] = start[3] = 0;
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

  if (warp < kDecWarps) {
    // --------------------------------------------------------------------- fetch and decode
    // the dims' half warp / 8 of rows 8 (warp % 8) .. + 7 of the chunk, four rows at a time: lane / 8 the row,
    // lane % 8 the group of 32.  Eight neighbouring lanes read a 128-byte line and store, in step k, the
    // 16-byte columns k ^ slot of their groups: four slots by two groups, all in different banks.
    const int half = warp >> 3, lr = lane >> 3, gi = lane & 7;
    const int ss = gi >> 1;                     // slot of 64 dims within the half
    // step k of the first row; of the second, 4 rows on: ^ 64, + 512
    uint32_t st_off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      st_off[k] = smem_u32(skv) + (uint32_t)((4 * half + ss) * kSlotBytes + (8 * (warp & 7) + lr) * 128 +
                                             ((((gi & 1) * 4 + (k ^ ss)) ^ lr) << 4));
    const uint8_t* codes = p.codes + half * 128 + gi * 16;
    const uint8_t* scales = p.scales + half * 8 + gi;
    uint4 d[2];
    uint32_t sc[2];
    // codes and scales of chunk x: a row without a slot reads slot 0 with a scale of 0
    auto load = [&](uint32_t x) {
      const bool got = wait_bar_warp(&slfull[x % kRing], (x / kRing) & 1, p.status, 80);
      const int* sl = slot_s + (x % kRing) * kRows + 8 * (warp & 7) + lr;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = sl[4 * i];
        d[i] = make_uint4(0, 0, 0, 0);
        sc[i] = 0;
        if (p.n_slots > 0) {
          d[i] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)max(at, 0) * kKv4CodeBytes));
          sc[i] = at < 0 ? 0u : __ldg(scales + (int64_t)at * kKv4ScaleBytes);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&slempty[x % kRing]);
      return got;
    };
    // q of token t as fp16 into the operand's layout; each warp 4 heads, 16-byte units lane and lane + 32
    auto load_q = [&](int qt, uint4 (&u)[4][2]) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((int64_t)qt * kHq + warp * 4) * kKv4Dim) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i][0] = __ldg(src + i * (kKv4Dim / 8));
        u[i][1] = __ldg(src + i * (kKv4Dim / 8) + 32);
      }
    };
    auto put_q = [&](uint4 (&u)[4][2], uint32_t qi) {
      const int h = warp * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f = p.scale * 1.4426950408889634f;
        if constexpr (kBf16) {
          // a head's exponent offset, from its largest magnitude (compared as bits); a logit in log2
          // units is the product times scale log2(e) 2^(offset - 112)
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            m = __vmaxu2(__vmaxu2(__vmaxu2(m, u[i][k].x & 0x7fff7fffu), __vmaxu2(u[i][k].y & 0x7fff7fffu, u[i][k].z & 0x7fff7fffu)),
                         u[i][k].w & 0x7fff7fffu);
          const uint32_t ex = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) >> 7;
          // the largest exponent field becomes 29; infinities and NaN stay what they are (field 31)
          const uint32_t off = ex == 255u ? 224u : ex > 29u ? ex - 29u : 0u;
          const uint32_t bias = (off << 7) | (off << 23);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            u[i][k] = make_uint4(bf16_to_fp16(u[i][k].x, bias), bf16_to_fp16(u[i][k].y, bias),
                                 bf16_to_fp16(u[i][k].z, bias), bf16_to_fp16(u[i][k].w, bias));
          f *= __uint_as_float((off + 15u) << 23);
        }
        if (lane == 0) cq[(qi % kItems) * kHq + h + i] = f;
      }
      const bool got = wait_bar_warp(qempty, (qi & 1) ^ 1, p.status, 91);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint8_t* dst = sq + (lane >> 3) * kQBlockBytes + (h + i) * 128 + (((lane & 7) ^ ((h + i) & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = u[i][0];
        *reinterpret_cast<uint4*>(dst + 4 * kQBlockBytes) = u[i][1];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      return got;
    };
    const uint32_t chunks = start[2];
    bool ok = true;
    uint32_t g = 0, item = 0;
    for (Walk w(rows_s, start); w.left > 0 && ok; w.next(), ++item) {
      uint4 u[4][2];
      load_q(w.t, u);
      if (item == 0) ok = load(0);
      ok = put_q(u, item) && ok;
#pragma unroll 1
      for (int ci = w.c0; ci < w.c1 && ok; ++ci, ++g) {
        const int b = g & 1;
        uint32_t v[2][16];  // decoded before the buffer is free
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __half2 s2 = __float2half2_rn(kv4_scale(sc[i]));
          // word k ^ slot of the group in step k
          const bool s0 = ss & 1, s1 = ss & 2;
          const uint32_t a0 = s0 ? d[i].y : d[i].x, a1 = s0 ? d[i].x : d[i].y;
          const uint32_t a2 = s0 ? d[i].w : d[i].z, a3 = s0 ? d[i].z : d[i].w;
          const uint32_t w4[4] = {s1 ? a2 : a0, s1 ? a3 : a1, s1 ? a0 : a2, s1 ? a1 : a3};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            kv4_decode8(w4[k], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][4 * k + e] = mul2(h[e], s2);
          }
        }
        if (g + 1 < chunks) ok = load(g + 1);
        ok = ok && wait_bar_warp(&kvempty[b * kHalves + half], ((g >> 1) & 1) ^ 1, p.status, 81);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = st_off[k] + b * kBufBytes, a4 = (st_off[k] ^ 64u) + b * kBufBytes;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0][4 * k]), "r"(v[0][4 * k + 1]),
                       "r"(v[0][4 * k + 2]), "r"(v[0][4 * k + 3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0 + 512], {%1, %2, %3, %4};" ::"r"(a4), "r"(v[1][4 * k]), "r"(v[1][4 * k + 1]),
                       "r"(v[1][4 * k + 2]), "r"(v[1][4 * k + 3])
                       : "memory");
        }
        fence_proxy_async();  // decoded rows -> visible to the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&kvfull[b * kHalves + half]);
      }
    }
  } else if (warp >= kSWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kSWarp) {
      // ------------------------------------------------------------------------ S = Q K^T
      uint32_t gc = 0, item = 0;
      bool ok = true;
      const uint32_t q_lo = (uint32_t)desc_sw128(smem_u32(sq), 16, 1024), kv_lo = (uint32_t)desc_sw128(smem_u32(skv), 16, 1024);
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++gc) {
          const int b = gc & 1;
          if (!wait_bar_warp(&sempty[b], ((gc >> 1) & 1) ^ 1, p.status, 82)) { ok = false; break; }
          if (c == w.c0) {
            if (lane == 0 && w.c1 == w.end && w.left > w.c1 - w.c0)
              prefetch_l2(p.q + (int64_t)(w.t + 1) * kHq * kKv4Dim, kHq * kKv4Dim * 2);
            if (!wait_bar_warp(qfull, item & 1, p.status, 83)) { ok = false; break; }
          }
#pragma unroll 1
          for (int half = 0; half < kHalves; ++half) {
            if (!wait_bar_warp(&kvfull[b * kHalves + half], (gc >> 1) & 1, p.status, 84)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a = q_lo + half * (4 * kQBlockBytes >> 4), k = kv_lo + (b * kBufBytes + half * 4 * kSlotBytes >> 4);
            mma_elect<false>(tmem + b * kHq, a, k, kIdescS, half);
#pragma unroll
            for (int i = 1; i < 16; ++i)
              mma_elect<true>(tmem + b * kHq, a + ((i >> 2) * kQBlockBytes + (i & 3) * 32 >> 4),
                              k + ((i >> 2) * kSlotBytes + (i & 3) * 32 >> 4), kIdescS, 1);
          }
          if (!ok) break;
          if (c == w.c1 - 1) tc_commit_elect(qempty);  // the next item's q may replace this one's
          // the arrival of this warp hands on what it waited for (the chunk's mask, the item's factors)
          if (lane == 0) mbar_arrive(&sfull[b]);
          tc_commit_elect(&sfull[b]);
        }
      }
    } else if (warp == kSlotWarp) {
      // --------------------------------------------------------- slots of the rows, a few chunks ahead
      uint32_t gc = 0;
      bool ok = true;
      for (Walk w(rows_s, start); w.left > 0 && ok; w.next()) {
        const int t = w.t, n = rows_s[t];
        const int32_t* list = p.indices ? p.indices + (int64_t)t * p.k_top : nullptr;
        auto row_of = [&](int c, int i) {
          const int j = c * kRows + lane + 32 * i;
          return j >= 0 && j < n ? (list ? __ldg(list + j) : j) : -1;
        };
        int next[2] = {row_of(w.c0, 0), row_of(w.c0, 1)};  // on their way while the request is looked up
        const int b = request_of(p, t);
        const int held = n > 0 && list ? __ldg(p.rows + b) : 0x7fffffff;
        const int32_t* table = p.tables + (int64_t)(n > 0 ? b : 0) * p.max_pages;
        for (int c = w.c0; c < w.c1; ++c, ++gc) {
          int slot[2];
          const int now[2] = {next[0], next[1]};
          if (c + 1 < w.c1) {
            next[0] = row_of(c + 1, 0);
            next[1] = row_of(c + 1, 1);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = now[i];
            const int pg = row >> p.log_page;
            slot[i] = -1;
            if (row >= 0 && pg < p.max_pages) {  // the table is read while the rows held are on their way
              const int page = __ldg(table + pg);
              const int64_t at = ((int64_t)page << p.log_page) + (row & ((1 << p.log_page) - 1));
              if (page >= 0 && at < p.n_slots && row < held) slot[i] = (int)at;
            }
          }
          const uint32_t m0 = __ballot_sync(0xffffffffu, slot[0] >= 0), m1 = __ballot_sync(0xffffffffu, slot[1] >= 0);
          ok = wait_bar_warp(&slempty[gc % kRing], ((gc / kRing) & 1) ^ 1, p.status, 79);
          if (!ok) break;
          slot_s[(gc % kRing) * kRows + lane] = slot[0];
          slot_s[(gc % kRing) * kRows + lane + 32] = slot[1];
          // a mask is overwritten eight chunks later: its slots were read then four chunks ago, by warps that
          // are at most two chunks ahead of the softmax
          if (lane == 0) *reinterpret_cast<uint2*>(mask_s + (gc % kMaskRing) * 2) = make_uint2(m0, m1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&slfull[gc % kRing]);
        }
      }
    } else if (warp == kOWarp) {
      // --------------------------------------------------------------------- O^T += V^T P^T
      uint32_t gc = 0, item = 0;
      uint32_t o_ph = 0;  // bit s: phase of O^T slot s's empty barrier
      bool ok = true;
      const uint32_t v_lo = (uint32_t)desc_sw128(smem_u32(skv), kSlotBytes, 1024), p_lo = (uint32_t)desc_sw128(smem_u32(sp), 16, 1024);
      for (Walk w(rows_s, start); __all_sync(0xffffffffu, w.left > 0 && ok); w.next(), ++item) {
        for (int c = w.c0; __all_sync(0xffffffffu, c < w.c1); ++c, ++gc) {
          const int b = gc & 1;
          if (!wait_bar_warp(&pfull[b], (gc >> 1) & 1, p.status, 85)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int db = 0; db < kPairs; ++db) {
            const int os = oslot(item, db);
            // an item's first product overwrites its slot: the output that last read it is done
            if (c == w.c0) {
              if (!wait_bar_warp(&oempty[os], ((o_ph >> os) & 1u) ^ 1u, p.status, 86)) { ok = false; break; }
              o_ph ^= 1u << os;
              tc_fence_after();
            }
            const uint32_t a = v_lo + (b * kBufBytes + 2 * db * kSlotBytes >> 4), k = p_lo + (b * kPBytes >> 4);
            mma_elect<false>(tmem + kColO + os * kHq, a, k, kIdescO, c > w.c0);
#pragma unroll
            for (int ks = 1; ks < kRows / 16; ++ks)
              mma_elect<true>(tmem + kColO + os * kHq, a + (ks * 2048 >> 4), k + 2 * ks, kIdescO, 1);
            if (db & 1) tc_commit_elect(&kvempty[b * kHalves + (db >> 1)]);  // this half of the chunk is free
            if (c == w.c1 - 1) tc_commit_elect(&ofull[os]);
          }
          if (!ok) break;
          tc_commit_elect(&pempty[b]);
        }
      }
    }
  } else if (warp < kOutWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------------------- softmax
    // S holds head 16 quad + i on TMEM lane 32 quad + i (i < 16).  The 16x256b load gives thread
    // (g = lane / 4, e = lane % 4) the heads hA = 16 quad + g and hB = hA + 8 and, of each, the
    // columns 8 r + 2 e + {0, 1}, r = 0..7: a head's 64 logits are spread over 4 threads.
    const int quad = warp - kSoftWarp;
    const int g = lane >> 2, e = lane & 3;
    const int hA = 16 * quad + g, hB = hA + 8;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t gc = 0, item = 0;
    // a wait that gave up is acted on where the four warps meet, so that they leave together
    bool ok = true, leave = false;
    for (Walk w(rows_s, start); w.left > 0 && !leave; w.next(), ++item) {
      float mA = -INFINITY, mB = -INFINITY;          // running maximum (log2 units)
      float lA = 0.f, lB = 0.f, rA = 0.f, rB = 0.f;  // sums of the weights, and of the rounded ones
      for (int ci = w.c0; ci < w.c1; ++ci, ++gc) {
        const int b = gc & 1;
        ok = ok && wait_bar_warp(&sfull[b], (gc >> 1) & 1, p.status, 87);
        tc_fence_after();
        float x[32];
        tmem_ld_16x256b_x8(tmem + t_lane + b * kHq, x);
        const uint2 live = *reinterpret_cast<const uint2*>(mask_s + (gc % kMaskRing) * 2);
        const float cA = cq[(item % kItems) * kHq + hA], cB = cq[(item % kItems) * kHq + hB];
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[b]);
        // scaled before the maximum is taken from them: a fused multiply-add would not cancel exactly
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          x[4 * r] *= cA;
          x[4 * r + 1] *= cA;
          x[4 * r + 2] *= cB;
          x[4 * r + 3] *= cB;
        }
        if ((live.x & live.y) != 0xffffffffu) {
          const uint32_t v0 = live.x >> (2 * e), v1 = live.y >> (2 * e);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const uint32_t bits = (r < 4 ? v0 : v1) >> (8 * (r & 3));
            if (!(bits & 1u)) x[4 * r] = x[4 * r + 2] = -INFINITY;
            if (!(bits & 2u)) x[4 * r + 1] = x[4 * r + 3] = -INFINITY;
          }
        }
        float mxA = -INFINITY, mxB = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
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
        // whether any head's maximum moves is said now and asked for when the weights are ready (the same
        // answer in all four warps: a later chunk's word is written after all have read this one's)
        const bool moved = __any_sync(0xffffffffu, needA || needB || !ok);
        if (lane == 0) {
          if (moved) *const_cast<volatile int*>(start + 3) = (int)(gc + 1);
          mbar_arrive(&looked[b]);
        }
        lA *= aA;
        rA *= aA;
        lB *= aB;
        rB *= aB;
        // weights 2^(x - m + 4), rounded to fp16 for the product
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
          add_halves(rA, hp);
          add_halves(rB, hq);
          pkA[r] = *reinterpret_cast<const uint32_t*>(&hp);
          pkB[r] = *reinterpret_cast<const uint32_t*>(&hq);
        }
        ok = ok && wait_bar_warp(&looked[b], (gc >> 1) & 1, p.status, 95);
        if (*const_cast<volatile int*>(start + 3) == (int)(gc + 1)) {
          leave = named_or(kSoftBar, kGroupThreads, !ok);
          if (leave) break;
          if (e == 0) {
            alpha_s[hA] = needA ? aA : 1.f;
            alpha_s[hB] = needB ? aB : 1.f;
          }
          named_sync(kSoftBar, kGroupThreads);
          // O^T must hold all of the previous chunk before its columns are rescaled
          const uint32_t prev = gc - 1;
          ok = wait_bar_warp(&pempty[prev & 1], (prev >> 1) & 1, p.status, 88);
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
        ok = ok && wait_bar_warp(&pempty[b], ((gc >> 1) & 1) ^ 1, p.status, 89);
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
      if (leave) break;
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        lA += __shfl_xor_sync(0xffffffffu, lA, d);
        lB += __shfl_xor_sync(0xffffffffu, lB, d);
        rA += __shfl_xor_sync(0xffffffffu, rA, d);
        rB += __shfl_xor_sync(0xffffffffu, rB, d);
      }
      // the slot of this item's parity was last read by the output of item - 2
      ok = ok && wait_bar_warp(&lfree[item & 1], ((item >> 1) & 1) ^ 1, p.status, 90);
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    // --------------------------------------------------------------------------- output
    const int quad = warp - kOutWarp;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    const bool odd = lane & 1;
    uint32_t item = 0;
    uint32_t f_ph = 0;  // bit s: phase of O^T slot s's full barrier
    bool ok = true;
    int from = 0;                                // the block's first chunk of the token
    for (Walk w(rows_s, start); w.left > 0; w.next(), ++item) {
      const int par = item & 1;
      ok = wait_bar_warp(&lready[par], (item >> 1) & 1, p.status, 92);
      if (!ok) break;
      const float* lrow = lm + par * 4 * kHq;
      // chunks before the block, or behind it: the sums go to the block's first or second part
      if (w.c0 == 0 || item == 0) from = w.c0;
      const bool begins = w.c0 == from, ends = w.c1 == w.end;
      const bool whole = ends && from == 0 && w.c1 == chunks_of(rows_s[w.t]);
      const int64_t part = 2 * (int64_t)blockIdx.x + (from == 0);
      if (!(begins && ends)) {
        // One of several items: its sums are joined to those so far, as kv4_combine_kernel joins parts.  They
        // lie where the part's go: the second part's own token is the block's last, behind all that lie whole
        // in the block.  A thread reads back only what it wrote.
        float* so_far = reinterpret_cast<float*>(smem + kOffJoin) + quad * 5 * kHq;
#pragma unroll 1
        for (int hh = lane; hh < kHq; hh += 32) {
          const float mi = lrow[2 * kHq + hh], m0 = begins ? -INFINITY : so_far[hh];
          const float m = fmaxf(m0, mi);
          const float f0 = begins ? 0.f : m == -INFINITY ? 1.f : ex2_approx(m0 - m);
          const float fi = m == -INFINITY ? 1.f : ex2_approx(mi - m);
          const float r = lrow[hh] * fi + (begins ? 0.f : so_far[kHq + hh] * f0);
          const float l = lrow[kHq + hh] * fi + (begins ? 0.f : so_far[2 * kHq + hh] * f0);
          so_far[hh] = m;
          so_far[kHq + hh] = r;
          so_far[2 * kHq + hh] = l;
          const float inv = !whole ? 1.f : r == 0.f ? 0.f : 1.f / r;
          so_far[3 * kHq + hh] = f0 * inv;
          so_far[4 * kHq + hh] = fi * inv;
          if (quad == 0 && ends && !whole) {
            float* st = p.stat + part * kStatFloats;
            st[hh] = r;
            st[kHq + hh] = l;
            st[2 * kHq + hh] = m;
          } else if (quad == 0 && whole && p.lse) {
            p.lse[(int64_t)w.t * kHq + hh] = l == 0.f ? -INFINITY : (m + (log2f(l) - kWeightLog2)) * 0.69314718055994531f;
          }
        }
        __syncwarp();
#pragma unroll 1
        for (int step = 0; step < 4 * kPairs; ++step) {  // quarters of the dims by quarters of the heads
          const int db = step >> 2, hb = (step & 3) * 16;
          const int os = oslot(item, db);
          if (hb == 0) {
            ok = wait_bar_warp(&ofull[os], (f_ph >> os) & 1u, p.status, 94);
            if (!ok) break;
            f_ph ^= 1u << os;
            tc_fence_after();
          }
          float v[16];
          tmem_ld16(tmem + t_lane + kColO + os * kHq + hb, v);
          tc_wait_ld();
          if (hb == 48) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&oempty[os]);
          }
          const int d = db * 128 + quad * 32 + lane;
          float* sums = p.part + part * kPartFloats + hb * kKv4Dim + d;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] *= so_far[4 * kHq + hb + i];
            if (!begins) v[i] += so_far[3 * kHq + hb + i] * sums[i * kKv4Dim];
          }
          uint16_t* orow = p.out + ((int64_t)w.t * kHq + hb) * kKv4Dim + d;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (whole) orow[i * kKv4Dim] = (uint16_t)pack16<kBf16>(v[i], 0.f);
            else sums[i * kKv4Dim] = v[i];
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfree[par]);
        continue;
      }
      if (lane < 16) {
        const int hh = quad * 16 + lane;
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
#pragma unroll 1
      for (int half = 0; half < 2 * kPairs; ++half) {  // quarters of the dims by halves of the heads
        const int db = half >> 1, hb = (half & 1) * 32;
        const int os = oslot(item, db);
        if (hb == 0) {
          ok = wait_bar_warp(&ofull[os], (f_ph >> os) & 1u, p.status, 93);
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
        const int d = db * 128 + quad * 32 + lane;
        if (whole) {
          // neighbouring lanes exchange, so that each writes two dims of one head
          uint32_t* orow = reinterpret_cast<uint32_t*>(p.out + ((int64_t)w.t * kHq + hb + (odd ? 1 : 0)) * kKv4Dim) + (d >> 1);
          const float4* inv = reinterpret_cast<const float4*>(lrow + 3 * kHq + hb);
          const uint32_t sel = odd ? 0x3276u : 0x5410u;  // even: both first heads; odd: both second ones
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 f = inv[i / 4];
            const uint32_t w0 = pack16<kBf16>(v[i] * f.x, v[i + 1] * f.y), w1 = pack16<kBf16>(v[i + 2] * f.z, v[i + 3] * f.w);
            orow[i * (kKv4Dim / 2)] = __byte_perm(w0, __shfl_xor_sync(0xffffffffu, w0, 1), sel);
            orow[(i + 2) * (kKv4Dim / 2)] = __byte_perm(w1, __shfl_xor_sync(0xffffffffu, w1, 1), sel);
          }
        } else {
          float* dst = p.part + part * kPartFloats + hb * kKv4Dim + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) dst[i * kKv4Dim] = v[i];
        }
      }
      if (!ok) break;
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

// Joins the parts of a token that several blocks worked on: part k holds O_k = sum_j 2^(x_j - m_k) kv_j and
// the sums r_k of its rounded weights and l_k of the exact ones, so with M = max_k m_k
//   out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) r_k,   lse = ln 2 (M + log2 sum_k 2^(m_k - M) l_k).
// A thread holds 4 dims; kGroups groups of threads take the parts in turn and are added up at the end, in
// an order that depends on the parts' number alone: the same bits on every run.
//   Many tokens (two or three parts each): a block per boundary between two blocks and four heads, one group
//   of 128 threads a head.
//   Few tokens (under a quarter of the blocks; one may have a part of every block): a block per token and head,
//   four groups.  Under 8 tokens four blocks a head, each a quarter of the dims, eight groups.  A block that
//   finds nothing to join costs its launch: 9664 of them about as much as the joining.
//   The rule looks at the number of tokens alone.  One request of 16384 rows among short ones, which has a part
//   of nearly every block: 26 us for 37 tokens (by token), 36 us for 38 (by boundary: its parts one after another);
//   64 requests of 320 rows: 23 us (by boundary).
constexpr int kMaxParts = 256;
template <bool kBf16, bool kByToken, int kGroups, int kHeads, int kDimBlocks>
__global__ void __launch_bounds__(kGroups * kHeads * kKv4Dim / 4 / kDimBlocks)
    kv4_combine_kernel(const int4* __restrict__ parts_of, int blocks, const float* __restrict__ part,
                       const float* __restrict__ stat, uint16_t* out, float* lse) {
  constexpr int kLane4 = kKv4Dim / 4 / kDimBlocks, kTeam = kGroups * kLane4;
  static_assert(kTeam >= 32 && (kHeads == 1 || kGroups == 1), "a team's first warp takes its statistics");
  __shared__ float weight[kHeads][kMaxParts], inv_s[kHeads];
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
  if (tid < 32) {
    float mx = -INFINITY, r = 0.f, l = 0.f;
    for (int k = tid; k < n; k += 32) mx = fmaxf(mx, stat[part_no(k) * kStatFloats + 2 * kHq + h]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    for (int k = tid; k < n; k += 32) {
      const float* st = stat + part_no(k) * kStatFloats + h;
      const float m = st[2 * kHq];
      const float f = mx == -INFINITY ? 1.f : exp2f(m - mx);  // without a maximum all is 0 (or NaN)
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
      inv_s[team] = r == 0.f ? 0.f : 1.f / r;
      if (lse && blockIdx.z == 0)
        lse[(int64_t)at.x * kHq + h] =
            l == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx) + (log2f(l) - kWeightLog2)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  const int group = tid / kLane4, lane4 = tid % kLane4, x = blockIdx.z * kLane4 + lane4;
  const float4* src = reinterpret_cast<const float4*>(part + h * kKv4Dim) + x;
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
  const float inv = inv_s[team];
  const uint32_t lo = pack16<kBf16>(acc.x * inv, acc.y * inv), hi = pack16<kBf16>(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(out + ((int64_t)at.x * kHq + h) * kKv4Dim + 4 * x) = make_uint2(lo, hi);
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
size_t kv4_attn_workspace_bytes(int T, int max_rows) {
  if (max_rows <= kRows) return kHeadBytes;
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
      const int4* po = p.parts_of;
      const float *pp = p.part, *ps = p.stat;
      cudaError_t e;
      if (4 * p.T < grid && p.T < 8)  // few tokens: four blocks a head fill more of the GPU
        e = launch_pdl(kv4_combine_kernel<kBf16, true, 8, 1, 4>, dim3(p.T, kHq, 4), dim3(256), 0, stream, po, grid, pp,
                       ps, p.out, p.lse);
      else if (4 * p.T < grid)
        e = launch_pdl(kv4_combine_kernel<kBf16, true, 4, 1, 1>, dim3(p.T, kHq), dim3(512), 0, stream, po, grid, pp, ps,
                       p.out, p.lse);
      else
        e = launch_pdl(kv4_combine_kernel<kBf16, false, 1, 4, 1>, dim3(grid - 1, kHq / 4), dim3(512), 0, stream, po,
                       grid, pp, ps, p.out, p.lse);
      if (e != cudaSuccess) return DS4X_ERR_CUDA;
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
                      out,    lse,                        need > 0 ? workspace : nullptr};
  return call_end(launch_kv4_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
