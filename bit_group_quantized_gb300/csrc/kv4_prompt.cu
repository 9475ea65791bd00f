// kv4_prompt.cu — attention over the 4-bit cache for many query rows a
// sequence (whole prompts, chunks of one, many drafted tokens): a dense
// contraction, on tcgen05.
//
// A unit is one key head of one sequence with kRows = 128 * NQ columns (a
// column being one (query row, query head) pair that shares the key head), as
// NQ tiles of 128 accumulator rows. Per 128 tokens:
//   S = Q K^T   both fp16 in shared memory, S fp32 in tensor memory. K's operand is (code - 8) * scale,
//               which fp16 holds exactly (for scales from 2^-17 on, or 2^-17 of a shifted block's); what is left of a key, bias + 8 * scale a group, is one more
//               step of 16 columns: (bias, bias, scale, scale) a group against the query's group sum in
//               two parts, and 8 times those. With code * scale + bias rounded to fp16 the logarithm of
//               the sum was 1.2e-6 off (relative, 24 sequences of up to 9000 tokens, head dim 256), so
//               it is 8e-8, for 3 % of the time;
//   P = exp2(S c - m), fp16, written over S in tensor memory;
//   O += P V    P from tensor memory, V fp16 in shared memory, O fp32. P and V are each rounded to fp16 once: half a step
//               is 2^-12, a sixteenth of the bf16 output's, of random sign over the tokens; the sum of P is fp32.
// The warps are specialised: eight dequantise K and V (a thread takes a token: its codes
// come by cp.async a tile ahead, V's value = code * scale + bias rounded to fp16 once,
// stored in the 128-byte swizzled layout: K as the K-major, V as the MN-major
// operand), four for each tile of rows do the softmax (a thread owns a row: its
// maximum and sum need no shuffles), and bring the next unit's queries while the last
// product runs, one warp issues the MMAs. With two row tiles the
// tensor cores multiply one while the other's softmax runs; with one (head dim 256,
// whose O fills tensor memory) S is double-buffered.
// What bounds it: a tile's chain of scores, softmax and product, which two row tiles fill by turns, and beside it shared
// memory, which the matrix instructions read at its full rate while they take Q and K from it (a tile of 2 x 128 rows
// takes 3600 cycles, of which the matrix instructions take 2200). 4096 tokens causal, 32 heads of 128 over 8: 154 us,
// 892 TFLOP/s; three chunks of 700 to 1100 rows behind up to 16000 tokens: 318 us, 1140 TFLOP/s (58 % of the matrix rate
// measured with a library product); 24 sequences of five rows, 16 heads of 256 over 2: 44 us, where dequantisation has
// too few rows to serve (5000 cycles a tile).
// P refers to 2^-7 of a row's maximum, which is raised, and O rescaled, only where
// scores pass it by 2^8: P then stays below 2^15, and a tail of tokens 2^-30 below the first one is still there. (Raised
// at 2^6, for two places more: 4096 tokens causal 166 us.)
//
// Half precision's range: queries are scaled by a power of two per row, K by
// one per 32 tokens where it leaves [2^-8, 2^15) (else none), or one a token where one for all would lose some; the softmax
// undoes it in the scores' factors. A group of 64 columns of V is
// scaled by one of three powers of two per 32 tokens, the unit of those columns of O. Tokens that it does not fit (far smaller or
// larger than the others' values) and blocks of other units than O's are left out of the product, and their softmax thread adds p V
// in fp32, slowly: no row's result depends on the size of values that it does not see, or of another group's. This and the care for
// very large scores cost ordinary values 2 to 4 % (4096 tokens causal: 154 us, 147.6 with one exponent for all that a row had met, which
// lost small values beside large ones; with the functions of the rare paths inlined it was 1 % more). In 4096 tokens, values of 2^-24 in one group of two: 261 us; in one token of
// 32: 1.8 ms; values of 2^-40 throughout, which no unit fits: 15 ms.
// A key or value pair that is not finite is stored as zeros, and the rows that see it are made NaN at the end.
//
// All (unit, key head, 128 tokens) triples form one list, which k_prompt_plan lays out from
// the lengths on the device; every CTA takes an equal, contiguous share, and units cut by a
// share are joined by k_prompt_join, in CTA order (the same bits every time).
// Every wait is bounded: on expiry the status word is set to BGQ_ERR_TIMEOUT and all
// later waits fall through, so the kernel ends by itself.
#include <cuda_fp16.h>

#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"
#include "kv4_seen.h"
#include "tc.cuh"

namespace bgq {

constexpr int kPrThreads = 640;  // warp 0: MMAs, 4-7: K's dequantisation, 8-11: V's, 12-15: rows 0-127, 16-19: rows 128-255
constexpr int kPrRegs = 96;      // of a thread at launch: 65536 / 640, in eights
constexpr int kPrTok = 128;      // tokens of a tile
constexpr long long kPrTimeoutNs = 1000000000ll;
constexpr int kPlanThreads = 256;
constexpr int kPlanSeqs = 4096;
// What bringing a unit's queries and writing its rows costs, in tiles: CTAs with many short units take fewer tiles (4096
// tokens causal: 157, 147, 145 us with 2, 3, 4; 24 sequences of five rows, which 4 serves worse: 42.1, 40.8, 43.4).
constexpr int kUnitCost = 3;
constexpr int kPanel = 128 * 128;  // bytes of an operand panel: 64 columns in 128-byte rows, 128-byte swizzle, 128 rows
constexpr int kExtra = 128 * 32;   // bytes of an operand's 16 extra columns: 8 x 8 cores, unswizzled

template <int D>
struct Prompt {
  static constexpr int G = D / kGroup;
  static constexpr int NQ = D == 256 ? 1 : 2;
  static constexpr int kRows = 128 * NQ;
  // K and V are held as rings of stages of some 64-column panels: two tiles of them, but at head dim 256, where a tile of
  // Q alone is 64 KB, three quarters of a K tile and one V tile.
  static constexpr int KP = D == 256 ? 1 : G, KST = D == 256 ? 3 : 2;
  static constexpr int VP = D == 256 ? 2 : G, VST = 2;
  static constexpr int kTile = kRows / NQ * D * 2;  // bytes of a Q tile
  static constexpr int kRaw = kPrTok * D / 2;       // bytes of a tile's K or V codes
  static constexpr int KE = G / KP > 1 ? 1 : KST;   // extra-column blocks of K held: each goes with its tile's first stage
  // more than half an SM's, so that no second CTA comes to wait for this one's tensor memory
  static constexpr int kNeed = 1024 + NQ * kTile + (KST * KP + VST * VP) * kPanel + 2 * kRaw + (NQ + KE) * kExtra;
  static constexpr int kSmem = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
  static constexpr int kOwn = 232448 - kSmem;  // bytes left for PrShared
  static constexpr int kSlot = 128 * D + 256;  // floats of a part: O by 4 columns and row, then m, then l
  // registers of a softmax, dequantisation and other warpgroup's threads: together at most the launch's
  static constexpr int kRegSoft = D == 256 ? 176 : 136, kRegDeq = D == 256 ? 104 : 80, kRegRest = 40;
  static_assert(NQ * kRegSoft + 2 * kRegDeq + (3 - NQ) * kRegRest <= 5 * kPrRegs, "more registers than the launch has");
};

// A unit: its sequence and row tile, its tokens' first and how many tiles of them, and the sequence's span.
struct __align__(16) PrUnit {
  int b, rt, tiles, begin;
  Span sp;
};
// n / (q_heads / kv_heads), n below 2^31: by ceil(2^64 / .), whose excess n times stays below 2^64.
__device__ __forceinline__ int pr_by_group(const AttnArgs& a, int n) {
  return a.group_inv ? (int)__umul64hi((unsigned long long)n, a.group_inv) : n;
}
// A sequence's row tiles, and the tokens of one of them.
__device__ __forceinline__ int pr_row_tiles(const AttnArgs& a, const Span& sp, int rows_unit) {
  return (min(sp.q_len, a.v.rows) * a.group + rows_unit - 1) / rows_unit;
}
__device__ __forceinline__ void pr_tokens(const AttnArgs& a, PrUnit& un, int rows_unit) {
  const int pos0 = un.sp.kv_len - un.sp.q_len;
  const int j0 = pr_by_group(a, un.rt * rows_unit);
  const int j1 = min(un.sp.q_len - 1, pr_by_group(a, un.rt * rows_unit + rows_unit - 1));
  un.begin = min(kv4_first_seen(pos0 + j0, a.window), un.sp.held) / 16 * 16;  // 16 tokens lie in one page
  const int end = kv4_end_seen(pos0 + j1, un.sp.kv_len, un.sp.held, a.causal);
  un.tiles = max(1, (end - un.begin + kPrTok - 1) / kPrTok);  // at least one: rows that see no token are written too
}
struct PrPlan {  // at the start of the workspace, behind the control block
  int units, pad;
  long long sum;  // cost of all units, for one key head
};

// A unit that CTA c0 began and did not end: CTAs c0 .. c1 have parts of it.
struct __align__(16) PrCut {
  int c0, c1;  // c1 -1: none
  int first, col0, cols;  // the sequence's first row, the unit's first column, the sequence's columns
  int h, pad[2];
};

struct PrWs {
  Ctrl* ctrl;
  PrPlan* plan;
  PrCut* cuts;        // [ncut]: by unit and key head, or where CTAs are fewer than those, by c0
  PrUnit* units;      // [cap]
  long long* prefix;  // [cap] cost of the units before a unit
  float* part;        // [grid][2][NQ][kSlot]
  int cap, ncut;
  size_t bytes;
};

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static PrWs carve_prompt(void* ws, int batch, int rows, int q_heads, int kv_heads, int d, int grid) {
  char* p = static_cast<char*>(ws);
  const int nq = d == 256 ? 1 : 2, group = q_heads / kv_heads;
  size_t at = 0;
  auto take = [&](size_t n) {
    char* r = p ? p + at : nullptr;
    at += up256(n);
    return r;
  };
  PrWs w;
  w.cap = (int)((long long)rows * group / (128 * nq)) + batch + 1;
  w.ncut = (int)std::min((long long)grid, (long long)w.cap * kv_heads);
  w.ctrl = reinterpret_cast<Ctrl*>(take(kAttnHead));
  w.plan = reinterpret_cast<PrPlan*>(take(sizeof(PrPlan)));
  w.cuts = reinterpret_cast<PrCut*>(take((size_t)w.ncut * sizeof(PrCut)));
  w.units = reinterpret_cast<PrUnit*>(take((size_t)w.cap * sizeof(PrUnit)));
  w.prefix = reinterpret_cast<long long*>(take((size_t)w.cap * 8));
  w.part = reinterpret_cast<float*>(take((size_t)grid * 2 * nq * (128 * d + 256) * 4));
  w.bytes = at;
  return w;
}

// ---------------------------------------------------------------------------
// The list: one CTA; row tiles per sequence, then tiles per unit.
// ---------------------------------------------------------------------------
__device__ __forceinline__ long long plan_scan(long long v, long long* warp_sum, long long& total) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const long long n = warp_sum[w];
    if (w < warp) before += n;
    total += n;
  }
  __syncthreads();
  return v + before - own;
}

__global__ void __launch_bounds__(kPlanThreads) k_prompt_plan(const __grid_constant__ AttnArgs a, PrWs w, int rows_unit) {
  __shared__ int first[kPlanSeqs + 1];  // units before a sequence
  __shared__ long long warp_sum[kPlanThreads / 32];
  pdl_wait();
  pdl_trigger();
  for (int c = threadIdx.x; c < w.ncut; c += kPlanThreads) w.cuts[c].c1 = -1;
  const int per = (a.v.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min((int)threadIdx.x * per, a.v.batch), b1 = min(b0 + per, a.v.batch);
  int own = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = pr_row_tiles(a, kv4_span(a.v, b), rows_unit);
    first[b] = own;  // so far within the thread's sequences
    own += n;
  }
  long long total;
  const int at = (int)plan_scan(own, warp_sum, total);
  for (int b = b0; b < b1; ++b) first[b] += at;
  const int units = (int)min(total, (long long)w.cap);  // never more, unless the rows of sequences overlap
  __syncthreads();
  long long sum = 0;
  for (int base = 0; base < units; base += kPlanThreads) {
    const int u = base + threadIdx.x;
    PrUnit un = {};
    if (u < units) {
      int lo = 0, hi = a.v.batch;  // the last sequence whose first unit is at or before u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u) lo = mid; else hi = mid;
      }
      un.sp = kv4_span(a.v, lo);
      un.b = lo;
      un.rt = u - first[lo];
      pr_tokens(a, un, rows_unit);
    }
    long long chunk;
    const int cost = u < units ? un.tiles + kUnitCost : 0;
    const long long pre = plan_scan(cost, warp_sum, chunk);
    if (u < units) {
      w.units[u] = un;
      w.prefix[u] = sum + pre;
    }
    sum += chunk;
  }
  if (threadIdx.x == 0) {
    w.plan->units = units;
    w.plan->sum = sum;
  }
}

// ---------------------------------------------------------------------------
// Tensor memory in 32 columns of the warp's 32 lanes, and waits
// ---------------------------------------------------------------------------
#define BGQ_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define BGQ_U8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
#define BGQ_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void pr_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : BGQ_R8(r, 0), BGQ_R8(r, 8), BGQ_R8(r, 16), BGQ_R8(r, 24)
      : "r"(t));
}
// Loads done: the registers pass through, so that nothing that uses them moves ahead.
__device__ __forceinline__ void pr_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(r, 0), BGQ_U8(r, 8), BGQ_U8(r, 16), BGQ_U8(r, 24)::"memory");
}
__device__ __forceinline__ void pr_st16(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      BGQ_I8(r, 0), BGQ_I8(r, 8)
      : "memory");
}
__device__ __forceinline__ void pr_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pr_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pr_bf2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// O of the warp's rows times f (a row's own), eight columns at a time: rare, and few registers.
template <int D>
__device__ __forceinline__ void pr_scale(uint32_t t, float f) {
#pragma unroll 1
  for (int d = 0; d < D; d += 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BGQ_R8(r, 0) : "r"(t + d));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(r, 0)::"memory");
#pragma unroll
    for (int x = 0; x < 8; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * f);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t + d), BGQ_I8(r, 0) : "memory");
  }
}
// 32 tokens' probabilities of the warp's rows times f.
__device__ __forceinline__ void pr_scale_p(uint32_t t, float f) {
  const uint32_t f2 = pr_half2(f, f);
#pragma unroll 1
  for (int d = 0; d < 16; d += 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BGQ_R8(r, 0) : "r"(t + d));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(r, 0)::"memory");
#pragma unroll
    for (int x = 0; x < 8; ++x) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r[x]) : "r"(r[x]), "r"(f2));
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t + d), BGQ_I8(r, 0) : "memory");
  }
}
// A score's factor: finite, so that zero times it stays zero, and not below normal numbers, so that -infinity times it stays that.
__device__ __forceinline__ float pr_factor(float f) { return fminf(fmaxf(f, 0x1p-126f), 3e38f); }
// 32 scores of the warp's rows times f, and the powers of two of their tokens' keys where those are given.
__device__ __noinline__ void pr_scale_s(uint32_t t, float f, const int8_t* ke) {
#pragma unroll 1
  for (int d = 0; d < 32; d += 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BGQ_R8(r, 0) : "r"(t + d));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(r, 0)::"memory");
#pragma unroll
    for (int x = 0; x < 8; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * (ke ? pr_factor(f * exp2i(ke[d + x])) : f));
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t + d), BGQ_I8(r, 0) : "memory");
  }
  pr_wait_st();
}
// Lanes m apart: the lower one's b for the upper one's a.
__device__ __forceinline__ void pr_swap(uint4& a, uint4& b, int m, int lane) {
  const bool upper = lane & m;
  auto one = [&](uint32_t& x, uint32_t& y) {
    const uint32_t got = __shfl_xor_sync(kFull, upper ? x : y, m);
    if (upper) x = got; else y = got;
  };
  one(a.x, b.x);
  one(a.y, b.y);
  one(a.z, b.z);
  one(a.w, b.w);
}
// Two fp32 values in one register pair, one instruction for both.
__device__ __forceinline__ uint64_t pr_pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void pr_split(uint64_t d, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t pr_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pr_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Registers of a warpgroup's threads, from the launch's.
template <int N>
__device__ __forceinline__ void pr_regs() {
  if (N > kPrRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if (N < kPrRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void pr_wait_loop(uint64_t* m, uint32_t parity, volatile int* fail) {
  const unsigned long long t0 = tc_time();
  while (!*fail && !tc_mbar_try_suspend(m, parity))
    if ((long long)(tc_time() - t0) > kPrTimeoutNs) *fail = 1;
}
__device__ __forceinline__ void pr_wait(uint64_t* m, uint32_t parity, volatile int* fail) {
  if (!tc_mbar_try(m, parity)) pr_wait_loop(m, parity, fail);
}

// Operand tiles: panels of 64 columns.
__device__ __forceinline__ uint64_t pr_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
__device__ __forceinline__ uint64_t pr_extra_desc(uint32_t saddr) {  // cores: 128 bytes to the next 8 columns, 256 to the next 8 rows
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(256 >> 4) << 32 | 1ull << 46;
}
__device__ __forceinline__ constexpr uint32_t pr_idesc(int n, bool b_mn) {  // fp16 x fp16 -> fp32, M = 128
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// Issued by the lane that has `lead`; the whole warp runs the code around them, so that addresses and descriptors stay
// in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* m, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc_smem(m)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pr_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Eight codes of a word as fp16 values (64 + code + off) * s + b, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 pr_values(uint32_t w, uint32_t off, uint32_t s2, uint32_t b2) {
  uint32_t o[4];
  const uint32_t r[4] = {w << 4, w, w >> 4, w >> 8};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 64 + code under the exponent of 64; exact, then one rounding
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(r[i]), "r"(0x00F000F0u), "r"(0x54005400u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(off));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(v), "r"(s2), "r"(b2));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A group of 64 columns of 32 tokens' values is held in fp16 divided by 2^E, one of three E by a rule on the pairs alone: a token
// fits where its 16 |s| + |b| (which no value of the group passes) is zero or in [2^(E - 8), 2^(E + 15)); there fp16 keeps
// 2^-17 of it, whatever the sizes beside it. The usual one is for 2^-14 to 2^9. E by two bits, of which a word has one pair a group:
constexpr int kVe = -6, kVeStep = 20;  // 0: kVe; 1: kVe - 20, for 2^-34 to 2^-11; 2: kVe + 20, for 2^6 to 2^29;
constexpr uint32_t kVeNone = 3;        // no token has a value but zero that any E fits
__device__ __forceinline__ int pr_unit(uint32_t word, int g) {
  const uint32_t k = word >> 2 * g & 3;
  return kVe + (k == 1 ? -kVeStep : k == 2 ? kVeStep : 0);
}
// What the softmax needs to know of 32 tokens. `odd` is zero for tokens all there, in half precision's range and
// finite: then nothing else is looked at.
struct __align__(16) PrMeta {
  float kf;        // 2^E of the keys: a score's factor; 0: each token has its own
  uint32_t ve;     // E of the values' groups
  uint32_t gap;    // tokens that are absent
  uint32_t bad;    // whether any pair is not finite (then the masks below)
  uint32_t side[4];  // by group: tokens whose values E does not fit, zeros in V's operand; the softmax adds them by itself
};
constexpr float kPrMost = 15.f, kPrLift = 7.f;  // log2 of the largest P; of P at a maximum that was raised
// A fused S c - m is as far from its value at the maximum as the product's rounding: 2^-4 at 2^20, but more than any exponent at
// 2^31. From here on a row's scores are multiplied and rounded first, as the maximum is.
constexpr float kPrLarge = 0x1p20f;
constexpr int kMetaTiles = 4;  // tiles whose notes are kept: the copies run at most two ahead of the softmax

template <int D>
struct PrShared {
  static constexpr int G = D / kGroup, NQ = Prompt<D>::NQ, KST = Prompt<D>::KST, VST = Prompt<D>::VST;
  uint64_t k_full[KST], k_free[KST], v_full[VST], v_free[VST];
  uint64_t q_full[NQ], s_full[2], p_full[2], o_full[NQ], drain, pv_done;
  PrMeta meta[kMetaTiles][4];
  __align__(16) uint32_t odd[kMetaTiles][4];
  uint32_t kbad[kMetaTiles][4], vbad[kMetaTiles][4][G];
  int8_t ke[kMetaTiles][kPrTok];  // tokens' E, where a block has no common one
  uint32_t tmem;
  int fail;
};

// A CTA's share of the list, unit by unit. A unit takes kUnitCost places of the list, then one for each tile; the
// CTA whose share holds a tile's place does the tile. Within a sequence the next unit is worked out, not loaded.
template <int D>
struct PrWalk {
  long long x, x1;  // the first tile's place of the unit in hand; the share's end
  int h, u, i0, i1, n0;  // tiles i0 .. i1 - 1 of unit u; tiles of the share before them
  PrUnit un;
  __device__ __forceinline__ void get(const PrWs& w) {
    const int4* p = reinterpret_cast<const int4*>(w.units + u);
    const int4 a = p[0], b = p[1];
    un = PrUnit{a.x, a.y, a.z, a.w, {b.x, b.y, b.z, b.w}};
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const PrWs& w, long long x0, long long x1_, long long sum, int units) {
    x1 = x1_;
    h = (int)(x0 / sum);
    const long long y = x0 - h * sum;
    int lo = 0, hi = units;  // the last unit that starts at or before y
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (w.prefix[mid] <= y) lo = mid; else hi = mid;
    }
    u = lo;
    get(w);
    n0 = 0;
    x = x0 - y + w.prefix[u] + kUnitCost;
    i0 = (int)max(0ll, x0 - x);
    i1 = (int)min((long long)un.tiles, x1 - x);
    if (i1 <= i0) {
      i0 = i1 = un.tiles;  // nothing of this unit
      next(a, w, units);
    }
  }
  __device__ __forceinline__ bool live() const { return i1 > i0; }
  __device__ __forceinline__ void next(const AttnArgs& a, const PrWs& w, int units) {
    x += un.tiles + kUnitCost;
    n0 += i1 - i0;
    i0 = i1 = 0;
    if (x >= x1) return;
    const bool same = un.rt + 1 < pr_row_tiles(a, un.sp, Prompt<D>::kRows);
    if (++u == units) {
      u = 0;
      ++h;
    }
    if (same && u > 0) {
      ++un.rt;
      pr_tokens(a, un, Prompt<D>::kRows);
    } else {
      get(w);
    }
    i1 = (int)min((long long)un.tiles, x1 - x);
  }
};

// ---------------------------------------------------------------------------
// Dequantisation: four warps for K, four for V, a token a thread.
// ---------------------------------------------------------------------------
// Codes come 16 bytes a lane, 16 tokens (of one page) at a time, into a buffer whose 16-byte pieces are
// swizzled so that 8 threads that read a piece each of their own token's row hit different banks.
template <int D>
__device__ __forceinline__ int pr_raw(int tok, int ch) {
  if (D == 64) return (tok >> 2) * 128 + (tok & 3) * 32 + ((ch ^ (tok >> 2)) & 1) * 16;
  if (D == 128) return (tok >> 1) * 128 + (tok & 1) * 64 + ((ch ^ (tok >> 1)) & 3) * 16;
  return tok * 128 + ((ch ^ tok) & 7) * 16;
}
__device__ __forceinline__ void pr_cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// The codes of the warp's 32 tokens. Lanes 0 and 16 hold in `base` the row of the first of their 16 tokens, which lie in
// one page; -1: absent, zeros.
template <int D>
__device__ __forceinline__ void pr_fetch(uint32_t raw, const uint32_t* q, long long base, int lane) {
  constexpr int CPT = D / 32;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const long long row = __shfl_sync(kFull, base, 16 * m);
    const char* src = reinterpret_cast<const char*>(q) + (row < 0 ? 0 : row) * (D / 2) + lane * 16;
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) {
      const int id = i * 32 + lane;
      pr_cp16(raw + m * (8 * D) + pr_raw<D>(id / CPT, id % CPT), src + i * 512, row >= 0);
    }
  }
}
template <int D>
__device__ __forceinline__ void pr_pairs(uint32_t (&sb)[D / kGroup], const uint16_t* p, long long row) {
#pragma unroll
  for (int i = 0; i < D / kGroup; ++i) sb[i] = 0;
  if (row >= 0) {
    const uint32_t* ss = reinterpret_cast<const uint32_t*>(p) + row * (D / kGroup);
#pragma unroll
    for (int i = 0; i < D / kGroup; ++i) sb[i] = ss[i];
  }
}
// Whether any of the warp's 32 tokens has a group whose 16 |s| + |b|, which none of its values passes, is outside [low, 2^23 low),
// low given as bits. A zero, an infinity or a NaN is outside too.
template <int D>
__device__ __forceinline__ bool pr_odd(const uint32_t (&sb)[D / kGroup], uint32_t low) {
  bool odd = false;
#pragma unroll
  for (int g = 0; g < D / kGroup; ++g) odd |= __float_as_uint(fmaf(16.f, fabsf(bf16lo(sb[g])), fabsf(bf16hi(sb[g])))) - low >= 23u << 23;
  return __any_sync(kFull, odd);
}
constexpr uint32_t kKeyLow = (uint32_t)(-8 + 127) << 23;        // keys: 2^-8 to 2^15 as they are
constexpr uint32_t kValueLow = (uint32_t)(kVe - 8 + 127) << 23;
// The same of a group, as bits; 0 where the pair is not finite.
__device__ __forceinline__ uint32_t pr_top(uint32_t sb, bool& fin) {
  const float s = fabsf(bf16lo(sb)), b = fabsf(bf16hi(sb));
  fin = s < INFINITY && b < INFINITY;
  return fin ? __float_as_uint(fminf(fmaf(16.f, s, b), 3e38f)) : 0u;
}
// What is divided out of the lane's token of odd keys: the exponent E that brings the block's largest into [2^13, 2^14), or, for
// tokens that it would put below 2^-6, the token's own one; `mix`: some have their own. `any`, `bad`: tokens whose pair (of which group) is not
// finite.
template <int D>
__device__ __forceinline__ int pr_key_range(const uint32_t (&sb)[D / kGroup], bool& mix, uint32_t& any, uint32_t (&bad)[D / kGroup]) {
  uint32_t own = 0;
#pragma unroll
  for (int g = 0; g < D / kGroup; ++g) {
    bool fin;
    own = max(own, pr_top(sb[g], fin));
    bad[g] = __ballot_sync(kFull, !fin);
    any |= bad[g];
  }
  if (!__any_sync(kFull, own && own - kKeyLow >= 23u << 23)) return 0;
  const int top = (int)(__reduce_max_sync(kFull, own) >> 23), it = (int)(own >> 23);
  const bool apart = own && it < top - 19;
  mix = __any_sync(kFull, apart);
  return min(max((apart ? it : top) - 127 - 13, -120), 120);
}
// E of odd values' groups, each the one of three that fits most of the block's tokens. `side`: by group, the tokens that it does not fit.
template <int D>
__device__ __forceinline__ uint32_t pr_value_range(const uint32_t (&sb)[D / kGroup], uint32_t (&side)[D / kGroup], uint32_t& any,
                                                   uint32_t (&bad)[D / kGroup]) {
  uint32_t word = 0;
#pragma unroll
  for (int g = 0; g < D / kGroup; ++g) {
    bool fin;
    const uint32_t top = pr_top(sb[g], fin);
    bad[g] = __ballot_sync(kFull, !fin);
    any |= bad[g];
    uint32_t f = 0, k = kVeNone;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t low = kValueLow + (uint32_t)((i == 1 ? -kVeStep : i == 2 ? kVeStep : 0) * (1 << 23));
      const uint32_t fits = __ballot_sync(kFull, top && top - low < 23u << 23);
      if (__popc(fits) > __popc(f)) {
        f = fits;
        k = i;
      }
    }
    side[g] = __ballot_sync(kFull, top != 0) & ~f;
    word |= k << 2 * g;
  }
  return word;
}
// O of the warp's rows in other units: rare.
template <int D>
__device__ __noinline__ void pr_rescale(uint32_t t, uint32_t from, uint32_t to) {
#pragma unroll 1
  for (int d = 0; d < D; d += 8) {
    const float f = exp2i(pr_unit(from, d / kGroup) - pr_unit(to, d / kGroup));  // at most 2^40 either way, which fp32 has to spare
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BGQ_R8(r, 0) : "r"(t + d));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(r, 0)::"memory");
#pragma unroll
    for (int x = 0; x < 8; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * f);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t + d), BGQ_I8(r, 0) : "memory");
  }
  pr_wait_st();
}
// Values that V's operand leaves out. They are summed in fp32 from their codes, in units of 2^15 (as P may be that large), in the place
// for a part that the CTA's segment has (whole units have the one that only the share's last unit writes): `sums`, the row's columns
// four by four, 512 floats apart, and, where a part has its maximum, what their probabilities refer to.
template <int D>
__device__ __forceinline__ float* pr_side_max(float* sums, int r) { return sums - r * 4 + 128 * D + r; }
struct PrMask4 {
  uint32_t of[4];
};
// Adds some of a block's tokens, by group, which are all there. `score` is the row's scores of the block in tensor memory.
template <int D>
__device__ __noinline__ void pr_side(const AttnArgs& a, int row0, int head, int t, PrMask4 side, uint32_t see, uint32_t score, float ck, float m,
                                     float* sums, int r, bool more) {
  const int lane = threadIdx.x & 31;
  int b = row0;
  if (a.v.q_start) {  // the last sequence that starts at or before the row
    int lo = 0, hi = a.v.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.v.q_start[mid] <= row0) lo = mid; else hi = mid;
    }
    b = lo;
  }
  b = __shfl_sync(kFull, b, 0);
  const int h = __shfl_sync(kFull, pr_by_group(a, head), 0);
  uint32_t some = 0;
#pragma unroll
  for (int g = 0; g < D / kGroup; ++g) some |= side.of[g];
  const int page = some >> lane & 1 ? kv4_page(a.v, b, t + lane) : -1;
  const long long mine = page < 0 ? 0 : ((long long)page * a.c.kv_heads + h) * a.c.page_size + (t + lane) % a.c.page_size;  // the lane's token
  const float mm = (m == -INFINITY ? 0.f : m) + kPrMost, was = more ? *pr_side_max<D>(sums, r) : m, f = was == m ? 1.f : pr_ex2(was - m);
  *pr_side_max<D>(sums, r) = m;
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    float4* const at = reinterpret_cast<float4*>(sums + d / 4 * 512);
    float acc[32];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 v = more ? at[x * 128] : make_float4(0.f, 0.f, 0.f, 0.f);
      acc[4 * x] = v.x * f; acc[4 * x + 1] = v.y * f; acc[4 * x + 2] = v.z * f; acc[4 * x + 3] = v.w * f;
    }
#pragma unroll 1
    for (uint32_t left = side.of[d / kGroup]; left; left &= left - 1) {
      const int x = __ffs(left) - 1;
      const long long row = __shfl_sync(kFull, mine, x);
      uint32_t s;
      __syncwarp();
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(s) : "r"(score + x));
      const uint4 q = *reinterpret_cast<const uint4*>(a.c.v_q + row * (D / 8) + d / 8);
      const uint32_t sb = reinterpret_cast<const uint32_t*>(a.c.v_sb)[row * (D / kGroup) + d / kGroup], w[4] = {q.x, q.y, q.z, q.w};
      asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(s)::"memory");
      const float p = see >> x & 1 ? pr_ex2(fmaf(__uint_as_float(s), ck, -mm)) : 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float v = fmaf(p, fmaf((float)(w[k / 8] >> k % 8 * 4 & 15u), bf16lo(sb), bf16hi(sb)), acc[k]);
        acc[k] = p == 0.f ? acc[k] : v;  // a hidden token adds nothing, whatever it holds
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) at[x * 128] = make_float4(acc[4 * x], acc[4 * x + 1], acc[4 * x + 2], acc[4 * x + 3]);
  }
}
// Adds the sums to O, whose columns come as 0 4 1 5 2 6 3 7. Returns whether they are so large that O's unit is 2^60 from here on.
template <int D>
__device__ __noinline__ bool pr_side_add(float* sums, int r, uint32_t o_t, float m, uint32_t units) {
  const float was = *pr_side_max<D>(sums, r);
  const float f = was == m ? 1.f : pr_ex2(was - m);
  float top = 0.f;
#pragma unroll 1
  for (int d = 0; d < D; d += 4) {
    const float4 v = *reinterpret_cast<const float4*>(sums + d / 4 * 512);
    top = fmaxf(fmaxf(fmaxf(top, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
  }
  const bool large = top * f > 0x1p30f;
#pragma unroll 1
  for (int d = 0; d < D; d += 8) {
    const int e = pr_unit(units, d / kGroup), unit = large ? 60 : e;
    const float fo = exp2i(e - unit), fs = exp2i((int)kPrMost - unit);
    const float4 lo = *reinterpret_cast<const float4*>(sums + d / 4 * 512), hi = *reinterpret_cast<const float4*>(sums + (d / 4 + 1) * 512);
    const float v[8] = {lo.x, hi.x, lo.y, hi.y, lo.z, hi.z, lo.w, hi.w};
    uint32_t o[8];
    __syncwarp();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BGQ_R8(o, 0) : "r"(o_t + d));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BGQ_U8(o, 0)::"memory");
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(fmaf(v[x] * f, fs, __uint_as_float(o[x]) * fo));
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(o_t + d), BGQ_I8(o, 0) : "memory");
  }
  pr_wait_st();
  return large;
}
// A token's values of group g into its row of a panel.
template <int D>
__device__ __forceinline__ void pr_store(const unsigned char* raw, int g, uint32_t off, uint32_t s2, uint32_t b2, unsigned char* panel, int t) {
  unsigned char* row = panel + t * 128;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q = *reinterpret_cast<const uint4*>(raw + pr_raw<D>(t & 31, g * 2 + h));
    *reinterpret_cast<uint4*>(row + (((h * 4) ^ (t & 7)) * 16)) = pr_values(q.x, off, s2, b2);
    *reinterpret_cast<uint4*>(row + (((h * 4 + 1) ^ (t & 7)) * 16)) = pr_values(q.y, off, s2, b2);
    *reinterpret_cast<uint4*>(row + (((h * 4 + 2) ^ (t & 7)) * 16)) = pr_values(q.z, off, s2, b2);
    *reinterpret_cast<uint4*>(row + (((h * 4 + 3) ^ (t & 7)) * 16)) = pr_values(q.w, off, s2, b2);
  }
}
// Byte of row t, columns 8 c of an operand's extra columns.
__device__ __forceinline__ int pr_extra(int t, int c) { return (t >> 3) * 256 + c * 128 + (t & 7) * 16; }

// The query row of a softmax thread in a unit.
struct PrRowOf {
  int row, head, pos;
  bool own, ok;  // a row of the unit; and one that may be read and written
};
template <int D>
__device__ __forceinline__ PrRowOf pr_row(const AttnArgs& a, const PrWalk<D>& wk, int group, int at) {
  const Span& sp = wk.un.sp;
  const int cols = min(sp.q_len, a.v.rows) * group;  // rows * group is below 2^31
  const int col = wk.un.rt * Prompt<D>::kRows + at;
  PrRowOf r;
  r.own = col < cols;
  const int cc = r.own ? col : cols - 1;  // rows behind the last see what it sees, and are dropped
  const int j = pr_by_group(a, cc);
  r.head = wk.h * group + cc - j * group;
  r.row = sp.first + j;
  r.ok = r.own && r.row >= 0 && r.row < a.v.rows;
  r.pos = sp.kv_len - sp.q_len + j;
  return r;
}
// The warp's 32 query rows on their way into the query tile as they are (bf16), 16 bytes a lane.
template <int D>
__device__ __forceinline__ void pr_query_fetch(const AttnArgs& a, const PrRowOf& q, uint32_t tile, int r0, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes of a row, rows at a time
  const long long mine = q.ok ? (long long)q.row * a.q_stride + q.head * D : -1;
  const int ch = lane % LPR;
#pragma unroll 8
  for (int k = 0; k < 32; k += RPW) {
    const int rl = k + lane / LPR, r = r0 + rl;
    const long long at = __shfl_sync(kFull, mine, rl);
    pr_cp16(tile + (ch >> 3) * kPanel + r * 128 + (((ch & 7) ^ (r & 7)) * 16), a.q + (at < 0 ? 0 : at) + ch * 8, at >= 0);
  }
}
// (A function of its own, once a unit: inlined, the same kernel was 0.5 us slower for 4096 tokens.)
// Row r of the tile, in place: fp16 scaled by a power of two, in the codes' order 0 4 1 5 2 6 3 7; and each group's sum,
// in two parts, for the extra columns. Returns the factor of its scores.
template <int D>
__device__ __noinline__ float pr_query_scale(const AttnArgs& a, unsigned char* tile, unsigned char* extra, int r) {
  auto chunk = [&](int ch) { return reinterpret_cast<uint4*>(tile + (ch >> 3) * kPanel + r * 128 + (((ch & 7) ^ (r & 7)) * 16)); };
  uint32_t t2[4] = {};
#pragma unroll 8
  for (int n = 0; n < D / 8; ++n) {
    const uint4 v = *chunk(n);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(t2[k]) : "r"(w[k]));
  }
  uint32_t top = 0;  // the largest magnitude's bits: without their signs they order like values (NaN is passed over)
#pragma unroll
  for (int k = 0; k < 4; ++k) top = max(top, max(t2[k] & 0x7fff0000u, t2[k] << 17 >> 1));
  const int e = top && top < 0x7f800000u ? min(max((int)(top >> 23) - 130, -110), 124) : 0;
  const float up = a.scale < 0.f ? -exp2i(-e) : exp2i(-e);
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    uint2 x = {};
    if (g < D / kGroup) {
      float sum[4] = {};
      uint4 v[8];  // all loads ahead of the stores
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = *chunk(g * 8 + n);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float f[8];
        unpack_bf16x8(v[n], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= up;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] += f[k] + f[k + 4];
        *chunk(g * 8 + n) = make_uint4(pr_half2(f[0], f[4]), pr_half2(f[1], f[5]), pr_half2(f[2], f[6]), pr_half2(f[3], f[7]));
      }
      const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);  // below 2^11
      const float top = __half2float(__float2half_rn(all)), rest = all - top;
      x = make_uint2(pr_half2(top, rest), pr_half2(8.f * top, 8.f * rest));
    }
    *reinterpret_cast<uint2*>(extra + pr_extra(r, g >> 1) + (g & 1) * 8) = x;
  }
  return fminf(fabsf(a.scale) * 1.4426950408889634f * exp2i(e), 3e38f);
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) k_attn_prompt(const __grid_constant__ AttnArgs a, const __grid_constant__ PrWs w) {
  using P = Prompt<D>;
  constexpr int G = P::G, NQ = P::NQ;
  extern __shared__ unsigned char smem_raw[];
  __shared__ PrShared<D> sh;
  static_assert(sizeof(sh) <= P::kOwn, "more shared memory than a CTA can have");
  unsigned char* const smem = smem_raw + ((1024 - (tc_smem(smem_raw) & 1023)) & 1023);
  unsigned char* const q_s = smem;
  unsigned char* const k_s = q_s + NQ * P::kTile;
  unsigned char* const v_s = k_s + P::KST * P::KP * kPanel;
  unsigned char* const raw_s = v_s + P::VST * P::VP * kPanel;
  unsigned char* const qe_s = raw_s + 2 * P::kRaw;   // extra columns
  unsigned char* const ke_s = qe_s + NQ * kExtra;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const fail = &sh.fail;
  if (tid == 0) {
    for (int i = 0; i < P::KST; ++i) {
      tc_mbar_init(&sh.k_full[i], 128);
      tc_mbar_init(&sh.k_free[i]);
    }
    for (int i = 0; i < P::VST; ++i) {
      tc_mbar_init(&sh.v_full[i], 128);
      tc_mbar_init(&sh.v_free[i]);
    }
    for (int i = 0; i < NQ; ++i) {
      tc_mbar_init(&sh.q_full[i], 128);
      tc_mbar_init(&sh.o_full[i]);
    }
    for (int i = 0; i < 2; ++i) {
      tc_mbar_init(&sh.s_full[i]);
      tc_mbar_init(&sh.p_full[i], 128);
    }
    tc_mbar_init(&sh.pv_done);
    tc_mbar_init(&sh.drain);
    sh.fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  const int units = w.plan->units;
  const long long sum = w.plan->sum, total = sum * a.c.kv_heads;
  // every CTA's share holds a tile, as its length is above kUnitCost
  const long long ctas = min((long long)gridDim.x, total / (kUnitCost + 1));
  const int cta = blockIdx.x;
  const int group = a.group;
  PrWalk<D> wk;
  wk.i0 = wk.i1 = 0;
  if (cta < ctas) wk.start(a, w, total * cta / ctas, total * (cta + 1) / ctas, sum, units);

  if (warp >= 12 && warp < 12 + 4 * NQ) {
    // ---------------------------------------------------------------- softmax: a thread owns a row
    pr_regs<P::kRegSoft>();
    const int i = (warp >> 2) - 3, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const uint32_t o_t = tmem + 256 + i * D + lanes;
    uint32_t s_par = 0, o_par = 0;  // parities: s_full (bit per slot), o_full
    uint32_t pv_par = 0;
    // A unit's end runs beside the next one's first product: the next queries are brought after the last
    // probabilities (the last scores are done then), before O is waited for. The first unit follows none.
    PrWalk<D> nw = wk;
    float c2 = 0.f, c2_next = 0.f;
    unsigned char* const q_tile = q_s + i * P::kTile;
    PrRowOf rw, next_row;
    bool none = true;
    for (;;) {
      const int row = rw.row, pos = rw.pos, head = rw.head;
      const Span& sp = wk.un.sp;
      const bool own = !none && rw.own, ok = rw.ok;
      const int hi = kv4_end_seen(pos, sp.kv_len, sp.held, a.causal), lo = kv4_first_seen(pos, a.window);
      const int hi_min = __reduce_min_sync(kFull, hi), hi_max = __reduce_max_sync(kFull, hi);
      const int lo_min = __reduce_min_sync(kFull, lo), lo_max = __reduce_max_sync(kFull, lo);
      const bool dead = !__any_sync(kFull, own);  // a warp without rows only keeps the barriers going

      float m = -INFINITY, mm = 0.f, l0 = 0.f, l1 = 0.f;  // m: what P refers to, 2^7 below the largest score when it was taken
      // Bit 0: a key that is not finite is seen; bit 1 + g: a value of group g. The same for all of a warp's rows: bits 8 to 15: O's units
      // (pr_unit); bit 30: scores are multiplied and rounded first (kPrLarge); bit 31: some values are summed apart.
      uint32_t rare = 0;
#pragma unroll 1
      for (int it = wk.i0; it < (none ? wk.i0 : wk.i1); ++it) {
        const int slot = NQ == 2 ? i : (it - wk.i0) & 1;
        const uint32_t s_t = tmem + slot * 128 + lanes;
        pr_wait(&sh.s_full[slot], s_par >> slot & 1, fail);
        s_par ^= 1u << slot;
        tc_fence_after();
        // tiles are numbered over the CTA's whole share, as in the dequantisation
        const int mt = (wk.n0 + it - wk.i0) & (kMetaTiles - 1);
        const int t0 = wk.un.begin + it * kPrTok;
        const uint4 odd4 = *reinterpret_cast<const uint4*>(sh.odd[mt]);
        const uint32_t odd_tile = odd4.x | odd4.y | odd4.z | odd4.w | (rare & 0x4000ff00u);
        const bool plain = !odd_tile && t0 >= lo_max && t0 + kPrTok <= hi_min;
        // Every row sees every token, and no factor but the row's: 64 tokens at a time. The probabilities are taken with the
        // maximum so far while the scores' own is found; where that is too far above (seldom), it is raised and they are taken again.
        int from = plain || dead ? 4 : 0;  // where the other way takes over
#pragma unroll 1
        for (int c = 0; c < (plain && !dead ? 4 : 0);) {
          uint32_t v[64], pk[32];
          pr_ld32(s_t + c * 32, v);
          pr_ld32(s_t + c * 32 + 32, v + 32);
          const float ck = fmaxf(c2, 0x1p-126f);
          uint64_t ll = pr_pair(l0, l1);
          const uint64_t ck2 = pr_pair(ck, ck), mm2 = pr_pair(-mm, -mm);
          pr_wait_ld(v);
          pr_wait_ld(v + 32);
          float tp[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) tp[k] = __uint_as_float(v[k]);
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float s0 = __uint_as_float(v[2 * x]), s1 = __uint_as_float(v[2 * x + 1]);
            float p0, p1;
            tp[x & 3] = pr_max3(tp[x & 3], s0, s1);
            pr_split(pr_fma2(pr_pair(s0, s1), ck2, mm2), p0, p1);
            p0 = pr_ex2(p0);
            p1 = pr_ex2(p1);
            ll = pr_add2(ll, pr_pair(p0, p1));
            pk[x] = pr_half2(p0, p1);
          }
          const float top = pr_max3(fmaxf(tp[0], tp[1]), tp[2], tp[3]) * ck;
          const bool raise = top > m + kPrMost;
          if (!__any_sync(kFull, raise)) {
            pr_split(ll, l0, l1);
            pr_st16(s_t + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(pk));
            pr_st16(s_t + c * 16 + 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16));
            c += 2;
            continue;
          }
          const float up = raise ? top - kPrLift : m;
          const float f = up == m ? 1.f : pr_ex2(m - up);
          m = up;
          mm = up == -INFINITY ? 0.f : up;
          l0 *= f;
          l1 *= f;
          pr_wait_st();
#pragma unroll 1
          for (int k = 0; k < c; ++k) pr_scale_p(s_t + k * 16, f);  // this tile's P so far
          if (it > wk.i0) {
            if (NQ == 1) {  // the product before this one may still be running
              pr_wait(&sh.pv_done, pv_par ^ 1, fail);
              tc_fence_after();
            }
            pr_scale<D>(o_t, f);
          }
          if (__any_sync(kFull, fabsf(mm) > kPrLarge)) {  // seldom: the tile's rest goes the other way
            rare |= 1u << 30;
            from = c;
            break;
          }
        }
        // otherwise 32 tokens at a time, in a short loop (the warps' loops share the instruction caches)
        uint32_t unit = 0;  // the tile's units: by group O's where a block has it, else that of the first block with any
        if (odd_tile) {
          const uint32_t now = rare >> 8 & 0xff, ve[4] = {sh.meta[mt][0].ve, sh.meta[mt][1].ve, sh.meta[mt][2].ve, sh.meta[mt][3].ve};
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t o = now >> 2 * g & 3;
            uint32_t u = kVeNone;
            bool keep = false;
#pragma unroll
            for (int c = 3; c >= 0; --c) {
              const uint32_t k = ve[c] >> 2 * g & 3;
              keep |= k == o;
              if (k != kVeNone) u = k;
            }
            unit |= (keep || u == kVeNone ? o : u) << 2 * g;
          }
        }
#pragma unroll 1
        for (int c = from; c < 4; ++c) {
          const int t = t0 + c * 32;
          if (t >= hi_max || t + 32 <= lo_min) {  // no row sees any
            const uint32_t none[16] = {};
            pr_st16(s_t + c * 16, none);
            continue;
          }
          uint32_t v[32];
          pr_ld32(s_t + c * 32, v);
          const uint32_t odd = sh.odd[mt][c];
          const bool look = odd || unit;
          const bool cut = t < lo_max || t + 32 > hi_min;
          float ck = c2;
          uint32_t see = 0xffffffffu;
          bool other = false;  // the block's operand is of another unit than O: all of its values are summed apart
          bool apart = false;  // some are
          bool mix = false;    // each token's key has its own factor
          if (look || cut) {
            const PrMeta me = sh.meta[mt][c];
            ck *= me.kf;
            mix = me.kf == 0.f;
            other = (me.ve ^ unit | (me.ve ^ unit) >> 1) & ~(me.ve & me.ve >> 1) & 0x55;
            apart = other || (me.side[0] | (G > 1 ? me.side[1] : 0) | (G > 2 ? me.side[2] | me.side[3] : 0));
            const int n0 = max(lo - t, 0), n1 = min(hi - t, 32);
            see = n1 > n0 ? (0xffffffffu >> (32 - n1)) & (0xffffffffu << n0) : 0u;
            see &= ~me.gap;
            if (me.bad) {
              if (see & sh.kbad[mt][c]) rare |= 1;
#pragma unroll
              for (int g = 0; g < G; ++g)
                if (see & sh.vbad[mt][c][g]) rare |= 2u << g;
            }
          }
          ck = pr_factor(ck);
          pr_wait_ld(v);
          if (mix || rare >> 30 & 1) {  // seldom
            pr_scale_s(s_t + c * 32, mix ? c2 : ck, mix ? sh.ke[mt] + c * 32 : nullptr);
            pr_ld32(s_t + c * 32, v);
            pr_wait_ld(v);
            ck = 1.f;
          }
          if (odd || cut) {
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = see >> x & 1 ? v[x] : 0xff800000u;
          }
          float ta = pr_max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
          float tb = pr_max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
#pragma unroll
          for (int x = 6; x < 30; x += 4) {
            ta = pr_max3(ta, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
            tb = pr_max3(tb, __uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
          }
          const float top = pr_max3(fmaxf(ta, tb), __uint_as_float(v[30]), __uint_as_float(v[31])) * ck;
          const bool raise = top - m > kPrMost;
          if (__any_sync(kFull, raise) || unit != (rare >> 8 & 0xff)) {
            const float up = raise ? top - kPrLift : m;
            const float f = up == m ? 1.f : pr_ex2(m - up);
            m = up;
            mm = up == -INFINITY ? 0.f : up;
            l0 *= f;
            l1 *= f;
            pr_wait_st();
#pragma unroll 1
            for (int k = 0; k < c; ++k) pr_scale_p(s_t + k * 16, f);  // this tile's P so far
            if (it > wk.i0) {
              if (NQ == 1) {  // the product before this one may still be running
                pr_wait(&sh.pv_done, pv_par ^ 1, fail);
                tc_fence_after();
              }
              pr_scale<D>(o_t, f);
              if (unit != (rare >> 8 & 0xff)) {
                pr_wait_st();
                pr_rescale<D>(o_t, rare >> 8, unit);
              }
            }
            rare = (rare & ~0xff00u) | unit << 8;
            if (!(rare >> 30 & 1) && __any_sync(kFull, fabsf(mm) > kPrLarge)) {
              rare |= 1u << 30;
              if (!mix) {  // these scores again
                --c;
                continue;
              }
            }
          }
          uint64_t ll = pr_pair(l0, l1);
          const uint64_t ck2 = pr_pair(ck, ck), mm2 = pr_pair(-mm, -mm);
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float p0, p1;
            // a hidden score is -infinity: its probability is zero
            pr_split(pr_fma2(pr_pair(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), ck2, mm2), p0, p1);
            p0 = pr_ex2(p0);
            p1 = pr_ex2(p1);
            ll = pr_add2(ll, pr_pair(p0, p1));
            pk[x] = pr_half2(p0, p1);
          }
          pr_split(ll, l0, l1);
          if (apart) {  // seldom
            const PrMeta& me = sh.meta[mt][c];
            PrMask4 by;
#pragma unroll
            for (int g = 0; g < 4; ++g) by.of[g] = g < G ? (other ? 0xffffffffu : me.side[g]) & ~me.gap : 0u;
            pr_side<D>(a, row, head, t, by, see, s_t + c * 32, ck, m, w.part + ((long long)(cta * 2 + (wk.i0 == 0)) * NQ + i) * P::kSlot + r * 4, r,
                       rare >> 31);
            rare |= 1u << 31;
#pragma unroll
            for (int x = 0; x < 16; ++x) pk[x] = other ? 0u : pk[x];
          }
          pr_st16(s_t + c * 16, pk);
        }
        pr_wait_st();
        pv_par ^= 1;
        tc_fence_before();
        tc_arrive(&sh.p_full[slot]);
      }

      if (!none) nw.next(a, w, units);
      if (nw.live()) {
        next_row = pr_row<D>(a, nw, group, i * 128 + r);
        pr_query_fetch<D>(a, next_row, tc_smem(q_tile), r & ~31, lane);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        c2_next = pr_query_scale<D>(a, q_tile, qe_s + i * kExtra, r);
        tc_fence_proxy();
        tc_arrive(&sh.q_full[i]);
      }
      // ---- the unit's end: O / l, or a part of it
      if (!none) {
      const bool whole = wk.i0 == 0 && wk.i1 == wk.un.tiles;
      float* const part = w.part + ((long long)(cta * 2 + (wk.i0 == 0)) * NQ + i) * P::kSlot;
      pr_wait(&sh.o_full[i], o_par, fail);
      o_par ^= 1;
      tc_fence_after();
      const bool large = rare >> 31 && pr_side_add<D>(part + r * 4, r, o_t, m, rare >> 8);
      float l = rare & 1 ? NAN : l0 + l1;
      const long long out_at = ok ? (long long)row * a.out_stride + head * D : -1;
      if (!dead) {
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t v[32];
          pr_ld32(o_t + d, v);
          pr_wait_ld(v);
          float f = inv * exp2i(large ? 60 : pr_unit(rare >> 8, d / kGroup));
          if (rare >> (1 + d / kGroup) & 1) f = NAN;
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * f);
          if (whole) {
            // Columns come as 0 4 1 5 2 6 3 7. Four lanes exchange their 16-byte pieces, so that together they write 64 bytes of a
            // row at a time, of eight rows a warp (4096 tokens causal: 147.8 us, 149.0 with each lane writing its own row).
            uint4 w4[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              auto b2 = [&](int p, int q) { return pr_bf2(__uint_as_float(v[x * 8 + p]), __uint_as_float(v[x * 8 + q])); };
              w4[x] = make_uint4(b2(0, 2), b2(4, 6), b2(1, 3), b2(5, 7));
            }
            pr_swap(w4[0], w4[1], 1, lane);
            pr_swap(w4[2], w4[3], 1, lane);
            pr_swap(w4[0], w4[2], 2, lane);
            pr_swap(w4[1], w4[3], 2, lane);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const long long at = __shfl_sync(kFull, out_at, lane & ~3 | x);
              if (at >= 0) *reinterpret_cast<uint4*>(a.out + at + d + (lane & 3) * 8) = w4[x];
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              *reinterpret_cast<uint4*>(part + ((d + x) / 4 * 128 + r) * 4) = make_uint4(v[x], v[x + 2], v[x + 4], v[x + 6]);
              *reinterpret_cast<uint4*>(part + ((d + x) / 4 * 128 + 128 + r) * 4) = make_uint4(v[x + 1], v[x + 3], v[x + 5], v[x + 7]);
            }
          }
        }
        if (whole) {
          if (ok && a.lse) a.lse[(long long)row * a.q_heads + head] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
        } else {
          part[128 * D + r] = m;
          part[128 * D + 128 + r] = l;
        }
      }
      tc_fence_before();
      if (!whole && wk.i0 == 0 && r == 0 && i == 0) {
        const long long last = wk.x + wk.un.tiles - 1;  // the unit's last tile's place in the list
        w.cuts[w.ncut < (int)gridDim.x ? wk.h * w.cap + wk.u : cta] = PrCut{cta, (int)(((last + 1) * ctas - 1) / total), sp.first, wk.un.rt * P::kRows, min(sp.q_len, a.v.rows) * group, wk.h, {}};
      }
      }
      if (!nw.live()) break;
      wk = nw;
      rw = next_row;
      c2 = c2_next;
      none = false;
    }
  } else if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------------- dequantisation
    pr_regs<P::kRegDeq>();
    // four warps take K, four V; a warp has 32 tokens, a lane one of them. As soon as a warp has read its codes of a
    // tile, the next tile's go on their way into the same place; the pages are looked up a tile earlier still.
    const bool val = warp >= 8;
    const int part = (warp & 3) * 32;
    uint64_t* const full = val ? sh.v_full : sh.k_full;
    uint64_t* const free_ = val ? sh.v_free : sh.k_free;
    unsigned char* const tiles = val ? v_s : k_s;
    const uint32_t* const codes = val ? a.c.v_q : a.c.k_q;
    const uint16_t* const pairs = val ? a.c.v_sb : a.c.k_sb;
    const unsigned char* const raw = raw_s + (val ? P::kRaw : 0) + (warp & 3) * (P::kRaw / 4);
    // panels of a stage, stages; what turns 64 + code into V's code or K's code - 8
    const int pan = val ? P::VP : P::KP, ring = val ? P::VST : P::KST;
    const uint32_t off = val ? 0xD400D400u : 0xD480D480u;
    if (!val && G < 4) {  // extra columns that no group has
#pragma unroll
      for (int i = 0; i < P::KE; ++i) *reinterpret_cast<uint4*>(ke_s + i * kExtra + pr_extra(part + lane, 1)) = make_uint4(0, 0, 0, 0);
    }
    const uint32_t raw_u = tc_smem(raw);
    int st = 0;
    uint32_t par = 1;  // the first pass over the ring finds it free
    PrWalk<D> fw = wk;
    int ft = fw.i0;
    int page = -1, place = 0, page_h = 0, left = 0;  // of the lane's own 16 tokens; tokens of the 32 that exist
    auto find = [&]() {  // false: the share ends
      page = -1;
      left = 0;
      if (!fw.live()) return false;
      const int tok0 = fw.un.begin + ft * kPrTok + part, tok = tok0 + (lane & 16);
      page_h = fw.h;
      left = fw.un.sp.held - tok0;
      int pg;
      if (a.page_shift >= 0) {
        pg = tok >> a.page_shift;
        place = tok & (a.c.page_size - 1);
      } else {
        pg = tok / a.c.page_size;
        place = tok - pg * a.c.page_size;
      }
      if (tok < fw.un.sp.held) page = a.v.pages ? a.v.pages[(long long)fw.un.b * a.v.max_pages + pg] : fw.un.b;
      if (++ft == fw.i1) {
        fw.next(a, w, units);
        ft = fw.i0;
      }
      return true;
    };
    uint32_t sb[G], vs[G];  // the token's pairs; a K warp has V's too, for the notes
    bool gone = true;
    bool more = find();
#pragma unroll 1
    for (int x = -1;; ++x) {  // tile x is stored, the next one fetched
      if (x >= 0) {
        const int mt = x & (kMetaTiles - 1);
        uint32_t any = 0, bad[G];
        bool mix = false;
        int e = 0;  // of the token's key
        const float down = val ? exp2i(-kVe) : 1.f;
        uint32_t s2[G], b2[G];
        const bool odd_own = pr_odd<D>(sb, val ? kValueLow : kKeyLow);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float sc = bf16lo(sb[g]) * down, bi = bf16hi(sb[g]) * down;
          s2[g] = pr_half2(sc, sc);
          b2[g] = pr_half2(bi, bi);
        }
        if (odd_own) {
          uint32_t apart[G] = {}, ve = 0;
          if (val) ve = pr_value_range<D>(sb, apart, any, bad);
          else e = pr_key_range<D>(sb, mix, any, bad);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float by = !val ? exp2i(-e) : apart[g] >> lane & 1 ? 0.f : exp2i(-pr_unit(ve, g));  // (without any, all is zero)
            float sc = bf16lo(sb[g]) * by, bi = bf16hi(sb[g]) * by;
            if (!(fabsf(sc) < INFINITY && fabsf(bi) < INFINITY)) sc = bi = 0.f;
            s2[g] = pr_half2(sc, sc);
            b2[g] = pr_half2(bi, bi);
          }
        }
        pr_wait(&free_[st], par, fail);
        if (!val) {  // the notes on both go out with K, for the softmax reads them with the scores
          uint32_t vside[G] = {}, vany = 0, vbad[G], ve = 0;
          const int c = part / 32;
          if (pr_odd<D>(vs, kValueLow)) ve = pr_value_range<D>(vs, vside, vany, vbad);
          const uint32_t gap = __ballot_sync(kFull, gone);
          if (lane == 0) {
            uint32_t odd = gap | any | vany | (uint32_t)e | (uint32_t)mix | ((ve ^ ve >> 1) & 0x55);  // (an E but the usual one)
#pragma unroll
            for (int g = 0; g < G; ++g) odd |= vside[g];
            sh.odd[mt][c] = odd;
            sh.meta[mt][c] = PrMeta{mix ? 0.f : exp2i(e), ve, gap, any | vany, {vside[0], G > 1 ? vside[1 % G] : 0, G > 2 ? vside[2 % G] : 0, G > 2 ? vside[3 % G] : 0}};
            if (odd) {
              sh.kbad[mt][c] = any;
#pragma unroll
              for (int g = 0; g < G; ++g) sh.vbad[mt][c][g] = vany ? vbad[g] : 0;
            }
          }
          if (mix) sh.ke[mt][part + lane] = (int8_t)e;
          unsigned char* const ext = ke_s + (P::KE > 1 ? st * kExtra : 0);
#pragma unroll
          for (int g = 0; g < G; g += 2)
            *reinterpret_cast<uint4*>(ext + pr_extra(part + lane, g >> 1)) =
                make_uint4(b2[g], s2[g], G > 1 ? b2[(g + 1) % G] : 0, G > 1 ? s2[(g + 1) % G] : 0);
#pragma unroll
          for (int g = 0; g < G; ++g) b2[g] = 0;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int p = g & (pan - 1);  // the group's panel of its stage
          if (g > 0 && p == 0) pr_wait(&free_[st], par, fail);
          pr_store<D>(raw, g, off, s2[g], b2[g], tiles + (st * pan + p) * kPanel, part + lane);
          if (p == pan - 1) {
            tc_fence_proxy();
            tc_arrive(&full[st]);
            if (++st == ring) {
              st = 0;
              par ^= 1;
            }
          }
        }
        __syncwarp();
      }
      // the next tile on its way, and the page of the one behind
      if (!more) break;
      long long row =
          (unsigned)page < (unsigned)a.c.n_pages ? (long long)(page * a.c.kv_heads + page_h) * a.c.page_size + place : -1;
      pr_fetch<D>(raw_u, codes, row, lane);
      row = row < 0 || lane >= left ? -1 : row + (lane & 15);
      gone = row < 0;
      pr_pairs<D>(sb, pairs, row);
      if (!val) pr_pairs<D>(vs, a.c.v_sb, row);
      more = find();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- MMAs, by one warp
    pr_regs<P::kRegRest>();
    if (__shfl_sync(kFull, warp, 0) == 0) {
      const uint32_t lead = elect_lane();
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      constexpr uint32_t id_s = pr_idesc(128, false), id_o = pr_idesc(P::VP * kGroup, true);
      // Short loops and few instructions per MMA: this thread's code competes with the other warps' for the
      // instruction caches. Only the low word of a descriptor changes (addresses stay below 2^18).
      const uint32_t hi_k = (uint32_t)(pr_desc(0, 16) >> 32), lo_k = (uint32_t)pr_desc(0, 16);
      const uint32_t hi_v = (uint32_t)(pr_desc(0, kPanel) >> 32), lo_v = (uint32_t)pr_desc(0, kPanel);
      const uint32_t hi_e = (uint32_t)(pr_extra_desc(0) >> 32), lo_e = (uint32_t)pr_extra_desc(0);
      const uint32_t qa = lo_k + (tc_smem(q_s) >> 4), ka = lo_k + (tc_smem(k_s) >> 4), va = lo_v + (tc_smem(v_s) >> 4);
      const uint32_t qe = lo_e + (tc_smem(qe_s) >> 4), ke = lo_e + (tc_smem(ke_s) >> 4);
      uint32_t q_par = 0, p_par = 0;          // bit per tile / slot
      int ks = 0, vs = 0;                      // ring places
      uint32_t k_par = 0, v_par = 0;
      auto k_next = [&]() {
        mma_commit(&sh.k_free[ks], lead);
        if (++ks == P::KST) {
          ks = 0;
          k_par ^= 1;
        }
      };
      auto v_next = [&]() {
        mma_commit(&sh.v_free[vs], lead);
        if (++vs == P::VST) {
          vs = 0;
          v_par ^= 1;
        }
      };
      // Q K^T of row tile i; one row tile: stage by stage of K, as they come
      auto scores = [&](int i, int slot) {
        const uint32_t d = tm + slot * 128;
        uint32_t qd = qa + i * (P::kTile >> 4), kd = ka + ks * (P::KP * kPanel >> 4);
        const uint32_t ked = ke + (P::KE > 1 ? ks * (kExtra >> 4) : 0);
#pragma unroll 1
        for (int p = 0; p < G; ++p) {
          if (NQ == 1) {
            pr_wait(&sh.k_full[ks], k_par, fail);
            tc_fence_after();
            kd = ka + ks * (kPanel >> 4);
          }
          if (p == 0) mma_ss(d, (uint64_t)hi_e << 32 | (qe + i * (kExtra >> 4)), (uint64_t)hi_e << 32 | ked, id_s, 0, lead);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(d, (uint64_t)hi_k << 32 | (qd + k * 2), (uint64_t)hi_k << 32 | (kd + k * 2), id_s, 1, lead);
          qd += kPanel >> 4;
          kd += kPanel >> 4;
          if (NQ == 1) k_next();
        }
        mma_commit(&sh.s_full[slot], lead);
      };
      // P V of row tile i: the columns of one stage of V
      auto product = [&](int i, int slot, int col, bool first) {
        const uint32_t d = tm + 256 + i * D + col;
        uint32_t pa = tm + slot * 128, vd = va + vs * (P::VP * kPanel >> 4), acc = !first;
#pragma unroll 1
        for (int k = 0; k < kPrTok / 64; ++k) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            mma_ts(d, pa + n * 8, (uint64_t)hi_v << 32 | (vd + n * 128), id_o, acc, lead);
            acc = 1;
          }
          pa += 32;
          vd += 512;
        }
      };
      for (; __shfl_sync(kFull, (int)wk.live(), 0); wk.next(a, w, units)) {
        const int n = __shfl_sync(kFull, wk.i1 - wk.i0, 0);
        for (int it = -1; it < n; ++it) {  // step it: the product of tile it, the scores of tile it + 1
          if (NQ == 2) {
            if (it >= 0) pr_wait(&sh.v_full[vs], v_par, fail);
#pragma unroll 1
            for (int i = 0; i < NQ; ++i) {
              if (it >= 0) {
                pr_wait(&sh.p_full[i], p_par >> i & 1, fail);
                p_par ^= 1u << i;
                tc_fence_after();
                product(i, i, 0, it == 0);
                if (it == n - 1) mma_commit(&sh.o_full[i], lead);
              } else {
                pr_wait(&sh.q_full[i], q_par >> i & 1, fail);
                q_par ^= 1u << i;
              }
              if (it + 1 < n) {
                if (i == 0) pr_wait(&sh.k_full[ks], k_par, fail);
                tc_fence_after();
                scores(i, i);
              }
            }
            if (it + 1 < n) k_next();
          } else {
            if (it < 0) {
              pr_wait(&sh.q_full[0], q_par & 1, fail);
              q_par ^= 1;
            }
            const int slot = it & 1;
            if (it + 1 < n) scores(0, (it + 1) & 1);
            if (it >= 0) {
              pr_wait(&sh.p_full[slot], p_par >> slot & 1, fail);
              p_par ^= 1u << slot;
#pragma unroll 1
              for (int col = 0; col < D; col += P::VP * kGroup) {
                pr_wait(&sh.v_full[vs], v_par, fail);
                tc_fence_after();
                product(0, slot, col, it == 0);
                v_next();
              }
              mma_commit(&sh.pv_done, lead);
              if (it == n - 1) mma_commit(&sh.o_full[0], lead);
            }
          }
          if (NQ == 2 && it >= 0) v_next();
        }
      }
      // nothing is left in flight, whatever ended the loop
      mma_commit(&sh.drain, lead);
      const unsigned long long t0 = tc_time();
      while (!tc_mbar_try_suspend(&sh.drain, 0) && (long long)(tc_time() - t0) < kPrTimeoutNs) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.fail) atomicExch(&w.ctrl->status, BGQ_ERR_TIMEOUT);
  if (warp == 0) tmem_free(tmem, 512);
}

// ---------------------------------------------------------------------------
// The units that a CTA's share cut: every CTA's part, weighted, in CTA order. A block takes eight rows of one such unit, a
// thread four columns (eight at head dim 256) of one row; neighbouring threads read neighbouring rows. Where units are
// few, one may have a part of every CTA: then PG groups of threads take every PG-th part, and are joined in their order.
// ---------------------------------------------------------------------------
constexpr int kJoinRows = 8;
constexpr int kJoinThreads = 256;
template <int D, int PG>
__global__ void __launch_bounds__(kJoinThreads * PG) k_prompt_join(const __grid_constant__ AttnArgs a, const __grid_constant__ PrWs w) {
  using P = Prompt<D>;
  constexpr int Q = D / 128 > 0 ? D / 128 : 1, N = 4 * Q + 2, U = 4;
  __shared__ float other[PG > 1 ? (PG - 1) * N * kJoinThreads : 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x % kJoinThreads, pg = threadIdx.x / kJoinThreads;
  const PrCut cut = w.cuts[blockIdx.x];
  const int c0 = cut.c0;
  const int at_row = blockIdx.y * kJoinRows + tid % kJoinRows, col = cut.col0 + at_row, d4 = tid / kJoinRows * Q;
  if (cut.c1 < 0 || blockIdx.y * kJoinRows + cut.col0 >= cut.cols) return;
  const bool live = col < cut.cols && d4 < D / 4;
  const int i = at_row >> 7, r = at_row & 127, group = a.q_heads / a.c.kv_heads;
  const int j = col / group, row = cut.first + j, head = cut.h * group + col - j * group;
  auto part = [&](int c) { return w.part + ((long long)(c * 2 + (c == c0)) * P::NQ + i) * P::kSlot; };
  float top = -INFINITY, sum = 0.f, v[4 * Q] = {};
  if (live) {
#pragma unroll 1
    for (int c = c0 + pg; c <= cut.c1; c += PG * U) {  // U parts' loads at once
      float mc[U], lc[U], up = top;
      float4 p[U][Q];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float* pp = part(min(c + k * PG, cut.c1));
        mc[k] = __ldcg(pp + 128 * D + r);
        lc[k] = __ldcg(pp + 128 * D + 128 + r);
#pragma unroll
        for (int x = 0; x < Q; ++x) p[k][x] = __ldcg(reinterpret_cast<const float4*>(pp) + (d4 + x) * 128 + r);
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (c + k * PG <= cut.c1) up = fmaxf(up, mc[k]);
      const float f0 = top == up ? 1.f : pr_ex2(top - up);
      top = up;
      sum *= f0;
#pragma unroll
      for (int x = 0; x < 4 * Q; ++x) v[x] *= f0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (c + k * PG > cut.c1) break;
        const float f = mc[k] == top ? 1.f : pr_ex2(mc[k] - top);
        sum = fmaf(f, lc[k], sum);
#pragma unroll
        for (int x = 0; x < Q; ++x) {
          v[4 * x] = fmaf(f, p[k][x].x, v[4 * x]);
          v[4 * x + 1] = fmaf(f, p[k][x].y, v[4 * x + 1]);
          v[4 * x + 2] = fmaf(f, p[k][x].z, v[4 * x + 2]);
          v[4 * x + 3] = fmaf(f, p[k][x].w, v[4 * x + 3]);
        }
      }
    }
  }
  if (PG > 1) {
    if (pg > 0) {
      float* o = other + (pg - 1) * N * kJoinThreads + tid;
      o[0] = top;
      o[kJoinThreads] = sum;
#pragma unroll
      for (int x = 0; x < 4 * Q; ++x) o[(2 + x) * kJoinThreads] = v[x];
    }
    __syncthreads();
    if (pg > 0) return;
#pragma unroll
    for (int g = 0; g < PG - 1; ++g) {
      const float* o = other + g * N * kJoinThreads + tid;
      const float m2 = o[0], up = fmaxf(top, m2);
      const float f = top == up ? 1.f : pr_ex2(top - up), f2 = m2 == up ? 1.f : pr_ex2(m2 - up);
      top = up;
      sum = sum * f + o[kJoinThreads] * f2;
#pragma unroll
      for (int x = 0; x < 4 * Q; ++x) v[x] = v[x] * f + o[(2 + x) * kJoinThreads] * f2;
    }
  }
  if (!live || row < 0 || row >= a.v.rows) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int x = 0; x < Q; ++x)
    *reinterpret_cast<uint2*>(a.out + (long long)row * a.out_stride + head * D + (d4 + x) * 4) =
        make_uint2(pr_bf2(v[4 * x] * inv, v[4 * x + 1] * inv), pr_bf2(v[4 * x + 2] * inv, v[4 * x + 3] * inv));
  if (a.lse && d4 == 0) a.lse[(long long)row * a.q_heads + head] = sum == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(sum));
}

static int prompt_grid() { return num_sms(); }

size_t prompt_workspace_bytes(int batch, int rows, int q_heads, int kv_heads, int d) {
  return carve_prompt(nullptr, batch, rows, q_heads, kv_heads, d, prompt_grid()).bytes;
}

template <int D>
static cudaError_t launch_prompt_t(const AttnArgs& a, cudaStream_t s) {
  using P = Prompt<D>;
  const PrWs w = carve_prompt(a.ws, a.v.batch, a.v.rows, a.q_heads, a.c.kv_heads, D, prompt_grid());
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem(k_attn_prompt<D>, P::kSmem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(k_prompt_plan, 1, kPlanThreads, 0, s, a, w, P::kRows);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(k_attn_prompt<D>, prompt_grid(), kPrThreads, P::kSmem, s, a, w);
  if (e != cudaSuccess) return e;
  const int rows = (int)std::min((long long)P::kRows, (long long)a.v.rows * (a.q_heads / a.c.kv_heads));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w.ncut, (rows + kJoinRows - 1) / kJoinRows);
  const bool few = w.ncut * 8 <= prompt_grid();  // a unit has parts of eight CTAs or more
  cfg.blockDim = dim3(few ? 4 * kJoinThreads : kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, k_prompt_join<D, 4>, a, w) : cudaLaunchKernelEx(&cfg, k_prompt_join<D, 1>, a, w);
}

cudaError_t launch_attn_prompt(const AttnArgs& a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch_prompt_t<64>(a, s);
    case 128: return launch_prompt_t<128>(a, s);
    default: return launch_prompt_t<256>(a, s);
  }
}

}  // namespace bgq
