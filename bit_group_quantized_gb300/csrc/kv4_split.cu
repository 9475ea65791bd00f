// kv4_split.cu — attention over the 4-bit cache for few query rows a sequence
// (decode steps, drafted tokens): bound by reading the cache once.
//
// A unit is one key head of one sequence with up to 8*NT columns, a column
// being one (query row, query head) pair that shares this key head, so the
// cache is read once for all of them. A unit's tokens are cut into tiles; all units' tiles
// form one list, and every CTA takes an equal, contiguous share of it, so
// ragged lengths balance by themselves and a single long sequence spreads over
// the whole GPU. The list is worked out on the device from the lengths there.
//
// In a CTA each warp runs on its own: it copies its next tiles into its own ring
// (cp.async), and takes tiles w, w + kWarps, ... of a segment (the part of a
// unit inside the CTA's share) with a running maximum and sum per column.
// Per tile, with mma.sync m16n8k16 (fp16 in, fp32 out):
//   scores  S[token][col] = sum_g s_g ((64 + codes) . x)_g + (b_g - 64 s_g) sum(x)_g: the A operand
//           is 64 + code, placed by masks under the exponent of 64, the query the B operand, scaled
//           by a power of two per column, which is exact;
//   output  O[dim][col] += (code - 8) (p s_g): the codes transposed by byte
//           permutes as the A operand, the probabilities times the token's scale
//           as the B operand; p (b_g + 8 s_g) is summed apart in fp32. Codes are
//           centred so that long sums stay small beside what is added to them.
// p s_g is rounded to fp16 (half a step 2^-12, a sixteenth of the bf16 output's, and of random sign); its exponent is kept in range by a power
// of two 2^E per warp that follows the largest scale of a tile; scales far from it, in tokens that a column may not even see, are
// multiplied apart. The maximum is only
// raised when a score passes it by 2^5, so that most tiles need no reduction over the warp.
// What bounds it is the issue of instructions and the length of a tile's chain, not memory: 400 instructions for 16 tokens of a head of
// 128, 55 for the copies among them (taken out, no time was saved). 64 sequences of 512 to 16384 tokens, 8 key
// heads of 128, 4 columns: 88.3 us, 3.8 TB/s (57 % of a copy's rate; issue slots 61 % full); one of 131071 tokens: 42.6 us, 3.5 TB/s
// (eight warps an SM, latency); one of 513: 8.8 us, a call's latency.
// A segment ends with the CTA's warps joined in shared memory; a unit cut by a
// CTA's share is joined by the last of its CTAs to arrive, in CTA order (the same
// bits every time).
#include <cuda_fp16.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"
#include "kv4_seen.h"
#include "split_join.h"

namespace bgq {

constexpr int kSplitWarps = 8;
constexpr int kSplitThreads = kSplitWarps * 32;
constexpr int kSplitMaxGrid = (kAttnHead - 256) / 8;  // two arrival counters a CTA, behind the control block
// What a unit costs beside its tiles (its queries, the joining of the warps), in tiles: 64 sequences of 512 to 16384 tokens
// took 103, 92, 88.7, 90.6 us with 6, 12, 20, 30.
constexpr int kSplitUnitCost = 20;

// CTAs: of an SM. Two of 128 registers a thread keep it busy while one joins its warps; one of 255 spares registers (at
// 128, a head dim times column tiles of 256 or more spills them) and halves the parts to join.
template <int D, int NT, int CTAS>
struct Split {
  static constexpr int G = D / kGroup;
  static constexpr int C = 8 * NT;                 // columns of a unit
  static constexpr int TT = D == 256 ? 16 : 32;    // tokens of a tile
  static constexpr int MT = TT / 16;
  static constexpr int ST = D == 64 ? 3 : CTAS == 1 ? 4 : 2;  // tiles of a warp's ring
  static constexpr int CPT = D / 32;               // 16-byte chunks of a token's codes
  static constexpr int kCode = TT * D / 2;         // bytes of a tile's K (or V) codes
  static constexpr int kSb = TT * D / 16;          // bytes of a tile's K (or V) pairs
  static constexpr int kStage = 2 * kCode + 2 * kSb;
  static constexpr int RD = D * NT >= 256 && NT == 2 ? 64 : (D < 128 ? D : 128);  // dims joined per round
  static constexpr int RS = RD + 4;                // row stride of the join area (floats)
  static constexpr bool kQs = D * NT > 64;         // query fragments in shared memory
  static constexpr int kQBytes = kQs ? NT * G * 4 * 32 * 8 : 0;
  static constexpr int kSmem = kSplitWarps * ST * kStage + kSplitWarps * C * RS * 4 + kQBytes;
  // the joining of CTAs keeps a weight for every part and column, and a column group for every thread
  static_assert((kSplitWarps * C * RS) >= 304 / (3 - CTAS) * C + 4 + kSplitThreads * 4, "join area too small");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with an accumulator that starts from zero.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Four 8x8 matrices of 16-bit units from shared memory, a row address a lane; TRANS: transposed.
template <bool TRANS>
__device__ __forceinline__ void ldmat4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// Constants of the code placement, kept in registers: instructions take one constant, and these are the second ones.
struct SplitK {
  uint32_t or64, or1024, by16, less72;
};
__device__ __forceinline__ SplitK split_constants() {
  SplitK k;
  asm volatile("mov.b32 %0, 0x54005400;" : "=r"(k.or64));
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k.or1024));
  asm volatile("mov.b32 %0, 0x2C002C00;" : "=r"(k.by16));
  asm volatile("mov.b32 %0, 0xD480D480;" : "=r"(k.less72));
  return k;
}
// Where 16-byte piece ch of token t (of 16) stands in a tile's codes: eight tokens' pieces lie in different banks.
template <int D>
__device__ __forceinline__ int split_at(int t, int ch) {
  if (D == 64) return (t >> 2) * 128 + (t & 3) * 32 + ((ch ^ (t >> 2)) & 1) * 16;
  if (D == 128) return (t >> 1) * 128 + (t & 1) * 64 + ((ch ^ (t >> 1)) & 3) * 16;
  return t * 128 + ((ch ^ t) & 7) * 16;
}
__device__ __forceinline__ uint32_t movm(uint32_t a) {  // transpose of an 8x8 fp16 matrix held by a warp
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(m), "r"(o));
  return d;
}

// A sequence's units and their tiles.
struct SeqTiles {
  Span sp;
  int begin;   // first token of its first tile
  int tiles;   // of one unit (at least one, so that rows that see no token are written)
  int rtiles;  // column tiles
};
template <int TT, int C>
__device__ __forceinline__ SeqTiles seq_tiles(const AttnArgs& a, int b) {
  SeqTiles s;
  s.sp = kv4_span(a.v, b);
  const int pos0 = s.sp.kv_len - s.sp.q_len;
  s.begin = min(kv4_first_seen(pos0, a.window), s.sp.held) / TT * TT;  // the look-up of pages runs up to 4064 tokens ahead of it
  s.tiles = max(1, (s.sp.held - s.begin + TT - 1) / TT);
  s.rtiles = (min(s.sp.q_len, a.v.rows) * (a.q_heads / a.c.kv_heads) + C - 1) / C;
  return s;
}

// A CTA's share of the list, segment by segment (tiles i0 .. i1 - 1 of a unit). A unit takes kSplitUnitCost places, then one
// for each tile, and the CTA whose share holds a tile's place does the tile; `flat`: every unit takes this
// many places, which is also a share's length.
template <int TT, int C>
struct Walk {
  long long x, x1;  // the place of the unit's first tile, the share's end
  int b, h, rt, i0, i1, flat;
  SeqTiles q;

  __device__ __forceinline__ bool live() const { return i1 > i0; }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    x += flat ? flat : q.tiles + kSplitUnitCost;
    i0 = i1 = 0;
    if (x >= x1) return;
    if (++rt >= q.rtiles) {
      rt = 0;
      ++h;
    }
    if (h >= a.c.kv_heads) {
      h = 0;
      q = seq_tiles<TT, C>(a, ++b);
      while (q.rtiles == 0 && b + 1 < a.v.batch) {  // sequences without rows: 32 are looked at together
        const int ahead = b + 1 + (threadIdx.x & 31);
        const uint32_t some = __ballot_sync(kFull, ahead < a.v.batch && kv4_span(a.v, ahead).q_len > 0);
        b = some ? b + __ffs(some) : min(b + 32, a.v.batch - 1);
        if (some || b + 1 == a.v.batch) q = seq_tiles<TT, C>(a, b);
      }
    }
    i1 = (int)min((long long)q.tiles, x1 - x);
  }
};

struct SplitWs {
  int* count;   // [grid] arrivals at the unit that CTA c began and did not end; left at zero
  float* part;  // [grid][2][C][D + 2]: slot 0 a unit begun by an earlier CTA, slot 1 a unit that goes on
};

// A warp's state over a segment; columns 2c and 2c + 1 of each eight.
template <int D, int NT>
struct SplitAcc {
  static constexpr int G = D / kGroup;
  // What the probabilities refer to, 0 before the first score; and what a score must pass to raise it: -infinity before the
  // first, and kSplitSteep, which all pass, where it is so large that products with cs are rounded first (in the masked form).
  float mm[NT][2], pass[NT][2];
  float l[NT][2], bias[NT][2][G];  // this lane's tokens' sums of p, and of p (b + 8 s)
  float o[NT][G][4][4];           // sum of (code - 8) p s, in units of 2^E
  float cs[NT][2];                // scale * log2(e) / 2^shift
  int hi[NT][2], lo[NT][2];       // the tokens that the columns see: lo <= t < hi
  float unit, inv;                // 2^E, 2^-E
  uint32_t less;                  // minus the bits of 2^E, the smallest scale that 2^-E takes in
};
// p s 2^-E has a place in fp16 for the scales s from 2^E to 2^(E + 9): p stays below 2^5, the product below 2^14, and only what is below
// 2^-25 is lost: a tail of tokens 2^-25 below the first one is still there, whatever their scales. E follows the
// largest scale of a tile, between -20 and 20, where fp32 has room for O in any such unit; scales that it does not take in (far
// smaller than others of the tile, or very large) are multiplied apart.
constexpr int kSplitTop = 8, kSplitMost = 20;
constexpr float kSplitRaise = 5.f;
constexpr uint32_t kSplitSpan = 9u << 23;
// A fused difference s cs - mm is as far from zero at the maximum as the product's rounding: 2^-4 at 2^20, but more than any exponent
// at 2^31. From kSplitLarge on scores are multiplied and rounded first, as the maximum is.
constexpr float kSplitLarge = 0x1p20f, kSplitSteep = -3e38f;

// Codes less 8 of dims 4g + j (row g) and 32 + 4g + j (row g + 8), from transposed words.
__device__ __forceinline__ void split_codes(uint32_t (&f)[4], const uint32_t (&w)[4], int j, const SplitK& k_) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = j & 2 ? w[i] >> 8 : w[i];
    f[i] = j & 1 ? hfma2_u(and_or(x, 0x00F000F0u, k_.or1024), k_.by16, k_.less72)  // (1024 + 16q)/16 - 72
                 : hadd2_u(and_or(x, 0x000F000Fu, k_.or1024), 0xE408E408u);              // 1024 + q - 1032
  }
}
// What the scales that 2^-E does not take in add to O and the sums beside it: token by token in fp32, a lane its own dims of O, with few registers.
// Seldom. The scores are multiplied by cs, hidden tokens' are -infinity.
template <int D, int NT>
__device__ __forceinline__ void split_far(SplitAcc<D, NT>& A, const float (&s)[Split<D, NT, 1>::MT][NT][4], const unsigned char* st, int t0, int held,
                                          int g) {
  using P = Split<D, NT, 1>;
  constexpr int G = P::G, MT = P::MT;
  asm volatile("" : "+r"(g), "+r"(t0), "+l"(st));  // nothing is worked out ahead, in registers of the loop around it
  const int c = threadIdx.x & 3;
#pragma unroll 1
  for (int mr = 0; mr < 2 * MT; ++mr) {  // eight tokens, of which the lane has one
    float p[NT][2], v[G];
    bool any = false;
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      const uint32_t pair = t0 + mr * 8 + g < held ? reinterpret_cast<const uint32_t*>(st + 2 * P::kCode + P::kSb)[(mr * 8 + g) * G + gr] : 0u;
      const uint32_t mag = (pair & 0x7fffu) << 16;
      const bool far = mag && mag < 0x7f800000u && mag + A.less >= kSplitSpan;
      v[gr] = far ? bf16lo(pair) : 0.f;
      any |= far;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = s[0][n][k];
#pragma unroll
        for (int i = 1; i < 2 * MT; ++i) x = mr == i ? s[i / 2][n][i % 2 * 2 + k] : x;
        p[n][k] = ex2(x - A.mm[n][k]);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) A.bias[n][k][gr] = fmaf(p[n][k], 8.f * v[gr], A.bias[n][k][gr]);
      }
#pragma unroll 1
    for (uint32_t left = __ballot_sync(kFull, any) & 0x11111111u; left; left &= left - 1) {
      const int from = __ffs(left) - 1, t = mr * 8 + (from >> 2);
      float f[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) f[n][k] = __shfl_sync(kFull, p[n][k], from + c) * A.inv;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const float vt = __shfl_sync(kFull, v[gr], from);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // dims 4g + j, then 32 + those
          const uint32_t w = *reinterpret_cast<const uint32_t*>(st + P::kCode + (t >> 4) * (8 * D) + split_at<D>(t & 15, gr * 2 + h) + (g >> 1) * 4) >> (g & 1) * 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float code = (float)(int)(w >> j * 4 & 15u) - 8.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k) A.o[n][gr][j][h * 2 + k] = fmaf(f[n][k] * vt, code, A.o[n][gr][j][h * 2 + k]);
          }
        }
      }
    }
  }
}

// What follows a tile's scores s; MASKED where some column does not see all of its tokens, some scale is far from the others or
// scores are very large: without it nothing is added then, and false returned.
template <int D, int NT, int CTAS, bool MASKED>
__device__ __forceinline__ bool split_finish(SplitAcc<D, NT>& A, float (&s)[Split<D, NT, 1>::MT][NT][4], const unsigned char* st,
                                             uint32_t st_u, int t0, int gaps, int held, int g, const SplitK& k_) {
  using P = Split<D, NT, 1>;  // a tile's layout does not go by the CTAs
  constexpr int G = P::G, MT = P::MT;
  // Where registers are short (128 a thread, or 16 columns of 256) the pairs are read again behind split_far, so that no register keeps
  // them over it (64 sequences of 512 to 16384 tokens: 88.3 us, else 89.6); elsewhere the registers are there (131071 tokens:
  // 42.6 us, else 43.4).
  constexpr bool kAgain = CTAS == 2 || D * NT >= 512;
  uint32_t vp[MT][2][G], big = 0;  // V's pairs; how far their scales' bits pass the smallest
  bool raise = false;
  if (MASKED) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][n][i] = __fmul_rn(s[mt][n][i], A.cs[n][i & 1]);
  }
  auto cs = [&](int n, int k) { return MASKED ? 1.f : A.cs[n][k]; };
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(st + 2 * P::kCode + P::kSb) + (mt * 16 + r * 8 + g) * G;
      const int t = t0 + mt * 16 + r * 8 + g;
      const bool some = !MASKED || (!(gaps >> mt & 1) && t < held);
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        vp[mt][r][gr] = src[gr];
        const uint32_t over = vp[mt][r][gr] * 65536u + A.less;
        if (MASKED && !some) vp[mt][r][gr] = 0u;
        else big = max(big, over);
      }
      if (MASKED) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!some || t < A.lo[n][k] || t >= A.hi[n][k]) s[mt][n][r * 2 + k] = -INFINITY;
          }
      }
    }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float top = s[0][n][k];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, mt ? fmaxf(s[mt][n][k], s[mt][n][2 + k]) : s[mt][n][2 + k]);
      raise |= top * cs(n, k) > A.pass[n][k];
    }
  // a scale of zero or with its sign set, an infinity or a NaN passes the span: looked at more closely there
  if (__any_sync(kFull, raise || big >= kSplitSpan)) {
    uint32_t most = 0, least = ~0u;  // largest and (less one) smallest of the finite scales but zero
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          const uint32_t mag = (vp[mt][r][gr] & 0x7fffu) << 16;
          if (mag < 0x7f800000u) {
            most = max(most, mag);
            least = min(least, mag - 1);
          }
        }
    most = __reduce_max_sync(kFull, most);
    least = __reduce_min_sync(kFull, least) + 1;
    int e = (int)(__float_as_uint(A.unit) >> 23) - 127;
    uint32_t less = A.less;
    if (most && most + less >= kSplitSpan) {
      e = min(max((int)(most >> 23) - 127 - kSplitTop, -kSplitMost), kSplitMost);
      less = 0u - __float_as_uint(exp2i(e + kSplitTop - 8));
    }
    const bool far = most && (most + less >= kSplitSpan || least < 0u - less);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, fmaxf(s[mt][n][k], s[mt][n][2 + k]));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
        const float m = A.pass[n][k] == -INFINITY ? -INFINITY : A.mm[n][k];
        top = fmaxf(m, top * cs(n, k));
        const float f = m == top ? 1.f : ex2(m - top);
        A.mm[n][k] = top == -INFINITY ? 0.f : top;
        A.pass[n][k] = fabsf(A.mm[n][k]) > kSplitLarge ? kSplitSteep : top + kSplitRaise;
        A.l[n][k] *= f;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          A.bias[n][k][gr] *= f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            A.o[n][gr][j][k] *= f;
            A.o[n][gr][j][2 + k] *= f;
          }
        }
      }
    if (!MASKED) {
      bool steep = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) steep |= A.pass[n][0] == kSplitSteep || A.pass[n][1] == kSplitSteep;
      if (far || __any_sync(kFull, steep)) return false;  // what was raised stays so
    }
    if (less != A.less) {
      const float f = A.unit * exp2i(-e);
      A.unit = exp2i(e);
      A.inv = exp2i(-e);
      A.less = less;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) A.o[n][gr][j][i] *= f;
    }
    if (MASKED && far) {
      split_far<D, NT>(A, s, st, t0, held, g);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const int t = mt * 16 + r * 8 + g;
            if (kAgain) vp[mt][r][gr] = !(gaps >> mt & 1) && t0 + t < held ? reinterpret_cast<const volatile uint32_t*>(st + 2 * P::kCode + P::kSb)[t * G + gr] : 0u;
            const uint32_t mag = (vp[mt][r][gr] & 0x7fffu) << 16;
            if (mag < 0x7f800000u && mag + A.less >= kSplitSpan) vp[mt][r][gr] &= 0xffff0000u;
          }
    }
  }
  // ---- probabilities, and the output
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    uint32_t bf[NT][G][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sc[G], vb[G];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const float v = bf16lo(vp[mt][r][gr]);
        sc[gr] = v * A.inv;
        vb[gr] = fmaf(8.f, v, bf16hi(vp[mt][r][gr]));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[k] = ex2(MASKED ? s[mt][n][r * 2 + k] - A.mm[n][k] : fmaf(s[mt][n][r * 2 + k], A.cs[n][k], -A.mm[n][k]));
          A.l[n][k] += p[k];
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          // a token that the mask hides adds nothing, whatever its pair holds
          float ps[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            ps[k] = p[k] * sc[gr];
            const float bs = fmaf(p[k], vb[gr], A.bias[n][k][gr]);
            const bool gone = MASKED && s[mt][n][r * 2 + k] == -INFINITY;
            if (gone) ps[k] = 0.f;
            A.bias[n][k][gr] = gone ? A.bias[n][k][gr] : bs;
          }
          bf[n][gr][r] = movm(half2_of(ps[0], ps[1]));
        }
      }
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      // four codes (dims 4g .. 4g + 3, then 32 + those) of tokens 2c and 2c + 1, then 8 + those, side by side
      uint32_t r[4];
      ldmat4<true>(r, (st_u + P::kCode + mt * (8 * D)) ^ (gr * 32));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t f[4];
        split_codes(f, r, j, k_);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(A.o[n][gr][j], f[0], f[2], f[1], f[3], bf[n][gr][0], bf[n][gr][1]);
      }
    }
  }
  return true;
}

template <int D, int NT, int CTAS>
__global__ void __launch_bounds__(kSplitThreads, CTAS) k_attn_split(const __grid_constant__ AttnArgs a) {
  using P = Split<D, NT, CTAS>;
  constexpr int G = P::G, C = P::C, TT = P::TT, MT = P::MT, ST = P::ST, RD = P::RD, RS = P::RS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_m[kSplitWarps][C], s_l[kSplitWarps][C];
  __shared__ long long s_scan[kSplitWarps], s_units[kSplitWarps], s_base;
  __shared__ int s_b, s_last, s_most[kSplitWarps], s_gaps[kSplitWarps][ST];
  unsigned char* const ring = smem + (threadIdx.x >> 5) * (ST * P::kStage);
  float* const area = reinterpret_cast<float*>(smem + kSplitWarps * ST * P::kStage);
  uint2* const qf_s = reinterpret_cast<uint2*>(smem + kSplitWarps * ST * P::kStage + kSplitWarps * C * RS * 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();

  // ---- the list: how long it is, and where this CTA's share begins
  const int per = (a.v.batch + kSplitThreads - 1) / kSplitThreads;
  const int b_lo = min((int)threadIdx.x * per, a.v.batch), b_hi = min(b_lo + per, a.v.batch);
  long long own = 0, own_units = 0;
  int most = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const SeqTiles s = seq_tiles<TT, C>(a, b);
    const long long n = (long long)s.rtiles * a.c.kv_heads;
    own_units += n;
    own += n * (s.tiles + kSplitUnitCost);
    if (n) most = max(most, s.tiles);
  }
  most = __reduce_max_sync(kFull, most);
  long long pre = own, pre_units = own_units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(kFull, pre, o), vu = __shfl_up_sync(kFull, pre_units, o);
    if (lane >= o) {
      pre += v;
      pre_units += vu;
    }
  }
  if (lane == 31) {
    s_scan[warp] = pre;
    s_units[warp] = pre_units;
    s_most[warp] = most;
  }
  __syncthreads();
  long long total = 0, before = 0, units = 0, before_units = 0;
#pragma unroll
  for (int w = 0; w < kSplitWarps; ++w) {
    if (w < warp) {
      before += s_scan[w];
      before_units += s_units[w];
    }
    total += s_scan[w];
    units += s_units[w];
    most = max(most, s_most[w]);
  }
  // Few short units: one a CTA, and nothing to join between CTAs. Otherwise equal shares, of at least a tile a warp.
  Walk<TT, C> wk;
  long long ctas;
  if (units <= gridDim.x && most <= 4 * kSplitWarps) {
    wk.flat = most;
    total = units * most;
    ctas = units;
    pre = (pre_units + before_units - own_units) * most;
    own = own_units * most;
  } else {
    wk.flat = 0;
    ctas = max(1ll, min((long long)gridDim.x, total / (kSplitWarps + kSplitUnitCost)));
    pre += before - own;
  }
  const int cta = blockIdx.x;
  if (cta >= ctas || total == 0) return;
  const long long x0 = total * cta / ctas;
  wk.x1 = total * (cta + 1) / ctas;
  if (x0 >= pre && x0 < pre + own) {
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const SeqTiles s = seq_tiles<TT, C>(a, b);
      const long long n = (long long)s.rtiles * a.c.kv_heads * (wk.flat ? wk.flat : s.tiles + kSplitUnitCost);
      if (x0 < pre + n) break;
      pre += n;
    }
    s_b = b;
    s_base = pre;
  }
  __syncthreads();
  wk.b = s_b;
  wk.q = seq_tiles<TT, C>(a, wk.b);
  {
    const int cost = wk.flat ? wk.flat : wk.q.tiles + kSplitUnitCost, unit0 = (int)((x0 - s_base) / cost);
    wk.h = unit0 / wk.q.rtiles;
    wk.rt = unit0 - wk.h * wk.q.rtiles;
    wk.x = s_base + (long long)unit0 * cost + (wk.flat ? 0 : kSplitUnitCost);
    wk.i0 = (int)max(0ll, x0 - wk.x);
    wk.i1 = (int)min((long long)wk.q.tiles, wk.x1 - wk.x);
    if (wk.i1 <= wk.i0) wk.next(a);
  }

  const int heads = a.c.kv_heads, group = a.q_heads / heads;
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);
  // the lane's part of 16 tokens' copies
  const char* const lane_k = reinterpret_cast<const char*>(a.c.k_q) + lane * 16;
  const char* const lane_v = reinterpret_cast<const char*>(a.c.v_q) + lane * 16;
  const char* const lane_sb = reinterpret_cast<const char*>(lane < 16 ? a.c.k_sb : a.c.v_sb) + (lane & 15) * 16;
  const uint32_t lane_dst = split_at<D>(lane / P::CPT, lane % P::CPT);
  const uint32_t pair_dst = ring_u + 2 * P::kCode + (lane < 16 ? 0 : P::kSb) + (lane & 15) * 16;

  // ---- copies: the warp's next tile of its share into ring slot `slot`. Lane l looks up the l-th 16 tokens (which lie in one
  // page) of the warp's next tiles, 32 at a time.
  Walk<TT, C> fw = wk;
  int fi = fw.i0 + warp, blk = -1, blk_at = 32;
  auto fetch = [&](int slot) {
    while (fw.live() && fi >= fw.i1) {
      fw.next(a);
      fi = fw.i0 + warp;
      blk_at = 32;
    }
    if (fw.live()) {
      if (blk_at == 32) {
        const int t = fw.q.begin + (fi + lane / MT * kSplitWarps) * TT + lane % MT * 16;
        blk = -1;
        if (t < fw.q.sp.held) {
          int pg, place;  // page of the list, 16 tokens of it
          if (a.page_shift >= 0) {
            pg = t >> a.page_shift;
            place = (t & (a.c.page_size - 1)) >> 4;
          } else {
            pg = t / a.c.page_size;
            place = (t - pg * a.c.page_size) >> 4;
          }
          const int page = a.v.pages ? a.v.pages[(long long)fw.b * a.v.max_pages + pg] : fw.b;
          if ((unsigned)page < (unsigned)a.c.n_pages) blk = (page * heads + fw.h) * (a.c.page_size >> 4) + place;
        }
        blk_at = 0;
      }
      const uint32_t dst = ring_u + slot * P::kStage + lane_dst;
      int gaps = 0;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int bk = __shfl_sync(kFull, blk, blk_at + m);
        const bool ok = bk >= 0;
        gaps |= ok ? 0 : 1 << m;
        const long long at = ok ? bk : 0;
        const char* ks = lane_k + at * (8 * D);
        const char* vs = lane_v + at * (8 * D);
#pragma unroll
        for (int i = 0; i < P::CPT / 2; ++i) {  // 16 tokens are 16 * CPT pieces
          // 32 pieces are whole periods of the swizzle, or (head dim 256) half of one, which flips its third bit
          const uint32_t to = (D == 256 && (i & 1) ? dst ^ 64 : dst) + m * (8 * D) + i * 512;
          cp16(to, ks + i * 512, ok);
          cp16(to + P::kCode, vs + i * 512, ok);
        }
        // pairs: D bytes per 16 tokens, K by the low lanes, V by the high ones
        if ((lane & 15) < D / 16) cp16(pair_dst + slot * P::kStage + m * D, lane_sb + at * D, ok);
      }
      blk_at += MT;
      if (lane == 0) s_gaps[warp][slot] = gaps;
      fi += kSplitWarps;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) fetch(i);
  int slot = 0;

  const SplitK k_ = split_constants();
  // the row address that the lane gives ldmatrix: token lane % 16, piece lane / 16 of a group
  const uint32_t mat_at = split_at<D>(lane & 15, lane >> 4);

  for (; wk.live(); wk.next(a)) {
    const int h = wk.h, col0 = wk.rt * C;
    // a sequence's columns may pass 2^32 where it claims more rows than there are
    const int ncol = __umulhi(wk.q.sp.q_len, group) ? C : (int)min((unsigned)C, (unsigned)wk.q.sp.q_len * group - col0);
    const int pos0 = wk.q.sp.kv_len - wk.q.sp.q_len;

    // ---- the query: fp16 fragments of column g, scaled by a power of two
    uint32_t qf[P::kQs ? 1 : NT * G * 8];
    float xs[NT][2][G];             // group sums of columns 2c, 2c + 1
    SplitAcc<D, NT> A;
    if (P::kQs) __syncthreads();    // the last segment's fragments are read
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = n * 8 + g;
      const int j = (col0 + col) / group, hh = (col0 + col) - j * group;
      const int row = wk.q.sp.first + j;
      const bool ok = col < ncol && row >= 0 && row < a.v.rows;
      const uint16_t* src = a.q + (long long)(ok ? row : 0) * a.q_stride + (h * group + hh) * D + c * 8;
      uint32_t raw[G][8];
      float top = 0.f;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (ok) v = *reinterpret_cast<const uint4*>(src + gr * 64 + i * 32);
          raw[gr][i * 4] = v.x; raw[gr][i * 4 + 1] = v.y; raw[gr][i * 4 + 2] = v.z; raw[gr][i * 4 + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf16lo(raw[gr][i])), fabsf(bf16hi(raw[gr][i]))));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // largest magnitude into [8, 16): fp16 keeps 2^-28 of it
      const int e = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 130, -110), 124) : 0;
      const float up = a.scale < 0.f ? -exp2i(-e) : exp2i(-e);
      float sum[G];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        sum[gr] = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w) {  // word w of the lane: dims 32w + 8c + 0..7; pair i is dims (i, i + 4)
          const uint32_t* r = raw[gr] + w * 4;
          uint32_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = i & 1 ? bf16hi(r[i >> 1]) : bf16lo(r[i >> 1]);
            const float x1 = i & 1 ? bf16hi(r[2 + (i >> 1)]) : bf16lo(r[2 + (i >> 1)]);
            f[i] = half2_of(x0 * up, x1 * up);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
            sum[gr] += back.x + back.y;
          }
          if (P::kQs) {
            if (warp == n % kSplitWarps) {
              qf_s[((n * G + gr) * 4 + w * 2) * 32 + lane] = make_uint2(f[0], f[1]);
              qf_s[((n * G + gr) * 4 + w * 2 + 1) * 32 + lane] = make_uint2(f[2], f[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[((n * G + gr) * 4 + w * 2) * 2 + i] = f[i];
          }
        }
        sum[gr] += __shfl_xor_sync(kFull, sum[gr], 1);
        sum[gr] += __shfl_xor_sync(kFull, sum[gr], 2);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = (2 * c + k) * 4;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) xs[n][k][gr] = __shfl_sync(kFull, sum[gr], from);
        // at least the smallest normal number, so that -infinity times it stays -infinity, and finite, so that zero times it stays zero
        A.cs[n][k] = fminf(fmaxf(fabsf(a.scale) * 1.4426950408889634f * exp2i(__shfl_sync(kFull, e, from)), 0x1p-126f), 3e38f);
        const int cc = n * 8 + 2 * c + k, jj = (col0 + cc) / group;
        const int pos = pos0 + jj;
        // columns behind the last see what the first one sees, and are dropped at the end
        const int p2 = cc < ncol ? pos : pos0 + col0 / group;
        A.hi[n][k] = kv4_end_seen(p2, wk.q.sp.kv_len, wk.q.sp.held, a.causal);
        A.lo[n][k] = kv4_first_seen(p2, a.window);
      }
    }
    if (P::kQs) __syncthreads();
    int all_lo = A.lo[0][0], all_hi = A.hi[0][0];  // what every column sees
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        all_lo = max(all_lo, A.lo[n][k]);
        all_hi = min(all_hi, A.hi[n][k]);
      }
    all_lo = __reduce_max_sync(kFull, all_lo);
    all_hi = __reduce_min_sync(kFull, all_hi);

#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        A.pass[n][k] = -INFINITY;
        A.mm[n][k] = A.l[n][k] = 0.f;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) A.bias[n][k][gr] = 0.f;
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) A.o[n][gr][j][i] = 0.f;
    }
    A.unit = A.inv = 1.f;
    A.less = 0u - 0x7f800000u;  // takes no scale in

    for (int it = wk.i0 + warp; it < wk.i1; it += kSplitWarps) {
      cp_wait<ST - 1>();
      __syncwarp();
      const unsigned char* st = ring + slot * P::kStage;
      const uint32_t st_u = ring_u + slot * P::kStage + mat_at;
      const int t0 = wk.q.begin + it * TT;
      const int gaps = s_gaps[warp][slot];
      const bool masked = gaps || t0 < all_lo || t0 + TT > all_hi;

      // ---- scores
      float s[MT][NT][4];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        uint32_t w[MT][4];  // word c of tokens g and g + 8, then word 4 + c
        float acc[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) ldmat4<false>(w[mt], (st_u + mt * (8 * D)) ^ (gr * 32));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t f[MT][4];  // 64 + code, pairs (2i, 2i + 4), (2i + 1, 2i + 5) of both tokens
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t r0 = w[mt][2 * k], r1 = w[mt][2 * k + 1];
              f[mt][0] = and_or(i ? r0 >> 4 : r0 << 4, 0x00F000F0u, k_.or64);
              f[mt][1] = and_or(i ? r1 >> 4 : r1 << 4, 0x00F000F0u, k_.or64);
              f[mt][2] = and_or(i ? r0 >> 8 : r0, 0x00F000F0u, k_.or64);
              f[mt][3] = and_or(i ? r1 >> 8 : r1, 0x00F000F0u, k_.or64);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int step = (n * G + gr) * 4 + k * 2 + i;
              uint32_t b0, b1;
              if (P::kQs) {
                const uint2 q2 = qf_s[step * 32 + lane];
                b0 = q2.x;
                b1 = q2.y;
              } else {
                b0 = qf[step * 2];
                b1 = qf[step * 2 + 1];
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if (k + i == 0) mma16816_zero(acc[mt][n], f[mt][0], f[mt][1], f[mt][2], f[mt][3], b0, b1);
                else mma16816(acc[mt][n], f[mt][0], f[mt][1], f[mt][2], f[mt][3], b0, b1);
              }
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t* kp = reinterpret_cast<const uint32_t*>(st + 2 * P::kCode) + mt * 16 * G;
          const uint32_t p0 = kp[g * G + gr], p1 = kp[(g + 8) * G + gr];
          // the operand was 64 + code
          const float b0 = fmaf(-64.f, bf16lo(p0), bf16hi(p0)), b1 = fmaf(-64.f, bf16lo(p1), bf16hi(p1));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float x0 = xs[n][0][gr], x1 = xs[n][1][gr];
            if (gr == 0) {
              s[mt][n][0] = fmaf(bf16lo(p0), acc[mt][n][0], b0 * x0);
              s[mt][n][1] = fmaf(bf16lo(p0), acc[mt][n][1], b0 * x1);
              s[mt][n][2] = fmaf(bf16lo(p1), acc[mt][n][2], b1 * x0);
              s[mt][n][3] = fmaf(bf16lo(p1), acc[mt][n][3], b1 * x1);
            } else {
              s[mt][n][0] = fmaf(bf16lo(p0), acc[mt][n][0], fmaf(b0, x0, s[mt][n][0]));
              s[mt][n][1] = fmaf(bf16lo(p0), acc[mt][n][1], fmaf(b0, x1, s[mt][n][1]));
              s[mt][n][2] = fmaf(bf16lo(p1), acc[mt][n][2], fmaf(b1, x0, s[mt][n][2]));
              s[mt][n][3] = fmaf(bf16lo(p1), acc[mt][n][3], fmaf(b1, x1, s[mt][n][3]));
            }
          }
        }
      }
      if (masked || !split_finish<D, NT, CTAS, false>(A, s, st, st_u, t0, gaps, wk.q.sp.held, g, k_))
        split_finish<D, NT, CTAS, true>(A, s, st, st_u, t0, gaps, wk.q.sp.held, g, k_);
      __syncwarp();
      fetch(slot);
      slot = slot + 1 == ST ? 0 : slot + 1;
    }

    // ---- join the CTA's warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          A.l[n][k] += __shfl_xor_sync(kFull, A.l[n][k], x);
#pragma unroll
          for (int gr = 0; gr < G; ++gr) A.bias[n][k][gr] += __shfl_xor_sync(kFull, A.bias[n][k][gr], x);
        }
        if (A.pass[n][k] == -INFINITY) A.mm[n][k] = -INFINITY;  // no score: the warp's part counts for nothing
        if (g == 0) s_m[warp][n * 8 + 2 * c + k] = A.mm[n][k];
      }
    __syncthreads();
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) top = fmaxf(top, s_m[w][n * 8 + 2 * c + k]);
        f[n][k] = A.mm[n][k] == top ? 1.f : ex2(A.mm[n][k] - top);
        if (g == 0) s_l[warp][n * 8 + 2 * c + k] = A.l[n][k] * f[n][k];
      }
    const bool whole = wk.i0 == 0 && wk.i1 == wk.q.tiles;
    const SplitWs ws{reinterpret_cast<int*>(static_cast<char*>(a.ws) + 256), reinterpret_cast<float*>(static_cast<char*>(a.ws) + kAttnHead)};
    float* part = ws.part + ((long long)cta * 2 + (wk.i0 == 0)) * (C * (D + 2));
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += RD) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int gr = d0 / 64; gr < (d0 + RD) / 64; ++gr) {
            float* dst = area + (warp * C + n * 8 + 2 * c + k) * RS + (gr - d0 / 64) * 64 + g * 4;
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = fmaf(A.o[n][gr][j][k], A.unit, A.bias[n][k][gr]) * f[n][k];
              v[4 + j] = fmaf(A.o[n][gr][j][2 + k], A.unit, A.bias[n][k][gr]) * f[n][k];
            }
            *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(dst + 32) = make_float4(v[4], v[5], v[6], v[7]);
          }
      __syncthreads();
      for (int i = threadIdx.x; i < ncol * (RD / 4); i += kSplitThreads) {
        const int col = i / (RD / 4), d4 = i % (RD / 4) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(area + (w * C + col) * RS + d4);
          acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
          sum += s_l[w][col];
        }
        if (whole) {
          const int j = (col0 + col) / group, hh = col0 + col - j * group, row = wk.q.sp.first + j;
          const float r = sum == 0.f ? 0.f : 1.f / sum;
          if (row >= 0 && row < a.v.rows)
            *reinterpret_cast<uint2*>(a.out + (long long)row * a.out_stride + (h * group + hh) * D + d0 + d4) =
                make_uint2((uint32_t)f2bf(acc.x * r) | (uint32_t)f2bf(acc.y * r) << 16,
                           (uint32_t)f2bf(acc.z * r) | (uint32_t)f2bf(acc.w * r) << 16);
        } else {
          *reinterpret_cast<float4*>(part + col * D + d0 + d4) = acc;
        }
      }
      if (d0 + RD < D) __syncthreads();
    }
    if ((int)threadIdx.x < ncol) {
      const int col = threadIdx.x;
      float sum = 0.f, top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) {
        sum += s_l[w][col];
        top = fmaxf(top, s_m[w][col]);
      }
      if (whole) {
        const int j = (col0 + col) / group, hh = col0 + col - j * group, row = wk.q.sp.first + j;
        if (a.lse && row >= 0 && row < a.v.rows)
          a.lse[(long long)row * a.q_heads + h * group + hh] = sum == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(sum));
      } else {
        part[C * D + col] = top;
        part[C * D + C + col] = sum;
      }
    }
    if (!whole) {  // the last CTA to arrive joins the unit's parts
      const long long u0 = wk.x, u1 = u0 + wk.q.tiles - 1;  // the places of the unit's first and last tile
      const int c0 = split_cta(u0, ctas, total), c1 = split_cta(u1, ctas, total);
      bool top_level = !split_two_levels(c1 - c0 + 1, ncol, D);
      SplitJoin join = top_level ? split_all(c0, c1, false) : split_eight(c0, c1, cta, gridDim.x);
      if (join.counter < 0) {  // an eight of one part is joined as it stands
        join = split_all(c0, c1, true);
        top_level = true;
      }
      for (;;) {
        const int first = join.first, step = join.step, n = join.n;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
          int* const count = ws.count + join.counter;
          const int last = atomicAdd(count, 1) == n - 1;
          if (last) *count = 0;
          s_last = last;
        }
        __syncthreads();
        if (!s_last) break;
        __threadfence();
        auto at = [&](int i) {
          const int p = first + i * step;
          return ws.part + ((long long)(c0 + p) * 2 + (p == 0)) * (C * (D + 2));
        };
        // the parts' weights: 2^(m - largest m), over the sum at last; a warp a column
        float* const wm = area;
        for (int i = threadIdx.x; i < n * ncol; i += kSplitThreads) wm[i] = __ldcg(at(i / ncol) + C * D + i % ncol);
        __syncthreads();
        for (int col = warp; col < ncol; col += kSplitWarps) {
          float top = -INFINITY, sum = 0.f;
          for (int p = lane; p < n; p += 32) top = fmaxf(top, wm[p * ncol + col]);
          top = warp_max(top);
          for (int p = lane; p < n; p += 32) {
            const float mp = wm[p * ncol + col];
            sum = fmaf(mp == top ? 1.f : ex2(mp - top), __ldcg(at(p) + C * D + C + col), sum);
          }
          sum = warp_sum(sum);
          const float r = !top_level ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
          for (int p = lane; p < n; p += 32) {
            const float mp = wm[p * ncol + col];
            wm[p * ncol + col] = (mp == top ? 1.f : ex2(mp - top)) * r;
          }
          const int j = (col0 + col) / group, hh = col0 + col - j * group, row = wk.q.sp.first + j;
          if (lane == 0) {
            if (!top_level) {  // the eight's first part becomes all of it
              at(0)[C * D + col] = top;
              at(0)[C * D + C + col] = sum;
            } else if (a.lse && row >= 0 && row < a.v.rows) {
              a.lse[(long long)row * a.q_heads + h * group + hh] = sum == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(sum));
            }
          }
        }
        __syncthreads();
        // every thread four columns of a row; with threads to spare, the parts are dealt out over them
        const int items = ncol * (D / 4), deal = max(1, kSplitThreads / items);
        float4* const sums = reinterpret_cast<float4*>(area + (n * ncol + 3) / 4 * 4);
        for (int i0 = 0; i0 < items; i0 += kSplitThreads) {
          const int i = i0 + (int)threadIdx.x % (items < kSplitThreads ? items : kSplitThreads);
          const int share = items < kSplitThreads ? threadIdx.x / items : 0;
          const int col = i / (D / 4), d4 = i % (D / 4) * 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < items && share < deal) {
#pragma unroll 8
            for (int p = share; p < n; p += deal) {
              const float w = wm[p * ncol + col];
              const float4 v = __ldcg(reinterpret_cast<const float4*>(at(p) + col * D + d4));
              acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
              acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
            }
            if (deal > 1) sums[share * items + i] = acc;
          }
          if (deal > 1) __syncthreads();
          if (i < items && share == 0) {
            for (int k = 1; k < deal; ++k) {
              const float4 v = sums[k * items + i];
              acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
            }
            const int j = (col0 + col) / group, hh = col0 + col - j * group, row = wk.q.sp.first + j;
            if (!top_level)
              *reinterpret_cast<float4*>(at(0) + col * D + d4) = acc;
            else if (row >= 0 && row < a.v.rows)
              *reinterpret_cast<uint2*>(a.out + (long long)row * a.out_stride + (h * group + hh) * D + d4) =
                  make_uint2((uint32_t)f2bf(acc.x) | (uint32_t)f2bf(acc.y) << 16, (uint32_t)f2bf(acc.z) | (uint32_t)f2bf(acc.w) << 16);
          }
        }
        if (top_level) break;
        join = split_all(c0, c1, true);
        top_level = true;
      }
    }
    __syncthreads();  // the join area and the sums are free again
  }
  cp_wait<0>();
}

// Columns a unit takes: the smallest of 8 and 16 that holds a whole sequence's, else 16.
static int split_nt(int max_q, int q_heads, int kv_heads) { return (long long)max_q * (q_heads / kv_heads) <= 8 ? 1 : 2; }

// CTAs per SM: two, but one where units are few (then each has parts of many CTAs) or registers would be spilled. In us,
// two and one: 131071 tokens, 8 key heads of 128, 4 columns: 44.7, 43.2; 8000 tokens: 18.8, 15.3; 65536 tokens, 2 key heads, 8
// columns: 24.3, 20.0; 64 sequences of 512 to 16384 tokens, 8 key heads, 4 columns: 86.1, 92.3. Head dim 256, 131071 tokens:
// 108, 70.
static int split_ctas(int d, int nt, int batch, int kv_heads) {
  return d * nt >= 256 || (long long)batch * kv_heads <= num_sms() ? 1 : 2;
}
static int split_grid(int ctas) {
  const int n = num_sms() * ctas;
  return n < kSplitMaxGrid ? n : kSplitMaxGrid;
}

size_t split_workspace_bytes(int batch, int max_q, int q_heads, int kv_heads, int d) {
  const int nt = split_nt(max_q, q_heads, kv_heads);
  const int grid = split_grid(split_ctas(d, nt, batch, kv_heads));
  return kAttnHead + (((size_t)grid * 2 * 8 * nt * (d + 2) * 4 + 255) & ~(size_t)255);
}

template <int D, int NT, int CTAS>
static cudaError_t launch_split_t(const AttnArgs& a, cudaStream_t s) {
  using P = Split<D, NT, CTAS>;
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem(k_attn_split<D, NT, CTAS>, P::kSmem, allowed);
  if (e != cudaSuccess) return e;
  return launch_overlapped(k_attn_split<D, NT, CTAS>, split_grid(CTAS), kSplitThreads, P::kSmem, s, a);
}

cudaError_t launch_attn_split(const AttnArgs& a, cudaStream_t s) {
  const int nt = split_nt(a.max_q, a.q_heads, a.c.kv_heads), d = a.c.head_dim;
  const bool two = split_ctas(d, nt, a.v.batch, a.c.kv_heads) == 2;
  if (d == 64 && nt == 1) return two ? launch_split_t<64, 1, 2>(a, s) : launch_split_t<64, 1, 1>(a, s);
  if (d == 64) return two ? launch_split_t<64, 2, 2>(a, s) : launch_split_t<64, 2, 1>(a, s);
  if (d == 128 && nt == 1) return two ? launch_split_t<128, 1, 2>(a, s) : launch_split_t<128, 1, 1>(a, s);
  if (d == 128) return launch_split_t<128, 2, 1>(a, s);
  return nt == 1 ? launch_split_t<256, 1, 1>(a, s) : launch_split_t<256, 2, 1>(a, s);
}

}  // namespace bgq
