// f8_mid.cu — products of e4m3 matrices for a batch of rows, on tcgen05, the sum over columns split.
//
// Here W is the operand of 128 rows and x the other, of as many rows (a multiple of 16) as there are, so that a batch of
// 40 costs the matrix instructions 48 rows and W is read once. A tile of 128 rows of W is the work of a cluster of CTAs, each
// with a share of the columns: enough of them to have all SMs reading W at once. Their sums meet in distributed shared
// memory, where CTA r adds the rows r, r + split, ... of x over the shares, in order (the same bits every time), a warp a row: its 128
// sums lie side by side, so gated products find a block's largest magnitude in one step, and stores are whole lines. (Sent to the
// adding CTA instead, 64 rows took 7.7 us where they took 7.2.)
// The warps are specialised: one copies, one issues, four keep the scales in tensor memory (f8_tc.cuh); all eight write the
// results. Copies and scales start before tensor memory is there.
// What bounds it: W's bytes (1 row, 12288 x 4096: 10.5 to 11 us, of which 7.5 at 6.7 TB/s) behind 3 us of start, first loads and end; with
// more rows the shares' sums, which cross between SMs at 20 bytes a ns each (64 rows, 4096 x 4096: 7.0 us; gated 64 rows, 2 x 1024 x
// 4096: 6.7 to 7.0). Half the shared memory, so that the next launch's CTAs start beside this one's, gave nothing (12.0 us for 11.5), nor did asking
// W into L2 ahead of the wait for the kernel before.
#include <algorithm>

#include "f8_tc.cuh"

namespace bgq {

constexpr int kMidThreads = 256, kMidSets = 4;  // warp 0: copies, 1: instructions, 2: tensor memory, 4-7: scales; all: results
constexpr int kMidRing = 224 * 1024;  // bytes
constexpr int kMidMaxStages = 8, kMidMaxSplit = 8;  // 2^3

struct MidShape {
  int rows;    // of x a tile: a multiple of 16, at most 256 (gated 128)
  int split;   // CTAs that share a tile's columns
  int stages;  // each of DEEP blocks
  uint32_t tmem;  // columns of tensor memory
};

template <bool GATED>
__host__ __device__ inline int mid_block(int rows) { return (GATED ? 2 : 1) * kF8Tile + rows * 128; }

__device__ __forceinline__ float4 mid_ld_peer(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// DEEP: blocks a stage (one barrier for two saves the issuing warp a third of a block's time, where it is what bounds).
template <bool GATED, int DEEP>
__global__ void __launch_bounds__(kMidThreads, 1)
    k_f8_mid(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw0,
             const __grid_constant__ CUtensorMap mw1, const F8Prod p, const MidShape sh) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint64_t full[kMidMaxStages], empty[kMidMaxStages], sf_full[kMidSets], sf_free[kMidSets], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  unsigned char* stages = smem_raw + (1024 - (tc_smem(smem_raw) & 1023)) % 1024;
  volatile int* fail = &s_fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x / sh.split, share = blockIdx.x - tile * sh.split, n0 = tile * 128, m0 = blockIdx.y * sh.rows;
  const int all = f8_blocks(p.K), b0 = all * share / sh.split, b1 = all * (share + 1) / sh.split;
  const int block_bytes = mid_block<GATED>(sh.rows), stage_bytes = DEEP * block_bytes;
  constexpr int kAligned = ~(DEEP - 1);  // a stage's blocks end at a multiple of its depth, so that they lie in one word of scales
  const uint32_t scales = GATED ? 2 * sh.rows : sh.rows;  // columns behind the sums: W's 4 (and 4 of up), then x's 8
  if (tid == 0) {
    for (int i = 0; i < sh.stages; ++i) {
      tc_mbar_init(&full[i]);
      tc_mbar_init(&empty[i]);
    }
    for (int i = 0; i < kMidSets; ++i) {
      tc_mbar_init(&sf_full[i], 4);
      tc_mbar_init(&sf_free[i]);
    }
    tc_mbar_init(&done);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc_fence_proxy();
    f8_map_ahead(&mx);
    f8_map_ahead(&mw0);
    if (GATED) f8_map_ahead(&mw1);
  }
  pdl_wait();
  // Scales: a lane has those of x's rows l, 32 + l, ...; W's are the same for its whole tile. Words of four groups of blocks at a
  // time, the first while tensor memory is taken.
  const int c0 = b0 >> 2, c1 = (b1 + 3) >> 2;
  uint32_t xs[4][8], wsc[4][2];
  auto load = [&](int c) {
    const uint8_t* x = p.xs + (int64_t)(m0 + lane) * p.xs_stride + 4 * c;
    const uint8_t *w0 = p.ws[0] + tile * p.ws_stride[0] + 4 * c, *w1 = p.ws[1] + tile * p.ws_stride[1] + 4 * c;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const bool there = c + g < c1;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        xs[g][j] = there && 32 * j < sh.rows && m0 + lane + 32 * j < p.M ? *reinterpret_cast<const uint32_t*>(x + 32 * j * p.xs_stride + 4 * g) : 0u;
      wsc[g][0] = there ? *reinterpret_cast<const uint32_t*>(w0 + 4 * g) : 0u;
      wsc[g][1] = there && GATED ? *reinterpret_cast<const uint32_t*>(w1 + 4 * g) : 0u;
    }
  };
  if (warp >= 4) load(c0);
  // Copies, by the thread that set the barriers up.
  int next = b0, stage = 0;
  uint32_t par = 1;
  auto copy = [&] {
    unsigned char* st = stages + stage * stage_bytes;
    uint64_t* bar = &full[stage];
    const int end = min(b1, (next + DEEP) & kAligned);
    f8_expect(bar, (end - next) * block_bytes);
    for (; next < end; ++next, st += block_bytes) {
      f8_load<1>(st, &mw0, next * 128, n0, tc_smem(bar));
      if (GATED) f8_load<1>(st + kF8Tile, &mw1, next * 128, n0, tc_smem(bar));
      f8_load<1>(st + (GATED ? 2 : 1) * kF8Tile, &mx, next * 128, m0, tc_smem(bar));
    }
    if (++stage == sh.stages) {
      stage = 0;
      par ^= 1;
    }
  };
  if (warp == 2) tmem_alloc(&s_tmem, sh.tmem);
  // warp 0 tells that the barriers are there, and needs nothing of the others (waited for, its copies held them up: gated 64 x 2 *
  // 1024 x 4096 took 7.7 us)
  if (warp == 0) {
    asm volatile("bar.arrive 1, 256;" ::: "memory");
  } else {
    tc_fence_before();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    tc_fence_after();
    pdl_trigger();
  }

  if (warp == 0) {
    while (lane == 0 && next < b1 && f8_wait(&empty[stage], par, fail)) copy();
  } else if (warp == 1) {
    const uint32_t lead = f8_elect(), tmem = s_tmem;
    int s = 0, set = 0;
    uint32_t par = 0, sf_par = 0;
    bool ok = true;
    for (int b = b0; b < b1;) {
      if (((b & 3) == 0 || b == b0) && !(ok = __all_sync(kFull, f8_wait(&sf_full[set], sf_par, fail)))) break;
      if (!(ok = __all_sync(kFull, f8_wait(&full[s], par, fail)))) break;
      tc_fence_after();
      const uint32_t at = tc_smem(stages + s * stage_bytes), sc = tmem + scales + set * 16;
      const int end = min(b1, (b + DEEP) & kAligned), first = b;
#pragma unroll
      for (int i = 0; i < DEEP; ++i) {
        if (first + i >= end) break;
        const uint64_t w = f8_desc(at + i * block_bytes), u = f8_desc(at + i * block_bytes + kF8Tile),
                       x = f8_desc(at + i * block_bytes + (GATED ? 2 : 1) * kF8Tile);
        const uint32_t idesc = f8_idesc(128, sh.rows, (first + i) & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t acc = first + i > b0 || k ? 1u : 0u;
          f8_tc_mma<1>(tmem, w + 2 * k, x + 2 * k, idesc, sc, sc + 8, acc, lead);
          if (GATED) f8_tc_mma<1>(tmem + sh.rows, u + 2 * k, x + 2 * k, idesc, sc + 4, sc + 8, acc, lead);
        }
      }
      b = end;
      f8_commit<1>(&empty[s], lead);
      if (++s == sh.stages) {
        s = 0;
        par ^= 1;
      }
      if ((b & 3) == 0) {
        f8_commit<1>(&sf_free[set], lead);
        if (++set == kMidSets) {
          set = 0;
          sf_par ^= 1;
        }
      }
    }
    if (ok) f8_commit<1>(&done, lead);
  } else if (warp >= 4) {
    const uint32_t at = s_tmem + ((uint32_t)(warp & 3) << 21) + scales;
    int set = 0;
    uint32_t par = 1;
    bool ok = true;
    for (int c = c0; ok && c < c1; c += 4) {
      if (c > c0) load(c);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (!ok || c + g >= c1) continue;
        if (!(ok = __all_sync(kFull, f8_wait(&sf_free[set], par, fail)))) continue;
        tc_fence_after();
        f8_tmem_st4(at + set * 16, wsc[g][0], wsc[g][0], wsc[g][0], wsc[g][0]);
        if (GATED) f8_tmem_st4(at + set * 16 + 4, wsc[g][1], wsc[g][1], wsc[g][1], wsc[g][1]);
        f8_tmem_st4(at + set * 16 + 8, xs[g][0], xs[g][1], xs[g][2], xs[g][3]);
        if (sh.rows > 128) f8_tmem_st4(at + set * 16 + 12, xs[g][4], xs[g][5], xs[g][6], xs[g][7]);
        f8_tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_arrive(&sf_full[set]);
        if (++set == kMidSets) {
          set = 0;
          par ^= 1;
        }
      }
    }
  }
  __syncwarp();
  const bool ok = __all_sync(kFull, f8_wait(&done, 0, fail));
  tc_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&s_tmem;
  // the sums, a row of x after the other; every stage has been read by now
  float* sums = reinterpret_cast<float*>(stages);
  if (ok)
    for (int c = 16 * (warp >> 2); c < (int)scales; c += 32) {
      float v[16];
      f8_tmem_ld16(tmem + ((uint32_t)(warp & 3) << 21) + c, v);
      f8_tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[(c + i) * 128 + (warp & 3) * 32 + lane] = v[i];
    }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_free(tmem, sh.tmem);
  if (sh.split > 1) f8_cluster_sync();
  const int here = min(sh.rows, p.M - m0);
  for (int r = share + sh.split * warp; r < here; r += sh.split * (kMidThreads / 32)) {
    const uint32_t at = tc_smem(sums + r * 128 + lane * 4), up = at + sh.rows * 512;
    float4 g, u;
    if (sh.split > 1) {
      float4 gs[kMidMaxSplit], us[kMidMaxSplit];
#pragma unroll
      for (int q = 0; q < kMidMaxSplit; ++q)
        if (q < sh.split) {
          uint32_t peer;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(q));
          gs[q] = mid_ld_peer(peer);
          if (GATED) us[q] = mid_ld_peer(peer + (up - at));
        }
      g = gs[0];
      u = us[0];
#pragma unroll
      for (int q = 1; q < kMidMaxSplit; ++q)
        if (q < sh.split) {
          g = make_float4(g.x + gs[q].x, g.y + gs[q].y, g.z + gs[q].z, g.w + gs[q].w);
          if (GATED) u = make_float4(u.x + us[q].x, u.y + us[q].y, u.z + us[q].z, u.w + us[q].w);
        }
    } else {
      g = *reinterpret_cast<const float4*>(sums + r * 128 + lane * 4);
      if (GATED) u = *reinterpret_cast<const float4*>(sums + (sh.rows + r) * 128 + lane * 4);
    }
    if (GATED) g = f8_swiglu4(g, u);
    const int64_t row = m0 + r;
    const int n = n0 + lane * 4, left = p.N - n;
    if (p.y && left > 0) {
      const uint32_t lo = (uint32_t)f2bf(g.x) | ((uint32_t)f2bf(g.y) << 16), hi = (uint32_t)f2bf(g.z) | ((uint32_t)f2bf(g.w) << 16);
      uint16_t* y = p.y + row * p.y_stride + n;
      if (left >= 4) {
        *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
      } else {
        y[0] = (uint16_t)lo;
        if (left > 1) y[1] = (uint16_t)(lo >> 16);
        if (left > 2) y[2] = (uint16_t)hi;
      }
    }
    if (p.yf && left > 0) {
      float* y = p.yf + row * p.y_stride + n;
      if (left >= 4) {
        *reinterpret_cast<float4*>(y) = g;
      } else {
        y[0] = g.x;
        if (left > 1) y[1] = g.y;
        if (left > 2) y[2] = g.z;
      }
    }
    if (GATED && p.h) {
      const uint32_t abs = 0x7fffffffu;
      const uint32_t m = max(max(__float_as_uint(g.x) & abs, __float_as_uint(g.y) & abs),
                             max(__float_as_uint(g.z) & abs, __float_as_uint(g.w) & abs));
      const uint32_t top = __reduce_max_sync(kFull, left > 0 ? m : 0u);
      const bool fine = f8_finite(top);
      const int byte = fine ? f8_scale_byte(top) : kF8One;
      const float inv = f8_inverse(byte);
      if (left > 0)  // a multiple of 16
        *reinterpret_cast<uint32_t*>(p.h + row * p.h_stride + n) = fine ? f8_codes4(g.x * inv, g.y * inv, g.z * inv, g.w * inv) : kF8Nan4;
      if (lane == 0) p.hs[row * p.hs_stride + tile] = (uint8_t)byte;
    }
  }
  __syncwarp();
  // the peers' sums have been read, and this CTA's by them (nothing is written for another CTA, so nothing is released)
  if (sh.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (*fail) {  // a wait has run out: copies in flight land before the CTA ends
    if (tid == 0) atomicExch(&p.ctrl->status, BGQ_ERR_TIMEOUT);
    for (const unsigned long long t0 = tc_time(); tc_time() - t0 < 5000000ull;) __nanosleep(10000);
  }
  __syncwarp();
  if (sh.split > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Clusters of 2^n CTAs that the device can hold at once, one CTA an SM (`known`: by device and n, asked for once).
static int mid_clusters(const void* kern, size_t smem, int n, std::atomic<int> (&known)[64][4]) {
  int dev = 0, count = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (count = known[dev][n].load(std::memory_order_relaxed)) > 0) return count;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1 << n);
  cfg.blockDim = dim3(kMidThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1u << n;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&count, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 64) known[dev][n].store(count, std::memory_order_relaxed);
  return count;
}

template <bool GATED, int DEEP>
static cudaError_t mid_of(const F8Prod& p, const F8MidPlan& plan, MidShape sh, cudaStream_t s) {
  const int tiles = (p.N + 127) / 128, stage = DEEP * mid_block<GATED>(sh.rows);
  sh.stages = std::min(kMidRing / stage, kMidMaxStages);
  const uint32_t cols = (GATED ? 2 : 1) * sh.rows + 16 * kMidSets;
  for (sh.tmem = 32; sh.tmem < cols;) sh.tmem <<= 1;
  const int sums = (GATED ? 2 : 1) * sh.rows * 512;  // take the ring's place
  const size_t smem = 1024 + std::max(sh.stages * stage, sums);
  const void* kern = (const void*)k_f8_mid<GATED, DEEP>;
  static_assert(kMidRing >= 2 * 128 * 512, "the ring holds the most sums");
  static std::atomic<uint64_t> known;
  const cudaError_t e = f8_room(kern, 1024 + kMidRing, known);
  if (e != cudaSuccess) return e;
  // as many CTAs a tile as planned, if all are there at once
  static std::atomic<int> clusters[64][4];
  int n = __builtin_ctz(plan.split);
  while (n > 0 && tiles * plan.down > mid_clusters(kern, 1024 + kMidRing, n, clusters)) --n;
  sh.split = 1 << n;
  CUtensorMap mx, mw[2];
  if (!f8_map(&mx, p.x, p.M, p.K, p.x_stride, sh.rows)) return cudaErrorInvalidValue;
  for (int i = 0; i < 2; ++i)
    if (!f8_map(&mw[i], p.w[i], p.N, p.K, p.w_stride[i])) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * sh.split, plan.down);
  cfg.blockDim = dim3(kMidThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)sh.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_f8_mid<GATED, DEEP>, mx, mw[0], mw[1], p, sh);
}

template <bool GATED>
static cudaError_t mid(const F8Prod& p, const F8MidPlan& plan, cudaStream_t s) {
  MidShape sh = {};
  sh.rows = plan.rows;
  return 6 * mid_block<GATED>(sh.rows) <= kMidRing ? mid_of<GATED, 2>(p, plan, sh, s) : mid_of<GATED, 1>(p, plan, sh, s);
}

cudaError_t launch_f8_mid(const F8Prod& p, bool gated, const F8MidPlan& plan, cudaStream_t s) {
  return gated ? mid<true>(p, plan, s) : mid<false>(p, plan, s);
}

}  // namespace bgq
