// f8_many.cu — products of e4m3 matrices for many rows, on tcgen05.
//
// Tiles of 256 rows of x by 256 rows of W (gated: 128 of gate beside the same 128 of up; fewer rows of W where that keeps more SMs busy),
// each the work of two CTAs that share their matrix instructions: a CTA brings 128 rows of x and half of W's for every block of 128
// columns, and has the sums of its 128 rows of x and all of W's in tensor memory. A pair of CTAs on every two SMs walks through the tiles.
// The warps are specialised: one copies, one (of the first CTA) issues, four keep the scales in tensor memory
// (f8_tc.cuh), four write the results, a thread a row; of a pair's last tile the scales' warps write half.
//
// Tensor memory has 512 columns: two tiles' sums of 256 and four sets of scales of 12 do not fit beside each other. The second
// tile's sums start kManyShared columns before the first's end, and a tile's epilogue reads those columns first: the next tile's
// instructions wait for them alone.
//
// What bounds it: the matrix instructions, 128 cycles for 256 x 256 x 32, beside them the operands' bytes (64 KB a pair in 512 cycles, where an
// SM takes 62 bytes a cycle), and the power that all of it draws. 8191 x 12288 x 4096: 226 to 244 us, 3.5 PFLOP/s, 373k cycles of which the
// instructions take 344k, at 1.6 GHz where the SMs could run at 2.07; the rest is the wait between tiles (1800 cycles for the last
// instructions and the shared columns). Gated 4095 x 2 * 12288 x 4096: 238 to 264 us. For seconds on end (1.4 kW): 267 and 271 to 283 us.
// A launch of one tile a pair spends 5 to 8 us besides its instructions (777 x 4096 x 8192: 25 us).
// What it took: instructions issued by a whole warp with one elected lane, so that descriptors stay in uniform registers (358 -> 313 us);
// scales in four sets, loaded far ahead (267); arrivals that release nothing (243); results by TMA stores (235).
#include "f8_tc.cuh"

namespace bgq {

constexpr int kManyThreads = 384;  // warp 0: copies, 1: instructions, 2: tensor memory, 4-7: scales, 8-11: results
constexpr int kManyStages = 6, kManyStage = 2 * kF8Tile;
constexpr int kManySets = 4;                 // sets of scales, 16 columns apart: x's 4, then W's 8
constexpr int kManyScales = 512 - 16 * kManySets;
constexpr int kManyShared = 16 * kManySets;  // columns that both tiles' sums use
constexpr int kManyBars = 2 * kManyStages + 2 * kManySets + 3;
constexpr size_t kManySmem = 1024 + (size_t)kManyStages * kManyStage + 4 * 2 * kF8Room;

struct ManyWork {
  int tiles, down, group;  // tiles; tiles of x's rows; of which `group` are walked through beside each other
  int across;
  int wide;  // rows of W a tile: 256, or less (in thirty-twos, as the instructions of two CTAs take them) where that leaves fewer SMs idle at the end; gated 128 of each
  // Tile i: groups of `group` tiles of x's rows by all of W's, so that what runs at a time shares both operands.
  __device__ __forceinline__ void at(int i, int& m, int& n) const {
    const int wide = group * across, g = i / wide, in = i - g * wide, h = min(group, down - g * group);
    n = in / h;
    m = g * group + in - n * h;
  }
};

struct ManyOut {
  CUtensorMap y, yf, h;  // those that are wanted
};

// WHOLE: tiles of 256 rows of W (gated ones always; known to the compiler, they take 1 to 2 % less time).
template <bool GATED, bool WHOLE>
__global__ void __launch_bounds__(kManyThreads, 1)
    k_f8_many(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw0,
              const __grid_constant__ CUtensorMap mw1, const __grid_constant__ ManyOut out, const F8Prod p, const ManyWork work) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint64_t bars[kManyBars];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  unsigned char* stages = smem_raw + (1024 - (tc_smem(smem_raw) & 1023)) % 1024;
  uint64_t *full = bars, *empty = full + kManyStages, *sf_full = empty + kManyStages, *sf_free = sf_full + kManySets,
           *acc_full = sf_free + kManySets, *acc_free = acc_full + 2;
  volatile int* fail = &s_fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = f8_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int blocks = f8_blocks(p.K), groups = (blocks + 3) >> 2;
  const int cols = WHOLE ? kManyCols : work.wide;  // of a tile's sums
  if (tid == 0) {
    for (int i = 0; i < kManyStages; ++i) {
      tc_mbar_init(&full[i]);
      tc_mbar_init(&empty[i]);
    }
    for (int i = 0; i < kManySets; ++i) {
      tc_mbar_init(&sf_full[i], 8);  // four warps of each CTA
      tc_mbar_init(&sf_free[i]);
    }
    for (int i = 0; i < 2; ++i) tc_mbar_init(&acc_full[i]);
    tc_mbar_init(acc_free, 8);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    f8_map_ahead(&mx);
    f8_map_ahead(rank ? &mw1 : &mw0);
  }
  // The other CTA's barriers are there before anything is copied for them. (That its tensor memory is there, too, its scales tell.)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();  // tensor memory, too, is taken only once earlier kernels have given theirs back
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // Scales: a lane has those of x's rows l, 32 + l, ...; W's are the same for a whole block of 128 rows.
  // A chunk: the words of four groups of blocks. They are loaded a chunk ahead, of this tile or the next (loaded a group
  // or two ahead, they held the instructions up: 8191 x 12288 x 4096 took 298 us, 267 so).
  const int wbs = f8_blocks(p.N);
  // A tile's rows of W lie in up to three blocks of 128 (gated: a block of gate, then one of up): `pick` has two bits for each 32 of
  // them, which of the three words this lane's row takes.
  struct Chunk {
    uint32_t x[4][4], w[4][3], pick;
  } cur = {}, next = {};
  int li = pair, lg = 0;  // tile and first group of the next chunk
  auto load = [&](Chunk& v) {
    if (li >= work.tiles) return;
    int tm, tn;
    work.at(li, tm, tn);
    const int m0 = tm * kManyRows + (int)rank * 128 + lane, n0 = GATED ? tn * 128 : tn * cols, wb = n0 / kF8Block;
    const uint8_t* x = p.xs + (int64_t)m0 * p.xs_stride + 4 * lg;
    const uint8_t* w0 = p.ws[0] + wb * p.ws_stride[0] + 4 * lg;
    const uint8_t* w1 = GATED ? p.ws[1] + wb * p.ws_stride[1] + 4 * lg : w0 + (wb + 1 < wbs ? p.ws_stride[0] : 0);
    const uint8_t* w2 = WHOLE ? w1 : w0 + (wb + 2 < wbs ? 2 * p.ws_stride[0] : 0);
    if (!WHOLE) {
      v.pick = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) v.pick |= (uint32_t)(((n0 & 127) + 32 * j + lane) >> 7) << 2 * j;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const bool there = lg + g < groups;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v.x[g][j] = there && m0 + 32 * j < p.M ? *reinterpret_cast<const uint32_t*>(x + 32 * j * p.xs_stride + 4 * g) : 0u;
      v.w[g][0] = there ? *reinterpret_cast<const uint32_t*>(w0 + 4 * g) : 0u;
      v.w[g][1] = there ? *reinterpret_cast<const uint32_t*>(w1 + 4 * g) : 0u;
      v.w[g][2] = there && !WHOLE ? *reinterpret_cast<const uint32_t*>(w2 + 4 * g) : 0u;
    }
    if ((lg += 4) >= groups) {
      lg = 0;
      li += pairs;
    }
  };
  if (warp >= 4 && warp < 8) load(cur);
  if (warp == 2) f8_tmem_alloc(&s_tmem, 512);
  if (warp > 0) {  // warp 0 needs none of it
    tc_fence_before();
    asm volatile("bar.sync 1, 352;" ::: "memory");
    tc_fence_after();
    pdl_trigger();
  }
  const uint32_t tmem = s_tmem;

  // Results. A warp that writes them has two rooms; the scales' warps, which share a pair's last tile, have theirs in the ring.
  unsigned char* rooms = stages + (warp >= 8 ? kManyStages * kManyStage : 0) + (warp & 3) * 2 * kF8Room;
  const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
  int room = 0;
  auto store = [&](const uint4(&line)[8], const CUtensorMap* map, int col, int row) {
    f8_store_rows(rooms + room * kF8Room, line, map, col, row);
    room ^= 1;
  };
  // 64 columns of the warp's rows, of which a thread has a row. (A TMA store writes 16 bytes or nothing: where the columns end
  // within that, the last pieces are written value by value.)
  auto store64 = [&](const float(&lo)[32], const float(&hi)[32], int col, int row) {
    uint4 line[8];
    if (row >= p.M) return;
    const int left = row + lane < p.M ? p.N - col : 0;
    if (p.y && col < p.N) {
      if (col + 64 <= p.N || p.N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) line[i] = f8_bf16x8(i < 4 ? &lo[8 * i] : &hi[8 * i - 32]);
        store(line, &out.y, col, row);
      } else {
        uint16_t* y = p.y + (int64_t)(row + lane) * p.y_stride + col;
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i < left) y[i] = f2bf(i < 32 ? lo[i & 31] : hi[i & 31]);
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c = col + 32 * half;
      if (!p.yf || c >= p.N) continue;
      if (c + 32 <= p.N || p.N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) line[i] = f8_fp32x4(half ? &hi[4 * i] : &lo[4 * i]);
        store(line, &out.yf, c, row);
      } else {
        float* y = p.yf + (int64_t)(row + lane) * p.y_stride + c;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < left - 32 * half) y[i] = half ? hi[i] : lo[i];
      }
    }
  };
  // 64 columns, the c-th, of a tile's sums at `acc`, from the end or from the beginning (what is left of less than 64 is written again
  // with columns beside it).
  const int chunks = (cols + 63) / 64;
  auto sums64 = [&](int c, bool back, uint32_t acc, int tn, int row, auto read) {
    const int first = back ? max(0, cols - 64 * (c + 1)) : min(64 * c, cols - 64);
    float v[2][32];
    f8_tmem_ld32(acc + first, v[0]);
    f8_tmem_ld32(acc + first + 32, v[1]);
    read(v);
    store64(v[0], v[1], tn * cols + first, row);
  };
  auto plain_read = [](float(&)[2][32]) { f8_tmem_ld_wait(); };

  if (warp == 0) {
    if (lane == 0) {
      const CUtensorMap* mw = GATED && rank ? &mw1 : &mw0;
      int s = 0;
      uint32_t par = 1;
      bool ok = true;
      for (int i = pair; ok && i < work.tiles; i += pairs) {
        int tm, tn;
        work.at(i, tm, tn);
        const int m0 = tm * kManyRows + (int)rank * 128;
        const int n0 = GATED ? tn * 128 : tn * cols + (int)rank * (cols / 2);
        for (int b = 0; b < blocks; ++b) {
          if (!(ok = f8_wait(&empty[s], par, fail))) break;
          unsigned char* st = stages + s * kManyStage;
          const uint32_t bar = f8_at(&full[s], 0);
          if (rank == 0) f8_expect(&full[s], 2 * kF8Tile + 128 * cols);
          f8_load<2>(st, &mx, b * 128, m0, bar);
          f8_load<2>(st + kF8Tile, mw, b * 128, n0, bar);
          if (++s == kManyStages) {
            s = 0;
            par ^= 1;
          }
        }
      }
      // every stage's last use is over, and told, before the CTA may end
      for (int i = 0; ok && i < kManyStages; ++i) {
        ok = f8_wait(&empty[s], par, fail);
        if (++s == kManyStages) {
          s = 0;
          par ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t lead = f8_elect();
      int s = 0, set = 0, t = 0;
      uint32_t par = 0, sf_par = 0;
      bool ok = true;
      for (int i = pair; ok && i < work.tiles; i += pairs, ++t) {
        if (t && !(ok = __all_sync(kFull, f8_wait(acc_free, (t - 1) & 1, fail)))) break;
        const uint32_t d = tmem + (t & 1 ? kManyCols - kManyShared : 0);
        for (int b = 0; b < blocks; ++b) {
          const int sf = b & 3;
          if (sf == 0 && !(ok = __all_sync(kFull, f8_wait(&sf_full[set], sf_par, fail)))) break;
          if (!(ok = __all_sync(kFull, f8_wait(&full[s], par, fail)))) break;
          tc_fence_after();
          const uint32_t at = tc_smem(stages + s * kManyStage), scales = tmem + kManyScales + set * 16;
          const uint64_t a = f8_desc(at), w = f8_desc(at + kF8Tile);
          const uint32_t idesc = f8_idesc(kManyRows, cols, sf);
#pragma unroll
          for (int k = 0; k < 4; ++k) f8_tc_mma<2>(d, a + 2 * k, w + 2 * k, idesc, scales, scales + 4, (b | k) ? 1u : 0u, lead);
          f8_commit<2>(&empty[s], lead);
          if (++s == kManyStages) {
            s = 0;
            par ^= 1;
          }
          if (sf == 3 || b == blocks - 1) {
            f8_commit<2>(&sf_free[set], lead);
            if (++set == kManySets) {
              set = 0;
              sf_par ^= 1;
            }
          }
        }
        if (ok) f8_commit<2>(&acc_full[t & 1], lead);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21) + kManyScales, ready = f8_at(&sf_full[0], 0);
    int set = 0;
    uint32_t par = 1;
    bool ok = true;
    for (int i = pair; ok && i < work.tiles; i += pairs)
      for (int g0 = 0; ok && g0 < groups; g0 += 4) {
        load(next);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (!ok || g0 + g >= groups) continue;
          if (!(ok = __all_sync(kFull, f8_wait(&sf_free[set], par, fail)))) continue;
          tc_fence_after();
          f8_tmem_st4(at + set * 16, cur.x[g][0], cur.x[g][1], cur.x[g][2], cur.x[g][3]);
          auto word = [&](int j) {
            if (WHOLE) return cur.w[g][j >> 2];
            const uint32_t k = cur.pick >> 2 * j & 3;
            return k == 0 ? cur.w[g][0] : k == 1 ? cur.w[g][1] : cur.w[g][2];
          };
          f8_tmem_st4(at + set * 16 + 4, word(0), word(1), word(2), word(3));
          f8_tmem_st4(at + set * 16 + 8, word(4), word(5), word(6), word(7));
          f8_tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) f8_arrive_at(ready + 8 * set);
          if (++set == kManySets) {
            set = 0;
            par ^= 1;
          }
        }
        cur = next;
      }
    for (int i = 0; ok && i < kManySets; ++i) {
      ok = __all_sync(kFull, f8_wait(&sf_free[set], par, fail));
      if (++set == kManySets) {
        set = 0;
        par ^= 1;
      }
    }
    if (!GATED && ok) {
      const int t = (work.tiles - 1 - pair) / pairs;
      int tm, tn;
      work.at(pair + t * pairs, tm, tn);
      ok = __all_sync(kFull, f8_wait(&acc_full[t & 1], (t >> 1) & 1, fail));
      tc_fence_after();
      const bool back = (t & 1) == 0;
#pragma unroll 1
      for (int c = (chunks + 1) / 2; ok && c < chunks; ++c)
        sums64(c, back, lanes + (back ? 0 : kManyCols - kManyShared), tn, tm * kManyRows + (int)rank * 128 + (warp & 3) * 32, plain_read);
      f8_stores_done();
    }
  } else if (warp >= 8) {
    const uint32_t freed = f8_at(acc_free, 0);
    int t = 0;
    for (int i = pair; i < work.tiles; i += pairs, ++t) {
      int tm, tn;
      work.at(i, tm, tn);
      const int row = tm * kManyRows + (int)rank * 128 + (warp & 3) * 32;  // the warp's first
      if (!__all_sync(kFull, f8_wait(&acc_full[t & 1], (t >> 1) & 1, fail))) break;
      tc_fence_after();
      // the columns that the next tile wants come first: the last ones of the first sums, the first of the second
      const bool back = (t & 1) == 0;
      const uint32_t acc = lanes + (back ? 0 : kManyCols - kManyShared);
      auto drained = [&](float(&v)[2][32]) {
        f8_tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) f8_arrive_at(freed);
#pragma unroll
        for (int j = 0; j < 64; ++j) asm volatile("" : "+f"(v[j >> 5][j & 31]));  // what is done with them comes behind the arrival
      };
      static_assert(kManyShared == 64, "two chunks of 32 columns");
      if (!GATED) {
        // (of a pair's last tile the scales' warps, which are done, have the second half)
        const int most = i + pairs < work.tiles ? chunks : (chunks + 1) / 2;
        sums64(0, back, acc, tn, row, drained);
#pragma unroll 1
        for (int c = 1; c < most; ++c) sums64(c, back, acc, tn, row, plain_read);
      } else {
        // columns 64 c .. of the result, c = 1, 0 or 0, 1
        float h[2][2][32];
        float most = 0.f;
        auto column = [&](int c) { return 64 * (back ? 1 - c : c); };
        auto join = [&](auto& g, auto& u) {  // 32 columns, or 16
          constexpr int n = sizeof(g) / sizeof(float);
          float least = fminf(g[0], g[1]);
#pragma unroll
          for (int j = 2; j < n; j += 2) least = f8_min3(least, g[j], g[j + 1]);
          if (__any_sync(kFull, least < kF8Far)) {  // one branch for all of the warp: far gates are rare
#pragma unroll
            for (int j = 0; j < n; ++j) f8_nearer(g[j], u[j]);
          }
#pragma unroll
          for (int j = 0; j < n; ++j) g[j] = f8_swiglu_near(g[j], u[j]);
#pragma unroll
          for (int j = 0; j < n; j += 2) most = f8_most3(most, g[j], g[j + 1]);
        };
        // the shared columns are the second half of up's sums, or the first of gate's
        float u[2][32];
        if (back) {
          f8_tmem_ld32(acc + 128 + 64, u[0]);
          f8_tmem_ld32(acc + 128 + 96, u[1]);
          drained(u);
          f8_tmem_ld32(acc + 64, h[0][0]);
          f8_tmem_ld32(acc + 96, h[0][1]);
        } else {
          f8_tmem_ld32(acc, h[0][0]);
          f8_tmem_ld32(acc + 32, h[0][1]);
          drained(h[0]);
          f8_tmem_ld32(acc + 128, u[0]);
          f8_tmem_ld32(acc + 128 + 32, u[1]);
        }
        f8_tmem_ld_wait();
        join(h[0][0], u[0]);
        join(h[0][1], u[1]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // (32 at a time the registers do not suffice: 2048 x 2 * 4096 x 1024 22.5 us, 20.5 so)
          auto& g = *reinterpret_cast<float(*)[16]>(&h[1][c >> 1][16 * (c & 1)]);
          auto& v = *reinterpret_cast<float(*)[16]>(&u[0][0]);
          f8_tmem_ld16(acc + column(1) + 16 * c, g);
          f8_tmem_ld16(acc + 128 + column(1) + 16 * c, v);
          f8_tmem_ld_wait();
          join(g, v);
        }
        if (p.y)
#pragma unroll
          for (int c = 0; c < 2; ++c) store64(h[c][0], h[c][1], tn * 128 + column(c), row);
        if (p.h) {
          const uint32_t top = __float_as_uint(most);
          const bool fine = f8_finite(top);
          const int byte = fine ? f8_scale_byte(top) : kF8One;
          const float inv = f8_inverse(byte);
          if (row + lane < p.M) p.hs[(int64_t)(row + lane) * p.hs_stride + tn] = (uint8_t)byte;
          uint4 line[8], codes[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float* v = &h[j >> 2][(j >> 1) & 1][16 * (j & 1)];
            codes[j] = make_uint4(kF8Nan4, kF8Nan4, kF8Nan4, kF8Nan4);
            if (fine)
              codes[j] = make_uint4(f8_codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv), f8_codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv),
                                    f8_codes4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
                                    f8_codes4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) line[j] = back ? codes[(j + 4) & 7] : codes[j];
          if (row < p.M) store(line, &out.h, tn * 128, row);
        }
      }
    }
    f8_stores_done();
  }
  __syncwarp();
  if (*fail && lane == 0)  // a wait has run out: the other CTA's end too
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(f8_at(&s_fail, rank ^ 1)), "r"(1) : "memory");
  tc_fence_before();
  if (__syncthreads_or(*fail)) {  // copies in flight land before the CTA ends
    if (tid == 0) atomicExch(&p.ctrl->status, BGQ_ERR_TIMEOUT);
    for (const unsigned long long t0 = tc_time(); tc_time() - t0 < 5000000ull;) __nanosleep(10000);
    __syncwarp();
  }
  f8_cluster_sync();
  if (warp == 2) f8_tmem_free(tmem, 512);
}

cudaError_t launch_f8_many(const F8Prod& p, bool gated, cudaStream_t s) {
  const int pairs = num_sms() / 2 > 0 ? num_sms() / 2 : 1, wide = gated ? 128 : f8_many_wide({p.M, p.N, p.K, gated}, pairs);
  CUtensorMap mx, mw[2];
  if (!f8_map(&mx, p.x, p.M, p.K, p.x_stride)) return cudaErrorInvalidValue;
  for (int i = 0; i < (gated ? 2 : 1); ++i)
    if (!f8_map(&mw[i], p.w[i], p.N, p.K, p.w_stride[i], gated ? 128 : wide / 2)) return cudaErrorInvalidValue;
  ManyOut out = {};
  if (p.y && !f8_out_map(&out.y, p.y, 2, p.M, p.N, p.y_stride)) return cudaErrorInvalidValue;
  if (p.yf && !f8_out_map(&out.yf, p.yf, 4, p.M, p.N, p.y_stride)) return cudaErrorInvalidValue;
  if (p.h && !f8_out_map(&out.h, p.h, 1, p.M, p.N, p.h_stride)) return cudaErrorInvalidValue;
  ManyWork work;
  work.down = (p.M + kManyRows - 1) / kManyRows;
  work.across = (p.N + wide - 1) / wide;
  work.wide = wide;
  work.tiles = work.down * work.across;
  work.group = work.down < 8 ? work.down : 8;
  static std::atomic<uint64_t> known[3];
  const int which = gated ? 0 : wide == kManyCols ? 1 : 2;
  const auto kern = gated ? k_f8_many<true, true> : which == 1 ? k_f8_many<false, true> : k_f8_many<false, false>;
  const cudaError_t e = f8_room((const void*)kern, (int)kManySmem, known[which]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (work.tiles < pairs ? work.tiles : pairs));
  cfg.blockDim = dim3(kManyThreads);
  cfg.dynamicSmemBytes = kManySmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mx, mw[0], mw[gated ? 1 : 0], out, p, work);
}

}  // namespace bgq
