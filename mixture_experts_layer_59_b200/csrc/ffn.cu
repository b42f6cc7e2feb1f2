// Shared (dense) gated feed-forward block, forward and backward: the expert
// every token passes, next to the routed ones.
//   UP    H = [x W1 | x W3], A = silu(H1) * H3   both projections, the
//                                                activation and the product
//   DOWN  y = A W2 (+ addend)
//   DAP   dA = dout W2^T; epilogue: A again from H, SwiGLU backward -> dH
//   DX    dx = dH1 W1^T + dH3 W3^T (+ addend)
//   DW    dW1 = x^T dH1, dW3 = x^T dH3, dW2 = A^T dout in one launch
// bf16 operands, fp32 accumulation; H, A, dH and the results are rounded
// once each to bf16 (they are stored, or feed the next product).
//
// One persistent kernel template, laid out as the grouped GEMMs are: a TMA
// producer warp, an MMA warp (tcgen05, 128 x BN x 16), eight epilogue warps,
// the accumulator double-buffered in TMEM.  Against the grouped kernels there
// is no row space: the tensor maps end at T, d and f, loads past them read
// zeros and stores past them are clipped, so any T and any d, f that are
// multiples of 8 (the 16-byte row strides TMA needs) work.
#include "common.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

enum FKind : int { F_UP = 0, F_DOWN = 1, F_DAP = 2, F_DX = 3, F_DW = 4 };

struct FfnArgs {
  CUtensorMap mA[3];   // DX: dH1, dH3; DW: the three products' A
  CUtensorMap mB[3];   // UP: W1, W3; DX: W1, W3; DW: the three products' B
  CUtensorMap sO[3];   // outputs (UP: H1, H3, A; DAP: dH1, dH3, A; DW: dW1, dW3, dW2)
  int T, d, f;
  int M[3], N[3];      // output rows and columns (UP: N counts the W1 columns)
  int mtiles[3], ntiles[3];
  int tile0, tiles;    // this launch: output tiles tile0 .. tiles - 1
  int kbs, kbh;        // k-blocks per tile; DX: of them with dH1
  int a4, b4;          // operand widths are multiples of 64: one box per stage
  int save_h;          // UP: write H
  const __nv_bfloat16* hin;     // DAP
  const __nv_bfloat16* addend;  // DOWN, DX: [T, d] or null
  // split tiles write their results from registers: rows of o0 / o1 / o2 at
  // strides ldo, ldo, ldo2 (UP: H1, H3, A; DAP: dH1, dH3, A; DW: per product)
  __nv_bfloat16* out[3];
  int ldo[3];
  int* status;
  uint64_t wait_ns;
  int dbg_no_load;
};

template <int KIND> struct FK {
  static constexpr bool A_MN = KIND == F_DW;
  static constexpr bool B_MN = KIND == F_UP || KIND == F_DOWN || KIND == F_DW;
};

template <int BN> struct FCfg {
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : 6;
  static constexpr int OUT_BYTES = 8 * 2 * 2048;
  static constexpr int SMEM = STAGES * STAGE + OUT_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(STAGE % 1024 == 0, "stages must keep 1 KB alignment");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct FTile {
  int p, m0, n0;
};

// Tiles in groups of 16 row tiles, columns outside rows within a group: the
// 148 tiles in flight then cover about as many rows as columns, and both
// operands' share of them stays in L2.
template <int KIND, int BN>
__device__ __forceinline__ FTile f_tile(int t, const FfnArgs& a) {
  FTile ti;
  ti.p = 0;
  if (KIND == F_DW) {
    while (ti.p < 2 && t >= a.mtiles[ti.p] * a.ntiles[ti.p]) {
      t -= a.mtiles[ti.p] * a.ntiles[ti.p];
      ++ti.p;
    }
  }
  constexpr int GM = 16;
  const int nt = a.ntiles[ti.p], per = GM * nt, g = t / per, r = t - g * per;
  const int gs = min(GM, a.mtiles[ti.p] - g * GM);
  ti.m0 = (g * GM + r % gs) * BM;
  ti.n0 = (r / gs) * (KIND == F_UP ? BN / 2 : BN);
  return ti;
}

// One operand tile of 64 k-rows x 64 * ATOMS columns, k-rows outermost.
template <int ATOMS>
__device__ __forceinline__ void load_mn(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int k0,
                                        int c0, bool one_box) {
  if (one_box) {
    tma_load_4d(dst, m, bar, 0, k0, c0 / 64, 0);
  } else {
#pragma unroll
    for (int i = 0; i < ATOMS; ++i) tma_load_2d(dst + i * ATOM, m, bar, c0 + 64 * i, k0);
  }
}

// 32 bf16 at p[col..], zeros at and past `limit` (a multiple of 8) and for dead rows.
__device__ __forceinline__ void ld_row32(const __nv_bfloat16* p, int col, int limit, bool live,
                                         uint4 (&q)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = live && col + 8 * i < limit ? *reinterpret_cast<const uint4*>(p + col + 8 * i)
                                       : make_uint4(0, 0, 0, 0);
}

// 8 bf16 results to p (16-byte aligned).
__device__ __forceinline__ void st_bf16x8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  memcpy(&u, h, 16);
  *reinterpret_cast<uint4*>(p) = u;
}

// Split tiles: a tile's fp32 partial lies in each CTA's shared memory as rows
// of BN, 16-byte chunk c of row r at chunk c ^ (r & 7), so that a warp's
// row-per-lane writes and the row-wise reads both spread over the banks.
template <int BN>
__device__ __forceinline__ uint32_t part_off(int row, int chunk) {
  return (uint32_t)(row * BN * 4 + ((chunk ^ (row & 7)) << 4));
}

// Columns c .. c+7 of a row, summed over the cluster's partials in rank order.
template <int BN>
__device__ __forceinline__ void part_sum8(uint32_t base, int nranks, int row, int c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int r = 0; r < nranks; ++r) {
    const uint32_t b = map_shared(base, r);
    const float4 x = ld_cluster_v4(b + part_off<BN>(row, c / 4));
    const float4 y = ld_cluster_v4(b + part_off<BN>(row, c / 4 + 1));
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
}

// SPLIT: the CTAs of a cluster share one tile, each takes a slice of its
// k-blocks, and the partial sums meet in distributed shared memory: for the
// tiles that do not fill the SMs (few rows, or the last wave of many).
template <int KIND, int BN, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) k_ffn(const __grid_constant__ FfnArgs a) {
  using C = FCfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) record_status(a.status, 0x1ff);
    return;
  }
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull_bar[s], 1);
      mbar_init(&tempty_bar[s], EPI_THREADS);
    }
    fence_mbar_init();
    prefetch_tmap(&a.mA[0]);
    prefetch_tmap(&a.mB[0]);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem_base = s_tmem;
  grid_dependency_wait();      // the previous product's results
  grid_launch_dependents();
  const int nranks = SPLIT ? (int)cluster_size() : 1, rank = SPLIT ? (int)cluster_rank() : 0;
  const int t_first = a.tile0 + (SPLIT ? (int)blockIdx.x / nranks : (int)blockIdx.x);
  const int t_end = SPLIT ? t_first + 1 : a.tiles, t_step = SPLIT ? 1 : (int)gridDim.x;
  const int kb_begin = SPLIT ? (int)((int64_t)a.kbs * rank / nranks) : 0;
  const int kb_end = SPLIT ? (int)((int64_t)a.kbs * (rank + 1) / nranks) : a.kbs;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && !a.dbg_no_load) {
      int stage = 0;
      uint32_t phase = 0;
      for (int t = t_first; t < t_end; t += t_step) {
        const FTile ti = f_tile<KIND, BN>(t, a);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!bounded_wait(&empty_bar[stage], phase ^ 1, &s_abort, a.status, 1, a.wait_ns))
            goto producer_done;
          uint8_t* sA = smem + stage * C::STAGE;
          uint8_t* sB = sA + A_BYTES;
          uint64_t* bar = &full_bar[stage];
          mbar_arrive_expect_tx(bar, C::STAGE);
          const int k0 = kb * BK;
          if constexpr (KIND == F_UP) {
            tma_load_2d(sA, &a.mA[0], bar, k0, ti.m0);
            load_mn<BN / 128>(sB, &a.mB[0], bar, k0, ti.n0, a.b4);
            load_mn<BN / 128>(sB + (BN / 128) * ATOM, &a.mB[1], bar, k0, ti.n0, a.b4);
          } else if constexpr (KIND == F_DOWN) {
            tma_load_2d(sA, &a.mA[0], bar, k0, ti.m0);
            load_mn<BN / 64>(sB, &a.mB[0], bar, k0, ti.n0, a.b4);
          } else if constexpr (KIND == F_DAP) {
            tma_load_2d(sA, &a.mA[0], bar, k0, ti.m0);
            tma_load_2d(sB, &a.mB[0], bar, k0, ti.n0);
          } else if constexpr (KIND == F_DX) {
            const int h = kb >= a.kbh;
            const int kk = h ? k0 - a.kbh * BK : k0;
            tma_load_2d(sA, &a.mA[h], bar, kk, ti.m0);
            tma_load_2d(sB, &a.mB[h], bar, kk, ti.n0);
          } else {
            load_mn<BM / 64>(sA, &a.mA[ti.p], bar, k0, ti.m0, (a.a4 >> ti.p) & 1);
            load_mn<BN / 64>(sB, &a.mB[ti.p], bar, k0, ti.n0, (a.b4 >> ti.p) & 1);
          }
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
    producer_done:;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16(BM, BN, FK<KIND>::A_MN, FK<KIND>::B_MN);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      for (int t = t_first; t < t_end; t += t_step, ++it) {
        const int acc = it & 1;
        if (!bounded_wait(&tempty_bar[acc], ((it >> 1) & 1) ^ 1, &s_abort, a.status, 2, a.wait_ns)) break;
        fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!bounded_wait(&full_bar[stage], phase, &s_abort, a.status, 3, a.wait_ns)) goto mma_done;
          fence_after_sync();
          const uint32_t sA = smem_u32(smem + stage * C::STAGE);
          const uint32_t sB = sA + A_BYTES;
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks) {
            const uint64_t ad = FK<KIND>::A_MN ? sdesc_sw128(sA + ks * 2048, ATOM, 1024)
                                               : sdesc_sw128(sA + ks * 32, 16, 1024);
            const uint64_t bd = FK<KIND>::B_MN ? sdesc_sw128(sB + ks * 2048, ATOM, 1024)
                                               : sdesc_sw128(sB + ks * 32, 16, 1024);
            umma_bf16(d_tmem, ad, bd, IDESC, kb > kb_begin || ks > 0);
          }
          umma_commit(&empty_bar[stage]);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
        umma_commit(&tfull_bar[acc]);
      }
    mma_done:;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    const int half = (warp - 2) >> 2;            // which half of the tile's columns
    const int rloc = q * 32 + lane;              // row of the tile owned by this thread
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    if constexpr (SPLIT) {
      // this slice's partial, fp32, over the pipeline's stages: every copy
      // into them has landed and every MMA that reads them is done
      const FTile ti = f_tile<KIND, BN>(t_first, a);
      if (bounded_wait(&tfull_bar[0], 0, &s_abort, a.status, 4, a.wait_ns) &&
          ti.m0 + q * 32 < a.M[ti.p]) {
        fence_after_sync();
#pragma unroll 1
        for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
          uint32_t r[32];
          tmem_ld32(tlane + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(smem + part_off<BN>(rloc, c / 4 + i)) =
                make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
    } else {
      uint8_t* otile = smem + C::STAGES * C::STAGE + (warp - 2) * 4096;
      int obuf = 0;
      int it = 0;
      // what the epilogue reads of memory (H; the addend) is loaded ahead in
      // 32-column chunks, across tiles: PRE chunks before they are needed
      constexpr int CH = (KIND == F_UP ? BN / 4 : BN / 2) / 32;   // chunks of a tile per warp
      constexpr int PRE = KIND == F_DAP ? 2 : CH;
      constexpr bool RD1 = KIND == F_DAP || KIND == F_DOWN || KIND == F_DX;
      uint4 n1[RD1 ? PRE : 1][4], n3[KIND == F_DAP ? PRE : 1][4];
      const bool rd = KIND == F_DAP || (RD1 && a.addend != nullptr);
      auto fetch = [&](int t, int j, int slot) {   // chunk j of tile t
        if (t >= t_end) return;
        const FTile ti = f_tile<KIND, BN>(t, a);
        const int row = ti.m0 + rloc, col = ti.n0 + (half * CH + j) * 32;
        const bool live = row < a.M[0];
        if constexpr (KIND == F_DAP) {
          const __nv_bfloat16* rp = a.hin + (size_t)row * 2 * a.f;
          ld_row32(rp, col, a.N[0], live, n1[slot]);
          ld_row32(rp + a.f, col, a.N[0], live, n3[slot]);
        } else if constexpr (RD1) {
          ld_row32(a.addend + (size_t)row * a.N[0], col, a.N[0], live, n1[slot]);
        }
      };
      if (rd) {
#pragma unroll
        for (int j = 0; j < PRE; ++j) fetch(t_first, j, j);
      }
      for (int t = t_first; t < t_end; t += t_step, ++it) {
        const FTile ti = f_tile<KIND, BN>(t, a);
        const int acc = it & 1;
        const int row0 = ti.m0 + q * 32;
        const int M = a.M[ti.p], N = a.N[ti.p];
        if (!bounded_wait(&tfull_bar[acc], (it >> 1) & 1, &s_abort, a.status, 4, a.wait_ns)) break;
        fence_after_sync();
        const uint32_t tbase = tlane + acc * BN;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int c = (half * CH + j) * 32, col = ti.n0 + c;
          const bool inside = col < N && row0 < M;   // else the whole box lies outside
          float v[32];
          uint32_t r[32];
          tmem_ld32(tbase + c, r);
          if constexpr (KIND == F_UP) {
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            float h3[32];
            tmem_ld32(tbase + BN / 2 + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) h3[i] = __uint_as_float(r[i]);
            if (!inside) continue;
            if (a.save_h) {
              stage_store(otile, obuf, v, &a.sO[0], col, row0, lane);
              stage_store(otile, obuf, h3, &a.sO[1], col, row0, lane);
            }
            // A from the accumulator, not from the rounded H: one rounding less
            // between x and y (2-norm error of y 2.4e-3 instead of 3.1e-3)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = v[i] * sigmoid_fast(v[i]) * h3[i];
            stage_store(otile, obuf, v, &a.sO[2], col, row0, lane);
          } else if constexpr (KIND == F_DAP) {
            tmem_ld_wait();
            float d3[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float h1 = bf16_lane(n1[j % PRE], i), h3 = bf16_lane(n3[j % PRE], i);
              const float da = __uint_as_float(r[i]);
              const float sg = sigmoid_fast(h1);
              const float sl = h1 * sg;
              v[i] = da * h3 * (sg * (1.0f + h1 * (1.0f - sg)));
              d3[i] = da * sl;
              r[i] = __float_as_uint(sl * h3);
            }
            if (j + PRE < CH) fetch(t, j + PRE, j % PRE);
            else fetch(t + t_step, j + PRE - CH, j % PRE);
            if (!inside) continue;
            stage_store(otile, obuf, v, &a.sO[0], col, row0, lane);
            stage_store(otile, obuf, d3, &a.sO[1], col, row0, lane);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            stage_store(otile, obuf, v, &a.sO[2], col, row0, lane);
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            if constexpr (RD1) {
              if (rd) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += bf16_lane(n1[j], i);
                fetch(t + t_step, j, j);
              }
            }
            if (!inside) continue;
            stage_store(otile, obuf, v, &a.sO[KIND == F_DW ? ti.p : 0], col, row0, lane);
          }
        }
        fence_before_sync();
        mbar_arrive(&tempty_bar[acc]);
      }
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();            // every partial of the tile is in place
    const FTile ti = f_tile<KIND, BN>(t_first, a);
    const int M = a.M[ti.p], N = a.N[ti.p];
    const int rows = min(BM, M - ti.m0);
    constexpr int UNITS = (KIND == F_UP ? BN / 2 : BN) / 8;   // 8-column units of a row
    const uint32_t base = smem_u32(smem);
    for (int i = rank * THREADS + threadIdx.x; i < rows * UNITS; i += nranks * THREADS) {
      const int rl = i / UNITS, c = (i % UNITS) * 8, col = ti.n0 + c;
      if (col >= N) continue;
      const size_t row = (size_t)(ti.m0 + rl);
      float v[8];
      if constexpr (KIND == F_UP) {
        float h3[8];
        part_sum8<BN>(base, nranks, rl, c, v);
        part_sum8<BN>(base, nranks, rl, BN / 2 + c, h3);
        if (a.save_h) {
          st_bf16x8(a.out[0] + row * a.ldo[0] + col, v);
          st_bf16x8(a.out[1] + row * a.ldo[1] + col, h3);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * sigmoid_fast(v[k]) * h3[k];
        st_bf16x8(a.out[2] + row * a.ldo[2] + col, v);
      } else if constexpr (KIND == F_DAP) {
        uint4 p1[4], p3[4];
        const __nv_bfloat16* rp = a.hin + row * 2 * a.f + col;
        p1[0] = *reinterpret_cast<const uint4*>(rp);
        p3[0] = *reinterpret_cast<const uint4*>(rp + a.f);
        part_sum8<BN>(base, nranks, rl, c, v);
        float d3[8], av[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h1 = bf16_lane(p1, k), h3 = bf16_lane(p3, k), da = v[k];
          const float sg = sigmoid_fast(h1);
          const float sl = h1 * sg;
          v[k] = da * h3 * (sg * (1.0f + h1 * (1.0f - sg)));
          d3[k] = da * sl;
          av[k] = sl * h3;
        }
        st_bf16x8(a.out[0] + row * a.ldo[0] + col, v);
        st_bf16x8(a.out[1] + row * a.ldo[1] + col, d3);
        st_bf16x8(a.out[2] + row * a.ldo[2] + col, av);
      } else {
        uint4 p1[4];
        const bool add = (KIND == F_DOWN || KIND == F_DX) && a.addend != nullptr;
        if (add) p1[0] = *reinterpret_cast<const uint4*>(a.addend + row * N + col);
        part_sum8<BN>(base, nranks, rl, c, v);
        if (add) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += bf16_lane(p1, k);
        }
        const int o = KIND == F_DW ? ti.p : 0;
        st_bf16x8(a.out[o] + row * a.ldo[o] + col, v);
      }
    }
    __syncwarp();
    cluster_sync();            // no CTA leaves while its partial is still read
  }
  if (!SPLIT && warp >= 2 && lane == 0) bulk_wait_all();   // the stores end before the CTA does
  if (s_abort) {   // aborted: let copies and MMAs in flight land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int KIND, int BN, bool SPLIT>
int f_go(const FfnArgs& a, int grid, int cluster, bool dependent, cudaStream_t s) {
  using C = FCfg<BN>;
  static const char* kNames[] = {"ffn_up", "ffn_down", "ffn_dap", "ffn_dx", "ffn_dw"};
  if (cudaError_t e = cudaFuncSetAttribute(k_ffn<KIND, BN, SPLIT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM))
    return cuda_fail(e, "ffn smem attribute");
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = THREADS;
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = at;
  if (SPLIT) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (dependent) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  ProfScope _ps(kNames[KIND], s);
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, k_ffn<KIND, BN, SPLIT>, a)) return cuda_fail(e, "ffn");
  return MOE_OK;
}

// Whole waves of tiles run one tile per CTA.  What is left over (all tiles,
// when there are few rows) is split along K over clusters of 2, 4 or 8 CTAs,
// as wide as the SMs hold at once: clusters do not straddle GPCs, so about
// 128 CTAs in clusters of 8 and 140 in smaller ones are resident.
int split_width(int rem, int kbs) {
  for (int c = 8; c >= 2; c /= 2)
    if (rem * c <= (c == 8 ? 128 : 140) && kbs >= c) return c;
  return 1;
}

template <int KIND, int BN>
int f_launch_bn(FfnArgs& a, bool dependent, cudaStream_t s) {
  a.status = status_ptr();
  a.wait_ns = WAIT_LIMIT_NS;
  a.dbg_no_load = 0;
  if (const long long dbg = take_debug_expire(); dbg > 0) {
    a.wait_ns = (uint64_t)dbg;
    a.dbg_no_load = 1;
  }
  int tiles = 0;
  for (int p = 0; p < (KIND == F_DW ? 3 : 1); ++p) {
    a.mtiles[p] = (a.M[p] + BM - 1) / BM;
    const int bn = KIND == F_UP ? BN / 2 : BN;
    a.ntiles[p] = (a.N[p] + bn - 1) / bn;
    tiles += a.mtiles[p] * a.ntiles[p];
  }
  const int sms = device_sm_count();
  const int rem = tiles % sms, c = rem ? split_width(rem, a.kbs) : 1;
  const int whole = c > 1 ? tiles - rem : tiles;
  if (whole > 0) {
    a.tile0 = 0;
    a.tiles = whole;
    if (int rc = f_go<KIND, BN, false>(a, whole < sms ? whole : sms, 1, dependent, s)) return rc;
    dependent = true;
  }
  if (whole < tiles) {
    a.tile0 = whole;
    a.tiles = tiles;
    return f_go<KIND, BN, true>(a, rem * c, c, dependent, s);
  }
  return MOE_OK;
}

// An MN-major operand [rows, cols]: one box of `atoms` 64-column blocks where
// the width allows it (*one_box), else one 64 x 64 box per block.
int map_mn(CUtensorMap* m, const void* p, int cols, int rows, int ld, int atoms, bool* one_box) {
  *one_box = cols % 64 == 0;
  return *one_box ? make_map_atoms(m, p, cols, rows, 1, atoms, ld)
                  : make_map_2d(m, p, cols, rows, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B, ld);
}

void set_out(FfnArgs& a, int i, void* p, int ld) {
  a.out[i] = (__nv_bfloat16*)p;
  a.ldo[i] = ld;
}

}  // namespace

int ffn_fwd(const FfnDense& p, const void* addend, void* H, void* act, void* y, cudaStream_t s) {
  const int T = p.T, d = p.d, f = p.f;
  int rc;
  bool b4;
  {  // UP
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T; a.d = d; a.f = f;
    a.M[0] = T; a.N[0] = f;
    a.kbs = (d + BK - 1) / BK;
    a.save_h = H != nullptr;
    const __nv_bfloat16* h = (const __nv_bfloat16*)H;
    if ((rc = make_map_2d(&a.mA[0], p.x, d, T, 64, BM))) return rc;
    if ((rc = map_mn(&a.mB[0], p.w1, f, d, f, 256 / 128, &b4))) return rc;
    if ((rc = map_mn(&a.mB[1], p.w3, f, d, f, 256 / 128, &b4))) return rc;
    a.b4 = b4;
    if (H) {
      if ((rc = make_map_2d(&a.sO[0], h, f, T, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, 2 * f))) return rc;
      if ((rc = make_map_2d(&a.sO[1], h + f, f, T, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, 2 * f))) return rc;
    }
    if ((rc = make_store_map(&a.sO[2], act, f, T))) return rc;
    set_out(a, 0, (void*)h, 2 * f);
    set_out(a, 1, (void*)(h + f), 2 * f);
    set_out(a, 2, act, f);
    if ((rc = f_launch_bn<F_UP, 256>(a, false, s))) return rc;
  }
  {  // DOWN
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T; a.d = d; a.f = f;
    a.M[0] = T; a.N[0] = d;
    a.kbs = (f + BK - 1) / BK;
    a.addend = (const __nv_bfloat16*)addend;
    if ((rc = make_map_2d(&a.mA[0], act, f, T, 64, BM))) return rc;
    if ((rc = map_mn(&a.mB[0], p.w2, d, f, d, 256 / 64, &b4))) return rc;
    a.b4 = b4;
    if ((rc = make_store_map(&a.sO[0], y, d, T))) return rc;
    set_out(a, 0, y, d);
    if ((rc = f_launch_bn<F_DOWN, 256>(a, true, s))) return rc;
  }
  return MOE_OK;
}

int ffn_bwd(const FfnDense& p, const void* dout, const void* H, const void* addend, void* dH,
            void* act, void* dx, void* dw1, void* dw3, void* dw2, cudaStream_t s) {
  const int T = p.T, d = p.d, f = p.f;
  __nv_bfloat16* dh = (__nv_bfloat16*)dH;
  int rc;
  {  // DAP
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T; a.d = d; a.f = f;
    a.M[0] = T; a.N[0] = f;
    a.kbs = (d + BK - 1) / BK;
    a.hin = (const __nv_bfloat16*)H;
    if ((rc = make_map_2d(&a.mA[0], dout, d, T, 64, BM))) return rc;
    if ((rc = make_map_2d(&a.mB[0], p.w2, d, f, 64, 256))) return rc;
    if ((rc = make_map_2d(&a.sO[0], dh, f, T, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, 2 * f))) return rc;
    if ((rc = make_map_2d(&a.sO[1], dh + f, f, T, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, 2 * f))) return rc;
    if ((rc = make_store_map(&a.sO[2], act, f, T))) return rc;
    set_out(a, 0, dh, 2 * f);
    set_out(a, 1, dh + f, 2 * f);
    set_out(a, 2, act, f);
    if ((rc = f_launch_bn<F_DAP, 256>(a, false, s))) return rc;
  }
  {  // DX
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T; a.d = d; a.f = f;
    a.M[0] = T; a.N[0] = d;
    a.kbh = (f + BK - 1) / BK;
    a.kbs = 2 * a.kbh;
    a.addend = (const __nv_bfloat16*)addend;
    for (int h = 0; h < 2; ++h) {
      if ((rc = make_map_2d(&a.mA[h], dh + h * f, f, T, 64, BM, CU_TENSOR_MAP_SWIZZLE_128B, 2 * f))) return rc;
      if ((rc = make_map_2d(&a.mB[h], h ? p.w3 : p.w1, f, d, 64, 256))) return rc;
    }
    if ((rc = make_store_map(&a.sO[0], dx, d, T))) return rc;
    set_out(a, 0, dx, d);
    if ((rc = f_launch_bn<F_DX, 256>(a, true, s))) return rc;
  }
  {  // DW
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T; a.d = d; a.f = f;
    a.kbs = (T + BK - 1) / BK;
    const struct { const void *A, *B; void* o; int M, N, lda, ldb; } w[3] = {
        {p.x, dh, dw1, d, f, d, 2 * f}, {p.x, dh + f, dw3, d, f, d, 2 * f}, {act, dout, dw2, f, d, f, d}};
    for (int i = 0; i < 3; ++i) {
      bool a4, b4;
      a.M[i] = w[i].M;
      a.N[i] = w[i].N;
      if ((rc = map_mn(&a.mA[i], w[i].A, w[i].M, T, w[i].lda, BM / 64, &a4))) return rc;
      if ((rc = map_mn(&a.mB[i], w[i].B, w[i].N, T, w[i].ldb, 256 / 64, &b4))) return rc;
      a.a4 |= (int)a4 << i;
      a.b4 |= (int)b4 << i;
      if ((rc = make_store_map(&a.sO[i], w[i].o, w[i].N, w[i].M))) return rc;
      set_out(a, i, w[i].o, w[i].N);
    }
    if ((rc = f_launch_bn<F_DW, 256>(a, true, s))) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
