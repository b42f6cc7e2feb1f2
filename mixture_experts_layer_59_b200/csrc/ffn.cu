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
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

enum FKind : int { F_UP = 0, F_DOWN = 1, F_DAP = 2, F_DX = 3, F_DW = 4 };

struct FfnArgs {
  CUtensorMap mA[3];   // DX: dH1, dH3; DW: the three products' A
  CUtensorMap mB[3];   // UP: W1, W3; DX: W1, W3; DW: the three products' B
  int T, d, f;
  int M[3], N[3];      // output rows and columns (UP: N counts the W1 columns)
  int mtiles[3], ntiles[3];
  int tiles;           // output tiles
  int whole, share;    // pairs: tiles below `whole` are one pair's each; the k-blocks
                       // of the others, end to end, are cut into shares (0: none)
  int span;            // k-blocks a shared tile counts for (>= kbs; a multiple of
                       // share: its cuts fall at the same k-blocks in every tile)
  float4* part;        // pairs: fp32 partials [pair][first or second segment][rank][PART4]
  int* count;          // pairs: arrivals [shared tile][rank], zero at the start
  int kbs, kbh;        // k-blocks per tile; DX: of them with dH1
  int stages;          // split: stages of the pipeline in use
  int a_rows;          // split: rows of A that a stage brings (the MMA's others are never read)
  const uint8_t* next[2];   // split: weights of the next product (or null) and their bytes
  int64_t next_bytes;
  int a4, b4;          // operand widths are multiples of 64: one box per stage
  int save_h;          // UP: write H
  const __nv_bfloat16* hin;     // DAP
  const __nv_bfloat16* addend;  // DOWN, DX: [T, d] or null
  CUtensorMap eO, eI;  // pairs, DOWN and DX: the output and the addend in 32 x 64 boxes
  // outputs and their row strides (UP: H1, H3, A; DAP: dH1, dH3, A; DW: dW1,
  // dW3, dW2; DOWN, DX: one)
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
  static constexpr int SMEM = STAGES * STAGE;
  static constexpr int TMEM_COLS = BN;
  static_assert(STAGE % 1024 == 0, "stages must keep 1 KB alignment");
  static_assert(BM * BN * 4 <= SMEM && SMEM <= 227 * 1024, "partials reuse the stages");
};

// sigmoid(z) = 1 / (1 + 2^(-z log2 e)) from the hardware's approximate 2^x and
// reciprocal (each within 2^-22; results are rounded to bf16 afterwards).
// Flushing denormals saves their range handling: about a third of the
// epilogue's instructions.
__device__ __forceinline__ float sigmoid_ftz(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// SwiGLU backward of one element: from dA and H the two halves of dH, and A.
__device__ __forceinline__ void swiglu_bwd(float da, float h1, float h3, float& d1, float& d3,
                                           float& av) {
  const float sg = sigmoid_ftz(h1);
  const float sl = h1 * sg;
  d1 = da * h3 * fmaf(sl, 1.0f - sg, sg);   // silu'(h1) = sg (1 + h1 (1 - sg))
  d3 = da * sl;
  av = sl * h3;
}

struct FTile {
  int p, m0, n0;
};

// Tiles of ROWS x BN in groups of 2048 rows, columns outside rows within a
// group: the tiles in flight then cover about as many rows as columns, and
// both operands' share of them stays in L2.
template <int KIND, int BN, int ROWS>
__device__ __forceinline__ FTile f_tile(int t, const FfnArgs& a) {
  FTile ti;
  ti.p = 0;
  if (KIND == F_DW) {
    while (ti.p < 2 && t >= a.mtiles[ti.p] * a.ntiles[ti.p]) {
      t -= a.mtiles[ti.p] * a.ntiles[ti.p];
      ++ti.p;
    }
  }
  constexpr int GM = 2048 / ROWS;
  const int nt = a.ntiles[ti.p], per = GM * nt, g = t / per, r = t - g * per;
  const int gs = min(GM, a.mtiles[ti.p] - g * GM);
  ti.m0 = (g * GM + r % gs) * ROWS;
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

// The same for one CTA of a pair (two 64-column blocks).
__device__ __forceinline__ void load_mn_pair(uint8_t* dst, const CUtensorMap* m, uint32_t bar,
                                             int k0, int c0, bool one_box) {
  if (one_box) {
    tma_load_4d_pair(dst, m, bar, 0, k0, c0 / 64, 0);
  } else {
    tma_load_2d_pair(dst, m, bar, c0, k0);
    tma_load_2d_pair(dst + ATOM, m, bar, c0 + 64, k0);
  }
}

// 4 bf16 results to p (8-byte aligned); element k of 4 in a pair of words.
__device__ __forceinline__ void st_bf16x4(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
  uint2 u;
  memcpy(&u, h, 8);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ float bf16_of(const uint2& u, int k) {
  const uint32_t w = k < 2 ? u.x : u.y;
  return __uint_as_float((k & 1) ? (w & 0xffff0000u) : (w << 16));
}

// Split tiles: a tile's fp32 partial lies in each CTA's shared memory as rows
// of BN, 16-byte chunk c of row r at chunk c ^ (r & 7), so that a warp's
// row-per-lane writes and the row-wise reads both spread over the banks.
template <int BN>
__device__ __forceinline__ uint32_t part_off(int row, int chunk) {
  return (uint32_t)(row * BN * 4 + ((chunk ^ (row & 7)) << 4));
}

constexpr int MAX_RANKS = 8;

// Few rows: the CTAs of a cluster share one 128 x BN tile, each takes a slice
// of its k-blocks, and the partial sums meet in distributed shared memory.
template <int KIND, int BN>
__global__ void __launch_bounds__(THREADS, 1) k_ffn_split(const __grid_constant__ FfnArgs a) {
  using C = FCfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t tfull_bar;
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
    mbar_init(&tfull_bar, 1);
    fence_mbar_init();
    prefetch_tmap(&a.mA[0]);
    prefetch_tmap(&a.mB[0]);
    if (KIND == F_UP || KIND == F_DX) prefetch_tmap(&a.mB[1]);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem_base = s_tmem;
  grid_launch_dependents();
  const int nranks = (int)cluster_size(), rank = (int)cluster_rank();
  const FTile ti = f_tile<KIND, BN, BM>((int)blockIdx.x / nranks, a);
  const int kb_begin = (int)((int64_t)a.kbs * rank / nranks);
  const int kb_end = (int)((int64_t)a.kbs * (rank + 1) / nranks);
  const int stages = a.stages;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && !a.dbg_no_load) {
      auto load_a = [&](int stage, int kb) {
        uint8_t* sA = smem + stage * C::STAGE;
        uint64_t* bar = &full_bar[stage];
        const int k0 = kb * BK;
        if constexpr (KIND == F_DX) {
          const int h = kb >= a.kbh;
          tma_load_2d(sA, &a.mA[h], bar, h ? k0 - a.kbh * BK : k0, ti.m0);
        } else if constexpr (KIND == F_DW) {
          load_mn<BM / 64>(sA, &a.mA[ti.p], bar, k0, ti.m0, (a.a4 >> ti.p) & 1);
        } else {
          tma_load_2d(sA, &a.mA[0], bar, k0, ti.m0);
        }
      };
      auto load_b = [&](int stage, int kb) {
        uint8_t* sB = smem + stage * C::STAGE + A_BYTES;
        uint64_t* bar = &full_bar[stage];
        const int k0 = kb * BK;
        mbar_arrive_expect_tx(bar, C::B_BYTES + a.a_rows * BK * 2);
        if constexpr (KIND == F_UP) {
          load_mn<BN / 128>(sB, &a.mB[0], bar, k0, ti.n0, a.b4);
          load_mn<BN / 128>(sB + (BN / 128) * ATOM, &a.mB[1], bar, k0, ti.n0, a.b4);
        } else if constexpr (KIND == F_DOWN) {
          load_mn<BN / 64>(sB, &a.mB[0], bar, k0, ti.n0, a.b4);
        } else if constexpr (KIND == F_DAP) {
          tma_load_2d(sB, &a.mB[0], bar, k0, ti.n0);
        } else if constexpr (KIND == F_DX) {
          const int h = kb >= a.kbh;
          tma_load_2d(sB, &a.mB[h], bar, h ? k0 - a.kbh * BK : k0, ti.n0);
        } else {
          load_mn<BN / 64>(sB, &a.mB[ti.p], bar, k0, ti.n0, (a.b4 >> ti.p) & 1);
        }
      };
      // The weights do not come from the product before this one: the first
      // stages' are fetched while it still runs.
      constexpr bool EARLY = KIND != F_DW;
      const int early = EARLY ? min(stages, kb_end - kb_begin) : 0;
      for (int i = 0; i < early; ++i) load_b(i, kb_begin + i);
      grid_dependency_wait();
      for (int i = 0; i < early; ++i) load_a(i, kb_begin + i);
      int stage = early == stages ? 0 : early;
      uint32_t phase = early == stages ? 1 : 0;
      for (int kb = kb_begin + early; kb < kb_end; ++kb) {
        if (!bounded_wait(&empty_bar[stage], phase ^ 1, &s_abort, a.status, 1, a.wait_ns)) break;
        load_b(stage, kb);
        load_a(stage, kb);
        if (++stage == stages) { stage = 0; phase ^= 1; }
      }
      // the next product's weights on their way to L2 while this one's sums meet
      if constexpr (KIND == F_UP || KIND == F_DAP) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (a.next[i] != nullptr)
            for (int64_t o = (int64_t)blockIdx.x * 16384; o < a.next_bytes;
                 o += (int64_t)gridDim.x * 16384)
              l2_prefetch(a.next[i] + o, (uint32_t)min((int64_t)16384, a.next_bytes - o));
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16(BM, BN, FK<KIND>::A_MN, FK<KIND>::B_MN);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!bounded_wait(&full_bar[stage], phase, &s_abort, a.status, 3, a.wait_ns)) break;
        fence_after_sync();
        const uint32_t sA = smem_u32(smem + stage * C::STAGE);
        const uint32_t sB = sA + A_BYTES;
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
          const uint64_t ad = FK<KIND>::A_MN ? sdesc_sw128(sA + ks * 2048, ATOM, 1024)
                                             : sdesc_sw128(sA + ks * 32, 16, 1024);
          const uint64_t bd = FK<KIND>::B_MN ? sdesc_sw128(sB + ks * 2048, ATOM, 1024)
                                             : sdesc_sw128(sB + ks * 32, 16, 1024);
          umma_bf16(tmem_base, ad, bd, IDESC, kb > kb_begin || ks > 0);
        }
        umma_commit(&empty_bar[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1; }
      }
      umma_commit(&tfull_bar);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    const int half = (warp - 2) >> 2;            // which half of the tile's columns
    const int rloc = q * 32 + lane;              // row of the tile owned by this thread
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    grid_dependency_wait();   // before anything below reads or writes memory
    // this slice's partial, fp32, over the pipeline's stages: every copy into
    // them has landed and every MMA that reads them is done
    if (bounded_wait(&tfull_bar, 0, &s_abort, a.status, 4, a.wait_ns) &&
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
  }

  __syncwarp();
  grid_dependency_wait();
  cluster_sync();            // every partial of the tile is in place
  {
    // Each thread takes 4-column units of the rows (16 bytes of a partial: a
    // warp reads whole rows of banks), NI at a time, so that their loads from
    // all ranks are in flight together.  The sums run in rank order.
    const int M = a.M[ti.p], N = a.N[ti.p];
    const int rows = min(BM, M - ti.m0);
    constexpr int UNITS = (KIND == F_UP ? BN / 2 : BN) / 4;   // of a row
    constexpr int SUMS = KIND == F_UP ? 2 : 1, NI = KIND == F_UP ? 2 : 4;
    const uint32_t base = smem_u32(smem);
    const int step = nranks * THREADS;
    const bool add = (KIND == F_DOWN || KIND == F_DX) && a.addend != nullptr;
    for (int i0 = rank * THREADS + threadIdx.x; i0 < rows * UNITS; i0 += NI * step) {
      float v[NI][SUMS][4];
      uint2 p1[NI], p3[KIND == F_DAP ? NI : 1];
      int rl[NI], c[NI];
      bool in[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int i = i0 + j * step;
        rl[j] = i / UNITS;
        c[j] = (i % UNITS) * 4;
        in[j] = i < rows * UNITS && ti.n0 + c[j] < N;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][0][k] = v[j][SUMS - 1][k] = 0.f;
        if (!in[j]) continue;
        const size_t row = (size_t)(ti.m0 + rl[j]);
        const int col = ti.n0 + c[j];
        if constexpr (KIND == F_DAP) {
          const __nv_bfloat16* rp = a.hin + row * 2 * a.f + col;
          p1[j] = *reinterpret_cast<const uint2*>(rp);
          p3[j] = *reinterpret_cast<const uint2*>(rp + a.f);
        } else if (add) {
          p1[j] = *reinterpret_cast<const uint2*>(a.addend + row * N + col);
        }
      }
#pragma unroll
      for (int r = 0; r < MAX_RANKS; ++r) {
        if (r >= nranks) continue;
        const uint32_t b = map_shared(base, r);
        float4 x[NI][SUMS];
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (!in[j]) continue;
#pragma unroll
          for (int m = 0; m < SUMS; ++m)
            x[j][m] = ld_cluster_v4(b + part_off<BN>(rl[j], (c[j] + m * (BN / 2)) / 4));
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (!in[j]) continue;
#pragma unroll
          for (int m = 0; m < SUMS; ++m) {
            v[j][m][0] += x[j][m].x;
            v[j][m][1] += x[j][m].y;
            v[j][m][2] += x[j][m].z;
            v[j][m][3] += x[j][m].w;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        if (!in[j]) continue;
        const size_t row = (size_t)(ti.m0 + rl[j]);
        const int col = ti.n0 + c[j];
        float(&t)[4] = v[j][0];
        if constexpr (KIND == F_UP) {
          float(&h3)[4] = v[j][SUMS - 1];
          if (a.save_h) {
            st_bf16x4(a.out[0] + row * a.ldo[0] + col, t);
            st_bf16x4(a.out[1] + row * a.ldo[1] + col, h3);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = t[k] * sigmoid_ftz(t[k]) * h3[k];
          st_bf16x4(a.out[2] + row * a.ldo[2] + col, t);
        } else if constexpr (KIND == F_DAP) {
          float d3[4], av[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            swiglu_bwd(t[k], bf16_of(p1[j], k), bf16_of(p3[j], k), t[k], d3[k], av[k]);
          st_bf16x4(a.out[0] + row * a.ldo[0] + col, t);
          st_bf16x4(a.out[1] + row * a.ldo[1] + col, d3);
          st_bf16x4(a.out[2] + row * a.ldo[2] + col, av);
        } else {
          if (add) {
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] += bf16_of(p1[j], k);
          }
          const int o = KIND == F_DW ? ti.p : 0;
          st_bf16x4(a.out[o] + row * a.ldo[o] + col, t);
        }
      }
    }
  }
  __syncwarp();
  cluster_sync_relaxed();    // no CTA leaves while its partial is still read
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

// ============================================================== CTA pairs
// The kernel of the many-row sizes.  Two CTAs of a cluster share a 256 x 256
// tile (cta_group::2): each holds 128 rows of A and of the accumulator and
// half of B's columns, so a k-block brings 32 KB into an SM instead of the
// 48 KB of a 128 x 256 tile, which the SM's 64 bytes per clock from L2 could
// not deliver in the 512 clocks the MMAs take.  Persistent; the accumulator is
// double-buffered in TMEM, six 32 KB stages.
//
// The tiles of the last partial wave are shared: their k-blocks, end to end,
// are cut into equal shares, one per pair, so that all pairs end together.  A
// share covers parts of one or two tiles; every part's epilogue leaves its
// fp32 partial in global memory (L2), and the part that arrives last (a
// counter; nobody waits) sums them in part order and runs the epilogue, so the
// result does not depend on who is last.
//
// Epilogue reads and writes pass through small boxes in shared memory, a few
// per warp, so that global accesses are whole rows of a box (64 or 128 bytes)
// while each thread computes on its own row.  What is read (H; the addend)
// comes ahead of the accumulator, what is written replaces it.  DOWN and DX,
// one box in and out per warp and tile, move them by TMA (addend and result
// at 18944 x 2048 x 256: 42 us; by the threads' own accesses 49).  DAP has two
// in and three out, which by TMA queued behind the operand tiles' loads: its
// threads move them (dA at 18944 x 2048 x 2048: 162 us; by TMA 183), and so
// do UP's and DW's, for which it makes no difference.
constexpr int PN = 256;                       // tile columns
constexpr int PSTAGE = 2 * A_BYTES;
constexpr int PART4 = BM * PN / 4;            // float4s of one CTA's partial
constexpr int MAX_PAIRS = 74;

// A box: 32 rows of 16 * CPR bytes (CPR 16-byte chunks: 4 or 8), chunk c of
// row r at chunk c ^ swizzle(r), so that a thread per row and a row per CPR
// threads both spread over the banks.
template <int CPR>
__device__ __forceinline__ int box_off(int r, int c) {
  return r * CPR * 16 + ((c ^ (CPR == 8 ? r & 7 : (r >> 1) & 3)) << 4);
}
// Columns 32 h .. of row `lane`.
template <int CPR>
__device__ __forceinline__ void box_get(const uint8_t* box, int lane, int h, uint4 (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const uint4*>(box + box_off<CPR>(lane, 4 * h + i));
}
template <int CPR>
__device__ __forceinline__ void box_put(uint8_t* box, int lane, int h, const float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = __floats2bfloat162_rn(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
    uint4 u;
    memcpy(&u, b, 16);
    *reinterpret_cast<uint4*>(box + box_off<CPR>(lane, 4 * h + i)) = u;
  }
}
// The warp copies a box to or from rows 0 .. rows - 1 and columns 0 .. cols - 1
// (a multiple of 8; at most the box's) of p, rows ld elements apart.
template <int CPR>
__device__ __forceinline__ void box_load(uint8_t* box, const __nv_bfloat16* p, int64_t ld, int rows,
                                         int cols, int lane) {
  const int c = lane % CPR;
#pragma unroll
  for (int i = 0; i < CPR; ++i) {
    const int r = i * (32 / CPR) + lane / CPR;
    const bool ok = r < rows && c * 8 < cols;
    cp_async16(box + box_off<CPR>(r, c), ok ? p + r * ld + c * 8 : p, ok);
  }
}
template <int CPR>
__device__ __forceinline__ void box_store(const uint8_t* box, __nv_bfloat16* p, int64_t ld, int rows,
                                          int cols, int lane) {
  const int c = lane % CPR;
#pragma unroll
  for (int i = 0; i < CPR; ++i) {
    const int r = i * (32 / CPR) + lane / CPR;
    if (r < rows && c * 8 < cols)
      *reinterpret_cast<uint4*>(p + r * ld + c * 8) =
          *reinterpret_cast<const uint4*>(box + box_off<CPR>(r, c));
  }
}

template <int KIND> struct PCfg {
  // Epilogue warps: 16 for DOWN and DX, whose K may be short (their way
  // through a box is latency), else 8.
  static constexpr int EW = KIND == F_DOWN || KIND == F_DX ? 16 : 8;
  static constexpr int BLOCK = 64 + 32 * EW;
  // Bytes of boxes per epilogue warp: UP H1, H3 and A of 64 columns; DAP two
  // sets of H1 and H3 of 32 columns, replaced by dH, and one for A; DOWN and
  // DX the addend of 64 columns, replaced by the result; DW 64 columns.
  static constexpr int BOXB = KIND == F_UP ? 12288 : (KIND == F_DAP ? 10240 : 4096);
  static constexpr int STAGES = KIND == F_DW ? 6 : (EW == 16 ? 5 : 4);
  static constexpr int SMEM = STAGES * PSTAGE + EW * BOXB;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int EW>
__device__ __forceinline__ void epi_barrier() {   // the epilogue warps
  asm volatile("bar.sync 1, %0;" ::"n"(EW * 32) : "memory");
}

// The walk of one pair over its work: whole tiles, then its share.
struct FWalk {
  int u, step, lim;      // next whole tile
  int pos, end;          // k-blocks left of the share
  int tile, kb0, kb1;    // the current unit
  int seg;               // shared: 0 or 1, whole: -1
  __device__ __forceinline__ FWalk(const FfnArgs& a, int pair, int npairs) {
    u = pair;
    step = npairs;
    lim = a.whole;
    pos = pair * a.share;
    end = min(pos + a.share, (a.tiles - a.whole) * a.span);
    seg = -1;
  }
  __device__ __forceinline__ bool next(const FfnArgs& a) {
    if (u < lim) {
      tile = u;
      u += step;
      kb0 = 0;
      kb1 = a.kbs;
      return true;
    }
    if (pos >= end) return false;
    const int t = pos / a.span;
    tile = a.whole + t;
    kb0 = pos - t * a.span;
    kb1 = min(a.span, end - t * a.span);
    pos = t * a.span + kb1;
    kb1 = min(kb1, a.kbs);
    ++seg;
    return true;
  }
};

template <int KIND>
__global__ void __launch_bounds__(PCfg<KIND>::BLOCK, 1) k_ffn_pair(const __grid_constant__ FfnArgs a) {
  using C = PCfg<KIND>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];    // used in the even CTA: both CTAs' bytes
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];        // used in the even CTA: both CTAs' warps
  __shared__ __align__(8) uint64_t box_bar[C::EW];       // TMA boxes: a warp's box has arrived
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;
  // 128-byte swizzled tiles need a 1 KB aligned base (the same in every CTA)
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
      mbar_init(&tempty_bar[s], 2 * C::EW);
    }
    for (int i = 0; i < C::EW; ++i) mbar_init(&box_bar[i], 1);
    fence_mbar_init();
    prefetch_tmap(&a.mA[0]);
    prefetch_tmap(&a.mB[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem, 512);
    tmem_relinquish_pair();
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();              // the peer's barriers are initialised
  fence_after_sync();
  const uint32_t tmem_base = s_tmem;
  grid_dependency_wait();      // the previous product's results
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0 && !a.dbg_no_load) {
      int stage = 0;
      uint32_t phase = 0;
      for (FWalk w(a, pair, npairs); w.next(a);) {
        const FTile ti = f_tile<KIND, PN, 2 * BM>(w.tile, a);
        const int m0 = ti.m0 + rank * BM;
        const int n0 = KIND == F_UP ? ti.n0 : ti.n0 + rank * (PN / 2);   // UP: W1 here, W3 there
        // rows of different tiles start at different k-blocks, so that the loads
        // in flight spread over the DRAM pages of a row; the weight gradients
        // keep in step (all tiles read the same rows)
        const int nkb = w.kb1 - w.kb0;
        int kr = KIND == F_DW ? 0 : (ti.m0 / (2 * BM) * 5) % nkb;
        for (int i = 0; i < nkb; ++i, kr = kr + 1 == nkb ? 0 : kr + 1) {
          const int kb = w.kb0 + kr;
          if (!bounded_wait(&empty_bar[stage], phase ^ 1, &s_abort, a.status, 1, a.wait_ns))
            goto producer_done;
          uint8_t* sA = smem + stage * PSTAGE;
          uint8_t* sB = sA + A_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * PSTAGE);
          const uint32_t bar = map_shared(smem_u32(&full_bar[stage]), 0);
          const int k0 = kb * BK;
          if constexpr (KIND == F_DX) {
            const int h = kb >= a.kbh;
            const int kk = h ? k0 - a.kbh * BK : k0;
            tma_load_2d_pair(sA, &a.mA[h], bar, kk, m0);
            tma_load_2d_pair(sB, &a.mB[h], bar, kk, n0);
          } else if constexpr (KIND == F_DW) {
            load_mn_pair(sA, &a.mA[ti.p], bar, k0, m0, (a.a4 >> ti.p) & 1);
            load_mn_pair(sB, &a.mB[ti.p], bar, k0, n0, (a.b4 >> ti.p) & 1);
          } else {
            tma_load_2d_pair(sA, &a.mA[0], bar, k0, m0);
            if constexpr (KIND == F_DAP) tma_load_2d_pair(sB, &a.mB[0], bar, k0, n0);
            else load_mn_pair(sB, &a.mB[KIND == F_UP ? rank : 0], bar, k0, n0, a.b4);
          }
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
    producer_done:;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t IDESC = idesc_bf16(2 * BM, PN, FK<KIND>::A_MN, FK<KIND>::B_MN);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      for (FWalk w(a, pair, npairs); w.next(a); ++it) {
        const int acc = it & 1;
        if (!bounded_wait(&tempty_bar[acc], ((it >> 1) & 1) ^ 1, &s_abort, a.status, 2, a.wait_ns)) break;
        fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * PN;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!bounded_wait(&full_bar[stage], phase, &s_abort, a.status, 3, a.wait_ns)) goto mma_done;
          fence_after_sync();
          const uint32_t sA = smem_u32(smem + stage * PSTAGE);
          const uint32_t sB = sA + A_BYTES;
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks) {
            const uint64_t ad = FK<KIND>::A_MN ? sdesc_sw128(sA + ks * 2048, ATOM, 1024)
                                               : sdesc_sw128(sA + ks * 32, 16, 1024);
            const uint64_t bd = FK<KIND>::B_MN ? sdesc_sw128(sB + ks * 2048, ATOM, 1024)
                                               : sdesc_sw128(sB + ks * 32, 16, 1024);
            umma_bf16_pair(d_tmem, ad, bd, IDESC, kb > w.kb0 || ks > 0);
          }
          umma_commit_pair(&empty_bar[stage]);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
        umma_commit_pair(&tfull_bar[acc]);
      }
    mma_done:;
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    const int slice = (warp - 2) >> 2;           // which of SL slices of the tile's columns
    constexpr int SL = C::EW / 4;
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    uint8_t* boxes = smem + C::STAGES * PSTAGE + (warp - 2) * C::BOXB;
    constexpr int CPR = KIND == F_DAP ? 4 : 8;                    // 16-byte chunks of a box's row
    constexpr int BOX = 512 * CPR, BOXW = 8 * CPR;                // a box's bytes and columns
    constexpr int CH = (KIND == F_UP ? PN / 2 : PN) / SL / BOXW;  // boxes of a tile per warp
    constexpr bool READS = KIND == F_DAP || KIND == F_DOWN || KIND == F_DX;
    constexpr bool TMA = KIND == F_DOWN || KIND == F_DX;
    constexpr int SETS = KIND == F_DAP ? 2 : 1;                   // loaded ahead
    const bool rd = KIND == F_DAP || (READS && a.addend != nullptr);
    int it = 0, g = 0;                  // g: boxes so far
    // The loads run ahead of the accumulator on a walk of their own.
    FWalk wl(a, pair, npairs);
    int lj = CH, lg = 0, lrow = 0, lcol = 0;
    auto load_next = [&]() {            // the addend's next box; H1's and H3's into set lg % SETS
      bool more = true;
      if (lj == CH) {
        more = wl.next(a);
        if (more) {
          const FTile ti = f_tile<KIND, PN, 2 * BM>(wl.tile, a);
          lrow = ti.m0 + rank * BM + q * 32;
          lcol = ti.n0 + slice * CH * BOXW;
          lj = 0;
        }
      }
      if constexpr (TMA) {
        if (lane == 0 && !a.dbg_no_load) {
          bulk_wait_read_all();         // the result has left the box
          if (more) {
            mbar_arrive_expect_tx(&box_bar[warp - 2], BOX);
            tma_load_2d(boxes, &a.eI, &box_bar[warp - 2], lcol, lrow);
            // one box ahead does not cover HBM's latency: the next tile's comes to L2
            FWalk wn = wl;
            if (wn.next(a)) {
              const FTile tn = f_tile<KIND, PN, 2 * BM>(wn.tile, a);
              const int prow = tn.m0 + rank * BM + q * 32, pcol = tn.n0 + slice * CH * BOXW;
              if (prow < a.M[0] && pcol < a.N[0]) tma_prefetch_2d(&a.eI, pcol, prow);
            }
          }
        }
        lj = CH;
      } else {
        if (more) {
          const int rows = a.M[0] - lrow, cols = a.N[0] - lcol;
          uint8_t* set = boxes + (lg % SETS) * 2 * BOX;
          const __nv_bfloat16* p = a.hin + (size_t)lrow * 2 * a.f + lcol;
          box_load<CPR>(set, p, 2 * a.f, rows, cols, lane);
          box_load<CPR>(set + BOX, p + a.f, 2 * a.f, rows, cols, lane);
          lcol += BOXW;
          ++lj;
          ++lg;
        }
        cp_async_commit();
      }
    };
    if (READS && rd) {
#pragma unroll
      for (int i = 0; i < SETS; ++i) load_next();
    }
    // Every epilogue warp walks every unit, also after a wait expired (the
    // waits then return at once): the barriers of shared tiles need all of them.
    for (FWalk w(a, pair, npairs); w.next(a); ++it) {
      const FTile ti = f_tile<KIND, PN, 2 * BM>(w.tile, a);
      const int acc = it & 1;
      const int row0 = ti.m0 + rank * BM + q * 32;
      const int M = a.M[ti.p], N = a.N[ti.p];
      bounded_wait(&tfull_bar[acc], (it >> 1) & 1, &s_abort, a.status, 4, a.wait_ns);
      fence_after_sync();
      const uint32_t tbase = tlane + acc * PN;
      float v[32];
      int first = 0, parts = 0;     // shared: the tile's first pair and number of parts
      bool finish = true;
      const int toff = (w.tile - a.whole) * a.span;
      auto partial = [&](int pr) {  // this warp's corner of pair pr's partial of the tile
        const int sg = pr * a.share < toff ? 1 : 0;   // its share began in an earlier tile
        return a.part + (((size_t)pr * 2 + sg) * 2 + rank) * PART4 + (q * 8) * 8 * 32 + lane;
      };
      if (w.seg >= 0) {
        first = toff / a.share;
        parts = (toff + a.kbs - 1) / a.share - first + 1;
        if (parts > 1) {
          float4* pb = partial(pair);
#pragma unroll 1
          for (int c = slice * (8 / SL); c < (slice + 1) * (8 / SL); ++c) {
            uint32_t r[32];
            tmem_ld32(tbase + c * 32, r);
            tmem_ld_wait();
            if (row0 < M) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                __stcg(pb + (c * 8 + i) * 32,
                       make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                   __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
            }
          }
          __threadfence();
          epi_barrier<C::EW>();
          if (threadIdx.x == 64) {
            s_last = atomicAdd(&a.count[(w.tile - a.whole) * 2 + rank], 1) == parts - 1;
            __threadfence();
          }
          epi_barrier<C::EW>();
          finish = s_last != 0;
        }
      }
      // columns 32 cc .. of this thread's row, over all parts in part order
      auto chunk = [&](int cc, float (&x)[32]) {
        if (parts <= 1) {
          uint32_t r[32];
          tmem_ld32(tbase + cc * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
          return;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
        if (row0 >= M) return;
#pragma unroll 1
        for (int p = 0; p < parts; ++p) {
          const float4* op = partial(first + p) + cc * 8 * 32;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 y = __ldcg(op + i * 32);
            x[4 * i] += y.x; x[4 * i + 1] += y.y; x[4 * i + 2] += y.z; x[4 * i + 3] += y.w;
          }
        }
      };
#pragma unroll 1
      for (int j = 0; j < CH; ++j, ++g) {
        const int cb = (slice * CH + j) * BOXW, col = ti.n0 + cb;
        const bool inside = finish && col < N && row0 < M;   // else nothing of the box is stored
        const int rows = M - row0, cols = N - col;
        uint8_t* box = boxes + (KIND == F_DAP ? (g % SETS) * 2 * BOX : 0);
        if constexpr (TMA) {
          static_assert(!TMA || CH == 1, "one box per warp and tile");
          if (rd) {
            bounded_wait(&box_bar[warp - 2], g & 1, &s_abort, a.status, 5, a.wait_ns);
          } else {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
        } else if (READS) {
          cp_async_wait<SETS - 1>();
          __syncwarp();
        }
        if constexpr (KIND == F_DAP) {
          if (inside) {
            uint4 p1[4], p3[4];
            box_get<CPR>(box, lane, 0, p1);
            box_get<CPR>(box + BOX, lane, 0, p3);
            chunk(cb / 32, v);
            float d3[32], av[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              swiglu_bwd(v[i], bf16_lane(p1, i), bf16_lane(p3, i), v[i], d3[i], av[i]);
            uint8_t* ab = boxes + 4 * BOX;
            box_put<CPR>(box, lane, 0, v);
            box_put<CPR>(box + BOX, lane, 0, d3);
            box_put<CPR>(ab, lane, 0, av);
            __syncwarp();
            box_store<CPR>(box, a.out[0] + (size_t)row0 * a.ldo[0] + col, a.ldo[0], rows, cols, lane);
            box_store<CPR>(box + BOX, a.out[1] + (size_t)row0 * a.ldo[1] + col, a.ldo[1], rows, cols, lane);
            box_store<CPR>(ab, a.out[2] + (size_t)row0 * a.ldo[2] + col, a.ldo[2], rows, cols, lane);
          }
        } else if (inside) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int cc = cb / 32 + h;
            if constexpr (KIND == F_UP) {
              float h3[32];
              chunk(cc, v);
              chunk(PN / 64 + cc, h3);
              if (a.save_h) {
                box_put<CPR>(boxes, lane, h, v);
                box_put<CPR>(boxes + BOX, lane, h, h3);
              }
              // A from the accumulator, not from the rounded H: one rounding less
              // between x and y (2-norm error of y 2.4e-3 instead of 3.1e-3)
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = v[i] * sigmoid_ftz(v[i]) * h3[i];
              box_put<CPR>(boxes + 2 * BOX, lane, h, v);
            } else {
              uint4 p1[4] = {};
              if (READS && rd) box_get<CPR>(box, lane, h, p1);
              chunk(cc, v);
              if (READS && rd) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += bf16_lane(p1, i);
              }
              box_put<CPR>(box, lane, h, v);
            }
          }
          if constexpr (TMA) fence_proxy_async_smem();
          __syncwarp();
          if constexpr (KIND == F_UP) {
            if (a.save_h) {
              box_store<CPR>(boxes, a.out[0] + (size_t)row0 * a.ldo[0] + col, a.ldo[0], rows, cols, lane);
              box_store<CPR>(boxes + BOX, a.out[1] + (size_t)row0 * a.ldo[1] + col, a.ldo[1], rows, cols, lane);
            }
            box_store<CPR>(boxes + 2 * BOX, a.out[2] + (size_t)row0 * a.ldo[2] + col, a.ldo[2], rows, cols, lane);
          } else if constexpr (TMA) {
            if (lane == 0) {
              tma_store_2d(&a.eO, box, col, row0);
              bulk_commit();
            }
          } else {
            const int o = KIND == F_DW ? ti.p : 0;
            box_store<CPR>(box, a.out[o] + (size_t)row0 * a.ldo[o] + col, a.ldo[o], rows, cols, lane);
          }
        }
        __syncwarp();      // the box has been read: it may be filled again
        if (READS && !TMA) load_next();
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_shared(smem_u32(&tempty_bar[acc]), 0));
      if (TMA && rd) load_next();   // waits for the result to leave the box
    }
    if (TMA && lane == 0) bulk_wait_all();   // the stores end before the CTA does
  }

  if (s_abort) {   // aborted: let copies and MMAs in flight land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();              // nothing arrives at a CTA that has left
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ============================================================== launches
const char* f_name(int kind) {
  static const char* n[] = {"ffn_up", "ffn_down", "ffn_dap", "ffn_dx", "ffn_dw"};
  return n[kind];
}

template <auto* KERNEL>
int f_go(const FfnArgs& a, int kind, int grid, int block, int cluster, int smem, int most_smem,
         bool dependent, cudaStream_t s) {
  if (cudaError_t e = smem_limit<KERNEL>(most_smem)) return cuda_fail(e, "ffn smem attribute");
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 2 : 1;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  ProfScope _ps(f_name(kind), s);
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, KERNEL, a)) return cuda_fail(e, "ffn");
  return MOE_OK;
}

// How one product is cut: BN columns and `cluster` CTAs per 128-row tile
// (k_ffn_split, few tiles), or pairs that share the last `tiles - whole`
// tiles in shares of `share` k-blocks (k_ffn_pair).
struct FPlan {
  bool split;
  int bn, cluster;
  int whole, share, span, tiles;
};

// CTAs of clusters of that size that are resident at once, one per SM
// (cudaOccupancyMaxActiveClusters: clusters do not straddle the GPCs).
int resident(int cluster) {
  static const int n[] = {0, 148, 148, 135, 132, 130, 132, 105, 120};
  return n[cluster];
}

int count_tiles(int kind, int d, int f, int T, int rows, int cols) {
  auto up = [](int a, int b) { return (a + b - 1) / b; };
  switch (kind) {
    case F_UP: return up(T, rows) * up(f, cols / 2);
    case F_DAP: return up(T, rows) * up(f, cols);
    case F_DW: return 2 * up(d, rows) * up(f, cols) + up(f, rows) * up(d, cols);
    default: return up(T, rows) * up(d, cols);
  }
}

// Rows of A's boxes: what exists, in the 8-row units of the swizzle.
int a_box_rows(int T) { return T >= BM ? BM : (T + 7) / 8 * 8; }

// k-blocks of a tile of one product.
int count_kbs(int kind, int T, int d, int f) {
  const int kd = (d + BK - 1) / BK, kf = (f + BK - 1) / BK, kt = (T + BK - 1) / BK;
  return kind == F_DW ? kt : (kind == F_DX ? 2 * kf : (kind == F_DOWN ? kf : kd));
}

FPlan f_plan(int kind, int T, int d, int f) {
  FPlan p = {};
  const int kbs = count_kbs(kind, T, d, f);
  // Clocks, for comparison only.  A pair's k-block takes 700 (measured at
  // 8192 x 7168 x 2048; 512 of MMAs), a split CTA's what 64 bytes per clock
  // bring in.  Whole waves of pairs; the rest shared where that ends the wave
  // earlier.  A partial's way through L2 costs each part about 2000, in the
  // unit that sums them.  Tiles cut alike keep their pairs on the same
  // k-blocks, which the weight gradients' long operands, streaming from HBM,
  // need (32768 x 1536 x 256: 75 us, with cuts anywhere 92); where fewer than
  // two parts per tile fit, cuts anywhere are what is left.
  p.tiles = count_tiles(kind, d, f, T, 2 * BM, PN);
  const int rem = p.tiles % MAX_PAIRS, waves = p.tiles / MAX_PAIRS;
  p.whole = p.tiles;
  int64_t best = (int64_t)(waves + (rem > 0)) * kbs * 700;
  auto share = [&](int k, int span, int parts) {
    const int64_t t = ((int64_t)waves * kbs + k) * 700 + 3000 + parts * 2000;
    if (t < best) {
      best = t;
      p.whole = p.tiles - rem;
      p.share = k;
      p.span = span;
    }
  };
  if (rem > 0) {
    for (int parts = 2; parts <= MAX_PAIRS / rem && parts <= kbs; ++parts) {
      const int k = (kbs + parts - 1) / parts;
      share(k, (kbs + k - 1) / k * k, parts);
    }
    if (2 * rem > MAX_PAIRS) share((rem * kbs + MAX_PAIRS - 1) / MAX_PAIRS, kbs, 3);
  }
  // Few tiles: clusters of at most 8 along K, all resident at once; the sums'
  // way between SMs costs them a start and a clock per 16 bytes (measured 18
  // and 13 per clock: 96 rows, 4 ranks, 128 and 256 columns).
  const int rows = kind == F_DW ? BM : a_box_rows(T);
  for (int bn = 256; bn >= 128; bn /= 2) {
    const int tiles = count_tiles(kind, d, f, T, BM, bn);
    for (int c = 1; c <= MAX_RANKS && c <= kbs && tiles * c <= resident(c); ++c) {
      const int64_t t = (int64_t)((kbs + c - 1) / c) * 2 * (rows + bn) + (c > 1 ? 1500 + rows * bn / 4 : 0);
      if (t < best) {
        best = t;
        p.split = true;
        p.bn = bn;
        p.cluster = c;
        p.tiles = tiles;
        p.whole = p.share = 0;
      }
    }
  }
  return p;
}

template <int KIND>
int f_launch(FfnArgs& a, const FPlan& p, bool dependent, cudaStream_t s) {
  a.status = status_ptr();
  a.wait_ns = WAIT_LIMIT_NS;
  a.dbg_no_load = 0;
  if (const long long dbg = take_debug_expire(); dbg > 0) {
    a.wait_ns = (uint64_t)dbg;
    a.dbg_no_load = 1;
  }
  const int rows = p.split ? BM : 2 * BM, bn = p.split ? p.bn : PN, cols = KIND == F_UP ? bn / 2 : bn;
  for (int i = 0; i < (KIND == F_DW ? 3 : 1); ++i) {
    a.mtiles[i] = (a.M[i] + rows - 1) / rows;
    a.ntiles[i] = (a.N[i] + cols - 1) / cols;
  }
  a.tiles = p.tiles;
  a.whole = p.whole;
  a.share = p.share;
  a.span = p.span;
  if (p.split) {
    // Shared memory: the stages in use (all of a CTA's slice, where it fits),
    // which then hold the partial of the rows that exist.  At least 448 bytes
    // per TMEM column, so that the CTAs of an SM never ask for more than its
    // 512 columns: a CTA that waited for columns could hold up its cluster.
    const int rows32 = KIND == F_DW ? BM : (a_box_rows(a.T) + 31) / 32 * 32;
    a.a_rows = KIND == F_DW ? BM : a_box_rows(a.T);
    const int grid = p.tiles * p.cluster, slice = (a.kbs + p.cluster - 1) / p.cluster;
    auto go = [&](auto cfg, auto launch) {
      typedef decltype(cfg) C;
      a.stages = std::min(slice, (int)C::STAGES);
      return launch(std::max(std::max(a.stages * C::STAGE, rows32 * p.bn * 4), 448 * p.bn));
    };
    if (p.bn == 256)
      return go(FCfg<256>{}, [&](int smem) {
        return f_go<k_ffn_split<KIND, 256>>(a, KIND, grid, THREADS, p.cluster, smem,
                                            FCfg<256>::SMEM, dependent, s);
      });
    return go(FCfg<128>{}, [&](int smem) {
      return f_go<k_ffn_split<KIND, 128>>(a, KIND, grid, THREADS, p.cluster, smem, FCfg<128>::SMEM,
                                          dependent, s);
    });
  }
  const int pairs = p.share || p.whole > MAX_PAIRS ? MAX_PAIRS : p.whole;
  return f_go<k_ffn_pair<KIND>>(a, KIND, 2 * pairs, PCfg<KIND>::BLOCK, 2, PCfg<KIND>::SMEM,
                                PCfg<KIND>::SMEM, dependent, s);
}

// An MN-major operand [rows, cols]: one box of `atoms` 64-column blocks where
// the width allows it (*one_box), else one 64 x 64 box per block.
int map_mn(CUtensorMap* m, const void* p, int cols, int rows, int ld, int atoms, bool* one_box) {
  *one_box = cols % 64 == 0;
  return *one_box ? make_map_atoms(m, p, cols, rows, 1, atoms, ld)
                  : make_map_2d(m, p, cols, rows, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B, ld);
}

// A matrix in the epilogue's TMA boxes.
int box_map(CUtensorMap* m, const void* p, int cols, int rows) {
  return make_map_2d(m, p, cols, rows, 64, 32);
}

// Output i at p, rows ld elements apart.
void set_out(FfnArgs& a, int i, void* p, int ld) {
  a.out[i] = (__nv_bfloat16*)p;
  a.ldo[i] = ld;
}

}  // namespace

// Partials and counters of the shared tiles of a call's products (one region,
// used by one product after the other); the counters are zeroed first.
namespace {
struct FScratch {
  FPlan plan[5];       // of the call's kinds
  size_t part_bytes = 0, counts = 0;
};
FScratch ffn_scratch(int T, int d, int f, bool bwd) {
  FScratch z;
  for (int k = bwd ? F_DAP : F_UP; k <= (bwd ? F_DW : F_DOWN); ++k) {
    const FPlan p = z.plan[k] = f_plan(k, T, d, f);
    if (p.share == 0) continue;
    z.part_bytes = (size_t)MAX_PAIRS * 2 * 2 * PART4 * sizeof(float4);
    z.counts += (size_t)(p.tiles - p.whole) * 2;
  }
  return z;
}

// Hands the scratch out to the products of one call.
struct FCall {
  FScratch z;
  int* count = nullptr;
  char* base;
  int T, d, f;
  cudaStream_t s;
  bool first = true;
  FCall(const FfnDense& p, bool bwd, void* scratch, cudaStream_t st)
      : z(ffn_scratch(p.T, p.d, p.f, bwd)), base((char*)scratch), T(p.T), d(p.d), f(p.f), s(st) {}
  int begin() {
    count = (int*)(base + z.part_bytes);
    if (z.counts)
      if (cudaError_t e = cudaMemsetAsync(count, 0, z.counts * sizeof(int), s))
        return cuda_fail(e, "ffn counters");
    return MOE_OK;
  }
  FfnArgs args() const {
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T;
    a.d = d;
    a.f = f;
    return a;
  }
  bool pairs(int kind) const { return !z.plan[kind].split; }
  // Rows of A that one CTA loads per stage.
  int a_rows(int kind) const { return z.plan[kind].split ? a_box_rows(T) : BM; }
  // Columns of B that one CTA loads per stage.
  int b_cols(int kind) const {
    const FPlan& p = z.plan[kind];
    const int n = p.split ? p.bn : PN / 2;
    return kind == F_UP && p.split ? n / 2 : n;
  }
  template <int KIND>
  int go(FfnArgs& a) {
    const FPlan& p = z.plan[KIND];
    a.part = (float4*)base;
    a.count = count;
    if (p.share) count += (p.tiles - p.whole) * 2;
    const bool dependent = !first;
    first = false;
    return f_launch<KIND>(a, p, dependent, s);
  }
};
}  // namespace

size_t ffn_scratch_bytes(int T, int d, int f, bool bwd) {
  const FScratch z = ffn_scratch(T, d, f, bwd);
  return z.part_bytes + align_up(z.counts * sizeof(int), 256);
}

void ffn_debug_plan(int T, int d, int f, int product, int* out) {
  const FPlan p = f_plan(product, T, d, f);
  const int v[] = {p.split ? p.bn : 0, p.split ? p.cluster : 2, p.tiles, p.whole, p.share, p.span,
                   count_kbs(product, T, d, f)};
  std::copy(std::begin(v), std::end(v), out);
}

int ffn_fwd(const FfnDense& p, const void* addend, void* H, void* act, void* y, void* scratch,
            cudaStream_t s) {
  const int T = p.T, d = p.d, f = p.f;
  int rc;
  bool b4;
  FCall call(p, false, scratch, s);
  if ((rc = call.begin())) return rc;
  {  // UP
    FfnArgs a = call.args();
    a.M[0] = T; a.N[0] = f;
    a.kbs = (d + BK - 1) / BK;
    a.save_h = H != nullptr;
    __nv_bfloat16* h = (__nv_bfloat16*)H;
    const int atoms = call.b_cols(F_UP) / 64;
    if ((rc = make_map_2d(&a.mA[0], p.x, d, T, 64, call.a_rows(F_UP)))) return rc;
    if ((rc = map_mn(&a.mB[0], p.w1, f, d, f, atoms, &b4))) return rc;
    if ((rc = map_mn(&a.mB[1], p.w3, f, d, f, atoms, &b4))) return rc;
    a.b4 = b4;
    set_out(a, 0, h, 2 * f);
    set_out(a, 1, H ? h + f : nullptr, 2 * f);
    set_out(a, 2, act, f);
    a.next[0] = (const uint8_t*)p.w2;
    a.next_bytes = (int64_t)d * f * 2;
    if ((rc = call.go<F_UP>(a))) return rc;
  }
  {  // DOWN
    FfnArgs a = call.args();
    a.M[0] = T; a.N[0] = d;
    a.kbs = (f + BK - 1) / BK;
    a.addend = (const __nv_bfloat16*)addend;
    if ((rc = make_map_2d(&a.mA[0], act, f, T, 64, call.a_rows(F_DOWN)))) return rc;
    if ((rc = map_mn(&a.mB[0], p.w2, d, f, d, call.b_cols(F_DOWN) / 64, &b4))) return rc;
    a.b4 = b4;
    set_out(a, 0, y, d);
    if (call.pairs(F_DOWN))
      if ((rc = box_map(&a.eO, y, d, T))) return rc;
    if (addend && call.pairs(F_DOWN))
      if ((rc = box_map(&a.eI, addend, d, T))) return rc;
    if ((rc = call.go<F_DOWN>(a))) return rc;
  }
  return MOE_OK;
}

int ffn_bwd(const FfnDense& p, const void* dout, const void* H, const void* addend, void* dH,
            void* act, void* dx, void* dw1, void* dw3, void* dw2, void* scratch, cudaStream_t s) {
  const int T = p.T, d = p.d, f = p.f;
  __nv_bfloat16* dh = (__nv_bfloat16*)dH;
  int rc;
  FCall call(p, true, scratch, s);
  if ((rc = call.begin())) return rc;
  {  // DAP
    FfnArgs a = call.args();
    a.M[0] = T; a.N[0] = f;
    a.kbs = (d + BK - 1) / BK;
    a.hin = (const __nv_bfloat16*)H;
    if ((rc = make_map_2d(&a.mA[0], dout, d, T, 64, call.a_rows(F_DAP)))) return rc;
    if ((rc = make_map_2d(&a.mB[0], p.w2, d, f, 64, call.b_cols(F_DAP)))) return rc;
    set_out(a, 0, dh, 2 * f);
    set_out(a, 1, dh + f, 2 * f);
    set_out(a, 2, act, f);
    a.next[0] = (const uint8_t*)p.w1;
    a.next[1] = (const uint8_t*)p.w3;
    a.next_bytes = (int64_t)d * f * 2;
    if ((rc = call.go<F_DAP>(a))) return rc;
  }
  {  // DX
    FfnArgs a = call.args();
    a.M[0] = T; a.N[0] = d;
    a.kbh = (f + BK - 1) / BK;
    a.kbs = 2 * a.kbh;
    a.addend = (const __nv_bfloat16*)addend;
    for (int h = 0; h < 2; ++h) {
      if ((rc = make_map_2d(&a.mA[h], dh + h * f, f, T, 64, call.a_rows(F_DX), CU_TENSOR_MAP_SWIZZLE_128B,
                            2 * f)))
        return rc;
      if ((rc = make_map_2d(&a.mB[h], h ? p.w3 : p.w1, f, d, 64, call.b_cols(F_DX)))) return rc;
    }
    set_out(a, 0, dx, d);
    if (call.pairs(F_DX))
      if ((rc = box_map(&a.eO, dx, d, T))) return rc;
    if (addend && call.pairs(F_DX))
      if ((rc = box_map(&a.eI, addend, d, T))) return rc;
    if ((rc = call.go<F_DX>(a))) return rc;
  }
  {  // DW
    FfnArgs a = call.args();
    a.kbs = (T + BK - 1) / BK;
    const struct { const void *A, *B; void* o; int M, N, lda, ldb; } w[3] = {
        {p.x, dh, dw1, d, f, d, 2 * f}, {p.x, dh + f, dw3, d, f, d, 2 * f}, {act, dout, dw2, f, d, f, d}};
    for (int i = 0; i < 3; ++i) {
      bool a4, b4;
      a.M[i] = w[i].M;
      a.N[i] = w[i].N;
      if ((rc = map_mn(&a.mA[i], w[i].A, w[i].M, T, w[i].lda, BM / 64, &a4))) return rc;
      if ((rc = map_mn(&a.mB[i], w[i].B, w[i].N, T, w[i].ldb, call.b_cols(F_DW) / 64, &b4))) return rc;
      a.a4 |= (int)a4 << i;
      a.b4 |= (int)b4 << i;
      set_out(a, i, w[i].o, w[i].N);
    }
    if ((rc = call.go<F_DW>(a))) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
