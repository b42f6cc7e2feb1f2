// Layer norm, forward and backward, over the rows of an activation [T, d].
//
//   y  = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//   g  = dy w,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ addend)
//   dw = sum_t dy xh,  db = sum_t dy
//
// Both directions are bound by HBM: a row is read once, its statistics are
// taken from registers (fp32; the variance from the centred values, a second
// pass over registers, so an offset does not cancel) and its result leaves
// from the same registers (backward: from shared memory).  Results are rounded
// once, to the activations' type.  At these rates the instructions count: the
// arithmetic runs on pairs (two fp32 per instruction).
#include <math.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

// V elements moved as one access of at most 16 bytes (fp32 parameters beside
// bf16 rows: two), held as raw bits and converted where they are used.
template <int BYTES> struct Bits;
template <> struct Bits<2> { typedef uint16_t type; };
template <> struct Bits<4> { typedef uint32_t type; };
template <> struct Bits<8> { typedef uint2 type; };
template <> struct Bits<16> { typedef uint4 type; };

template <class T, int V>
struct Pack {
  static constexpr int BYTES = V * (int)sizeof(T);
  static constexpr int UNIT = BYTES > 16 ? 16 : BYTES;
  typename Bits<UNIT>::type raw[BYTES / UNIT];
};

// A thread's share of a row: NV packs of V columns, computed on in pairs (of
// neighbours; of two packs where V is 1).  Columns past the row read zero.
template <class T, int V, int NV>
struct Vals {
  static constexpr int NP = NV * V / 2;   // pairs
  static_assert(V > 1 || NV % 2 == 0, "packs of one come in pairs");
  Pack<T, V> p[NV];
  // pack i holds columns col + i * step ..
  __device__ __forceinline__ void load(const T* row, int col, int step, int d) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col + i * step;
#pragma unroll
      for (int u = 0; u < Pack<T, V>::BYTES / Pack<T, V>::UNIT; ++u) {
        typedef typename Bits<Pack<T, V>::UNIT>::type B;
        p[i].raw[u] = c < d ? reinterpret_cast<const B*>(row + c)[u] : B{};
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int col, int step, int d) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col + i * step;
      if (c < d) {
#pragma unroll
        for (int u = 0; u < Pack<T, V>::BYTES / Pack<T, V>::UNIT; ++u)
          reinterpret_cast<typename Bits<Pack<T, V>::UNIT>::type*>(row + c)[u] = p[i].raw[u];
      }
    }
  }
  __device__ __forceinline__ F2 pair(int m) const {
    if constexpr (V == 1) {
      return f2(one(p[2 * m]), one(p[2 * m + 1]));
    } else {
      const Pack<T, V>& k = p[m / (V / 2)];
      const int j = m % (V / 2);
      if constexpr (sizeof(T) == 4) {
        const float* e = reinterpret_cast<const float*>(k.raw);
        return f2(e[2 * j], e[2 * j + 1]);
      } else {
        return f2_from_bf16x2(reinterpret_cast<const uint32_t*>(k.raw)[j]);
      }
    }
  }
  __device__ __forceinline__ void set_pair(int m, F2 v) {
    if constexpr (V == 1) {
      const float2 t = f2_get(v);
      put(p[2 * m], t.x);
      put(p[2 * m + 1], t.y);
    } else {
      Pack<T, V>& k = p[m / (V / 2)];
      const int j = m % (V / 2);
      if constexpr (sizeof(T) == 4) {
        const float2 t = f2_get(v);
        float* e = reinterpret_cast<float*>(k.raw);
        e[2 * j] = t.x;
        e[2 * j + 1] = t.y;
      } else {
        reinterpret_cast<uint32_t*>(k.raw)[j] = f2_to_bf16x2(v);
      }
    }
  }
  // Values derived from this share before and after this point are computed
  // anew rather than kept in registers.
  __device__ __forceinline__ void forget() {
    constexpr int WORDS = NV * Pack<T, V>::BYTES / 4;
    if constexpr (WORDS * 4 == NV * Pack<T, V>::BYTES && Pack<T, V>::UNIT >= 4) {
      uint32_t* w = reinterpret_cast<uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) asm volatile("" : "+r"(w[i]));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        asm volatile("" : "+h"(*reinterpret_cast<uint16_t*>(p[i].raw)));
    }
  }
  // column of pair m's first (h = 0) or second element
  __device__ __forceinline__ static int column(int m, int h, int col, int step) {
    if (V == 1) return col + (2 * m + h) * step;
    return col + m / (V > 1 ? V / 2 : 1) * step + 2 * (m % (V > 1 ? V / 2 : 1)) + h;
  }

 private:
  __device__ __forceinline__ static float one(const Pack<T, V>& k) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float*>(k.raw);
    else return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(k.raw) << 16);
  }
  __device__ __forceinline__ static void put(Pack<T, V>& k, float v) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float*>(k.raw) = v;
    } else {
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      memcpy(k.raw, &h, 2);
    }
  }
};

// Sum over the `lanes` (a power of two) neighbours that share a row; every
// lane of the warp calls it.
__device__ __forceinline__ float warp_sum(float v, int lanes = 32) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the wpr warps of a row's group; every thread of the block calls it.
__device__ __forceinline__ float group_sum(float v, float* red, int wpr, int warp, int lane) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int w0 = warp / wpr * wpr;
  float s = 0.f;
  for (int i = 0; i < wpr; ++i) s += red[w0 + i];
  return s;
}

constexpr int LN_SMS = 148;

// ============================================================== forward
// A group of WPR warps holds one row: NV packs of V elements per thread.
// 16384 x 2048 bf16: 27.5 us, 4.9 TB/s (a plain copy of that size 25 us).
// Narrow rows: LPR lanes to a row, several rows in a warp (200000 x 128: 29 us,
// a warp to a row 59).
template <class T, class W, int V, int NV, int WPR, int LPR = 32>
__global__ void __launch_bounds__(WPR > 8 ? 1024 : 256)
k_ln_fwd(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, T* y,
         float* __restrict__ mean, float* __restrict__ rstd, int T_, int d, float inv_d, float eps) {
  __shared__ float red[2][32];
  static_assert(LPR == 32 || WPR == 1, "a row lies in a part of a warp or in whole warps");
  constexpr int wpr = WPR, G = WPR * LPR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpb = blockDim.x / G;
  const int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / G;
  const int lin = threadIdx.x % G;
  const bool live = row < T_;
  typedef Vals<T, V, NV> X;
  const F2 zero = f2(0.f, 0.f);
  const int col = lin * V, step = G * V;
  X raw;
  raw.load(x + row * ldx, col, step, live ? d : 0);
  F2 v[X::NP], acc = zero;
#pragma unroll
  for (int m = 0; m < X::NP; ++m) {
    v[m] = raw.pair(m);
    acc = f2_add(acc, v[m]);
  }
  const float2 a1 = f2_get(acc);
  auto sum = [&](float e, float* r) {
    return LPR < 32 ? warp_sum(e, LPR) : group_sum(e, r, wpr, warp, lane);
  };
  const float mu = sum(a1.x + a1.y, red[0]) * inv_d;
  const F2 nmu = f2(-mu, -mu);
  acc = zero;
#pragma unroll
  for (int m = 0; m < X::NP; ++m) {
    v[m] = f2_add(v[m], nmu);
    if constexpr (V == 1) {
      const float2 t = f2_get(v[m]);
      v[m] = f2(X::column(m, 0, col, step) < d ? t.x : 0.f, X::column(m, 1, col, step) < d ? t.y : 0.f);
    } else if (X::column(m, 0, col, step) >= d) {
      v[m] = zero;
    }
    acc = f2_fma(v[m], v[m], acc);
  }
  const float2 a2 = f2_get(acc);
  const float rs = rsqrtf(sum(a2.x + a2.y, red[1]) * inv_d + eps);
  if (!live) return;
  const F2 rs2 = f2(rs, rs);
  // the parameters pack by pack (of pairs of packs where V is 1): few registers
  constexpr int PG = V == 1 ? 2 : 1;
#pragma unroll
  for (int i = 0; i < NV; i += PG) {
    const int c = col + i * step;
    Vals<W, V, PG> pw, pb;
    Vals<T, V, PG> o;
    if (w) pw.load(w, c, step, d);
    if (b) pb.load(b, c, step, d);
#pragma unroll
    for (int j = 0; j < Vals<T, V, PG>::NP; ++j) {
      F2 e = f2_mul(v[i / PG * Vals<T, V, PG>::NP + j], rs2);
      if (w && b) e = f2_fma(e, pw.pair(j), pb.pair(j));
      else if (w) e = f2_mul(e, pw.pair(j));
      else if (b) e = f2_add(e, pb.pair(j));
      o.set_pair(j, e);
    }
    o.store(y + row * d, c, step, d);
  }
  if (lin == 0 && mean) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

// Many wide bf16 rows that do not start at 4-byte units, x and y alike.  Each row is
// walked in the 16-byte units that hold it: unit j holds columns V j - o ..,
// o the row's offset in its first unit; columns outside the row count as
// nothing, and whole units leave as one store.  The columns of a thread thus
// move from row to row, so w and b lie in shared memory as fp32, V columns and
// a word to spare: element k of unit j is word (V + 1) j - o + k, less one
// where k < o (a choice that the whole row shares), and a warp's 32 units hit
// 32 banks.  Persistent blocks of 8 warps, gw to a row.  9563 x 7017 in 107 us
// (by single elements 178), 32000 x 1037 in 63 (76); narrower rows and fp32 ones
// are faster by single elements, which need no shared memory: 60000 x 767 in
// 68 (84), 32000 x 1037 fp32 in 53 (76).
template <class W, int NV>
__global__ void __launch_bounds__(256, 3)
k_ln_fwd_units(const __nv_bfloat16* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b,
               __nv_bfloat16* y, float* __restrict__ mean, float* __restrict__ rstd, int T_,
               int d, float inv_d, float eps, int gw) {
  extern __shared__ float params[];              // w, then b
  __shared__ float red[2][2][8];
  typedef __nv_bfloat16 T;
  constexpr int V = 8, HV = V / 2;
  typedef Vals<T, V, 1> P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / gw, groups = 8 / gw, lin = (warp % gw) * 32 + lane, G = gw * 32;
  float *sw = params, *sb = params + (d / V + 1) * (V + 1);
  for (int c = threadIdx.x; c < d; c += 256) {
    const int i = c / V * (V + 1) + c % V;
    if (w) sw[i] = to_f(w[c]);
    if (b) sb[i] = to_f(b[c]);
  }
  __syncthreads();
  auto sum = [&](float v, float* r) {            // over the row's warps
    v = warp_sum(v);
    if (gw == 1) return v;
    if (lane == 0) r[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(G) : "memory");
    v = 0.f;
    for (int i = 0; i < gw; ++i) v += r[grp * gw + i];
    return v;
  };
  int odd = 0;
  const int64_t rstep = (int64_t)gridDim.x * groups;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < T_; row += rstep, odd ^= 1) {
    const T* xr = x + row * ldx;
    const int o = (int)((reinterpret_cast<uintptr_t>(xr) & 15u) / sizeof(T));
    const T* xa = xr - o;                        // the row's first unit
    T* ya = y + row * d - o;
    P raw[NV];
    F2 v[NV * HV], acc = f2(0.f, 0.f);
    // column of element k of unit i: inside the row?
    auto in = [&](int i, int k) { return (unsigned)((lin + i * G) * V - o + k) < (unsigned)d; };
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i].load(xa, (lin + i * G) * V, 0, o + d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool whole = in(i, 0) && in(i, V - 1);
#pragma unroll
      for (int j = 0; j < HV; ++j) {
        F2 e = raw[i].pair(j);
        if (!whole) {
          const float2 t = f2_get(e);
          e = f2(in(i, 2 * j) ? t.x : 0.f, in(i, 2 * j + 1) ? t.y : 0.f);
        }
        v[i * HV + j] = e;
        acc = f2_add(acc, e);
      }
    }
    const float2 a1 = f2_get(acc);
    const float mu = sum(a1.x + a1.y, red[odd][0]) * inv_d;
    const F2 nmu = f2(-mu, -mu);
    acc = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool whole = in(i, 0) && in(i, V - 1);
#pragma unroll
      for (int j = 0; j < HV; ++j) {
        F2 e = f2_add(v[i * HV + j], nmu);
        if (!whole) {
          const float2 t = f2_get(e);
          e = f2(in(i, 2 * j) ? t.x : 0.f, in(i, 2 * j + 1) ? t.y : 0.f);
        }
        v[i * HV + j] = e;
        acc = f2_fma(e, e, acc);
      }
    }
    const float2 a2 = f2_get(acc);
    const float rs = rsqrtf(sum(a2.x + a2.y, red[odd][1]) * inv_d + eps);
    const F2 rs2 = f2(rs, rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int base = (lin + i * G) * (V + 1) - o;   // word of element k: base + k - (k < o)
      auto word = [&](const float* p, int k) { return (k < o ? p + base - 1 : p + base)[k]; };
      if (in(i, 0) && in(i, V - 1)) {
        P out;
#pragma unroll
        for (int j = 0; j < HV; ++j) {
          F2 e = f2_mul(v[i * HV + j], rs2);
          if (w && b) e = f2_fma(e, f2(word(sw, 2 * j), word(sw, 2 * j + 1)),
                                 f2(word(sb, 2 * j), word(sb, 2 * j + 1)));
          else if (w) e = f2_mul(e, f2(word(sw, 2 * j), word(sw, 2 * j + 1)));
          else if (b) e = f2_add(e, f2(word(sb, 2 * j), word(sb, 2 * j + 1)));
          out.set_pair(j, e);
        }
        out.store(ya, (lin + i * G) * V, 0, o + d);
      } else {
        // a unit that the row shares with its neighbour, or none of it
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (in(i, k)) {
            const float2 t = f2_get(v[i * HV + k / 2]);
            float e = (k & 1 ? t.y : t.x) * rs;
            if (w && b) e = fmaf(e, word(sw, k), word(sb, k));
            else if (w) e *= word(sw, k);
            else if (b) e += word(sb, k);
            ya[(lin + i * G) * V + k] = from_f<T>(e);
          }
      }
    }
    if (lin == 0 && mean) {
      mean[row] = mu;
      rstd[row] = rs;
    }
  }
}

// A thread's sums over a row or column too long for registers: f adds element i
// to the N sums, for i = first, first + step, .. below end.  LONG: more than
// LONG_SUM elements, of which that many at a time add up in fp32 and those sums
// in fp64, so that the roundings stay as few as elsewhere (a constant row of
// 2^28 columns added up in fp32 alone: its mean 0.25 % off).
constexpr int LONG_SUM = 64;
template <bool LONG, int N, class F>
__device__ __forceinline__ void strided_sums(int64_t first, int64_t step, int64_t end,
                                             float (&sums)[N], F f) {
  int64_t i = first;
  double total[N] = {};
  if (LONG)
    while (i + (LONG_SUM - 1) * step < end) {
      float s[N] = {};
#pragma unroll 4
      for (int k = 0; k < LONG_SUM; ++k, i += step) f(i, s);
#pragma unroll
      for (int n = 0; n < N; ++n) total[n] += s[n];
    }
#pragma unroll
  for (int n = 0; n < N; ++n) sums[n] = 0.f;
  for (; i < end; i += step) f(i, sums);
  if (LONG)
#pragma unroll
    for (int n = 0; n < N; ++n) sums[n] = (float)(total[n] + sums[n]);
}

// Rows wider than the registers of a block: three passes over the row, the
// second and third from the caches, by single elements (2000 x 40000 bf16: 248
// us, the bytes' floor 49).
template <class T, class W, bool LONG>
__global__ void __launch_bounds__(1024)
k_ln_fwd_wide(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, T* y,
              float* __restrict__ mean, float* __restrict__ rstd, int d, float eps) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  float s[1];
  strided_sums<LONG>(threadIdx.x, blockDim.x, d, s, [&](int64_t c, float* a) { a[0] += to_f(xr[c]); });
  const float inv_d = 1.0f / (float)d;
  const float mu = group_sum(s[0], red[0], 32, warp, lane) * inv_d;
  strided_sums<LONG>(threadIdx.x, blockDim.x, d, s, [&](int64_t c, float* a) {
    const float e = to_f(xr[c]) - mu;
    a[0] = fmaf(e, e, a[0]);
  });
  const float rs = rsqrtf(group_sum(s[0], red[1], 32, warp, lane) * inv_d + eps);
  for (int64_t c = threadIdx.x; c < d; c += blockDim.x) {
    float e = (to_f(xr[c]) - mu) * rs;
    if (w) e *= to_f(w[c]);
    if (b) e += to_f(b[c]);
    y[row * d + c] = from_f<T>(e);
  }
  if (threadIdx.x == 0 && mean) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

// ============================================================== backward
// Any rows of up to 8192 columns.  A block walks rows; a group of G threads
// (whole warps, or 4, 8 or 16 lanes) owns a row at a time and each thread the
// same 8 columns of every row, so that the column sums of dy xh and dy stay in
// registers until the block's last row and leave as one partial row per block.
template <class T, class W, int V, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 512 ? 1 : (V > 1 && MAXT == 128 ? 6 : 512 / MAXT))
k_ln_bwd(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* __restrict__ w,
         const float* __restrict__ mean, const float* __restrict__ rstd, const T* add,
         int64_t ldadd, T* dx, float* __restrict__ part, int T_, int d, float inv_d, int G) {
  extern __shared__ float colsum[];        // [2][d], where a block has several groups
  __shared__ float2 red[2][32];
  constexpr int NV = 8 / V;
  typedef Vals<T, V, NV> X;
  constexpr int PG = V == 1 ? 2 : 1, GP = X::NP / (NV / PG);   // pairs of PG packs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = threadIdx.x / G, lin = threadIdx.x - grp * G;
  const int groups = blockDim.x / G, wpg = G >> 5;
  const int col = lin * V, step = G * V;
  const F2 zero = f2(0.f, 0.f), one = f2(1.f, 1.f);
  F2 aw[X::NP], ab[X::NP];
#pragma unroll
  for (int m = 0; m < X::NP; ++m) aw[m] = ab[m] = zero;
  int64_t row = (int64_t)blockIdx.x * groups + grp;
  const int64_t rstep = (int64_t)gridDim.x * groups;
  for (int it = 0; (int64_t)blockIdx.x * groups + it * rstep < T_; ++it, row += rstep) {
    // a row past the last has no columns: zeros
    const int dd = row < T_ ? d : 0;
    X vx, vd, va;
    vx.load(x + row * ldx, col, step, dd);
    vd.load(dy + row * lddy, col, step, dd);
    if (add) va.load(add + row * ldadd, col, step, dd);
    const float mu = dd ? mean[row] : 0.f, r = dd ? rstd[row] : 0.f;
    const F2 nmu = f2(-mu, -mu), rs = f2(r, r);
    // columns past the row have dy = 0 and add nothing to the sums
    F2 t1 = zero, t2 = zero;
#pragma unroll
    for (int i = 0; i < NV / PG; ++i) {
      Vals<W, V, PG> pw;
      if (w) pw.load(w, col + i * PG * step, step, d);
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const int m = i * GP + j;
        const F2 dyv = vd.pair(m);
        const F2 xh = f2_mul(f2_add(vx.pair(m), nmu), rs);
        const F2 g = w ? f2_mul(dyv, pw.pair(j)) : dyv;
        aw[m] = f2_fma(dyv, xh, aw[m]);
        ab[m] = f2_add(ab[m], dyv);
        t1 = f2_add(t1, g);
        t2 = f2_fma(g, xh, t2);
      }
    }
    const float2 p1 = f2_get(t1), p2 = f2_get(t2);
    const float u1 = p1.x + p1.y, u2 = p2.x + p2.y;
    float s1, s2;
    if (G < 32) {
      s1 = warp_sum(u1, G);
      s2 = warp_sum(u2, G);
    } else {
      // both sums over the warp: each half goes on with one
      const bool hi = lane & 16;
      float u = (hi ? u2 : u1) + __shfl_xor_sync(0xffffffffu, hi ? u1 : u2, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      s1 = __shfl_sync(0xffffffffu, u, 0);
      s2 = __shfl_sync(0xffffffffu, u, 16);
    }
    if (wpg > 1) {                         // two buffers: one barrier per row
      if (lane == 0) red[it & 1][warp] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.f;
      for (int i = 0; i < wpg; ++i) {
        const float2 v = red[it & 1][grp * wpg + i];
        s1 += v.x;
        s2 += v.y;
      }
    }
    const F2 ns1 = f2(-s1 * inv_d, -s1 * inv_d), ns2 = f2(-s2 * inv_d, -s2 * inv_d);
    vx.forget();
    vd.forget();
#pragma unroll
    for (int i = 0; i < NV / PG; ++i) {
      Vals<W, V, PG> pw;
      if (w) pw.load(w, col + i * PG * step, step, d);
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const int m = i * GP + j;
        const F2 xh = f2_mul(f2_add(vx.pair(m), nmu), rs);
        const F2 e = f2_fma(xh, ns2, f2_fma(vd.pair(m), w ? pw.pair(j) : one, ns1));
        vx.set_pair(m, add ? f2_fma(e, rs, va.pair(m)) : f2_mul(e, rs));
      }
    }
    vx.store(dx + row * d, col, step, dd);
  }
  if (part == nullptr) return;
  // the groups' sums, added in order: those of a warp by shuffles first
  if (G < 32)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o >= G)
#pragma unroll
        for (int m = 0; m < X::NP; ++m) {
          aw[m].v = f2_add(aw[m], F2{__shfl_xor_sync(0xffffffffu, aw[m].v, o)}).v;
          ab[m].v = f2_add(ab[m], F2{__shfl_xor_sync(0xffffffffu, ab[m].v, o)}).v;
        }
  const int owners = G < 32 ? (int)blockDim.x / 32 : groups;
  const int own = G < 32 ? (lane < G ? warp : -1) : grp;
  float* pr = part + (size_t)blockIdx.x * 2 * d;
  for (int k = 0; k < owners; ++k) {
    if (own == k) {
#pragma unroll
      for (int m = 0; m < X::NP; ++m) {
        const float2 sw = f2_get(aw[m]), sb = f2_get(ab[m]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = X::column(m, h, col, step);
          if (c < d) {
            float u = h ? sw.y : sw.x, v = h ? sb.y : sb.x;
            if (k > 0) {
              u += colsum[c];
              v += colsum[d + c];
            }
            float* to = k == owners - 1 ? pr : colsum;
            to[c] = u;
            to[d + c] = v;
          }
        }
      }
    }
    if (owners > 1) __syncthreads();
  }
}

// Many rows.  The same sums in three roles that never meet at a barrier of the
// block, so that the loads, the rows' sums and the columns' sums of different
// rows overlap: one thread brings stages of R rows by bulk copies; a few warps
// take each row's two sums over its columns; CW warps, a thread to the same E
// columns of all rows, take rows to dx and to the column sums in their
// registers.  (The kernel above, whose warps all wait for each row's sums, 86
// us at 32768 x 1536 bf16 with an addend; with all 8 warps first at the rows'
// sums, then at the columns, 87; this one 74 and 4 for the partial rows' sums:
// 5.4 TB/s; a plain sum of two such tensors runs at 6.5.)
// Rows that do not start and end at 16-byte units come with the bytes around
// them (never another 16-byte unit than one that holds a byte of the row) and
// are read from shared memory in pairs (V = 2, rows at 4-byte units: 16000 x
// 2046 66 us) or by single elements (x 2047: 82), neighbouring threads
// neighbouring columns.
constexpr int LN_STAGES = 6;                     // at most
// Row-sum warps: with 16 column warps three, so that 20 warps leave each
// thread 96 registers; bf16 in accesses of less than 16 bytes needs more of
// them (9563 x 7017: 212 us with 7, 280 with 3; 12000 x 3002: 68 and 103; fp32
// loses by it, 6000 x 4341: 140 and 113).  With 8 column warps four (32000 x
// 1038 bf16: 84 us, with 6 102).
constexpr int ln_sum_warps(int cw, int v, int es) {
  return cw < 16 ? 4 : (es == 2 && v < 8 ? 7 : 3);
}
constexpr int ln_ws_threads(int cw, int v, int es) { return 32 * (cw + ln_sum_warps(cw, v, es) + 1); }

template <class T, class W, int V, int E, int CW>
__global__ void __launch_bounds__(ln_ws_threads(CW, V, sizeof(T)), CW == 8 ? 2 : 1)
k_ln_bwd_ws(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* __restrict__ w,
            const float* __restrict__ mean, const float* __restrict__ rstd, const T* add,
            int64_t ldadd, T* dx, float* __restrict__ part, int T_, int d, float inv_d, int R,
            int stages, int ct, int* status, uint64_t wait_ns, int dbg_no_load) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[LN_STAGES], ready[LN_STAGES], empty[LN_STAGES];
  // per row of a stage, as pairs of the same value: -mean, rstd, -s1 / d, -s2 / d
  __shared__ __align__(16) F2 stat[LN_STAGES][8][4];
  __shared__ volatile int s_abort;
  constexpr int SW = ln_sum_warps(CW, V, sizeof(T));
  constexpr int PG = V == 1 ? 2 : 1;             // packs at a time: a pair at least
  typedef Vals<T, V, PG> P;
  constexpr int NG = E / (V * PG), GP = P::NP;   // groups of packs per thread, pairs in one
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rb = (uint32_t)d * sizeof(T);
  constexpr bool UNITS = V * sizeof(T) == 16;    // rows start and end at 16-byte units
  const uint32_t slot = UNITS ? rb : (rb + 15) / 16 * 16 + 16;   // a row's bytes in a stage
  const int na = add ? 3 : 2;
  const uint32_t stage_bytes = (uint32_t)(na * R) * slot;
  const int64_t tiles = ((int64_t)T_ + R - 1) / R;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < LN_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&ready[i], SW);
      mbar_init(&empty[i], CW);
    }
    fence_mbar_init();
  }
  __syncthreads();
  int st = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++st == stages) { st = 0; phase ^= 1; }
  };
  auto rows_of = [&](int64_t t) { return (int)(T_ - t * R < R ? T_ - t * R : R); };
  // where row r of array `arr` of the current stage begins (its source: p)
  auto in_stage = [&](int arr, int r, const T* p) {
    const uint32_t off = UNITS ? 0u : (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
    return reinterpret_cast<const T*>(smem + (size_t)st * stage_bytes + (size_t)(arr * R + r) * slot + off);
  };
  if (warp == CW + SW) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && !dbg_no_load) {
      auto bytes_of = [&](const T* p) {
        return UNITS ? rb : (((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u) + rb + 15) / 16 * 16;
      };
      auto bring = [&](int arr, int r, const T* p) {
        bulk_load(smem + (size_t)st * stage_bytes + (size_t)(arr * R + r) * slot,
                  reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15),
                  bytes_of(p), &full[st]);
      };
      for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, advance()) {
        if (!bounded_wait(&empty[st], phase ^ 1, &s_abort, status, 6, wait_ns)) break;
        const int rows = rows_of(t);
        uint32_t bytes = 0;
        for (int r = 0; r < rows; ++r) {
          const int64_t row = t * R + r;
          bytes += bytes_of(x + row * ldx) + bytes_of(dy + row * lddy);
          if (add) bytes += bytes_of(add + row * ldadd);
        }
        mbar_arrive_expect_tx(&full[st], bytes);
        for (int r = 0; r < rows; ++r) {
          const int64_t row = t * R + r;
          bring(0, r, x + row * ldx);
          bring(1, r, dy + row * lddy);
          if (add) bring(2, r, add + row * ldadd);
        }
      }
    }
  } else if (warp >= CW) {
    // ------------------------------------------------------------ the rows' sums
    // the block's rows go round the warps, across the stages
    int turn = warp - CW;                          // this warp's first row of the stage
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, advance()) {
      const int rows = rows_of(t);
      const bool any = turn < rows;                // its statistics early
      const float mu0 = any ? mean[t * R + turn] : 0.f, rs0 = any ? rstd[t * R + turn] : 0.f;
      // a warp without a row waits too: it must not run ahead of the stage
      bounded_wait(&full[st], phase, &s_abort, status, 7, wait_ns);
      for (int r = turn; r < rows; r += SW) {
        const bool first = r == turn;
        const int64_t row = t * R + r;
        const float mu = first ? mu0 : mean[row], rs = first ? rs0 : rstd[row];
        const F2 nmu = f2(-mu, -mu);
        const T *xr = in_stage(0, r, x + row * ldx), *dr = in_stage(1, r, dy + row * lddy);
        F2 t1 = f2(0.f, 0.f), t2 = t1;
        // columns past the row read zero and have dy = 0
#pragma unroll 4
        for (int c = lane * V; c < d; c += 32 * V * PG) {
          P px, pd;
          Vals<W, V, PG> pw;
          px.load(xr, c, 32 * V, d);
          pd.load(dr, c, 32 * V, d);
          if (w) pw.load(w, c, 32 * V, d);
#pragma unroll
          for (int j = 0; j < GP; ++j) {
            const F2 g = w ? f2_mul(pd.pair(j), pw.pair(j)) : pd.pair(j);
            t1 = f2_add(t1, g);
            t2 = f2_fma(g, f2_add(px.pair(j), nmu), t2);   // rstd times this: sum g xh
          }
        }
        const float2 p1 = f2_get(t1), p2 = f2_get(t2);
        const float s1 = warp_sum(p1.x + p1.y) * inv_d, s2 = warp_sum(p2.x + p2.y) * rs * inv_d;
        if (lane == 0) {
          stat[st][r][0] = f2(-mu, -mu);
          stat[st][r][1] = f2(rs, rs);
          stat[st][r][2] = f2(-s1, -s1);
          stat[st][r][3] = f2(-s2, -s2);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[st]);
      turn = (turn + SW - R % SW) % SW;            // all stages but the last hold R rows
    }
  } else {
    // ------------------------------------------------------------ dx and the columns' sums
    // ct threads side by side cover a row; the next ct take the next row
    const int nsg = 32 * CW / ct, sg = threadIdx.x / ct;
    const int c0 = (threadIdx.x % ct) * V, cstep = ct * V;
    F2 aw[NG * GP], ab[NG * GP], wv[NG * GP];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      Vals<W, V, PG> pw;
      if (w) pw.load(w, c0 + i * PG * cstep, cstep, d);
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        aw[i * GP + j] = ab[i * GP + j] = f2(0.f, 0.f);
        wv[i * GP + j] = w ? pw.pair(j) : f2(1.f, 1.f);
      }
    }
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, advance()) {
      const int rows = sg < nsg ? rows_of(t) : 0;   // threads past the last whole ct rest
      bounded_wait(&ready[st], phase, &s_abort, status, 8, wait_ns);
#pragma unroll 2
      for (int r = sg; r < rows; r += nsg) {
        const int64_t row = t * R + r;
        const F2 nmu = stat[st][r][0], rs2 = stat[st][r][1], ns1 = stat[st][r][2], ns2 = stat[st][r][3];
        const T *xr = in_stage(0, r, x + row * ldx), *dr = in_stage(1, r, dy + row * lddy);
        const T* ar = in_stage(2, r, add + (add ? row * ldadd : 0));
        T* orow = dx + row * d;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const int c = c0 + i * PG * cstep;
          if (c < d) {
            P px, pd, pa, o;
            px.load(xr, c, cstep, d);
            pd.load(dr, c, cstep, d);
            if (add) pa.load(ar, c, cstep, d);
#pragma unroll
            for (int j = 0; j < GP; ++j) {
              const int m = i * GP + j;
              const F2 dyv = pd.pair(j);
              const F2 xh = f2_mul(f2_add(px.pair(j), nmu), rs2);
              aw[m] = f2_fma(dyv, xh, aw[m]);
              ab[m] = f2_add(ab[m], dyv);
              const F2 e = f2_fma(xh, ns2, f2_fma(dyv, wv[m], ns1));
              o.set_pair(j, add ? f2_fma(e, rs2, pa.pair(j)) : f2_mul(e, rs2));
            }
            o.store(orow, c, cstep, d);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (part != nullptr) {
      // the row subgroups' sums, added in order; every stage has been read by
      // then, so its memory holds them
      auto columns = []() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CW) : "memory"); };
      float* acc = reinterpret_cast<float*>(smem);   // [2][d]
      float* pr = part + (size_t)blockIdx.x * 2 * d;
      columns();
      for (int k = 0; k < nsg; ++k) {
        if (sg == k) {
          float* to = k == nsg - 1 ? pr : acc;
#pragma unroll
          for (int m = 0; m < NG * GP; ++m) {
            const float2 sw = f2_get(aw[m]), sb = f2_get(ab[m]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = Vals<T, V, NG * PG>::column(m, h, c0, cstep);
              if (c < d) {
                float u = h ? sw.y : sw.x, v = h ? sb.y : sb.x;
                if (k > 0) {
                  u += acc[c];
                  v += acc[d + c];
                }
                to[c] = u;
                to[d + c] = v;
              }
            }
          }
        }
        columns();
      }
    }
  }
  if (s_abort) {   // a wait expired: let copies in flight land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
}

// out[c] = sum of the partial rows in a fixed order: 32 columns per block,
// 32 threads share a column's rows and are joined in order.
__global__ void __launch_bounds__(1024)
k_ln_reduce(const float* __restrict__ part, int nparts, int d, float* __restrict__ dw,
            float* __restrict__ db) {
  __shared__ float sm[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  tc::grid_dependency_wait();
  float s = 0.f;
  if (c < 2 * (int64_t)d)
#pragma unroll 8
    for (int r = threadIdx.y; r < nparts; r += 32) s += part[(size_t)r * 2 * d + c];
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * (int64_t)d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sm[i][threadIdx.x];
    if (c < d) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - d] = s;
    }
  }
}

// Rows wider than a block's registers: the column sums first (a strip of 256
// columns over a slice of the rows per block), then dx row by row.  Single
// elements, x and dy read three times, twice from HBM: 4096 x 12288 bf16 256 us
// (floor 46), fp32 293 (92).
template <class T, bool LONG>
__global__ void __launch_bounds__(256)
k_ln_bwd_cols(const T* dy, int64_t lddy, const T* x, int64_t ldx, const float* __restrict__ mean,
              const float* __restrict__ rstd, float* __restrict__ part, int T_, int d) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float s[2];
  strided_sums<LONG>(blockIdx.y, gridDim.y, T_, s, [&](int64_t t, float* a) {
    const float dyv = to_f(dy[t * lddy + c]);
    a[0] = fmaf(dyv, (to_f(x[t * ldx + c]) - mean[t]) * rstd[t], a[0]);
    a[1] += dyv;
  });
  part[(size_t)blockIdx.y * 2 * d + c] = s[0];
  part[(size_t)blockIdx.y * 2 * d + d + c] = s[1];
}

template <class T, class W, bool LONG>
__global__ void __launch_bounds__(1024)
k_ln_bwd_wide(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* __restrict__ w,
              const float* __restrict__ mean, const float* __restrict__ rstd, const T* add,
              int64_t ldadd, T* dx, int d) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row];
  float s[2];
  strided_sums<LONG>(threadIdx.x, blockDim.x, d, s, [&](int64_t c, float* a) {
    const float g = to_f(dy[row * lddy + c]) * (w ? to_f(w[c]) : 1.f);
    a[0] += g;
    a[1] = fmaf(g, (to_f(x[row * ldx + c]) - mu) * rs, a[1]);
  });
  const float inv_d = 1.0f / (float)d;
  const float s1 = group_sum(s[0], red[0], 32, warp, lane) * inv_d;
  const float s2 = group_sum(s[1], red[1], 32, warp, lane) * inv_d;
  for (int64_t c = threadIdx.x; c < d; c += blockDim.x) {
    const float g = to_f(dy[row * lddy + c]) * (w ? to_f(w[c]) : 1.f);
    float v = rs * (g - s1 - (to_f(x[row * ldx + c]) - mu) * rs * s2);
    if (add) v += to_f(add[row * ldadd + c]);
    dx[row * d + c] = from_f<T>(v);
  }
}

// Widest pack (in elements of at most 16 bytes) that every pointer, row
// stride and the width allow.
template <class T, class W>
int pick_pack(int d, std::initializer_list<int64_t> lds, std::initializer_list<const void*> tp,
              std::initializer_list<const void*> wp) {
  int v = 16 / (int)sizeof(T);
  auto fits = [&](int n) {
    if (d % n) return false;
    for (int64_t l : lds)
      if (l % n) return false;
    for (const void* p : tp)
      if (reinterpret_cast<uintptr_t>(p) % (n * sizeof(T))) return false;
    const size_t wb = n * sizeof(W) > 16 ? 16 : n * sizeof(W);
    for (const void* p : wp)
      if (reinterpret_cast<uintptr_t>(p) % wb) return false;
    return true;
  };
  while (v > 1 && !fits(v)) v = sizeof(T) == 2 && v == 8 ? 2 : 1;
  return v;
}

template <class T, class W, int V>
int ln_fwd_v(const T* x, int64_t ldx, const W* w, const W* b, int T_, int d, float eps, T* y,
             float* mean, float* rstd, cudaStream_t s) {
  const int npack = d / V;
  // Warps per row: as few as hold the row in 32 columns a thread (16384 x 2048
  // bf16: 2 warps 36 us, 1 warp with 64 columns 44, 4 warps 38), in 12 by
  // single fp32 elements (8: 32000 x 1037 80 us, 12: 53), 8 by bf16 ones (60000
  // x 767: 68 us, 12: 104); more while the rows alone do not give the SMs 16
  // warps each (few rows: latency).
  constexpr int PT = V * sizeof(T) == 16 ? 32 / V : (V == 1 && sizeof(T) == 4 ? 12 : 8);
  int wpr = 1;
  while (wpr < 32 && npack > wpr * 32 * PT) wpr *= 2;
  while (wpr < 32 && npack > wpr * 32 && (int64_t)T_ * wpr < LN_SMS * 16) wpr *= 2;
  const int nv = (int)(((int64_t)npack + wpr * 32 - 1) / (wpr * 32));   // npack may be 2^31 - 1
  const float inv_d = 1.0f / (float)d;
  ProfScope _ps("layernorm_fwd", s);
  // Many rows, each in a warp or a part of it, 256 threads to a block: two packs of
  // 16 bytes (four of 4) per lane, or 8 single elements (200000 x 127 bf16: 37 us, 94 by units).
  constexpr int PL = V == 1 ? 8 : (V * sizeof(T) == 16 ? 2 : 4);
  if (npack <= 32 * PL && T_ >= LN_SMS * 16) {
#define LN_GO(LPR)                                                                             \
  k_ln_fwd<T, W, V, PL, 1, LPR><<<(T_ + (int64_t)(256 / LPR) - 1) / (256 / LPR), 256, 0, s>>>( \
      x, ldx, w, b, y, mean, rstd, T_, d, inv_d, eps)
    if (npack <= 4 * PL) LN_GO(4);
    else if (npack <= 8 * PL) LN_GO(8);
    else if (npack <= 16 * PL) LN_GO(16);
    else LN_GO(32);
#undef LN_GO
    MOE_CHECK_LAUNCH("layernorm_fwd");
    return MOE_OK;
  }
#define LN_GO(NV, WPR)                                                                        \
  do {                                                                                        \
    const int rpb = WPR == 1 ? 2 : 1;   /* rows per block */                                  \
    k_ln_fwd<T, W, V, NV, WPR><<<(T_ + (int64_t)rpb - 1) / rpb, rpb * WPR * 32, 0, s>>>(      \
        x, ldx, w, b, y, mean, rstd, T_, d, inv_d, eps);                                      \
  } while (0)
#define LN_W(NV)                                                                              \
  do {                                                                                        \
    if (wpr == 1) {                                                                           \
      /* one pack per lane, or many rows of more than PL: rows between were launched above */ \
      if constexpr (NV <= 2 || NV > PL) LN_GO(NV, 1);                                         \
    } else if (wpr == 2) LN_GO(NV, 2);                                                        \
    else if (wpr == 4) LN_GO(NV, 4);                                                          \
    else if (wpr == 8) LN_GO(NV, 8);                                                          \
    else if (wpr == 16) LN_GO(NV, 16);                                                        \
    else LN_GO(NV, 32);                                                                       \
  } while (0)
  if (nv > PT) {
    auto* kernel = d <= LONG_SUM * 1024 ? k_ln_fwd_wide<T, W, false> : k_ln_fwd_wide<T, W, true>;
    kernel<<<T_, 1024, 0, s>>>(x, ldx, w, b, y, mean, rstd, d, eps);
  } else if (nv <= 2) LN_W(2);
  else if (nv <= 4) LN_W(4);
  else if constexpr (PT == 8 && V * sizeof(T) == 16) LN_W(8);
  else if constexpr (PT > 4) {
    if (nv <= 6) LN_W(6);
    else if (nv <= 8) LN_W(8);
    else if constexpr (PT > 8) {
      if (nv <= 10) LN_W(10);
      else LN_W(12);
    }
  }
#undef LN_W
#undef LN_GO
  MOE_CHECK_LAUNCH("layernorm_fwd");
  return MOE_OK;
}

// k_ln_fwd_units' launch; 1 where it does not fit or there are too few rows.
constexpr int LN_UNITS = 1024;    // columns from which it is the faster one
template <class W>
int ln_fwd_units(const __nv_bfloat16* x, int64_t ldx, const W* w, const W* b, int T_, int d,
                 float eps, __nv_bfloat16* y, float* mean, float* rstd, cudaStream_t s) {
  constexpr int V = 8, MAXNV = 5;                // up to 40 columns per thread
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15u) ||
      (ldx - d) % V)
    return 1;
  const int units = (int)(((int64_t)d + 2 * V - 2) / V);   // at most, over the offsets
  int gw = 1;
  while (gw < 8 && units > gw * 32 * MAXNV) gw *= 2;
  if (units > gw * 32 * MAXNV || (int64_t)T_ * gw < LN_SMS * 8) return 1;
  const size_t bytes = (size_t)2 * (d / V + 1) * (V + 1) * sizeof(float);
  const int per_sm = (int)std::min<size_t>(216 * 1024 / bytes, 3);
  const int64_t want = ((int64_t)T_ * gw + 7) / 8;
  const int grid = (int)std::min<int64_t>(want, LN_SMS * per_sm);
  ProfScope _ps("layernorm_fwd", s);
#define LN_GO(NV)                                                                              \
  do {                                                                                         \
    if (cudaError_t e = smem_limit<k_ln_fwd_units<W, NV>>(100 * 1024))                         \
      return cuda_fail(e, "layernorm smem attribute");                                         \
    k_ln_fwd_units<W, NV><<<grid, 256, bytes, s>>>(x, ldx, w, b, y, mean, rstd, T_, d,         \
                                                   1.0f / (float)d, eps, gw);                  \
  } while (0)
  const int nv = (units + gw * 32 - 1) / (gw * 32);
  if (nv <= 3) LN_GO(3);
  else if (nv <= 4) LN_GO(4);
  else LN_GO(5);
#undef LN_GO
  MOE_CHECK_LAUNCH("layernorm_fwd");
  return MOE_OK;
}

template <class T, class W>
int ln_fwd_t(const void* x, int64_t ldx, const void* w, const void* b, int T_, int d, float eps,
             void* y, float* mean, float* rstd, cudaStream_t s) {
  const T* xt = (const T*)x;
  const W *wt = (const W*)w, *bt = (const W*)b;
  T* yt = (T*)y;
  const int v = pick_pack<T, W>(d, {ldx}, {x, y}, {w, b});
  if constexpr (sizeof(T) == 2) {
    if (v == 1 && d > LN_UNITS) {
      const int rc = ln_fwd_units<W>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
      if (rc <= 0) return rc;
    }
    if (v == 8) return ln_fwd_v<T, W, 8>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
    if (v == 2) return ln_fwd_v<T, W, 2>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
  } else {
    if (v == 4) return ln_fwd_v<T, W, 4>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
  }
  return ln_fwd_v<T, W, 1>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
}

constexpr int LN_COLS = 8192;     // widest row of k_ln_bwd: 8 columns x 1024 threads
// Columns up to which k_ln_bwd takes many rows as well: a stage of k_ln_bwd_ws
// is too few bytes there (200000 rows of 128 bf16: 57 us against 134 by
// k_ln_bwd_ws; of 256: 97 and 138; 100000 of 512: 130 and 95).
constexpr int LN_NARROW = 256;
// Most blocks of either kernel.
int ln_blocks(int d) { return LN_SMS * (d <= LN_NARROW ? 6 : 4); }
constexpr int LN_SLICES = 64;     // row slices of k_ln_bwd_cols
// Launch shape of k_ln_bwd_ws for packs of v; R = 0 where rows are too wide or
// too few to give every block a few stages.
struct LnWs {
  int R = 0, stages, ct, E, cw, grid;
  size_t bytes;
};
LnWs ln_bwd_ws(int T_, int d, int es, int v, bool add) {
  LnWs p;
  if (d > LN_COLS) return p;
  // 8 column warps and two blocks per SM for up to 8 columns per thread, 16
  // warps and one block beyond; fp32 as few columns per thread as there are
  // threads, bf16 at least 4 (100000 x 511: 143 us, with 2 155)
  p.cw = (d + 255) / 256 <= 8 ? 8 : 16;
  p.E = es == 2 ? std::max(v, 4) : (v == 1 ? 2 : 4);
  while ((d + p.E - 1) / p.E > 32 * p.cw) p.E *= 2;
  p.ct = ((d + p.E - 1) / p.E + 31) / 32 * 32;
  // stages of a row or two per row-sum warp where three of them fit
  const int sw = ln_sum_warps(p.cw, v, es);
  const size_t rb = v * es < 16 ? ((size_t)d * es + 15) / 16 * 16 + 16 : (size_t)d * es;
  const size_t row = rb * (add ? 3 : 2), room = (p.cw == 8 ? 108 : 216) * 1024;
  p.grid = LN_SMS * (p.cw == 8 ? 2 : 1);
  int r = std::min(2 * sw, 8);
  if (3 * r * row > room || T_ < 4 * (int64_t)p.grid * r) r = std::min(sw, 4);
  while (r > 1 && 2 * r * row > room) --r;
  p.stages = (int)std::min<size_t>(room / (r * row), LN_STAGES);
  p.bytes = std::max((size_t)p.stages * r * row, (size_t)8 * d);
  if (p.stages < 2 || T_ < 2 * (int64_t)p.grid * r) return p;
  p.R = r;
  return p;
}

template <class T, class W, int V>
int ln_bwd_ws_go(const LnWs& p, const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* w,
                 const float* mean, const float* rstd, const T* add, int64_t ldadd, int T_, int d,
                 T* dx, float* part, cudaStream_t s) {
  ProfScope _ps("layernorm_bwd", s);
  const long long dbg = take_debug_expire();
#define LN_GO(E, CW)                                                                           \
  do {                                                                                         \
    if (cudaError_t e = smem_limit<k_ln_bwd_ws<T, W, V, E, CW>>((CW == 8 ? 108 : 216) * 1024)) \
      return cuda_fail(e, "layernorm smem attribute");                                         \
    k_ln_bwd_ws<T, W, V, E, CW><<<p.grid, ln_ws_threads(CW, V, sizeof(T)), p.bytes, s>>>(                  \
        dy, lddy, x, ldx, w, mean, rstd, add, ldadd, dx, part, T_, d, 1.0f / (float)d, p.R,    \
        p.stages, p.ct, status_ptr(), dbg > 0 ? (uint64_t)dbg : WAIT_LIMIT_NS, dbg > 0);       \
  } while (0)
  if (p.cw == 16) {
    if (p.E <= 8) LN_GO(8, 16);
    else LN_GO(16, 16);
  } else if constexpr (V == 8) {
    LN_GO(8, 8);
  } else {
    if (p.E <= 2) {
      if constexpr (V == 1 && sizeof(T) == 4) LN_GO(2, 8);
    } else if (p.E <= 4) {
      LN_GO(4, 8);
    } else {
      LN_GO(8, 8);
    }
  }
#undef LN_GO
  MOE_CHECK_LAUNCH("layernorm_bwd");
  return MOE_OK;
}

template <class T, class W, int V>
int ln_bwd_v(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* w, const float* mean,
             const float* rstd, const T* add, int64_t ldadd, int T_, int d, T* dx, float* part,
             int* nparts, cudaStream_t s) {
  const LnWs p = ln_bwd_ws(T_, d, sizeof(T), V, add != nullptr);
  if (p.R && d > LN_NARROW) {
    *nparts = p.grid;
    return ln_bwd_ws_go<T, W, V>(p, dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T_, d, dx, part, s);
  }
  // threads of a row: whole warps, or a power of two below
  int G = ((d + 7) / 8 + 31) / 32 * 32;
  while (G <= 32 && G > 4 && d <= G * 4) G /= 2;
  const int groups = G >= 128 ? 1 : 128 / G, block = G * groups;
  const size_t smem = groups > 1 ? (size_t)2 * d * sizeof(float) : 0;
  const int64_t steps = ((int64_t)T_ + groups - 1) / groups;
  // 200000 x 128 bf16: 6 blocks of 128 threads per SM 57 us, 4 69; by single
  // elements (V = 1) 6 cost registers, 200000 x 127: 119 and 101
  const int per_sm = block > 512 ? 1 : (V > 1 && G <= 32 ? 6 : std::min(4, 512 / block));
  const int grid = (int)std::min<int64_t>(steps, LN_SMS * per_sm);
  *nparts = grid;
  ProfScope _ps("layernorm_bwd", s);
#define LN_GO(MAXT)                                                         \
  k_ln_bwd<T, W, V, MAXT><<<grid, block, smem, s>>>(                        \
      dy, lddy, x, ldx, w, mean, rstd, add, ldadd, dx, part, T_, d, 1.0f / (float)d, G)
  if (block <= 128) LN_GO(128);
  else if (block <= 256) LN_GO(256);
  else if (block <= 512) LN_GO(512);
  else LN_GO(1024);
#undef LN_GO
  MOE_CHECK_LAUNCH("layernorm_bwd");
  return MOE_OK;
}

template <class T, class W>
int ln_bwd_t(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
             const float* mean, const float* rstd, const void* add, int64_t ldadd, int T_, int d,
             void* dx, float* part, int* nparts, cudaStream_t s) {
  const T *dyt = (const T*)dy, *xt = (const T*)x, *at = (const T*)add;
  const W* wt = (const W*)w;
  T* dxt = (T*)dx;
  if (d > LN_COLS) {
    *nparts = LN_SLICES;
    if (part) {
      ProfScope _ps("layernorm_bwd_cols", s);
      const dim3 grid((unsigned)(((int64_t)d + 255) / 256), LN_SLICES);
      auto* kernel = T_ <= LONG_SUM * LN_SLICES ? k_ln_bwd_cols<T, false> : k_ln_bwd_cols<T, true>;
      kernel<<<grid, 256, 0, s>>>(dyt, lddy, xt, ldx, mean, rstd, part, T_, d);
      MOE_CHECK_LAUNCH("layernorm_bwd_cols");
    }
    ProfScope _ps("layernorm_bwd", s);
    auto* kernel = d <= LONG_SUM * 1024 ? k_ln_bwd_wide<T, W, false> : k_ln_bwd_wide<T, W, true>;
    kernel<<<T_, 1024, 0, s>>>(dyt, lddy, xt, ldx, wt, mean, rstd, at, ldadd, dxt, d);
    MOE_CHECK_LAUNCH("layernorm_bwd");
    return MOE_OK;
  }
  const int v = pick_pack<T, W>(d, {lddy, ldx, add ? ldadd : 0}, {dy, x, add, dx}, {w});
#define LN_V(V) \
  return ln_bwd_v<T, W, V>(dyt, lddy, xt, ldx, wt, mean, rstd, at, ldadd, T_, d, dxt, part, nparts, s)
  if constexpr (sizeof(T) == 2) {
    if (v == 8) LN_V(8);
    if (v == 2) LN_V(2);
  } else {
    if (v == 4) LN_V(4);
  }
  LN_V(1);
#undef LN_V
}

int ln_parts(int T_, int d) { return d > LN_COLS ? LN_SLICES : std::min(T_, ln_blocks(d)); }

}  // namespace

int launch_layernorm_fwd(const void* x, int64_t ldx, const void* w, const void* b, int T, int d,
                         int dtype, int wdtype, float eps, void* y, float* mean, float* rstd,
                         cudaStream_t s) {
  if (dtype == MOE_BF16)
    return wdtype == MOE_BF16
               ? ln_fwd_t<__nv_bfloat16, __nv_bfloat16>(x, ldx, w, b, T, d, eps, y, mean, rstd, s)
               : ln_fwd_t<__nv_bfloat16, float>(x, ldx, w, b, T, d, eps, y, mean, rstd, s);
  return wdtype == MOE_BF16 ? ln_fwd_t<float, __nv_bfloat16>(x, ldx, w, b, T, d, eps, y, mean, rstd, s)
                            : ln_fwd_t<float, float>(x, ldx, w, b, T, d, eps, y, mean, rstd, s);
}

size_t layernorm_bwd_ws_bytes(int T, int d) {
  return T > 0 && d > 0 ? (size_t)ln_parts(T, d) * 2 * d * sizeof(float) : 0;
}

int launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                         const float* mean, const float* rstd, const void* add, int64_t ldadd,
                         int T, int d, int dtype, int wdtype, void* dx, float* dweight,
                         float* dbias, float* part, cudaStream_t s) {
  if (dweight == nullptr && dbias == nullptr) part = nullptr;
  int rc, nparts = 0;
  if (dtype == MOE_BF16)
    rc = wdtype == MOE_BF16
             ? ln_bwd_t<__nv_bfloat16, __nv_bfloat16>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, &nparts, s)
             : ln_bwd_t<__nv_bfloat16, float>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, &nparts, s);
  else
    rc = wdtype == MOE_BF16
             ? ln_bwd_t<float, __nv_bfloat16>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, &nparts, s)
             : ln_bwd_t<float, float>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, &nparts, s);
  if (rc || part == nullptr) return rc;
  // launched as a dependent: neither kernel above triggers it early, so its
  // blocks start when the last of theirs has left, before the stream's full wait
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)((2 * (int64_t)d + 31) / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  ProfScope _ps("layernorm_reduce", s);
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, k_ln_reduce, (const float*)part, nparts, d, dweight, dbias))
    return cuda_fail(e, "layernorm_reduce");
  return MOE_OK;
}

}  // namespace moe
