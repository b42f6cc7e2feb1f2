// Layer norm, forward and backward, over the rows of an activation [T, d].
//
//   y  = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//   g  = dy w,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)) (+ addend)
//   dw = sum_t dy xh,  db = sum_t dy
//
// Both directions are bound by HBM: a row is read once into registers, its
// statistics are taken there (fp32; the variance from the centred values, a
// second pass over registers, so an offset does not cancel) and its result
// leaves from the same registers.  Results are rounded once, to the
// activations' type.
#include <math.h>

#include <cstring>

#include "common.cuh"
#include "internal.h"

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
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(raw)[j];
    else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(raw)[j] << 16);
  }
  __device__ __forceinline__ void set(int j, float v) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float*>(raw)[j] = v;
    } else {
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      memcpy(reinterpret_cast<uint16_t*>(raw) + j, &h, 2);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < BYTES / UNIT; ++i)
      reinterpret_cast<typename Bits<UNIT>::type*>(p)[i] = raw[i];
  }
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
  Pack<T, V> r;
#pragma unroll
  for (int i = 0; i < Pack<T, V>::BYTES / Pack<T, V>::UNIT; ++i)
    r.raw[i] = reinterpret_cast<const typename Bits<Pack<T, V>::UNIT>::type*>(p)[i];
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

// ============================================================== forward
// A group of wpr warps holds one row: NV packs of V elements per thread.
template <class T, class W, int V, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT)
k_ln_fwd(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, T* y,
         float* __restrict__ mean, float* __restrict__ rstd, int T_, int d, float eps, int wpr) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpb = (blockDim.x >> 5) / wpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + warp / wpr;
  const int lin = (warp % wpr) * 32 + lane, G = wpr * 32;
  const bool live = row < T_;
  const T* xr = x + row * ldx;
  Pack<T, V> raw[NV];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
    if (live && c < d) raw[i] = ld_pack<T, V>(xr + c);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
    if (live && c < d) {
#pragma unroll
      for (int j = 0; j < V; ++j) s += raw[i].get(j);
    }
  }
  const float inv_d = 1.0f / (float)d;
  const float mu = group_sum(s, red[0], wpr, warp, lane) * inv_d;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
    if (live && c < d) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float e = raw[i].get(j) - mu;
        s = fmaf(e, e, s);
      }
    }
  }
  const float rs = 1.0f / sqrtf(group_sum(s, red[1], wpr, warp, lane) * inv_d + eps);
  if (!live) return;
  T* yr = y + row * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
    if (c < d) {
      Pack<W, V> pw, pb;
      if (w) pw = ld_pack<W, V>(w + c);
      if (b) pb = ld_pack<W, V>(b + c);
      Pack<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float e = (raw[i].get(j) - mu) * rs;
        if (w) e *= pw.get(j);
        if (b) e += pb.get(j);
        o.set(j, e);
      }
      o.store(yr + c);
    }
  }
  if (lin == 0 && mean) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

// Rows wider than the registers of a block: three passes over the row, the
// second and third from the caches.
template <class T, class W>
__global__ void __launch_bounds__(1024)
k_ln_fwd_wide(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, T* y,
              float* __restrict__ mean, float* __restrict__ rstd, int d, float eps) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < d; c += blockDim.x) s += to_f(xr[c]);
  const float inv_d = 1.0f / (float)d;
  const float mu = group_sum(s, red[0], 32, warp, lane) * inv_d;
  s = 0.f;
  for (int64_t c = threadIdx.x; c < d; c += blockDim.x) {
    const float e = to_f(xr[c]) - mu;
    s = fmaf(e, e, s);
  }
  const float rs = 1.0f / sqrtf(group_sum(s, red[1], 32, warp, lane) * inv_d + eps);
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
// A block walks rows; a group of G threads owns one row at a time and each
// thread the same columns of every row (NV packs of V), so that the column
// sums of dy xh and dy stay in registers until the block's last row and
// leave as one partial row per group.  The next row's loads are issued
// before this row's two sums are taken.
template <class T, class W, int V, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
k_ln_bwd(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* __restrict__ w,
         const float* __restrict__ mean, const float* __restrict__ rstd, const T* add,
         int64_t ldadd, T* dx, float* __restrict__ part, int T_, int d, int G) {
  __shared__ float2 red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = threadIdx.x / G, lin = threadIdx.x - grp * G;
  const int rpb = blockDim.x / G, wpg = G >> 5;
  const float inv_d = 1.0f / (float)d;
  float aw[NV * V], ab[NV * V], wv[NV * V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
    Pack<W, V> pw;
    if (w && c < d) pw = ld_pack<W, V>(w + c);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      aw[i * V + j] = ab[i * V + j] = 0.f;
      wv[i * V + j] = w && c < d ? pw.get(j) : 1.f;
    }
  }
  struct Row {
    Pack<T, V> x[NV], dy[NV], add[NV];
    float mu, rs;
  };
  auto load = [&](Row& q, int64_t row) {
    if (row < T_) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lin + i * G) * V;
        if (c < d) {
          q.x[i] = ld_pack<T, V>(x + row * ldx + c);
          q.dy[i] = ld_pack<T, V>(dy + row * lddy + c);
          if (add) q.add[i] = ld_pack<T, V>(add + row * ldadd + c);
        }
      }
      q.mu = mean[row];
      q.rs = rstd[row];
    }
  };
  int64_t row = (int64_t)blockIdx.x * rpb + grp;
  const int64_t step = (int64_t)gridDim.x * rpb;
  Row cur, next;
  load(cur, row);
  for (int it = 0; (int64_t)blockIdx.x * rpb + it * step < T_; ++it, row += step) {
    const bool live = row < T_;
    load(next, row + step);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (live && (lin + i * G) * V < d) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int q = i * V + j;
          const float dyv = cur.dy[i].get(j);
          const float xh = (cur.x[i].get(j) - cur.mu) * cur.rs;
          const float g = dyv * wv[q];
          aw[q] = fmaf(dyv, xh, aw[q]);
          ab[q] += dyv;
          s1 += g;
          s2 = fmaf(g, xh, s2);
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (wpg > 1) {
      float2* rb = red[it & 1];      // two buffers: one barrier per row
      if (lane == 0) rb[warp] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.f;
      for (int i = 0; i < wpg; ++i) {
        const float2 v = rb[grp * wpg + i];
        s1 += v.x;
        s2 += v.y;
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lin + i * G) * V;
      if (live && c < d) {
        Pack<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (cur.x[i].get(j) - cur.mu) * cur.rs;
          const float g = cur.dy[i].get(j) * wv[i * V + j];
          float v = cur.rs * (g - s1 - xh * s2);
          if (add) v += cur.add[i].get(j);
          o.set(j, v);
        }
        o.store(dx + row * d + c);
      }
    }
    cur = next;
  }
  if (part == nullptr) return;
  float* pr = part + ((size_t)blockIdx.x * rpb + grp) * 2 * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lin + i * G) * V;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < d) {
        pr[c + j] = aw[i * V + j];
        pr[d + c + j] = ab[i * V + j];
      }
  }
}

// out[c] = sum of the partial rows in a fixed order: 32 columns per block,
// 32 threads share a column's rows and are joined in order.
__global__ void __launch_bounds__(1024)
k_ln_reduce(const float* __restrict__ part, int nparts, int d, float* __restrict__ dw,
            float* __restrict__ db) {
  __shared__ float sm[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < 2 * (int64_t)d)
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
// columns over a slice of the rows per block), then dx row by row.
template <class T>
__global__ void __launch_bounds__(256)
k_ln_bwd_cols(const T* dy, int64_t lddy, const T* x, int64_t ldx, const float* __restrict__ mean,
              const float* __restrict__ rstd, float* __restrict__ part, int T_, int d) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t t = blockIdx.y; t < T_; t += gridDim.y) {
    const float dyv = to_f(dy[t * lddy + c]);
    aw = fmaf(dyv, (to_f(x[t * ldx + c]) - mean[t]) * rstd[t], aw);
    ab += dyv;
  }
  part[(size_t)blockIdx.y * 2 * d + c] = aw;
  part[(size_t)blockIdx.y * 2 * d + d + c] = ab;
}

template <class T, class W>
__global__ void __launch_bounds__(1024)
k_ln_bwd_wide(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* __restrict__ w,
              const float* __restrict__ mean, const float* __restrict__ rstd, const T* add,
              int64_t ldadd, T* dx, int d) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t c = threadIdx.x; c < d; c += blockDim.x) {
    const float g = to_f(dy[row * lddy + c]) * (w ? to_f(w[c]) : 1.f);
    s1 += g;
    s2 = fmaf(g, (to_f(x[row * ldx + c]) - mu) * rs, s2);
  }
  const float inv_d = 1.0f / (float)d;
  s1 = group_sum(s1, red[0], 32, warp, lane) * inv_d;
  s2 = group_sum(s2, red[1], 32, warp, lane) * inv_d;
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
  // Warps per row: as few as hold the row in 8 packs a thread; more while
  // the rows alone do not give the SMs 16 warps each (few rows: latency).
  int wpr = 1;
  while (wpr < 32 && npack > wpr * 32 * 8) wpr *= 2;
  while (wpr < 32 && npack > wpr * 32 && (int64_t)T_ * wpr < 148 * 16) wpr *= 2;
  const int nv = (npack + wpr * 32 - 1) / (wpr * 32);
  const int warps = wpr > 8 ? wpr : 8;
  const int rpb = warps / wpr;
  const unsigned grid = (unsigned)(((int64_t)T_ + rpb - 1) / rpb);
  ProfScope _ps("layernorm_fwd", s);
#define LN_GO(NV, MAXT)                                                                        \
  k_ln_fwd<T, W, V, NV, MAXT><<<grid, warps * 32, 0, s>>>(x, ldx, w, b, y, mean, rstd, T_, d,  \
                                                          eps, wpr)
  if (nv > 8) k_ln_fwd_wide<T, W><<<T_, 1024, 0, s>>>(x, ldx, w, b, y, mean, rstd, d, eps);
  else if (wpr <= 8 && nv > 4) LN_GO(8, 256);
  else if (wpr <= 8 && nv > 2) LN_GO(4, 256);
  else if (wpr <= 8) LN_GO(2, 256);
  else if (nv > 4) LN_GO(8, 1024);
  else if (nv > 2) LN_GO(4, 1024);
  else LN_GO(2, 1024);
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
    if (v == 8) return ln_fwd_v<T, W, 8>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
    if (v == 2) return ln_fwd_v<T, W, 2>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
  } else {
    if (v == 4) return ln_fwd_v<T, W, 4>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
  }
  return ln_fwd_v<T, W, 1>(xt, ldx, wt, bt, T_, d, eps, yt, mean, rstd, s);
}

constexpr int LN_COLS = 8192;     // widest row of k_ln_bwd: 16 elements x 512 threads
constexpr int LN_SLICES = 64;     // row slices of k_ln_bwd_cols
constexpr int LN_SMS = 148;

// Launch shape of k_ln_bwd: elements per thread, threads per row, rows per
// block, blocks.
struct LnShape {
  int per, G, rpb, grid;
};
LnShape ln_bwd_shape(int T_, int d) {
  LnShape p;
  p.per = d <= 4096 ? 8 : 16;
  const int packs = (d + p.per - 1) / p.per;
  p.G = (packs + 31) / 32 * 32;
  p.rpb = p.G >= 256 ? 1 : 256 / p.G;
  const int per_sm = p.G * p.rpb <= 256 ? 3 : 1;
  const int64_t rows = ((int64_t)T_ + p.rpb - 1) / p.rpb;
  p.grid = (int)(rows < LN_SMS * per_sm ? rows : LN_SMS * per_sm);
  return p;
}

template <class T, class W, int V>
int ln_bwd_v(const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* w, const float* mean,
             const float* rstd, const T* add, int64_t ldadd, int T_, int d, T* dx, float* part,
             cudaStream_t s) {
  const LnShape p = ln_bwd_shape(T_, d);
  const int threads = p.G * p.rpb;
  ProfScope _ps("layernorm_bwd", s);
#define LN_GO(NV, MAXT, MINB)                                                                   \
  k_ln_bwd<T, W, V, NV, MAXT, MINB><<<p.grid, threads, 0, s>>>(dy, lddy, x, ldx, w, mean, rstd, \
                                                               add, ldadd, dx, part, T_, d, p.G)
  if (p.per == 16) LN_GO(16 / V, 512, 1);
  else if (threads > 256) LN_GO(8 / V, 512, 1);
  else LN_GO(8 / V, 256, sizeof(T) == 2 ? 3 : 2);
#undef LN_GO
  MOE_CHECK_LAUNCH("layernorm_bwd");
  return MOE_OK;
}

template <class T, class W>
int ln_bwd_t(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
             const float* mean, const float* rstd, const void* add, int64_t ldadd, int T_, int d,
             void* dx, float* part, cudaStream_t s) {
  const T *dyt = (const T*)dy, *xt = (const T*)x, *at = (const T*)add;
  const W* wt = (const W*)w;
  T* dxt = (T*)dx;
  if (d > LN_COLS) {
    if (part) {
      ProfScope _ps("layernorm_bwd_cols", s);
      const dim3 grid((d + 255) / 256, LN_SLICES);
      k_ln_bwd_cols<T><<<grid, 256, 0, s>>>(dyt, lddy, xt, ldx, mean, rstd, part, T_, d);
      MOE_CHECK_LAUNCH("layernorm_bwd_cols");
    }
    ProfScope _ps("layernorm_bwd", s);
    k_ln_bwd_wide<T, W><<<T_, 1024, 0, s>>>(dyt, lddy, xt, ldx, wt, mean, rstd, at, ldadd, dxt, d);
    MOE_CHECK_LAUNCH("layernorm_bwd");
    return MOE_OK;
  }
  const int v = pick_pack<T, W>(d, {lddy, ldx, add ? ldadd : 0}, {dy, x, add, dx}, {w});
#define LN_V(V) \
  return ln_bwd_v<T, W, V>(dyt, lddy, xt, ldx, wt, mean, rstd, at, ldadd, T_, d, dxt, part, s)
  if constexpr (sizeof(T) == 2) {
    if (v == 8) LN_V(8);
    if (v == 2) LN_V(2);
  } else {
    if (v == 4) LN_V(4);
  }
  LN_V(1);
#undef LN_V
}

int ln_parts(int T_, int d) {
  if (d > LN_COLS) return LN_SLICES;
  const LnShape p = ln_bwd_shape(T_, d);
  return p.grid * p.rpb;
}

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
  int rc;
  if (dtype == MOE_BF16)
    rc = wdtype == MOE_BF16
             ? ln_bwd_t<__nv_bfloat16, __nv_bfloat16>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, s)
             : ln_bwd_t<__nv_bfloat16, float>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, s);
  else
    rc = wdtype == MOE_BF16
             ? ln_bwd_t<float, __nv_bfloat16>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, s)
             : ln_bwd_t<float, float>(dy, lddy, x, ldx, w, mean, rstd, add, ldadd, T, d, dx, part, s);
  if (rc || part == nullptr) return rc;
  ProfScope _ps("layernorm_reduce", s);
  k_ln_reduce<<<(unsigned)((2 * (int64_t)d + 31) / 32), dim3(32, 32), 0, s>>>(part, ln_parts(T, d), d,
                                                                              dweight, dbias);
  MOE_CHECK_LAUNCH("layernorm_reduce");
  return MOE_OK;
}

}  // namespace moe
