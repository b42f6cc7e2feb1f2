// Dropout from a counter-based generator, with the residual sum.
//
//   out[i] = residual[i] + (keep_i ? x[i] * 65536 / (65536 - thr) : 0)
//
// The mask is never stored: the backward pass draws it again.  keep_i comes
// from Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", 2011) with the seed as its key and the counter
// (i / 8, offset): eight elements share one block of 128 bits, 16 bits each
// (element i: half i % 2 of word (i % 8) / 2), kept where the 16 bits are at
// least thr = round(65536 p).  16 bits instead of 32 halve the integer work
// per element, which at 32 bits is about what the memory system leaves time
// for; the price is that p counts in steps of 2^-16, and the scale follows
// the rounded p, so the mean is exact.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

// The 8 draws of block `blk`: words.x..w, low half first.
__device__ __forceinline__ uint4 philox(uint64_t seed, uint64_t offset, uint64_t blk) {
  uint32_t c0 = (uint32_t)blk, c1 = (uint32_t)(blk >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Element j is kept where its 16 bits are >= thr; thr_hi = thr << 16, and a
// low half is compared after a shift (`any` false: thr = 65536, nothing is kept).
__device__ __forceinline__ bool kept(const uint4& w, int j, uint32_t thr_hi, bool any) {
  const uint32_t word = j < 2 ? w.x : (j < 4 ? w.y : (j < 6 ? w.z : w.w));
  return any && ((j & 1) ? word : word << 16) >= thr_hi;
}

// The 8 elements of one generator block as raw words, computed on in pairs.
template <class T>
struct Oct {
  static constexpr int U = 8 * (int)sizeof(T) / 16;
  uint4 r[U];
  __device__ __forceinline__ void load(const T* p, int64_t blk) {
    const uint4* s = reinterpret_cast<const uint4*>(p) + blk * U;
#pragma unroll
    for (int i = 0; i < U; ++i) r[i] = s[i];
  }
  __device__ __forceinline__ void store(T* p, int64_t blk) const {
    uint4* s = reinterpret_cast<uint4*>(p) + blk * U;
#pragma unroll
    for (int i = 0; i < U; ++i) s[i] = r[i];
  }
  __device__ __forceinline__ F2 pair(int j) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(r);
    if constexpr (sizeof(T) == 2) return f2_from_bf16x2(w[j]);
    else return f2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  }
  __device__ __forceinline__ void set_pair(int j, F2 v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(r);
    if constexpr (sizeof(T) == 2) {
      w[j] = f2_to_bf16x2(v);
    } else {
      const float2 t = f2_get(v);
      w[2 * j] = __float_as_uint(t.x);
      w[2 * j + 1] = __float_as_uint(t.y);
    }
  }
};

// One thread per generator block, 64 warps on an SM: at 16384 x 2048 bf16 with
// a residual 36 us, against 38 to 44 with 2 or 4 blocks per thread and fewer
// warps, or with a grid that walks (a plain sum of two tensors takes 33).
template <class T, bool RES>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 8 : 6)
k_dropout(const T* x, const T* res, int64_t n, uint32_t thr, float scale,
          const int64_t* __restrict__ rng, T* out) {
  const int64_t nb = n >> 3, b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const uint32_t thr_hi = thr << 16;
  const bool any = thr < 65536u;
  if (b < nb) {
    Oct<T> vx, vr;
    vx.load(x, b);
    if (RES) vr.load(res, b);
    const uint4 w = philox((uint64_t)rng[0], (uint64_t)rng[1], (uint64_t)b);
    const F2 sc = f2(scale, scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // a select, not a product with 0: what is dropped may be infinite
      const float2 t = f2_get(vx.pair(j));
      const F2 k = f2(kept(w, 2 * j, thr_hi, any) ? t.x : 0.f,
                      kept(w, 2 * j + 1, thr_hi, any) ? t.y : 0.f);
      vx.set_pair(j, f2_fma(k, sc, RES ? vr.pair(j) : f2(0.f, 0.f)));
    }
    vx.store(out, b);
  } else if (b < nb + (n & 7)) {   // the last, partial block: one element each
    const int j = (int)(b - nb);
    const int64_t i = (nb << 3) + j;
    const uint4 w = philox((uint64_t)rng[0], (uint64_t)rng[1], (uint64_t)nb);
    const float v = kept(w, j, thr_hi, any) ? to_f(x[i]) : 0.f;
    out[i] = from_f<T>(fmaf(v, scale, RES ? to_f(res[i]) : 0.f));
  }
}

// Buffers that are not 16-byte aligned: element accesses, a thread's eight side by
// side (16384 x 2048 bf16 with a residual, one element off: 92 us, aligned 32).
template <class T, bool RES>
__global__ void __launch_bounds__(256)
k_dropout_any(const T* x, const T* res, int64_t n, uint32_t thr, float scale,
              const int64_t* __restrict__ rng, T* out) {
  const uint64_t seed = (uint64_t)rng[0], offset = (uint64_t)rng[1];
  const uint32_t thr_hi = thr << 16;
  const bool any = thr < 65536u;
  const int64_t nb = (n + 7) >> 3, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < nb; b += stride) {
    const uint4 w = philox(seed, offset, (uint64_t)b);
    const int m = n - (b << 3) < 8 ? (int)(n - (b << 3)) : 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < m) {
        const int64_t i = (b << 3) + j;
        const float v = kept(w, j, thr_hi, any) ? to_f(x[i]) : 0.f;
        out[i] = from_f<T>(fmaf(v, scale, RES ? to_f(res[i]) : 0.f));
      }
  }
}

template <class T>
int dropout_t(const void* x, const void* res, int64_t n, uint32_t thr, float scale,
              const int64_t* rng, void* out, const char* name, cudaStream_t s) {
  const bool al = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) |
                    reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int64_t want = ((n >> 3) + (n & 7) + 255) / 256;
  if (want > 0x7fffffff) return fail(MOE_ERR_UNSUPPORTED, "dropout: n must be below 2^42");
  const unsigned grid = (unsigned)want;
  const T *xt = (const T*)x, *rt = (const T*)res;
  T* ot = (T*)out;
  ProfScope _ps(name, s);
  if (al && res) k_dropout<T, true><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
  else if (al) k_dropout<T, false><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
  else if (res) k_dropout_any<T, true><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
  else k_dropout_any<T, false><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
  MOE_CHECK_LAUNCH(name);
  return MOE_OK;
}

}  // namespace

int launch_dropout(const void* x, const void* residual, int64_t n, uint32_t thr, const int64_t* rng,
                   int dtype, void* out, const char* name, cudaStream_t s) {
  // nothing is kept at thr = 65536
  const float scale = thr < 65536u ? (float)(65536.0 / (65536.0 - thr)) : 0.f;
  return dtype == MOE_BF16 ? dropout_t<__nv_bfloat16>(x, residual, n, thr, scale, rng, out, name, s)
                           : dropout_t<float>(x, residual, n, thr, scale, rng, out, name, s);
}

}  // namespace moe
