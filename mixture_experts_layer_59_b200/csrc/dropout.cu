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

__device__ __forceinline__ bool kept(const uint4& w, int j, uint32_t thr) {
  const uint32_t word = j < 2 ? w.x : (j < 4 ? w.y : (j < 6 ? w.z : w.w));
  return ((j & 1) ? word >> 16 : word & 0xffffu) >= thr;
}

template <class T>
struct alignas(16) Oct {   // the 8 elements of one generator block
  T v[8];
};

// One thread per generator block and step; UN blocks in flight per thread.
template <class T, bool RES, int UN>
__global__ void __launch_bounds__(256)
k_dropout(const T* x, const T* res, int64_t n, uint32_t thr, float scale,
          const int64_t* __restrict__ rng, T* out) {
  const uint64_t seed = (uint64_t)rng[0], offset = (uint64_t)rng[1];
  const int64_t nb = n >> 3, stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t b0 = first; b0 < nb; b0 += UN * stride) {
    Oct<T> vx[UN], vr[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t b = b0 + u * stride;
      if (b < nb) {
        vx[u] = reinterpret_cast<const Oct<T>*>(x)[b];
        if (RES) vr[u] = reinterpret_cast<const Oct<T>*>(res)[b];
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t b = b0 + u * stride;
      if (b < nb) {
        const uint4 w = philox(seed, offset, (uint64_t)b);
        Oct<T> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // a select, not a product with 0: what is dropped may be infinite
          float v = kept(w, j, thr) ? to_f(vx[u].v[j]) * scale : 0.f;
          if (RES) v += to_f(vr[u].v[j]);
          o.v[j] = from_f<T>(v);
        }
        reinterpret_cast<Oct<T>*>(out)[b] = o;
      }
    }
  }
  const int tail = (int)(n & 7);
  if (first < tail) {
    const int64_t i = (nb << 3) + first;
    const uint4 w = philox(seed, offset, (uint64_t)nb);
    float v = kept(w, (int)first, thr) ? to_f(x[i]) * scale : 0.f;
    if (RES) v += to_f(res[i]);
    out[i] = from_f<T>(v);
  }
}

// Buffers that are not 16-byte aligned: element accesses.
template <class T, bool RES>
__global__ void __launch_bounds__(256)
k_dropout_any(const T* x, const T* res, int64_t n, uint32_t thr, float scale,
              const int64_t* __restrict__ rng, T* out) {
  const uint64_t seed = (uint64_t)rng[0], offset = (uint64_t)rng[1];
  const int64_t nb = (n + 7) >> 3, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < nb; b += stride) {
    const uint4 w = philox(seed, offset, (uint64_t)b);
    const int m = n - (b << 3) < 8 ? (int)(n - (b << 3)) : 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < m) {
        const int64_t i = (b << 3) + j;
        float v = kept(w, j, thr) ? to_f(x[i]) * scale : 0.f;
        if (RES) v += to_f(res[i]);
        out[i] = from_f<T>(v);
      }
  }
}

template <class T>
int dropout_t(const void* x, const void* res, int64_t n, uint32_t thr, float scale,
              const int64_t* rng, void* out, const char* name, cudaStream_t s) {
  constexpr int UN = 2;
  const bool al = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) |
                    reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int64_t blocks8 = (n + 7) >> 3;
  const int64_t want = (blocks8 + 255) / 256;
  const unsigned grid = (unsigned)(want < 148 * 8 ? want : 148 * 8);
  const T *xt = (const T*)x, *rt = (const T*)res;
  T* ot = (T*)out;
  ProfScope _ps(name, s);
  if (al && res) k_dropout<T, true, UN><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
  else if (al) k_dropout<T, false, UN><<<grid, 256, 0, s>>>(xt, rt, n, thr, scale, rng, ot);
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
