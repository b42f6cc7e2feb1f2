// What the tensor-core kernels share: tile sizes, bounded waits, the staged
// tile stores of the epilogues, and the host-side tensor maps.
#pragma once

#include <dlfcn.h>

#include <cstring>

#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

using namespace tc;

constexpr int BM = 128;
constexpr int BK = 64;                 // 64 bf16 = 128 bytes = one swizzle row
constexpr int ATOM = 8192;             // one 64 x 64 bf16 TMA box
constexpr int A_BYTES = BM * BK * 2;   // 16 KB
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int THREADS = 320;           // 2 control warps + 8 epilogue warps
constexpr int EPI_THREADS = 256;

// Sigmoid for the tensor-core epilogues (fast exponential and division; the
// results are rounded to bf16 afterwards).
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}

__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* s_abort,
                                             int* status, int code, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*s_abort) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        *s_abort = 1;
        record_status(status, 0x200 | code);
        return false;
      }
    }
  }
}

// Element i of 32 bf16 values packed in four uint4, as fp32.
__device__ __forceinline__ float bf16_lane(const uint4 (&p)[4], int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(&p[i >> 3])[(i >> 1) & 3];
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}

__device__ __forceinline__ void ld_bf16x32(const __nv_bfloat16* src, float* v) {
  const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 u = p[q];
    __nv_bfloat162 h[4];
    memcpy(h, &u, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f2 = __bfloat1622float2(h[i]);
      v[q * 8 + 2 * i] = f2.x;
      v[q * 8 + 2 * i + 1] = f2.y;
    }
  }
}

// Stage one warp's 32 rows x 32 columns (row = lane) in one of its two 2 KB
// shared tiles (64-byte swizzle: 16-byte chunk c of row r sits at chunk
// c ^ ((r >> 1) & 3)) and store it with one TMA tile store at (col, row0).
// The tiles alternate; before a tile is rewritten, the store issued from it
// two calls ago must have finished reading it.
template <int NT = 2>
__device__ __forceinline__ void stage_store(uint8_t* tiles, int& which, const float* v,
                                            const CUtensorMap* map, int col, int row0, int lane) {
  uint8_t* tile = tiles + which * 2048;
  if (NT == 2) which ^= 1;
  if (lane == 0) {
    if (NT == 2) bulk_wait_read_1();
    else bulk_wait_read_all();
  }
  __syncwarp();
  uint8_t* rowp = tile + lane * 64;
  const int sw = (lane >> 1) & 3;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[q * 8 + 2 * i], v[q * 8 + 2 * i + 1]);
    uint4 u;
    memcpy(&u, h, 16);
    *reinterpret_cast<uint4*>(rowp + ((q ^ sw) << 4)) = u;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, tile, col, row0);
    bulk_commit();
  }
}

// ============================================================== host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Looked up once; the initialisation of a function-local static is
// thread-safe, so host threads may make their first calls concurrently.
inline EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* h = dlopen("libcuda.so.1", RTLD_NOW | RTLD_GLOBAL);
    return h ? reinterpret_cast<EncodeTiledFn>(dlsym(h, "cuTensorMapEncodeTiled")) : nullptr;
  }();
  return fn;
}

// bf16 row-major [outer, inner] (rows ld elements apart; 0: inner) viewed in
// boxes of box_outer x box_inner.
inline int make_map_2d(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                       uint32_t box_inner, uint32_t box_outer,
                       CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B, uint64_t ld = 0) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {(ld ? ld : inner) * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (2d) failed: " + std::to_string((int)r));
  return MOE_OK;
}

// 8-bit [d2, d1, d0] (d0 innermost; d2 = 1 for a matrix) in boxes of box1 x
// box0 bytes, 128-byte swizzle (E4M3 operand tiles).
inline int make_map_u8(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2,
                       uint32_t box0, uint32_t box1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0, d0 * d1};
  cuuint32_t box[3] = {box0, box1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (u8) failed: " + std::to_string((int)r));
  return MOE_OK;
}

// Output map of the epilogue's TMA stores: 32 x 32 boxes, 64-byte swizzle.
inline int make_store_map(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer) {
  return make_map_2d(m, ptr, inner, outer, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// bf16 [batch, outer, inner] (inner contiguous, a multiple of 64; rows ld
// elements apart, 0: inner) as the
// 4-d view [batch][inner / 64][outer][64]: one box brings `atoms` adjacent
// 64-column blocks of BK rows, stored block after block (BK x 128 bytes
// each, 128-byte swizzle) -- the shared-memory layout of an MN-major
// operand -- so a stage's operand takes one copy instead of one per block.
inline int make_map_atoms(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                          uint64_t batch, uint32_t atoms, uint64_t ld = 0) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  if (inner % 64 != 0) return fail(MOE_ERR_INVALID_ARG, "operand width not a multiple of 64");
  cuuint64_t dims[4] = {64, outer, inner / 64, batch};
  if (ld == 0) ld = inner;
  cuuint64_t strides[3] = {ld * 2, 128, ld * outer * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)BK, atoms, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (atoms) failed: " + std::to_string((int)r));
  return MOE_OK;
}

// bf16 [d2, d1, d0] (d0 innermost) viewed in boxes of box1 x box0.
inline int make_map_3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2,
                       uint32_t box0, uint32_t box1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  cuuint32_t box[3] = {box0, box1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (3d) failed: " + std::to_string((int)r));
  return MOE_OK;
}

}  // namespace moe
