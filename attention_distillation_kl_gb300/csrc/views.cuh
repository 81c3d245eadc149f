// Host helpers of the entry points that take strided views: their checks,
// tensor maps and workspace layout.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host.cuh"
#include "kernels.cuh"
#include "streamkl.h"

namespace skl {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t up16(size_t n) { return (n + 15) / 16 * 16; }
inline int tiles(int n) { return (n + kTile - 1) / kTile; }
inline int tile_width(int d) { return d <= 64 ? 64 : 128; }

// Strides of [B][heads][n][d] with the last dimension dense.  A dimension of
// size 1 takes any stride.
inline bool view_ok(const streamkl_view& v, int B, int heads, int n) {
  if (v.data == nullptr || !aligned16(v.data)) return false;
  auto ok = [](long long s, int size) { return size <= 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38)); };
  return ok(v.stride_b, B) && ok(v.stride_h, heads) && ok(v.stride_n, n);
}

// A strided [B][heads][n][d] bf16 tensor: boxes of 64 elements x box_rows,
// 128-byte swizzle; rows past n and columns past d read as zeros.
inline bool map_bf16(CUtensorMap* m, const streamkl_view& v, int B, int heads, int n, int d, int box_rows = kTile) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  auto bytes = [&](long long s, int size) { return cuuint64_t(size <= 1 ? ((d + 7) / 8 * 16) : s * 2); };
  cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(n), cuuint64_t(heads), cuuint64_t(B)};
  cuuint64_t strides[3] = {bytes(v.stride_n, n), bytes(v.stride_h, heads), bytes(v.stride_b, B)};
  cuuint32_t box[4] = {64u, cuuint32_t(box_rows), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v.data), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Gradients in the workspace, [heads][n][pitch] fp32: boxes of 32 x 32, 128-byte swizzle.
inline bool map_f32(CUtensorMap* m, float* p, int heads, int n, int pitch) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {cuuint64_t(pitch), cuuint64_t(n), cuuint64_t(heads)};
  cuuint64_t strides[2] = {cuuint64_t(pitch) * 4, cuuint64_t(n) * pitch * 4};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes handed out of a workspace, 16-byte aligned; with a null base it only counts.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base == nullptr ? nullptr : reinterpret_cast<T*>(base + used);
    used += up16(count * sizeof(T));
    return p;
  }
};

inline int as_status(int cuda_err) { return cuda_err == 0 ? STREAMKL_OK : STREAMKL_CUDA_ERROR; }

}  // namespace skl
