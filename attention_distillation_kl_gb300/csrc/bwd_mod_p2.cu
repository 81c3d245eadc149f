// Instantiations of the backward over modified scores, mode P2 (see
// bwd_mod.cuh), and the kernels around it.  One translation unit per mode so
// the build compiles them in parallel.
#include <algorithm>

#include "bwd_mod.cuh"

namespace skl {

namespace {

// fp32 rows [heads][n][pitch] (null: zeros) rounded once to bf16, 8 values a thread.
__global__ void __launch_bounds__(256) mod_convert_kernel(const float* __restrict__ src, int per_batch, int n, int d,
                                                          int pitch, __nv_bfloat16* __restrict__ dst, long long sb,
                                                          long long sh, long long sn) {
  const int per_row = d / 8;
  const long long total = (long long)n * per_row;
  const int b = blockIdx.y / per_batch, h = blockIdx.y - b * per_batch;
  for (long long u = blockIdx.x * 256ll + threadIdx.x; u < total; u += gridDim.x * 256ll) {
    const int i = int(u / per_row), c = int(u - (long long)i * per_row) * 8;
    float4 x{0.f, 0.f, 0.f, 0.f}, y = x;
    if (src != nullptr) {
      const float4* p = reinterpret_cast<const float4*>(src + (size_t(blockIdx.y) * n + i) * pitch + c);
      x = __ldcs(p);
      y = __ldcs(p + 1);
    }
    uint4 o;
    o.x = pack_bf16(x.x, x.y);
    o.y = pack_bf16(x.z, x.w);
    o.z = pack_bf16(y.x, y.y);
    o.w = pack_bf16(y.z, y.w);
    *reinterpret_cast<uint4*>(dst + b * sb + h * sh + i * sn + c) = o;
  }
}

// dtable[h][k] = the warps' sums added in a fixed order: thread (g, k) takes
// every 4th of the head's rows, then the four shares are added.
__global__ void __launch_bounds__(256) mod_table_reduce_kernel(const float* __restrict__ dtab, int B, int H, int nkt,
                                                               int num_buckets, float* __restrict__ dtable) {
  __shared__ float part[4][kMaxBuckets];
  const int h = blockIdx.x, k = threadIdx.x % kMaxBuckets, g = threadIdx.x / kMaxBuckets;
  float s = 0.f;
  for (int b = 0; b < B; ++b) {
    const float* p = dtab + (size_t(b) * H + h) * nkt * 8 * kMaxBuckets;
    for (int u = g; u < nkt * 8; u += 4) s += p[size_t(u) * kMaxBuckets + k];
  }
  part[g][k] = s;
  __syncthreads();
  if (g == 0 && k < num_buckets) dtable[size_t(h) * num_buckets + k] = (part[0][k] + part[1][k]) + (part[2][k] + part[3][k]);
}

// kmax of a strided K (see kmax_kernel in dq_fixed.cu).
__global__ void __launch_bounds__(256) mod_kmax_kernel(const __nv_bfloat16* __restrict__ k, int per_batch, int n, int d,
                                                       long long sb, long long sh, long long sn, unsigned* kmax) {
  const int b = blockIdx.y / per_batch, h = blockIdx.y - b * per_batch;
  const __nv_bfloat16* p = k + b * sb + h * sh;
  const int per_row = d / 8;
  const long long total = (long long)n * per_row;
  uint32_t m = 0;
  for (long long u = blockIdx.x * 256ll + threadIdx.x; u < total; u += gridDim.x * 256ll) {
    const long long i = u / per_row;
    const uint4 w = *reinterpret_cast<const uint4*>(p + i * sn + (u - i * per_row) * 8);
    const uint32_t x = max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu), max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
    const uint32_t y = max(max(w.z & 0x7fffu, (w.z >> 16) & 0x7fffu), max(w.w & 0x7fffu, (w.w >> 16) & 0x7fffu));
    m = max(m, max(x, y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) atomicMax(kmax + blockIdx.y, m);
}

int row_blocks(long long total, int heads) {
  const long long want = (total + 255) / 256, share = (4864 + heads - 1) / heads;  // 32 blocks per SM over all heads
  return int(std::max(1ll, std::min(want, share)));
}

}  // namespace

int launch_bwd_mod_p2(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st) {
  return launch_bwd_mod_mode<STREAMKL_GRAD_P2>(m, d1, d2, a, st);
}

int launch_mod_convert(const float* src, int B, int per_batch, int n, int d, int pitch, void* dst, long long sb,
                       long long sh, long long sn, cudaStream_t st) {
  const int heads = B * per_batch;
  dim3 grid(row_blocks((long long)n * (d / 8), heads), heads);
  mod_convert_kernel<<<grid, 256, 0, st>>>(src, per_batch, n, d, pitch, static_cast<__nv_bfloat16*>(dst), sb, sh, sn);
  return cudaGetLastError();
}

int launch_mod_table_reduce(const float* dtab, int B, int H, int nkt, int num_buckets, float* dtable,
                            cudaStream_t st) {
  mod_table_reduce_kernel<<<H, 256, 0, st>>>(dtab, B, H, nkt, num_buckets, dtable);
  return cudaGetLastError();
}

int launch_kmax_strided(const void* k, int B, int per_batch, int n, int d, long long sb, long long sh, long long sn,
                        unsigned* kmax, cudaStream_t st) {
  const int heads = B * per_batch;
  dim3 grid(row_blocks((long long)n * (d / 8), heads), heads);
  mod_kmax_kernel<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(k), per_batch, n, d, sb, sh, sn, kmax);
  return cudaGetLastError();
}

}  // namespace skl
