// One key for each block of keys: the mean of those whose id is not negative,
// summed in fp32 and rounded to bf16 once.  A warp takes a block, its lanes 16
// bytes of a row each, as many rows at a time as 32 lanes hold.  Bound by the
// one read of K: 65536 keys x 8 heads x 128 take 22.6 us, 6.0 TB/s (24.4 without
// the hint that they are read once; 31 with 16 loads of a lane in flight instead
// of 8, and 27 with 8 warps a block).
#include <cuda_bf16.h>

#include "bwd_common.cuh"
#include "views.cuh"

namespace skl {

namespace {

constexpr int kPoolWarps = 4;

struct PoolArgs {
  const __nv_bfloat16* k;
  __nv_bfloat16* y;
  long long kb, kh, kn, yb, yh, yn;
  const int* ids;  // [B][NK] or null
  int heads, NK, d, block, blocks, units;
};

__global__ void __launch_bounds__(32 * kPoolWarps) pool_kernel(const __grid_constant__ PoolArgs a) {
  const int unit = blockIdx.x * kPoolWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit >= a.units) return;
  const int head = unit / a.blocks, j = unit - head * a.blocks, b = head / a.heads, h = head - b * a.heads;
  const int per_row = a.d / 8, at_once = 32 / per_row;  // lanes of a row, rows at a time
  const int sub = lane / per_row, c = lane - sub * per_row;
  const int first = j * a.block, rows = min(a.block, a.NK - first);
  const __nv_bfloat16* src = a.k + b * a.kb + h * a.kh + first * a.kn + 8 * c;
  const int* ids = a.ids == nullptr ? nullptr : a.ids + (long long)b * a.NK + first;
  float sum[8] = {};
  int n = 0;
  auto add = [&](const uint4& w) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[2 * e] += __uint_as_float(v[e] << 16);
      sum[2 * e + 1] += __uint_as_float(v[e] & 0xffff0000u);
    }
    ++n;
  };
  if (sub < at_once) {
    constexpr int kAtOnce = 8;
    for (int r0 = sub; r0 < rows; r0 += kAtOnce * at_once) {
      uint4 w[kAtOnce];
      bool on[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int r = r0 + e * at_once;
        on[e] = r < rows && (ids == nullptr || ids[r] >= 0);
        if (on[e]) w[e] = __ldcs(reinterpret_cast<const uint4*>(src + r * a.kn));
      }
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        if (on[e]) add(w[e]);
    }
  }
  // the shares of a row's lanes, in order
  float out[8] = {};
  int total = 0;
  for (int s = 0; s < at_once; ++s) {
    const int from = (s * per_row + c) & 31;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] += __shfl_sync(0xffffffffu, sum[e], from);
    total += __shfl_sync(0xffffffffu, n, from);
  }
  if (sub != 0) return;
  const float div = float(max(total, 1));
  uint4 o;
  o.x = pack_bf16(out[0] / div, out[1] / div);
  o.y = pack_bf16(out[2] / div, out[3] / div);
  o.z = pack_bf16(out[4] / div, out[5] / div);
  o.w = pack_bf16(out[6] / div, out[7] / div);
  *reinterpret_cast<uint4*>(a.y + b * a.yb + h * a.yh + j * a.yn + 8 * c) = o;
}

}  // namespace

}  // namespace skl

extern "C" int streamkl_pool_blocks(const streamkl_view* k, const int* doc_k, int B, int HK, int NK, int d, int block,
                                    const streamkl_view* kb, streamkl_stream_t stream) {
  using namespace skl;
  if (k == nullptr || kb == nullptr || B < 0 || HK < 0 || NK < 0) return STREAMKL_INVALID_ARG;
  if (block != 32 && block != 64 && block != 128) return STREAMKL_INVALID_ARG;
  if (d < 16 || d > 128 || d % 16 != 0) return STREAMKL_UNSUPPORTED;
  if (!aligned4(doc_k)) return STREAMKL_INVALID_ARG;
  if (B == 0 || HK == 0 || NK == 0) return STREAMKL_OK;
  const int blocks = int(((long long)NK + block - 1) / block);
  if (!view_ok(*k, B, HK, NK) || !view_ok(*kb, B, HK, blocks)) return STREAMKL_INVALID_ARG;
  if ((long long)B * HK > 65535 || (long long)B * HK * NK > (1ll << 31) - 1) return STREAMKL_INVALID_ARG;
  const int s = check_device();
  if (s != STREAMKL_OK) return s;
  auto stride = [](long long v, int size) { return size <= 1 ? 0ll : v; };
  PoolArgs a{};
  a.k = static_cast<const __nv_bfloat16*>(k->data);
  a.y = static_cast<__nv_bfloat16*>(kb->data);
  a.kb = stride(k->stride_b, B), a.kh = stride(k->stride_h, HK), a.kn = stride(k->stride_n, NK);
  a.yb = stride(kb->stride_b, B), a.yh = stride(kb->stride_h, HK), a.yn = stride(kb->stride_n, blocks);
  a.ids = doc_k;
  a.heads = HK;
  a.NK = NK;
  a.d = d;
  a.block = block;
  a.blocks = blocks;
  a.units = B * HK * blocks;
  pool_kernel<<<unsigned((a.units + kPoolWarps - 1) / kPoolWarps), 32 * kPoolWarps, 0,
                reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return as_status(cudaGetLastError());
}
