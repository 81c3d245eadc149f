// Instantiations of the forward over modified scores for a first side of tile
// width 64; see fwd_mod.cuh.  Two translation units so the build compiles
// them in parallel.
#include "fwd_mod.cuh"

namespace skl {

namespace {

// Merges the key splits: a warp per row, a lane for every 32nd split, then
// the lanes' states in pairs.  (A thread per row waited for each split's
// values in turn: 21 us for 512 rows of 19 splits.)
__global__ void __launch_bounds__(256) mod_reduce_kernel(const __grid_constant__ ModFwdArgs a) {
  const float* __restrict__ part = a.partial;
  const int rows = a.B * a.H * a.NQ;
  const int lane = threadIdx.x & 31;
  const long long i = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  if (i >= rows) return;
  const size_t R = size_t(rows);
  auto add = [](ModStats& st, const ModStats& o) {
    if (o.l1 == 0.f) return;
    if (st.l1 == 0.f) st = o;
    else merge_stats(st, o);
  };
  ModStats st{0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = lane; s < a.num_splits; s += 32) {
    const float* p = part + size_t(s) * 5 * R + i;
    add(st, ModStats{p[0], p[R], p[2 * R], p[3 * R], p[4 * R]});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const ModStats x{__shfl_down_sync(0xffffffffu, st.m1, o), __shfl_down_sync(0xffffffffu, st.m2, o),
                     __shfl_down_sync(0xffffffffu, st.l1, o), __shfl_down_sync(0xffffffffu, st.l2, o),
                     __shfl_down_sync(0xffffffffu, st.acc, o)};
    if (lane < o) add(st, x);
  }
  const int h = int(i / a.NQ) % a.H;
  auto masked = [&](const ModSide& s) {
    return s.kind == kBiasTable ? s.near[size_t(h) * near_row(s.reach) + near_len(s.reach) + 2] : -INFINITY;
  };
  if (lane == 0) write_row(st, masked(a.s1), masked(a.s2), a.kl + i, a.lse1 + i, a.lse2 + i);
}

}  // namespace

int launch_fwd_mod_64(const ModMaps& m, int d2, const ModFwdArgs& a, cudaStream_t st) {
  return d2 == 64 ? launch_fwd_mod_t<64, 64>(m, a, st) : launch_fwd_mod_t<64, 128>(m, a, st);
}

int launch_mod_reduce(const ModFwdArgs& a, cudaStream_t st) {
  const long long rows = (long long)a.B * a.H * a.NQ;
  mod_reduce_kernel<<<unsigned((rows + 7) / 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace skl
