// Instantiations of the forward over modified scores for a first side of tile
// width 128; see fwd_mod.cuh.  Two translation units so the build compiles
// them in parallel.
#include "fwd_mod.cuh"

namespace skl {

int launch_fwd_mod_128(const ModMaps& m, int d2, const ModFwdArgs& a, cudaStream_t st) {
  return d2 == 64 ? launch_fwd_mod_t<128, 64>(m, a, st) : launch_fwd_mod_t<128, 128>(m, a, st);
}

}  // namespace skl
