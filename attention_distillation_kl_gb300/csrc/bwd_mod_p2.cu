// Instantiations of the backward over modified scores, mode P2; see
// bwd_mod.cuh.  One translation unit per mode so the build compiles them in
// parallel.
#include "bwd_mod.cuh"

namespace skl {

int launch_bwd_mod_p2(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st) {
  return launch_bwd_mod_mode<STREAMKL_GRAD_P2>(m, d1, d2, a, st);
}

}  // namespace skl
