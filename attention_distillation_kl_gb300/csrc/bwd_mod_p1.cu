// Instantiations of the backward over modified scores, mode P1; see bwd_mod.cuh.
#include "bwd_mod.cuh"

namespace skl {

int launch_bwd_mod_p1(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st) {
  return launch_bwd_mod_mode<STREAMKL_GRAD_P1>(m, d1, d2, a, st);
}

}  // namespace skl
