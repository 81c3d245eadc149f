// Host helpers of the calls that take two sides and their masks (defined in
// api_mod.cu).
#pragma once

#include "mod_common.cuh"
#include "views.cuh"

namespace skl {

// Sizes, masks and both sides.  *empty: no query row (or head) to compute.
int check_call(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis, int B, int H, int NQ,
               int NK, bool data, bool* empty);
// The part of a workspace that holds padded ids and lookup rows.
void take_prep(Carver& c, ModPrepArgs& a, const streamkl_side* const p[2], const streamkl_visible& vis, int B, int H,
               int NQ, int NK, int table_grad_side);
ModVis vis_args(const streamkl_visible& v, const ModPrepArgs& p);

}  // namespace skl
