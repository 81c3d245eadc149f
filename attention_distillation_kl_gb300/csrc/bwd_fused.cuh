// What the fused backward kernels (bwd.cu and bwd_mod.cuh) share: their shared
// memory layout and barriers, and the waits between issuers and between CTAs.
#pragma once

#include "bwd_common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace skl {

constexpr int kDqBoxes = 2;          // dQ staging boxes per epilogue warp
constexpr uint32_t kDqBoxBytes = 4096;  // [32 rows][32 fp32], 128-byte swizzle

template <int D1, int D2, int MODE>
struct BwdLayout {
  static constexpr int DG = MODE == STREAMKL_GRAD_P2 ? D2 : D1;  // gradient side
  static constexpr int DO = MODE == STREAMKL_GRAD_P2 ? D1 : D2;  // other side
  // Mode P1 forms dS with one ex2 per pair, so the MMA issue chain is what
  // bounds it: dK and dQ then get an issuing thread each (16 warps).  In
  // mode P2 the dS warps bound the tile and one thread issues both (15).
  static constexpr bool kSplitIssue = MODE == STREAMKL_GRAD_P1;
  static constexpr int kThreads = 32 * (kSplitIssue ? 16 : 15);
  static constexpr uint32_t kDS = kTile * kTile * 2;
  static constexpr uint32_t kK1 = kTile * D1 * 2, kK2 = kTile * D2 * 2;
  static constexpr uint32_t kQo = kTile * DO * 2, kQg = kTile * DG * 2;
  enum {
    B_KFULL, B_QOFULL, B_QOEMPTY, B_QGFULL0, B_QGFULL1, B_QGFULL2, B_QGEMPTY0, B_QGEMPTY1, B_QGEMPTY2,
    B_SFULL, B_SFREE, B_DSFULL, B_DSEMPTY, B_DQFULL, B_DQEMPTY, B_DKFULL, B_DONE, kNumBars
  };
  // Q_g buffers: its buffer of tile t is free again only when the dK
  // product of tile t has run, and that product comes late in the tile (it
  // waits for dS and for the next tile's S to be queued), so two buffers
  // chain the reload of tile t + 2 to the dK of tile t; a third buffer,
  // where it fits (every pair of head dims but 128 and 128), takes the
  // reload off that chain
  static constexpr uint32_t kFixed = kDS + kK1 + kK2 + kQo + 4 * kDqBoxes * kDqBoxBytes + kNumBars * 8 + 32;
  static constexpr int kQgBufs = kFixed + 3 * kQg + 1024 <= 232448 ? 3 : 2;
  static constexpr uint32_t oDS = 0, oK1 = kDS, oK2 = oK1 + kK1, oQo = oK2 + kK2, oQg = oQo + kQo;
  static constexpr uint32_t oStage = oQg + kQgBufs * kQg;  // dQ staging: 4 warps x kDqBoxes x kDqBoxBytes
  static constexpr uint32_t oBar = oStage + 4 * kDqBoxes * kDqBoxBytes;
  static constexpr uint32_t oMisc = oBar + kNumBars * 8;
  static constexpr uint32_t kBytes = oMisc + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "over the 227 KB shared memory limit");
};

// The gradient products of tile t are issued only once the S products of
// tile t + 1 are queued: the tensor pipe takes them in issue order, and S is
// what the dS warps wait for, so S should not queue behind dK and dQ.  A
// scheduling hint only (the two groups touch different TMEM columns and
// operands), so the wait gives up after 20 us rather than reporting anything.
__device__ __forceinline__ void wait_s_queued(volatile int* s_queued, int want) {
  if (want <= 0 || *s_queued >= want) return;
  const uint64_t t0 = globaltimer();
  while (*s_queued < want && globaltimer() - t0 < 20000ull) {
  }
}

// Grouped key heads, deterministic mode: waits until the count of query
// heads that have added their dK to this (key head, key tile) reads `want`,
// polling with a short sleep.  Gives up when this CTA or another one has
// aborted, or after `limit_ns`; then this CTA aborts, and a time-out also
// aborts the launch and is reported in the status word.
static __device__ __noinline__ bool wait_turn(const int* turn, int want, int* launch_abort, Ctl ctl,
                                              uint64_t limit_ns = STREAMKL_WAIT_LIMIT_NS) {
  const uint64_t t0 = globaltimer();
  while (true) {
    if (ld_acquire_gpu(turn) == want) return true;
    if (*ctl.abort || *reinterpret_cast<volatile int*>(launch_abort)) {
      *ctl.abort = 1;
      return false;
    }
    if (globaltimer() - t0 > limit_ns) {
      *ctl.abort = 1;
      atomicExch(launch_abort, 1);
      atomicCAS(ctl.status, 0, (int)STREAMKL_DEVICE_TIMEOUT);
      return false;
    }
    __nanosleep(128);
  }
}

}  // namespace skl
