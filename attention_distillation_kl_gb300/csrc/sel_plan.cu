// The plan of attention over selected blocks (sel_common.cuh): for each block
// the queries that selected it, in order, and the items that cut these lists.
//
// Three kernels.  A warp owns a chunk of queries and the blocks' counters of
// that chunk, in shared memory; it takes 32 slots at a time, and lanes with the
// same block find one another by a warp match, so no order of atomics enters:
// count; then one CTA for each selection head turns counts into places and
// writes items; then the same walk again writes the entries.  A block that a
// query names twice counts once, and one that it cannot see, or that does not
// exist, does not count.
#include <algorithm>

#include "sel_common.cuh"

namespace skl {

namespace {

constexpr int kPlanWarps = 4;
constexpr int kScanThreads = 1024;

// Walks the slots of a chunk's queries.  counters: of this warp, by block.
// kFill: counters hold where the chunk's next entry of each block goes.
template <bool kFill>
__device__ __forceinline__ void walk(const SelPlan& p, int sel, int q0, int q1, unsigned* counters) {
  const int lane = threadIdx.x & 31;
  const int b = sel / p.HS;
  const int off = p.NK - p.NQ;
  const int prefix = p.prefix != nullptr ? p.prefix[b] : 0;
  const int* sel_rows = p.selected + size_t(sel) * p.NQ * p.T;
  const int* ids = p.doc_q != nullptr ? p.doc_q + size_t(b) * p.NQ : nullptr;
  unsigned* entries = p.entries + size_t(sel) * p.NQ * p.T;
  unsigned* slots = p.slots + size_t(sel) * p.NQ * p.words;
  int span = 1;  // lanes of a query: a power of two
  while (span < p.T && span < 32) span *= 2;
  const int per = 32 / span, q = lane / span, t0 = lane - q * span;
  const unsigned own = span == 32 ? 0xffffffffu : ((1u << span) - 1u) << (q * span);
  // what follows for 32 slots: j, or -1 where a slot does not count
  auto step = [&](int i, int j, bool on, int w, int t) {
    const unsigned same = __match_any_sync(0xffffffffu, on ? j : -2 - lane);
    const unsigned lower = same & ((1u << lane) - 1u);
    on = on && (lower & own) == 0u;
    const unsigned all = __ballot_sync(0xffffffffu, on);
    if (!kFill && t0 == 0 && i < q1) slots[size_t(i) * p.words + w] = (all & own) >> (q * span);
    const unsigned mine = same & all;  // (of a lane that counts)
    const unsigned at = on ? counters[j] : 0u;
    __syncwarp();
    if (on) {
      if ((mine & ((1u << lane) - 1u)) == 0u) counters[j] = at + __popc(mine);
      if (kFill) entries[at + __popc(lower & all)] = (unsigned(i) << kSlotBits) | unsigned(t);
    }
    __syncwarp();
  };
  auto counts = [&](int i, int j) {
    return j >= 0 && j < p.blocks && (!p.causal || j * p.bs <= i + off || j * p.bs < prefix);
  };
  if (p.words == 1) {
    constexpr int kAhead = 8;  // loads in flight
    for (int i0 = q0; i0 < q1; i0 += kAhead * per) {
      int j[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int i = i0 + s * per + q;
        const bool row = i < q1 && t0 < p.T && (ids == nullptr || ids[i] >= 0);
        j[s] = row ? sel_rows[size_t(i) * p.T + t0] : -1;
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int i = i0 + s * per + q;
        if (i0 + s * per < q1) step(i, j[s], counts(i, j[s]), 0, t0);
      }
    }
    return;
  }
  for (int i = q0; i < q1; ++i) {
    const bool row = ids == nullptr || ids[i] >= 0;
    int before[kMaxSlots / 32];
#pragma unroll
    for (int w = 0; w < kMaxSlots / 32; ++w) {
      if (w >= p.words) break;
      const int t = 32 * w + t0;
      const int j = row && t < p.T ? sel_rows[size_t(i) * p.T + t] : -1;
      bool on = counts(i, j);
      before[w] = on ? j : -1;
#pragma unroll
      for (int v = 0; v < w; ++v)  // named in the words before?
        for (int s = 0; s < 32; ++s)
          if (__shfl_sync(0xffffffffu, before[v], s) == j) on = false;
      step(i, j, on, w, t);
    }
  }
}

template <bool kFill>
__global__ void __launch_bounds__(32 * kPlanWarps) sel_walk_kernel(const __grid_constant__ SelPlan p) {
  extern __shared__ unsigned shared_counters[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sel = blockIdx.y, c = blockIdx.x * kPlanWarps + warp;
  if (!kFill && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.item_count = 0;
  if (c >= p.chunks) return;
  unsigned* counters = shared_counters + warp * p.blocks;
  unsigned* mine = p.counts + (size_t(sel) * p.chunks + c) * p.blocks;
  for (int j = lane; j < p.blocks; j += 32) counters[j] = kFill ? mine[j] : 0u;
  __syncwarp();
  walk<kFill>(p, sel, c * p.chunk, min(p.NQ, (c + 1) * p.chunk), counters);
  if (!kFill)
    for (int j = lane; j < p.blocks; j += 32) mine[j] = counters[j];
}

// Exclusive sums over the CTA's threads of two values; the totals in sum_a, sum_b.
__device__ __forceinline__ void scan2(unsigned a, unsigned b, unsigned& before_a, unsigned& before_b, unsigned& sum_a,
                                      unsigned& sum_b) {
  __shared__ uint2 part[kScanThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const unsigned u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  if (lane == 31) part[warp] = make_uint2(x, y);
  __syncthreads();
  if (warp == 0) {
    uint2 s = lane < kScanThreads / 32 ? part[lane] : make_uint2(0, 0);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned u = __shfl_up_sync(0xffffffffu, s.x, o), v = __shfl_up_sync(0xffffffffu, s.y, o);
      if (lane >= o) s.x += u, s.y += v;
    }
    if (lane < kScanThreads / 32) part[lane] = s;
  }
  __syncthreads();
  const uint2 up = warp > 0 ? part[warp - 1] : make_uint2(0, 0), all = part[kScanThreads / 32 - 1];
  before_a = up.x + x - a;
  before_b = up.y + y - b;
  sum_a = all.x;
  sum_b = all.y;
  __syncthreads();
}

__global__ void __launch_bounds__(kScanThreads) sel_scan_kernel(const __grid_constant__ SelPlan p) {
  __shared__ int region;
  const int sel = blockIdx.x;
  unsigned* counts = p.counts + size_t(sel) * p.chunks * p.blocks;
  const unsigned per_item = unsigned(p.queries_per_tile) * p.tiles_per_item;
  // items in all first: they are one stretch of the table
  unsigned total_items = 0;
  constexpr int kRounds = kMaxSelBlocks / kScanThreads;
  unsigned n[kRounds], entry[kRounds], item[kRounds];
  unsigned entries_before = 0;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (r * kScanThreads >= p.blocks) break;
    const int j = r * kScanThreads + threadIdx.x;
    n[r] = 0;
    if (j < p.blocks)
#pragma unroll 8
      for (int c = 0; c < p.chunks; ++c) n[r] += counts[size_t(c) * p.blocks + j];
    unsigned be, bi, se, si;
    scan2(n[r], (n[r] + per_item - 1) / per_item, be, bi, se, si);
    entry[r] = entries_before + be;
    item[r] = total_items + bi;
    entries_before += se;
    total_items += si;
  }
  if (threadIdx.x == 0) region = atomicAdd(p.item_count, int(total_items));
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int j = r * kScanThreads + threadIdx.x;
    if (j >= p.blocks) break;
    unsigned at = entry[r];
#pragma unroll 8
    for (int c = 0; c < p.chunks; ++c) {
      const unsigned k = counts[size_t(c) * p.blocks + j];
      counts[size_t(c) * p.blocks + j] = at;
      at += k;
    }
    if (p.ranges != nullptr)
      p.ranges[size_t(sel) * p.blocks + j] = make_int2(region + int(item[r]), int((n[r] + per_item - 1) / per_item));
    const unsigned base = unsigned(sel) * unsigned(p.NQ) * p.T + entry[r];
    for (unsigned k = 0; k * per_item < n[r]; ++k) {
      const int place = region + int(item[r] + k);
      if (place < p.max_items)
        p.items[place] = SelItem{sel, j, int(base + k * per_item), int(min(per_item, n[r] - k * per_item))};
    }
  }
}

}  // namespace

int launch_sel_plan(const SelPlan& p, cudaStream_t st) {
  const dim3 grid(unsigned((p.chunks + kPlanWarps - 1) / kPlanWarps), unsigned(p.B * p.HS));
  const int smem = kPlanWarps * p.blocks * int(sizeof(unsigned));
  for (auto kern : {sel_walk_kernel<false>, sel_walk_kernel<true>}) {
    // (always the most: threads that launch at once would set each other's size)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kPlanWarps * kMaxSelBlocks * int(sizeof(unsigned)));
    if (e != cudaSuccess) return e;
  }
  sel_walk_kernel<false><<<grid, 32 * kPlanWarps, smem, st>>>(p);
  sel_scan_kernel<<<p.B * p.HS, kScanThreads, 0, st>>>(p);
  sel_walk_kernel<true><<<grid, 32 * kPlanWarps, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace skl
