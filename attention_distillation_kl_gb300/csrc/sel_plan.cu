// The plan of attention over selected blocks (sel_common.cuh): for each block
// the queries that selected it, in order, and each CTA's part of these lists.
//
// A warp owns a chunk of queries and the blocks' counters of that chunk, in
// shared memory; it takes 32 slots at a time, and lanes with the same block find
// one another by a warp match, so no order of atomics enters: count; then one
// CTA for each selection head turns counts into places and lists; then the same
// walk again writes the entries.  With few queries one CTA does all three, its
// warps' counters in shared memory throughout.  A block that a query names twice
// counts once, and one that it cannot see, or that does not exist, does not
// count.
#include <algorithm>

#include "sel_common.cuh"

namespace skl {

namespace {

constexpr int kPlanWarps = 4;
constexpr int kScanThreads = 1024;
constexpr int kRowThreads = 256;

// Walks the slots of a chunk's queries.  counters: of this warp, by block.
// kFill: counters hold where the chunk's next entry of each block goes.  kWide:
// there may be more than 32 slots.
template <bool kFill, bool kWide>
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
  if (!kWide || p.words == 1) {
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
  if constexpr (kWide) {
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
}

// CTAs of a plan's launches that a backward has beside the plan: with what
// counts, those for max |K| of each key head; with what fills, those for the
// rows' parameters.
struct Beside {
  int plan;   // CTAs of the plan itself
  int each;   // a head's CTAs for max |K|
};

__device__ __forceinline__ void kmax_beside(const SelBwdArgs& a, const Beside& by) {
  const int x = blockIdx.x - by.plan, head = x / by.each, b = head / a.HK;
  kmax_share(static_cast<const __nv_bfloat16*>(a.k) + b * a.k_sb + (head - b * a.HK) * a.k_sh, a.p.NK, a.dg, a.k_sn,
             a.doc_k != nullptr ? a.doc_k + size_t(b) * a.p.NK : nullptr, x - head * by.each, by.each, a.kmax + head);
}

template <bool kFill>
__global__ void __launch_bounds__(32 * kPlanWarps)
    sel_walk_kernel(const __grid_constant__ SelPlan p, const __grid_constant__ SelBwdArgs bwd, const __grid_constant__ Beside by) {
  extern __shared__ unsigned shared_counters[];
  if (blockIdx.x >= by.plan) {
    if (kFill)
      row_params(bwd, (long long)(blockIdx.x - by.plan) * blockDim.x + threadIdx.x);
    else
      kmax_beside(bwd, by);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int walkers = (p.chunks + kPlanWarps - 1) / kPlanWarps;
  const int sel = blockIdx.x / walkers, c = (blockIdx.x - sel * walkers) * kPlanWarps + warp;
  if (c >= p.chunks) return;
  unsigned* counters = shared_counters + warp * p.blocks;
  unsigned* mine = p.counts + (size_t(sel) * p.chunks + c) * p.blocks;
  for (int j = lane; j < p.blocks; j += 32) counters[j] = kFill ? mine[j] : 0u;
  __syncwarp();
  walk<kFill, true>(p, sel, c * p.chunk, min(p.NQ, (c + 1) * p.chunk), counters);
  if (!kFill)
    for (int j = lane; j < p.blocks; j += 32) mine[j] = counters[j];
}

// Exclusive sums over the CTA's threads of three values (and of all in `sum`).
__device__ __forceinline__ uint3 scan3(uint3 v, uint3& sum) {
  __shared__ uint3 part[kScanThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto up = [&](uint3& x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o),
                     c = __shfl_up_sync(0xffffffffu, x.z, o);
      if (lane >= o) x.x += a, x.y += b, x.z += c;
    }
  };
  uint3 x = v;
  up(x);
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint3 s = part[lane];
    up(s);
    part[lane] = s;
  }
  __syncthreads();
  static_assert(kScanThreads == 1024, "a warp sums the warps");
  const uint3 before = warp > 0 ? part[warp - 1] : make_uint3(0, 0, 0);
  sum = part[kScanThreads / 32 - 1];
  __syncthreads();
  return make_uint3(before.x + x.x - v.x, before.y + x.y - v.y, before.z + x.z - v.z);
}

// A block's chunks are shared by as many threads as there are for it: `parts`,
// a power of two, neighbours of a block in threads `width` apart.
__global__ void __launch_bounds__(kScanThreads) sel_scan_kernel(const __grid_constant__ SelPlan p) {
  __shared__ unsigned share[kScanThreads];
  const int sel = blockIdx.x;
  unsigned* counts = p.counts + size_t(sel) * p.chunks * p.blocks;
  const unsigned per = p.queries_per_tile, base = unsigned(sel) * unsigned(p.NQ) * p.T;
  int width = 32;
  while (width < p.blocks && width < kScanThreads) width *= 2;
  const int parts = kScanThreads / width, part = threadIdx.x / width, len = (p.chunks + parts - 1) / parts;
  const int c0 = min(p.chunks, part * len), c1 = min(p.chunks, c0 + len);
  uint3 before{0, 0, 0};  // entries, lists, tiles
  for (int j0 = 0; j0 < p.blocks; j0 += width) {
    const int j = j0 + (threadIdx.x & (width - 1));
    unsigned mine = 0;
    if (j < p.blocks)
#pragma unroll 16
      for (int c = c0; c < c1; ++c) mine += counts[size_t(c) * p.blocks + j];
    share[threadIdx.x] = mine;
    __syncthreads();
    unsigned n = 0, to = 0;  // of the block; of the parts before this one
    for (int x = 0; x < parts; ++x) {
      const unsigned k = share[x * width + (threadIdx.x & (width - 1))];
      if (x < part) to += k;
      n += k;
    }
    const bool first = part == 0 && j < p.blocks;
    uint3 sum;
    uint3 at = scan3(first ? make_uint3(n, n != 0u ? 1u : 0u, (n + per - 1) / per) : make_uint3(0, 0, 0), sum);
    at = make_uint3(at.x + before.x, at.y + before.y, at.z + before.z);
    before = make_uint3(before.x + sum.x, before.y + sum.y, before.z + sum.z);
    if (part == 0) share[threadIdx.x] = at.x;
    __syncthreads();
    to += share[threadIdx.x & (width - 1)];
    if (first) {
      if (n != 0u) p.lists[size_t(sel) * p.cap + at.y] = make_int4(j, int(base + at.x), int(n), int(at.z));
      if (p.place != nullptr) p.place[size_t(sel) * p.blocks + j] = n != 0u ? int(at.y) : -1;
    }
    if (j < p.blocks)
#pragma unroll 16
      for (int c = c0; c < c1; ++c) {
        const unsigned k = counts[size_t(c) * p.blocks + j];
        counts[size_t(c) * p.blocks + j] = to;
        to += k;
      }
    __syncthreads();
  }
  if (threadIdx.x == 0) p.sizes[sel] = make_int2(int(before.y), int(before.z));
}

// All of it for one selection head, of up to 32 slots: `chunks` warps (32 at most) with a chunk each.
__global__ void __launch_bounds__(kScanThreads)
    sel_plan_kernel(const __grid_constant__ SelPlan p, const __grid_constant__ SelBwdArgs bwd, const __grid_constant__ Beside by) {
  extern __shared__ unsigned counters[];  // [chunks][blocks]
  if (blockIdx.x >= by.plan) {
    kmax_beside(bwd, by);
    return;
  }
  const int sel = blockIdx.x, warp = threadIdx.x >> 5;
  const unsigned per = p.queries_per_tile, base = unsigned(sel) * unsigned(p.NQ) * p.T;
  for (int x = threadIdx.x; x < p.chunks * p.blocks; x += kScanThreads) counters[x] = 0u;
  __syncthreads();
  if (warp < p.chunks) walk<false, false>(p, sel, warp * p.chunk, min(p.NQ, (warp + 1) * p.chunk), counters + warp * p.blocks);
  __syncthreads();
  uint3 before{0, 0, 0};  // entries, lists, tiles
  for (int j0 = 0; j0 < p.blocks; j0 += kScanThreads) {
    const int j = j0 + threadIdx.x;
    unsigned n = 0;
    if (j < p.blocks)
      for (int c = 0; c < p.chunks; ++c) n += counters[c * p.blocks + j];
    uint3 sum;
    uint3 at = scan3(make_uint3(n, n != 0u ? 1u : 0u, (n + per - 1) / per), sum);
    at = make_uint3(at.x + before.x, at.y + before.y, at.z + before.z);
    before = make_uint3(before.x + sum.x, before.y + sum.y, before.z + sum.z);
    if (j >= p.blocks) continue;
    if (n != 0u) p.lists[size_t(sel) * p.cap + at.y] = make_int4(j, int(base + at.x), int(n), int(at.z));
    if (p.place != nullptr) p.place[size_t(sel) * p.blocks + j] = n != 0u ? int(at.y) : -1;
    unsigned to = at.x;
    for (int c = 0; c < p.chunks; ++c) {
      const unsigned k = counters[c * p.blocks + j];
      counters[c * p.blocks + j] = to;
      to += k;
    }
  }
  if (threadIdx.x == 0) p.sizes[sel] = make_int2(int(before.y), int(before.z));
  __syncthreads();
  if (warp < p.chunks) walk<true, false>(p, sel, warp * p.chunk, min(p.NQ, (warp + 1) * p.chunk), counters + warp * p.blocks);
}

__global__ void __launch_bounds__(kRowThreads) sel_rows_kernel(const __grid_constant__ SelBwdArgs a) {
  row_params(a, (long long)blockIdx.x * kRowThreads + threadIdx.x);
}

}  // namespace

int launch_sel_plan(const SelPlan& p, const SelBwdArgs* bwd, cudaStream_t st) {
  static const SelBwdArgs kNone{};
  const SelBwdArgs& a = bwd != nullptr ? *bwd : kNone;
  const long long rows = bwd != nullptr ? (long long)p.B * p.H * p.NQ : 0;
  // CTAs of so many threads for max |K|, and so many heads' worth of them
  auto beside = [&](unsigned plan, int threads) {
    const long long blocks = loop_blocks((long long)p.NK * (a.dg / 8)) * 256ll / threads;
    return Beside{int(plan), bwd != nullptr ? int(std::max(1ll, blocks / (p.B * a.HK))) : 0};
  };
  // (always the most shared memory: threads that launch at once would set each other's size)
  if (p.counts == nullptr) {
    const cudaError_t e = cudaFuncSetAttribute(sel_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanShared);
    if (e != cudaSuccess) return e;
    const Beside by = beside(p.B * p.HS, kScanThreads);
    sel_plan_kernel<<<by.plan + p.B * a.HK * by.each, kScanThreads, p.chunks * p.blocks * int(sizeof(unsigned)), st>>>(p, a, by);
    if (rows > 0) sel_rows_kernel<<<unsigned((rows + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const unsigned walkers = unsigned((p.chunks + kPlanWarps - 1) / kPlanWarps * p.B * p.HS);
  const int smem = kPlanWarps * p.blocks * int(sizeof(unsigned));
  for (auto kern : {sel_walk_kernel<false>, sel_walk_kernel<true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kPlanWarps * kMaxSelBlocks * int(sizeof(unsigned)));
    if (e != cudaSuccess) return e;
  }
  constexpr int kThreads = 32 * kPlanWarps;
  const Beside by = beside(walkers, kThreads);
  sel_walk_kernel<false><<<walkers + unsigned(p.B * a.HK * by.each), kThreads, smem, st>>>(p, a, by);
  sel_scan_kernel<<<p.B * p.HS, kScanThreads, 0, st>>>(p);
  sel_walk_kernel<true><<<walkers + unsigned((rows + kThreads - 1) / kThreads), kThreads, smem, st>>>(p, a, by);
  return cudaGetLastError();
}

}  // namespace skl
