// Attention over selected blocks of keys: what the plan, the forward and the
// backward share.
//
// Every query has up to T blocks of its own, so a tile of consecutive queries
// shares no keys.  The work is turned round: for each block of keys, the
// queries that selected it, 128 rows (queries x the heads that share keys) at
// a time, their rows gathered.  K is then read once for a list of rows
// and every product is a full 128-row tile.  The attention KL's share of a
// (row, block) is five numbers, so what is written between the passes stays
// small; an output of d values a row would not allow this.
//
// The plan (sel_plan.cu) makes these lists, in query order.  All lists' tiles in
// a row are cut into as many parts of equal cost as there are CTAs, whatever
// block a cut falls into; several selection heads at a time, as many as L2 holds the rows
// of.  Nothing in the plan depends on the order in which blocks of a launch run.
#pragma once

#include "bwd_common.cuh"
#include "kernels.cuh"
#include "mod_common.cuh"
#include "ptx.cuh"

namespace skl {

constexpr int kMaxSlots = 128;    // blocks of one query
constexpr int kMaxSelBlocks = 4096;
constexpr int kSlotBits = 7;
constexpr int kPlanShared = 160 * 1024;  // counters of a plan made by one kernel

struct SelPlan {
  int B, H, NQ, NK, HS, T;
  int bs, blocks;        // keys of a block, blocks of a batch entry
  int G;                 // query heads of a tile, which share keys and selection
  int HU;                // units of G heads in a batch entry; HU / HS use the same lists
  int queries_per_tile;  // 128 / G
  int causal;
  const int* prefix;     // [B] or null
  const int* doc_q;      // [B][NQ] or null
  const int* selected;   // [B][HS][NQ][T]
  int chunk, chunks;     // queries whose entries one warp counts, and their number
  unsigned* counts;      // [B HS][chunks][blocks]: entries of a chunk; then where they start (null: made by one kernel)
  unsigned* entries;     // [B HS][NQ T]: query << kSlotBits | slot
  unsigned* slots;       // [B HS][NQ][words]: the slots that count
  int words;             // (T + 31) / 32
  // Lists that are not empty, of every selection head in block order:
  // block, first entry (of all), entries, tiles before it.  `cap` places a head.
  int4* lists;           // [B HS][cap]
  int cap;
  int2* sizes;           // [B HS]: lists, tiles
  int* place;            // [B HS][blocks]: a block's list, or -1 (null: not needed)
  int group, groups;     // selection heads at a time, and how many times
  int ctas;
};

// Where a group's tiles are cut.  What a list takes counts as a tile more than
// it has (its K, its start in the pipeline, its dK): CTA c begins at the tile of
// cost c total / ctas.
__device__ __forceinline__ long long sel_cost(const SelPlan& p, int s) {  // of a selection head's lists, all units
  const int2 n = __ldg(p.sizes + s);
  return (long long)(n.x + n.y) * (p.HU / p.HS);
}
// Sum over a group's heads before `s`, and over all of them.  By a whole warp.
__device__ __forceinline__ long long group_cost(const SelPlan& p, int g, int s, long long& total) {
  const int s0 = g * p.group, s1 = min(p.B * p.HS, s0 + p.group), lane = threadIdx.x & 31;
  long long all = 0, before = 0;
  for (int k = s0 + lane; k < s1; k += 32) {
    const long long x = sel_cost(p, k);
    all += x;
    if (k < s) before += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total = all;
  return before;
}
// (as many parts as there are CTAs, or less where that leaves nothing for one)
__device__ __forceinline__ long long sel_parts(const SelPlan& p, long long total) { return min((long long)p.ctas, total); }
struct SelCut {
  int s, sub, i, t;  // selection head, unit of it, list, its tile
};
// The tile at cost `at` of a group (below its total).  By a whole warp: 32
// places of the table at a time.
__device__ __forceinline__ SelCut find_cut(const SelPlan& p, int g, long long at) {
  const int lane = threadIdx.x & 31, per = p.HU / p.HS, s1 = min(p.B * p.HS, (g + 1) * p.group);
  SelCut k{g * p.group, 0, 0, 0};
  while (true) {  // the head: 32 at a time
    const long long mine = k.s + lane < s1 ? sel_cost(p, k.s + lane) : 0;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at < sum);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      at -= __shfl_sync(0xffffffffu, sum - mine, l);
      k.s += l;
      break;
    }
    at -= __shfl_sync(0xffffffffu, sum, 31);
    k.s += 32;
  }
  // the last list that starts at or before it
  const int4* lists = p.lists + size_t(k.s) * p.cap;
  int lo = 0, n = __ldg(p.sizes + k.s).x;  // among [lo, lo + n)
  while (n > 1) {
    const int stride = (n + 31) / 32, mid = lo + lane * stride;
    const bool in = lane * stride < n && (long long)(__ldg(lists + min(mid, lo + n - 1)).w + mid) * per <= at;
    const int l = 31 - __clz(__ballot_sync(0xffffffffu, in));  // (lane 0's starts before it)
    n = min(stride, n - l * stride);
    lo += l * stride;
  }
  const int4 l = __ldg(lists + lo);
  const int tiles = (l.z + p.queries_per_tile - 1) / p.queries_per_tile, in = int(at - (long long)(l.w + lo) * per);
  k.i = lo;
  k.sub = in / (tiles + 1);
  k.t = max(in - k.sub * (tiles + 1) - 1, 0);
  return k;
}

// A CTA's shares of lists, in order: `count` entries from `first` on.  What
// comes next is read ahead.  By a whole warp.
struct SelWalk {
  int first, count;
  int g;              // group
  SelCut k, end;      // where it is, and where this CTA's part of the group ends
  int n;              // the head's lists
  int4 cur, next;
  bool on;

  __device__ __forceinline__ explicit SelWalk(const SelPlan& p) : g(-1) { enter(p); }
  __device__ __forceinline__ bool more() const { return on; }
  __device__ __forceinline__ void list(const SelPlan& p, int4 now) {
    cur = now;
    next = k.i + 1 < n ? __ldg(p.lists + size_t(k.s) * p.cap + k.i + 1) : int4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void here(const SelPlan& p) {  // the current list's share
    const bool last = k.s == end.s && k.i == end.i && k.sub == end.sub;
    const int per = p.queries_per_tile, to = last ? end.t * per : cur.z;
    first = cur.y + k.t * per;
    count = min(to, cur.z) - k.t * per;
    on = count > 0;
  }
  __device__ __forceinline__ void enter(const SelPlan& p) {  // the next group's part
    on = false;
    count = first = 0;
    while (!on && ++g < p.groups) {
      long long total;
      group_cost(p, g, 0, total);
      const long long parts = sel_parts(p, total), a = blockIdx.x * total / max(parts, 1ll);
      if (blockIdx.x >= parts) continue;
      const long long b = (blockIdx.x + 1) * total / parts;
      k = find_cut(p, g, a);
      end = b < total ? find_cut(p, g, b) : SelCut{-1, 0, 0, 0};  // (nothing behind the last list)
      n = __ldg(p.sizes + k.s).x;
      list(p, __ldg(p.lists + size_t(k.s) * p.cap + k.i));
      here(p);
    }
  }
  __device__ __forceinline__ void advance(const SelPlan& p) {
    if (k.s == end.s && k.i == end.i && k.sub == end.sub) return enter(p);
    k.t = 0;
    if (++k.sub == p.HU / p.HS) {
      k.sub = 0;
      if (++k.i < n) {
        list(p, next);
      } else {
        k.i = 0;
        const int s1 = min(p.B * p.HS, (g + 1) * p.group);
        do {
          if (++k.s >= s1) return enter(p);
          n = __ldg(p.sizes + k.s).x;
        } while (n == 0);
        list(p, __ldg(p.lists + size_t(k.s) * p.cap));
      }
    }
    here(p);
    if (!on) enter(p);  // (the part ends where this list begins)
  }
  // A number of its own for every (list, CTA) that meet: along the parts one or
  // the other goes up.
  __device__ __forceinline__ long long meeting(const SelPlan& p) const {
    return ((long long)k.s * p.cap + k.i) * (p.HU / p.HS) + k.sub + (long long)g * p.ctas + blockIdx.x;
  }
};

// What the other warps of a CTA are told about a share; count 0: there are no more.
struct alignas(16) SelShare {
  int first, count, b, head0;
  int block, unit;             // unit of the batch entry: head0 / G
  unsigned long long meeting;  // SelWalk::meeting
};
constexpr int kShares = 8;  // told ahead

// One warp walks and tells; the others read every share once, when they come to
// it.  (A walk in every warp cost the statistics their registers: 783 us for
// the forward at 16384 queries x 32 heads, where 479 had been.)  Barriers: full
// [kShares] (1 arrival), then empty [kShares] (one for each reading warp).
__device__ __forceinline__ void tell_shares(const SelPlan& p, SelShare* shares, uint32_t bars, Ctl ctl) {
  SelWalk walk(p);
  for (int q = 0;; ++q) {
    const int at = q % kShares;
    if (!mbar_wait_warp(bars + 8u * (kShares + at), ((q / kShares) & 1) ^ 1, ctl)) return;
    const bool more = walk.more();
    if ((threadIdx.x & 31) == 0) {
      SelShare x{0, 0, 0, 0, 0, 0, 0ull};
      if (more) {
        const int unit = walk.k.s * (p.HU / p.HS) + walk.k.sub;
        x.first = walk.first;
        x.count = walk.count;
        x.b = unit / p.HU;
        x.unit = unit - x.b * p.HU;
        x.head0 = x.unit * p.G;
        x.block = walk.cur.x;
        x.meeting = walk.meeting(p);
      }
      shares[at] = x;
      mbar_arrive(bars + 8u * at);
    }
    if (!more) return;
    walk.advance(p);
  }
}

struct SelReader {
  const SelShare* shares;
  uint32_t bars;
  int q;
  int first, count, b, head0, block;
  unsigned long long meeting;

  __device__ __forceinline__ SelReader(const SelShare* s, uint32_t barriers) : shares(s), bars(barriers), q(0), count(0) {}
  // Called by a whole warp; false at the end (and on an abort).
  __device__ __forceinline__ bool next(Ctl ctl) {
    const int at = q % kShares;
    if (!mbar_wait_warp(bars + 8u * at, (q / kShares) & 1, ctl)) {
      count = 0;
      return false;
    }
    const int4 v = *reinterpret_cast<const int4*>(shares + at);
    first = v.x;
    count = v.y;
    b = v.z;
    head0 = v.w;
    block = shares[at].block;
    meeting = shares[at].meeting;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8u * (kShares + at));
    ++q;
    return count > 0;
  }
};
constexpr unsigned kNoEntry = 0xffffffffu;
// Entry e of the reader's share, for a row with a place in the tile.
__device__ __forceinline__ unsigned entry_of(const SelPlan& p, const SelReader& k, int e, bool place) {
  return place && e < k.count ? __ldg(p.entries + k.first + e) : kNoEntry;
}

// A [B][heads][N][d] bf16 view (strides in bytes).
struct SelRows {
  const uint8_t* base;
  long long sb, sh, sn;
  int chunks;  // 16-byte pieces of a row: d / 8
  __device__ __forceinline__ const uint8_t* at(int b, int h, int i) const { return base + b * sb + h * sh + i * sn; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros with size 0 (nothing is read).
__device__ __forceinline__ void cp_async16_size(uint32_t dst, const void* src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
// This thread's arrival on `bar` once its copies so far have landed.  The one
// that waits for them and hands them to the tensor core puts the proxy fence
// between the two: a fence of each copying warp held up its next copies (763
// us instead of 686, at the time, for 16384 queries x 32 heads).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Step kk of 16 along d of a K-major operand of `rows` rows.
__device__ __forceinline__ uint32_t step_off(int kk, int rows) { return (kk >> 2) * (rows * 128) + (kk & 3) * 32; }

// Slots of a ring that the sides' tiles (D1 and D2 columns) take in turn.  Columns past a head dim are zeros from the
// start on, but with an odd number of slots each holds tiles of both sides, and a side that is narrower than the other
// would find that one's values there: a NaN among them reaches products of rows that have nothing to do with it.  An
// even number keeps a slot with its side.  (Zeros written with each tile instead: the forward of 8192 tokens x 32 heads,
// 16 blocks of 64, took 272 us instead of 262 whatever the head dims; the backward of d 128 and 96 over blocks of 128,
// which is left 2 slots, 437 instead of 513.)
inline int slots_of_sides(int slots, const SelRows& r1, int d1, const SelRows& r2, int d2) {
  const bool mixed = (r1.chunks < d1 / 8 && r2.chunks > r1.chunks) || (r2.chunks < d2 / 8 && r1.chunks > r2.chunks);
  return mixed ? slots / 2 * 2 : slots;
}

// Copies 32 rows (lane r holds the address of row r; 0: not copied, or with
// ZERO zeros) into rows [first, first + 32) of a [128][D] operand tile,
// swizzled as TMA would: 64 bytes of 8 rows at a time, so that all but four
// addresses a lane are constants away, and no branch between them.  Called by
// a whole warp.
template <int D, bool ZERO>
__device__ __forceinline__ void gather_rows(uint32_t tile, int first, unsigned long long mine, const SelRows& rows) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t even = tile + (first + r) * 128 + ((c ^ r) << 4), odd = even ^ 64u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long row = __shfl_sync(0xffffffffu, mine, r + 8 * k);
    const uint8_t* p = (row != 0 ? reinterpret_cast<const uint8_t*>(row) : rows.base) + c * 16;
    const uint32_t size = row != 0 ? 16u : 0u;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint32_t to = (j & 1 ? odd : even) + k * 1024 + (j >> 1) * (kTile * 128);
      if (c + 4 * j < rows.chunks) {
        if (ZERO) cp_async16_size(to, p + 64 * j, size);
        else if (row != 0) cp_async16(to, p + 64 * j);
      }
    }
  }
}

// D (+)= A B^T for `steps` of 16 along the contraction: operand descriptors by
// their low words, which alone change (the address is their low 14 bits).
__device__ __forceinline__ void mma_step(uint32_t leader, uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, q;\n\t}" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

struct SelMaps {
  CUtensorMap k1, k2;  // 4-D (d, N, heads, B), boxes of 64 x block, 128-byte swizzle
};

struct SelFwdArgs {
  SelPlan p;
  SelRows r1, r2;
  int u1, u2;             // units per key head of each side
  float scale1, scale2;
  ModVis vis;
  float4* rec;            // [B H NQ][T]: m1, m2, l1, l2 of a row's keys in one block
  float* acc;             // [B H NQ][T]
  float* kl;
  float* lse1;
  float* lse2;
  int* status;
  int slots, k_bufs;
};

struct SelBwdArgs {
  SelPlan p;
  SelRows r1, r2;
  int u1, u2;
  float scale1, scale2;
  ModVis vis;
  const float* kl;
  const float* lse1;
  const float* lse2;
  const float* dkl;
  int dg, pitch;          // head dim of the gradient side; row length of dq32
  float* dq32;            // [B H NQ][pitch], zeroed: dQ contributions, on their rows' grids
  float* dk_part;         // [meetings][bs][dg]: a CTA's dK of a list
  unsigned* kmax;         // per key head of the gradient side, zeroed: max |K|, as bf16 bits
  void* dk;               // bf16 [B][HK][NK][dg]
  long long dk_sb, dk_sh, dk_sn;
  int HK;                 // of the gradient side
  int* status;
  float4* rows;           // [B H NQ], of row_params
  int mode;
  const void* k;          // K of the gradient side
  long long k_sb, k_sh, k_sn;
  const int* doc_k;
  int slots, k_bufs;
};

// What dS and dQ need of a row: na, nb, ws as in the dense kernels, and the
// exponent of its grid.  A row that saw nothing has na = -inf.
__device__ __forceinline__ void row_params(const SelBwdArgs& a, long long row) {
  if (row >= (long long)a.p.B * a.p.H * a.p.NQ) return;
  const bool p2 = a.mode == STREAMKL_GRAD_P2;
  const float l1 = a.lse1[row], l2 = a.lse2[row], kl = a.kl[row], dkl = a.dkl[row], sg = p2 ? a.scale2 : a.scale1;
  float4 par{-INFINITY, p2 ? -INFINITY : 0.f, 0.f, 0.f};
  if (l1 != -INFINITY) {
    const int bh = int(row / a.p.NQ), b = bh / a.p.H, h = bh - b * a.p.H;
    const float kmax = __uint_as_float(__ldcg(a.kmax + b * a.HK + h / (a.p.H / a.HK)) << 16);
    par.x = -l1 * kLog2e;
    par.y = p2 ? -l2 * kLog2e : -(l1 - l2 + kl);
    par.z = sg * dkl;
    par.w = float(dq_fixed_exp(a.mode, sg, dkl, kl, kmax));
  }
  a.rows[row] = par;
}

// The plan; of a backward (else null) max |K| and the rows' parameters too.
int launch_sel_plan(const SelPlan& p, const SelBwdArgs* bwd, cudaStream_t st);
int launch_sel_bwd(const SelMaps& m, int d1, int d2, const SelBwdArgs& a, cudaStream_t st);
// dK from its shares, and dq32 to bf16
int launch_sel_finish(const SelBwdArgs& a, const ModFinishArgs::Rows& dq, cudaStream_t st);
int launch_sel_fwd(const SelMaps& m, int d1, int d2, const SelFwdArgs& a, cudaStream_t st);
int launch_sel_merge(const SelFwdArgs& a, cudaStream_t st);

}  // namespace skl
