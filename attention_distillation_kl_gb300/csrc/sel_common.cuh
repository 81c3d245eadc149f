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
  unsigned* counts;      // [B HS][chunks][blocks]: entries of a chunk; then where they start
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
  int4* starts;          // [groups][ctas]: (selection head, unit), list, its tile, tiles of the part
};

// A CTA's shares of lists, in order: `count` entries from `first` on.  What
// comes next is read ahead.
struct SelWalk {
  int first, count;
  int g, left;        // group, tiles of the part from the current list on
  int s, sub, i, n;   // selection head, unit of it, list, the head's lists
  int tile, tiles;    // the current list's first tile and number of tiles here
  int4 cur, next, start;

  __device__ __forceinline__ explicit SelWalk(const SelPlan& p) : g(-1) {
    start = part(p, 0);
    enter(p);
  }
  __device__ __forceinline__ int4 part(const SelPlan& p, int at) const {
    return at < p.groups ? __ldg(p.starts + size_t(at) * p.ctas + blockIdx.x) : int4{0, 0, 0, 0};
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void list(const SelPlan& p, int4 now) {
    cur = now;
    next = i + 1 < n ? __ldg(p.lists + size_t(s) * p.cap + i + 1) : int4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void here(const SelPlan& p) {  // the current list's share
    const int per = p.queries_per_tile;
    tiles = min((cur.z + per - 1) / per - tile, left);
    first = cur.y + tile * per;
    count = min(cur.z - tile * per, tiles * per);
  }
  __device__ __forceinline__ void enter(const SelPlan& p) {  // the next group's part
    left = 0;
    count = first = tiles = tile = 0;
    while (left == 0 && ++g < p.groups) {
      const int4 v = start;
      start = part(p, g + 1);
      left = v.w;
      if (left == 0) continue;
      const int per = p.HU / p.HS;
      s = v.x / per;
      sub = v.x - s * per;
      i = v.y;
      tile = v.z;
      n = __ldg(p.sizes + s).x;
      list(p, __ldg(p.lists + size_t(s) * p.cap + i));
      here(p);
    }
  }
  __device__ __forceinline__ void advance(const SelPlan& p) {
    left -= tiles;
    if (left <= 0) return enter(p);
    tile = 0;
    if (++sub == p.HU / p.HS) {
      sub = 0;
      if (++i < n) {
        list(p, next);
      } else {
        i = 0;
        do n = __ldg(p.sizes + ++s).x;  // (tiles are left, so lists are)
        while (n == 0);
        list(p, __ldg(p.lists + size_t(s) * p.cap));
      }
    }
    here(p);
  }
  // A number of its own for every (list, CTA) that meet: along the parts one or
  // the other goes up.
  __device__ __forceinline__ long long meeting(const SelPlan& p) const {
    return ((long long)s * p.cap + i) * (p.HU / p.HS) + sub + (long long)g * p.ctas + blockIdx.x;
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
    if (!mbar_wait_polled(bars + 8u * (kShares + at), ((q / kShares) & 1) ^ 1, ctl)) return;
    SelShare x{0, 0, 0, 0, 0, 0, 0ull};
    const bool more = walk.more();
    if (more) {
      const int unit = walk.s * (p.HU / p.HS) + walk.sub;
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
// between the two: a fence of each copying warp held up its next copies (731
// us instead of @@ for the forward at 16384 queries x 32 heads).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Step kk of 16 along d of a K-major operand of `rows` rows.
__device__ __forceinline__ uint32_t step_off(int kk, int rows) { return (kk >> 2) * (rows * 128) + (kk & 3) * 32; }

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
  const unsigned* kmax;   // per key head of the gradient side (launch_kmax_strided)
  void* dk;               // bf16 [B][HK][NK][dg]
  long long dk_sb, dk_sh, dk_sn;
  int HK;                 // of the gradient side
  int* status;
  float4* rows;           // [B H NQ], of sel_rows_kernel
  int slots, k_bufs;
};

int launch_sel_bwd(const SelMaps& m, int d1, int d2, int mode, const SelBwdArgs& a, cudaStream_t st);
int launch_sel_dk(const SelBwdArgs& a, cudaStream_t st);
int launch_sel_plan(const SelPlan& p, cudaStream_t st);
int launch_sel_fwd(const SelMaps& m, int d1, int d2, const SelFwdArgs& a, cudaStream_t st);
int launch_sel_merge(const SelFwdArgs& a, cudaStream_t st);

}  // namespace skl
