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
// The plan (sel_plan.cu) makes these lists, in query order, and cuts them into
// items of at most tiles_per_item tiles.  Nothing in it depends on the order
// in which blocks of a launch run but the items' places in their table.
#pragma once

#include "bwd_common.cuh"
#include "kernels.cuh"
#include "mod_common.cuh"
#include "ptx.cuh"

namespace skl {

constexpr int kMaxSlots = 128;    // blocks of one query
constexpr int kMaxSelBlocks = 4096;
constexpr int kSlotBits = 7;

// A piece of one block's list: `count` queries from entries[first].
struct SelItem {
  int sel;    // b * HS + selection head
  int block;
  int first;  // of all entries
  int count;
};

struct SelPlan {
  int B, H, NQ, NK, HS, T;
  int bs, blocks;        // keys of a block, blocks of a batch entry
  int G;                 // query heads of a tile, which share keys and selection
  int HU;                // units of G heads in a batch entry; HU / HS use the same lists
  int queries_per_tile;  // 128 / G
  int tiles_per_item;
  int causal;
  const int* prefix;     // [B] or null
  const int* doc_q;      // [B][NQ] or null
  const int* selected;   // [B][HS][NQ][T]
  int chunk, chunks;     // queries whose entries one warp counts, and their number
  unsigned* counts;      // [B HS][chunks][blocks]: entries of a chunk; then where they start
  unsigned* entries;     // [B HS][NQ T]: query << kSlotBits | slot
  unsigned* slots;       // [B HS][NQ][words]: the slots that count
  int words;             // (T + 31) / 32
  SelItem* items;
  int* item_count;       // device
  int2* ranges;          // [B HS][blocks]: a block's first item and their number, or null
  int max_items;
};

// What an item is about.
struct SelWork {
  int b, head0, block, unit;
};

// A CTA's items, in order, every role for itself: works blockIdx.x,
// blockIdx.x + gridDim.x, ...; the one behind the current one is read ahead.
// (Read where they are used, items and entries put two trips to memory into
// every tile's chain: 731 us instead of what the copies allow.)
struct SelWalk {
  int w, works, first, count;  // entries of the current item
  int4 raw, next;

  __device__ __forceinline__ SelWalk(const SelPlan& p, int all) : w(blockIdx.x), works(all) {
    raw = read(p, w);
    next = read(p, w + gridDim.x);
    first = raw.z;
    count = raw.w;
  }
  __device__ __forceinline__ int4 read(const SelPlan& p, int at) const {
    return at < works ? __ldg(reinterpret_cast<const int4*>(p.items) + at / (p.HU / p.HS)) : int4{0, 0, 0, 0};
  }
  __device__ __forceinline__ bool more() const { return w < works; }
  __device__ __forceinline__ void advance(const SelPlan& p) {
    w += gridDim.x;
    raw = next;
    next = read(p, w + gridDim.x);
    first = raw.z;
    count = raw.w;
  }
  __device__ __forceinline__ SelWork get(const SelPlan& p) const {
    const int per = p.HU / p.HS;
    SelWork k;
    k.unit = raw.x * per + w % per;  // b * HU + unit of the batch entry
    k.b = k.unit / p.HU;
    k.head0 = (k.unit - k.b * p.HU) * p.G;
    k.block = raw.y;
    return k;
  }
};
constexpr unsigned kNoEntry = 0xffffffffu;
// Entry e of the walk's item, for a row with a place in the tile.
__device__ __forceinline__ unsigned entry_of(const SelPlan& p, const SelWalk& k, int e, bool place) {
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
  float* dk_part;         // [works][bs][dg]: dK of an item
  const unsigned* kmax;   // per key head of the gradient side (launch_kmax_strided)
  void* dk;               // bf16 [B][HK][NK][dg]
  long long dk_sb, dk_sh, dk_sn;
  int HK;                 // of the gradient side
  int* status;
  float4* rows;           // [B H NQ], of sel_rows_kernel
  int slots, k_bufs;
};

int launch_sel_bwd(const SelMaps& m, int d1, int d2, int mode, const SelBwdArgs& a, int sms, cudaStream_t st);
int launch_sel_dk(const SelBwdArgs& a, cudaStream_t st);
int launch_sel_plan(const SelPlan& p, cudaStream_t st);
int launch_sel_fwd(const SelMaps& m, int d1, int d2, const SelFwdArgs& a, int sms, cudaStream_t st);
int launch_sel_merge(const SelFwdArgs& a, cudaStream_t st);

}  // namespace skl
