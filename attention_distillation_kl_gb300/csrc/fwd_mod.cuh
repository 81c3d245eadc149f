// Forward over modified scores (see mod_common.cuh): KL, LSE1, LSE2 per query
// row in one pass over the visible key tiles, and the merge of key splits.
//
// The pipeline is the plain forward's (fwd_kernel.cuh): one CTA per 128-row
// query tile; a TMA warp streams K1_j, K2_j through a ring; the MMA warp
// multiplies S1 = Q1 K1_j^T and S2 = Q2 K2_j^T into one of two TMEM buffers;
// 16 statistics warps (thread = row, warpgroup w = columns [32 w, 32 w + 32)
// of every tile) turn the products into scores and keep running statistics.
//
// Scores are in base 2 and relative to a reference m_t per row and side:
//   e_t = S_t log2 e - m_t,  l_t = sum 2^e_t,  acc = sum 2^e1 (e1 - e2)
//   LSE_t = ln 2 m_t + ln l_t,  KL = ln 2 acc / l1 + ln(l2 / l1)
// (the references cancel in KL, so nothing of an LSE's size is rounded on the
// way to it).  -m_t is added with the bias, in the operation that finishes
// the score.  Any reference serves as long as no term overflows and the
// largest does not underflow: a row takes the rounded maximum of its first
// visible chunk, and a chunk whose sums reach 2^64 moves it; a chunk of scores
// much smaller than their distance to it is taken again, relative to its own
// maximum.  References are whole numbers, so moving one is exact: by d1, d2,
//   l_t <- l_t 2^-d_t,  acc <- 2^-d1 (acc - (d1 - d2) l1).
// Scores beyond 10^6 (mostly a mask written as a bias) give no usable
// reference: the chunks after them are taken relative to 0.
//
// Key tiles run from the last to the first: a causal row then takes its
// references where a distance bias is largest, and farther tiles only fall
// below them (the other way round, a steep slope moved them at every tile);
// and the diagonal tile is the first, which goes through the general path
// anyway.  With ids, the tiles outside the first and last that share an id
// with the query tile are never loaded, and tiles whose ids are all the same
// take no mask.
#pragma once

#include <climits>

#include "mod_common.cuh"
#include "tiles.cuh"

namespace skl {

namespace {

template <int D1, int D2>
struct ModFwdLayout {
  static_assert(D1 <= 128 && D2 <= 128, "tile widths up to 128");
  static constexpr int kWGs = 4;  // statistics warpgroups, kCols columns of every tile each
  static constexpr int kStatWarps = 4 * kWGs;
  static constexpr int kCols = kTile / kWGs;
  static constexpr int kProdWarp = kStatWarps, kMmaWarp = kStatWarps + 1;
  static constexpr int kThreads = 32 * (kStatWarps + 2);
  static constexpr uint32_t kQ1 = kTile * D1 * 2, kQ2 = kTile * D2 * 2;
  static constexpr uint32_t kK1 = kTile * D1 * 2, kStage = kK1 + kTile * D2 * 2;
  static constexpr int kStagesFit = int((210u * 1024u - kQ1 - kQ2) / kStage);
  static constexpr int kStages = kStagesFit > 4 ? 4 : kStagesFit;
  static constexpr uint32_t oQ1 = 0, oQ2 = kQ1, oK = kQ1 + kQ2;
  static constexpr uint32_t oBar = oK + kStages * kStage;
  // q_full, k_full[S], k_empty[S], s_full[2], s_empty[2], mma_done
  static constexpr int kNumBars = 1 + 2 * kStages + 4 + 1;
  static constexpr uint32_t oMisc = oBar + kNumBars * 8;  // tmem base, abort flag
  static constexpr uint32_t oRange = oMisc + 8;           // first and last key tile with a shared id
  static constexpr uint32_t oBias = (oRange + 8 + 15) / 16 * 16;  // HeadBias of both sides, of up to 8 heads
  static constexpr uint32_t oMerge = oBias + 16 * sizeof(HeadBias);
  static_assert(sizeof(HeadBias) % 16 == 0, "what follows stays aligned");
  static constexpr uint32_t oNear = oMerge + (kWGs - 1) * kTile * 5 * 4;  // lookup rows, where they fit
  static constexpr uint32_t kAlloc = oNear + 1024;
  static_assert(kStages >= 2, "shared memory ring needs two stages");
  static_assert(kCols == 32, "one word of visible bits for each row and tile");
  static_assert(kAlloc <= 232448, "over the 227 KB shared memory limit");
};

// The biases a kernel knows: none, slopes only, tables too.
enum { kNone = 0, kLinear = 1, kAny = 2 };

// Whether scores can be taken against m: beyond that (a mask's score, as a
// rule) 0 serves better, which loses nothing of scores that are nearer to it.
__device__ __forceinline__ bool usable(float m) { return fabsf(m) <= -kLow; }
// The reference that the next chunk's scores are taken against.
__device__ __forceinline__ float chunk_ref(float m) { return usable(m) ? m : 0.f; }

struct ModStats {
  float m1, m2, l1, l2, acc;  // l1 == 0: no key seen yet
};

// Sums of a chunk with every column visible, in two chains of pairs.
struct ChunkSums {
  uint64_t l1a, l1b, l2a, l2b, aa, ab;
};
template <int N>
__device__ __forceinline__ void sums_all(const uint64_t (&e1)[N], const uint64_t (&e2)[N], ChunkSums& s) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float a0, a1, b0, b1;
    f2_split(e1[k], a0, a1);
    f2_split(e2[k], b0, b1);
    const uint64_t P = f2(ex2(a0), ex2(a1));
    s.l1a = f2_add(s.l1a, P);
    s.l2a = f2_add(s.l2a, f2(ex2(b0), ex2(b1)));
    s.aa = f2_fma(P, f2_sub(e1[k], e2[k]), s.aa);
    f2_split(e1[k + 1], a0, a1);
    f2_split(e2[k + 1], b0, b1);
    const uint64_t Q = f2(ex2(a0), ex2(a1));
    s.l1b = f2_add(s.l1b, Q);
    s.l2b = f2_add(s.l2b, f2(ex2(b0), ex2(b1)));
    s.ab = f2_fma(Q, f2_sub(e1[k + 1], e2[k + 1]), s.ab);
  }
}
__device__ __forceinline__ float sum2(uint64_t a, uint64_t b) {
  float u, v;
  f2_split(f2_add(a, b), u, v);
  return u + v;
}

__device__ __forceinline__ void add_chunk(ModStats& st, float l1, float l2, float acc) {
  st.l1 += l1;
  st.l2 += l2;
  st.acc += acc;
}

// Moves the references of the state to m1, m2 (not below its own; set, not
// added up: the step from a mask's score rounds).
__device__ __forceinline__ void move_refs(ModStats& st, float m1, float m2) {
  const float d1 = m1 - st.m1, d2 = m2 - st.m2;
  const float a1 = ex2(-d1);
  st.acc = a1 * fmaf(-(d1 - d2), st.l1, st.acc);
  st.l1 *= a1;
  st.l2 *= ex2(-d2);
  st.m1 = m1;
  st.m2 = m2;
}

constexpr float kGone = -3.0e38f;  // 2^ that is 0 against any reference, and differences of it are 0

template <int N>
__device__ __forceinline__ void mask_products(uint32_t (&x1)[N], uint32_t (&x2)[N], uint32_t bits) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (!((bits >> k) & 1u)) x1[k] = x2[k] = 0u;
}
template <int N>
__device__ __forceinline__ void mask_scores(uint64_t (&e1)[N], uint64_t (&e2)[N], uint32_t bits) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const bool va = (bits >> (2 * k)) & 1u, vb = (bits >> (2 * k + 1)) & 1u;
    float a, b, c, d;
    f2_split(e1[k], a, b);
    f2_split(e2[k], c, d);
    e1[k] = f2(va ? a : kGone, vb ? b : kGone);
    e2[k] = f2(va ? c : kGone, vb ? d : kGone);
  }
}

// Whether the row has no weight on any key yet.  (While a chunk is taken again
// one side's sum alone may have become 0.)
__device__ __forceinline__ bool nothing(const ModStats& st) { return st.l1 == 0.f && st.l2 == 0.f; }

// The references after a chunk: its visible maxima (r1, r2: what its scores
// are relative to) where the row has seen nothing or these are above its own.
template <int N>
__device__ __forceinline__ void chunk_max(const ModStats& st, const uint64_t (&e1)[N], const uint64_t (&e2)[N], float r1,
                                          float r2, float& m1, float& m2) {
  float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float a, b, c, d;
    f2_split(e1[k], a, b);
    f2_split(e2[k], c, d);
    t1 = max3(t1, a, b);
    t2 = max3(t2, c, d);
  }
  m1 = rintf(t1) + r1;
  m2 = rintf(t2) + r2;
  if (!nothing(st)) {
    m1 = fmaxf(m1, st.m1);
    m2 = fmaxf(m2, st.m2);
  }
}

// Moves the references to m1, m2 (of chunk_max), or sets those of a row that has seen nothing.
__device__ __forceinline__ void take_refs(ModStats& st, float m1, float m2) {
  if (!nothing(st)) return move_refs(st, m1, m2);
  st.m1 = m1;
  st.m2 = m2;
}

// Adds a chunk, its masked columns at kGone, with the references at m1, m2.
template <int N>
__device__ __forceinline__ void fold_chunk(ModStats& st, uint64_t (&e1)[N], uint64_t (&e2)[N], float r1, float r2,
                                           float m1, float m2) {
  take_refs(st, m1, m2);
  const uint64_t D1 = f2(r1 - m1, r1 - m1), D2 = f2(r2 - m2, r2 - m2);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    e1[k] = f2_add(e1[k], D1);
    e2[k] = f2_add(e2[k], D2);
  }
  ChunkSums s{};
  sums_all(e1, e2, s);
  add_chunk(st, sum2(s.l1a, s.l1b), sum2(s.l2a, s.l2b), sum2(s.aa, s.ab));
}

// A tile with masked columns, the first of a row, or one above its references:
// the row's kCols columns at ts, 16 at a time (they leave the most registers
// free).  MASK = false: every column is visible; what a masked column holds
// does not matter.  Called by whole warps.
//
// Scores are rounded at the size of their distance to the reference.  Where a
// chunk's own are much smaller than that (the keys before were masked by a
// large finite bias, say: a whole chunk of entries of -65504 put errors of
// 0.004 into the scores of the next one, and up to 0.02 into KL), it is taken
// again, against its own maximum.
template <int kCols, bool CAP1, bool CAP2, int KIND, bool MASK>
__device__ __forceinline__ void fold_tile(ModStats& st, uint32_t ts, const ModFwdArgs& a, const SideRegs& p1,
                                          const SideRegs& p2, const HeadBias* hb, int rmin, int r0, uint32_t bits) {
  constexpr bool kBiased = KIND != kNone;
  constexpr float kFar = 64.f;
  TileBias tb1{kZero, 0.f, 0.f}, tb2 = tb1;
  if (kBiased) {
    tb1 = tile_bias(hb[0], rmin, rmin + 2 * kTile - 2);
    tb2 = tile_bias(hb[1], rmin, rmin + 2 * kTile - 2);
  }
  bool again = false;
#pragma unroll 1
  for (int c = 0; c < kCols;) {
    const uint32_t part = MASK ? (bits >> c) & 0xffffu : 0xffffu;
    if (MASK && __all_sync(0xffffffffu, part == 0u)) {
      c += 16;
      continue;
    }
    const float ref1 = chunk_ref(st.m1), ref2 = chunk_ref(st.m2);
    RowBias rb1{0.f, 0.f, -ref1, -ref1, nullptr}, rb2{0.f, 0.f, -ref2, -ref2, nullptr};
    if (kBiased) {
      rb1 = row_bias(hb[0], tb1, r0 + c, -ref1);
      rb2 = row_bias(hb[1], tb2, r0 + c, -ref2);
    }
    uint32_t x1[16], x2[16];
    uint64_t e1[8], e2[8];
    tmem_ld2x16(ts + c, ts + c + 128, x1, x2);
    if (MASK && (CAP1 || CAP2)) mask_products(x1, x2, part);  // a masked product must not choose the path below
    const float z1 = scores<CAP1, kBiased>(x1, e1, p1, tb1.how, rb1);
    const float z2 = scores<CAP2, kBiased>(x2, e2, p2, tb2.how, rb2);
    if ((CAP1 || CAP2) && __any_sync(0xffffffffu, z1 > a.s1.zmax || z2 > a.s2.zmax)) {  // beyond half of a cap
      tmem_ld2x16(ts + c, ts + c + 128, x1, x2);
      scores_any<CAP1, kBiased>(x1, e1, a.s1, tb1.how, rb1);
      scores_any<CAP2, kBiased>(x2, e2, a.s2, tb2.how, rb2);
    }
    if (MASK) mask_scores(e1, e2, part);
    float m1, m2;
    chunk_max(st, e1, e2, ref1, ref2, m1, m2);
    auto above = [&](float m, float ref) { return usable(m) && m - ref > fmaxf(kFar, fabsf(m)); };
    const bool far = part != 0u && (above(m1, ref1) || above(m2, ref2));
    if (!again && __any_sync(0xffffffffu, far)) {
      if (far) take_refs(st, m1, m2);
      again = true;
      continue;
    }
    if (!MASK || part != 0u) fold_chunk(st, e1, e2, ref1, ref2, m1, m2);
    again = false;
    c += 16;
  }
}

// Adds another part of the row; both have seen a key.
__device__ __forceinline__ void merge_stats(ModStats& st, ModStats o) {
  const float m1 = fmaxf(st.m1, o.m1), m2 = fmaxf(st.m2, o.m2);
  move_refs(st, m1, m2);
  move_refs(o, m1, m2);
  add_chunk(st, o.l1, o.l2, o.acc);
}

// The row's results.  A row that saw no key, or whose largest score on one
// side is a table's mask (masked1, masked2: HeadBias::masked; however low raw
// scores or slopes take it, a row without such an entry is computed): KL 0,
// LSE -inf.  (A row of NaNs has no maximum either: its sums say so.)
__device__ __forceinline__ void write_row(const ModStats& st, float masked1, float masked2, float* kl, float* lse1,
                                          float* lse2) {
  const bool low = st.m1 < masked1 || st.m2 < masked2;
  const bool seen = st.l1 != 0.f && (!low || st.l1 != st.l1 || st.l2 != st.l2);
  *lse1 = seen ? fmaf(st.m1, kLn2, logf(st.l1)) : -INFINITY;
  *lse2 = seen ? fmaf(st.m2, kLn2, logf(st.l2)) : -INFINITY;
  *kl = seen ? fmaf(kLn2, st.acc / st.l1, logf(st.l2 / st.l1)) : 0.f;
}

// The row's kCols columns of a tile, 16 at a time, against the references as
// they stand; MASK: only the columns in bits.  Returns false with the state
// untouched where that is not exact: the row has no usable reference, a sum
// reached 2^64 or a score is beyond half of its cap.
template <int kCols, bool CAP1, bool CAP2, int HOW1, int HOW2, bool MASK>
__device__ __forceinline__ bool add_tile(ModStats& st, uint32_t ts, const SideRegs& s1, const SideRegs& s2, float zmax1,
                                         float zmax2, RowBias rb1, RowBias rb2, uint32_t bits) {
  ChunkSums s{};
  float z1 = 0.f, z2 = 0.f;
#pragma unroll
  for (int c = 0; c < kCols; c += 16) {
    uint32_t x1[16], x2[16];
    uint64_t e1[8], e2[8];
    tmem_ld2x16(ts + c, ts + c + 128, x1, x2);
    if (MASK && (CAP1 || CAP2)) mask_products(x1, x2, bits >> c);
    z1 = fmaxf(z1, scores_how<CAP1, HOW1>(x1, e1, s1, rb1));
    z2 = fmaxf(z2, scores_how<CAP2, HOW2>(x2, e2, s2, rb2));
    if (HOW1 != kZero) rb1 = further(rb1, 16);
    if (HOW2 != kZero) rb2 = further(rb2, 16);
    if (MASK) mask_scores(e1, e2, bits >> c);
    sums_all(e1, e2, s);
  }
  const float l1 = sum2(s.l1a, s.l1b), l2 = sum2(s.l2a, s.l2b);
  bool ok = st.l1 != 0.f && usable(st.m1) && usable(st.m2);
  ok = ok && l1 < 18446744073709551616.f && l2 < 18446744073709551616.f;  // 2^64
  if (CAP1) ok = ok && z1 <= zmax1;
  if (CAP2) ok = ok && z2 <= zmax2;
  if (MASK) ok = ok || bits == 0u;
  ok = __all_sync(0xffffffffu, ok);
  if (ok && (!MASK || bits != 0u)) add_chunk(st, l1, l2, sum2(s.aa, s.ab));
  return ok;
}

// The same by the tile's kinds of bias (neither kFold).
template <int kCols, bool CAP1, bool CAP2, int KIND, bool MASK>
__device__ __forceinline__ bool add_tile_how(ModStats& st, uint32_t ts, const SideRegs& s1, const SideRegs& s2,
                                             float zmax1, float zmax2, int how1, int how2, const RowBias& rb1,
                                             const RowBias& rb2, uint32_t bits) {
  if (KIND == kNone) return add_tile<kCols, CAP1, CAP2, kZero, kZero, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits);
  if (KIND == kLinear) return add_tile<kCols, CAP1, CAP2, kFlat, kFlat, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits);
  if (how1 != kLook)
    return how2 != kLook ? add_tile<kCols, CAP1, CAP2, kFlat, kFlat, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits)
                         : add_tile<kCols, CAP1, CAP2, kFlat, kLook, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits);
  return how2 != kLook ? add_tile<kCols, CAP1, CAP2, kLook, kFlat, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits)
                       : add_tile<kCols, CAP1, CAP2, kLook, kLook, MASK>(st, ts, s1, s2, zmax1, zmax2, rb1, rb2, bits);
}

// MASKED: some tile besides a row's first may need a mask (ids, a prefix).
template <int D1, int D2, bool CAP1, bool CAP2, int KIND, bool MASKED>
__global__ void __launch_bounds__(ModFwdLayout<D1, D2>::kThreads, 1)
    fwd_mod_kernel(const __grid_constant__ CUtensorMap tq1, const __grid_constant__ CUtensorMap tk1,
                   const __grid_constant__ CUtensorMap tq2, const __grid_constant__ CUtensorMap tk2,
                   const __grid_constant__ ModFwdArgs a) {
  using L = ModFwdLayout<D1, D2>;
  using T1 = OpTile<D1>;
  using T2 = OpTile<D2>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int nqt = (a.NQ + kTile - 1) / kTile, nkt_rows = (a.NK + kTile - 1) / kTile;
  // a unit is a query tile of one head, or the rows of 2^pack_shift heads
  int unit, t;
  grouped_unit(int(blockIdx.y) * int(gridDim.x) + int(blockIdx.x), a.B * (a.H >> a.pack_shift), nqt, a.head_group,
               unit, t);
  const int bh = unit << a.pack_shift;  // the (first) head
  const int b = bh / a.H, h = bh - b * a.H;
  const int pack_rows = kTile >> a.pack_shift;
  const int qt = a.vis.causal ? (nqt - 1 - t) : t;  // longest rows first
  const int split = blockIdx.z;
  const int q0 = qt * kTile;
  const int off = a.NK - a.NQ;
  const int prefix = a.vis.prefix != nullptr ? min(max(a.vis.prefix[b], 0), a.NK) : 0;

  const uint32_t bar0 = sb + L::oBar;
  const uint32_t bar_q = bar0;
  auto bar_kfull = [&](int s) { return bar0 + 8u * (1 + s); };
  auto bar_kempty = [&](int s) { return bar0 + 8u * (1 + L::kStages + s); };
  auto bar_sfull = [&](int i) { return bar0 + 8u * (1 + 2 * L::kStages + i); };
  auto bar_sempty = [&](int i) { return bar0 + 8u * (3 + 2 * L::kStages + i); };
  const uint32_t bar_done = bar0 + 8u * (5 + 2 * L::kStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oMisc + 4);
  int* range = reinterpret_cast<int*>(smem + L::oRange);
  const Ctl ctl{abort_flag, a.status};

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar_kfull(s), 1);
      mbar_init(bar_kempty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_sfull(i), 1);
      mbar_init(bar_sempty(i), L::kStatWarps);
    }
    mbar_init(bar_done, 1);
    *abort_flag = 0;
    range[0] = INT_MAX;
    range[1] = -1;
    fence_barrier_init();
    // Q at once: it does not wait for the rest of the block's start
    mbar_arrive_expect_tx(bar_q, L::kQ1 + L::kQ2);
    for (int s = 0; s < (1 << a.pack_shift); ++s) {
      load_tile<T1>(sb + L::oQ1 + s * pack_rows * T1::kRowBytes, &tq1, bar_q, q0, h + s, b);
      load_tile<T2>(sb + L::oQ2 + s * pack_rows * T2::kRowBytes, &tq2, bar_q, q0, h + s, b);
    }
  }
  HeadBias* hbs = reinterpret_cast<HeadBias*>(smem + L::oBias);  // two for each head
  if (KIND != kNone && threadIdx.x < (2u << a.pack_shift))
    hbs[threadIdx.x] = head_bias(threadIdx.x & 1 ? a.s2 : a.s1, h + int(threadIdx.x >> 1));
  float* near_rows = reinterpret_cast<float*>(smem + L::oNear);
  if (KIND == kAny && a.near_smem) {
    __syncthreads();
    near_to_smem(hbs, 2 << a.pack_shift, near_rows);
    __syncthreads();
    if (threadIdx.x == 0) near_in_smem(hbs, 2 << a.pack_shift, near_rows);
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // the key tiles this query tile can see: [tlo, thi)
  int tlo = 0, thi = nkt_rows;
  if (a.vis.causal) {
    const int kend = max(min(q0 + kTile, a.NQ) + off, prefix);  // at most NK
    thi = kend <= 0 ? 0 : (kend + kTile - 1) / kTile;
  }
  int4 tq{0, 0, 1, 0};
  if (a.vis.ids_q != nullptr) {
    __syncthreads();
    tq = a.vis.tiles_q[size_t(b) * nqt + qt];
    int lo = INT_MAX, hi = -1;
    for (int j = threadIdx.x; j < thi; j += blockDim.x)
      if (tiles_meet(tq, a.vis.tiles_k[size_t(b) * nkt_rows + j])) {
        lo = min(lo, j);
        hi = max(hi, j);
      }
    if (hi >= 0) {
      atomicMin(range, lo);
      atomicMax(range + 1, hi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (a.vis.ids_q != nullptr) {
    thi = range[1] + 1;
    tlo = thi > 0 ? range[0] : 0;
  }
  const int kt_lo = tlo + int((long long)split * (thi - tlo) / a.num_splits);
  const int kt_hi = tlo + int((long long)(split + 1) * (thi - tlo) / a.num_splits);
  const int nkt = kt_hi - kt_lo;

  if (warp == L::kProdWarp) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0 && nkt > 0) {
      int issued = 0;
      for (int j = 0; j < nkt; ++j) {
        const int s = j % L::kStages;
        if (!mbar_wait(bar_kempty(s), ((j / L::kStages) & 1) ^ 1, ctl)) break;
        const int k0 = (kt_hi - 1 - j) * kTile;
        const uint32_t st = sb + L::oK + s * L::kStage;
        if (!SKL_CHECK(a.status, s < L::kStages && k0 < a.NK)) {
          *abort_flag = 1;
          break;
        }
        mbar_arrive_expect_tx(bar_kfull(s), L::kStage);
        load_tile<T1>(st, &tk1, bar_kfull(s), k0, h / a.g1, b);
        load_tile<T2>(st + L::kK1, &tk2, bar_kfull(s), k0, h / a.g2, b);
        issued = j + 1;
      }
      if (*abort_flag) {  // let the copies already started land before the CTA exits
        mbar_drain(bar_q, 0, 200000000ull);
        for (int j = issued > L::kStages ? issued - L::kStages : 0; j < issued; ++j)
          mbar_drain(bar_kfull(j % L::kStages), (j / L::kStages) & 1, 200000000ull);
      }
    }
    if (lane == 0 && nkt <= 0) mbar_drain(bar_q, 0, 200000000ull);  // no tile to wait for it
  } else if (warp == L::kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    // (the whole warp runs the loop; the elected lane issues)
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16(128, 128, 0, 0);
    if (nkt > 0 && mbar_wait_warp(bar_q, 0, ctl)) {
      for (int j = 0; j < nkt; ++j) {
        const int i = j & 1, s = j % L::kStages;
        const uint32_t d1 = tmem + i * 256, d2 = d1 + 128;
        if (!mbar_wait_warp(bar_kfull(s), (j / L::kStages) & 1, ctl)) break;
        if (!mbar_wait_warp(bar_sempty(i), ((j >> 1) & 1) ^ 1, ctl)) break;
        tc_fence_after();
        const uint32_t k1s = sb + L::oK + s * L::kStage, k2s = k1s + L::kK1;
#pragma unroll
        for (int kk = 0; kk < D1 / 16; ++kk) {
          const uint32_t o = T1::off_k(kk);
          mma_bf16_ss(leader, d1, T1::desc_k(sb + L::oQ1 + o), T1::desc_k(k1s + o), idesc, kk > 0);
        }
#pragma unroll
        for (int kk = 0; kk < D2 / 16; ++kk) {
          const uint32_t o = T2::off_k(kk);
          mma_bf16_ss(leader, d2, T2::desc_k(sb + L::oQ2 + o), T2::desc_k(k2s + o), idesc, kk > 0);
        }
        mma_commit(leader, bar_kempty(s));
        mma_commit(leader, bar_sfull(i));
      }
    }
    // every MMA this warp issued has finished before TMEM is released
    mma_commit(leader, bar_done);
    mbar_drain(bar_done, 0, 1000000000ull);
  } else {
    // ---------------------------------------------------------------- statistics
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int slot = row / pack_rows;      // the row's head is h + slot
    const int grow = q0 + row - slot * pack_rows;  // its query
    const HeadBias* hb = hbs + 2 * slot;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const int col = wg * L::kCols;
    const bool ids = MASKED && a.vis.ids_q != nullptr;
    const int id = ids ? a.vis.ids_q[size_t(b) * nqt * kTile + grow] : 0;
    const SideRegs p1 = side_regs<CAP1>(a.s1), p2 = side_regs<CAP2>(a.s2);
    const bool idle = __all_sync(0xffffffffu, grow >= a.NQ);  // this warp's rows are all past NQ
    ModStats st{0.f, 0.f, 0.f, 0.f, 0.f};
    // The first tiles, general and masked: the last keys, the diagonal, and
    // at least one, which gives the row its references.  (With ids or a
    // prefix any tile may need a mask.)
    int npeel = 1;
    if (!MASKED) {
      int full = a.NK / kTile;
      if (a.vis.causal) full = min(full, max(q0 + off + 1, 0) / kTile);
      npeel = max(1, kt_hi - full);
    }
    npeel = min(npeel, nkt);
    for (int j = 0; j < npeel; ++j) {
      const int i = j & 1;
      const int kt = kt_hi - 1 - j, k0 = kt * kTile;
      const bool same = !MASKED || !ids || tiles_same(tq, a.vis.tiles_k[size_t(b) * nkt_rows + kt]);
      const uint32_t bits = visible_bits<32>(grow, k0 + col, off, a.NK, a.vis.causal, prefix, id,
                                             same ? nullptr : a.vis.ids_k + size_t(b) * nkt_rows * kTile + k0 + col);
      if (!mbar_wait_warp(bar_sfull(i), (j >> 1) & 1, ctl)) break;
      tc_fence_after();
      if (!idle)
        fold_tile<L::kCols, CAP1, CAP2, KIND, true>(st, tmem + lane_off + uint32_t(i * 256 + col), a, p1, p2, hb,
                                                    k0 - (q0 + kTile - 1 + off), k0 + col - (grow + off), bits);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sempty(i));
    }
    // the id range of the tile after this one is fetched a tile ahead
    auto range_of = [&](int kt) { return ids ? a.vis.tiles_k[size_t(b) * nkt_rows + max(kt, 0)] : int4{0, 0, 1, 0}; };
    int4 tk = range_of(kt_hi - 1 - npeel);
    for (int j = npeel; j < nkt; ++j) {
      const int i = j & 1;
      const int kt = kt_hi - 1 - j, k0 = kt * kTile;
      // the tile's relative positions: key k0 + c against query q0 + r
      const int rmin = k0 - (q0 + kTile - 1 + off);
      const int r0 = k0 + col - (grow + off);
      const uint32_t ts = tmem + lane_off + uint32_t(i * 256 + col);
      bool need_mask = false;
      uint32_t bits = 0xffffffffu;
      if (MASKED) {
        const bool same = !ids || tiles_same(tq, tk);
        tk = range_of(kt - 1);
        need_mask = (k0 + kTile > a.NK) || !same || (a.vis.causal && rmin + 2 * kTile - 2 > 0 && k0 + kTile > prefix);
        if (need_mask)
          bits = visible_bits<32>(grow, k0 + col, off, a.NK, a.vis.causal, prefix, id,
                                  same ? nullptr : a.vis.ids_k + size_t(b) * nkt_rows * kTile + k0 + col);
      }
      RowBias rb1{0.f, 0.f, -st.m1, -st.m1, nullptr}, rb2{0.f, 0.f, -st.m2, -st.m2, nullptr};
      int how1 = kZero, how2 = kZero;
      if (KIND != kNone) {
        const TileBias tb1 = tile_bias(hb[0], rmin, rmin + 2 * kTile - 2);
        const TileBias tb2 = tile_bias(hb[1], rmin, rmin + 2 * kTile - 2);
        how1 = tb1.how;
        how2 = tb2.how;
        rb1 = row_bias(hb[0], tb1, r0, -st.m1);
        rb2 = row_bias(hb[1], tb2, r0, -st.m2);
      }
      if (!mbar_wait_warp(bar_sfull(i), (j >> 1) & 1, ctl)) break;
      tc_fence_after();
      if (!idle) {
        bool ok = KIND == kNone || (how1 != kFold && how2 != kFold);
        if (ok) {
          if (MASKED && need_mask)
            ok = add_tile_how<L::kCols, CAP1, CAP2, KIND, true>(st, ts, p1, p2, a.s1.zmax, a.s2.zmax, how1, how2, rb1,
                                                                rb2, bits);
          else
            ok = add_tile_how<L::kCols, CAP1, CAP2, KIND, false>(st, ts, p1, p2, a.s1.zmax, a.s2.zmax, how1, how2, rb1,
                                                                 rb2, bits);
        }
        if (!ok) fold_tile<L::kCols, CAP1, CAP2, KIND, MASKED>(st, ts, a, p1, p2, hb, rmin, r0, bits);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sempty(i));
    }
    // merge the column shares of every row (warpgroups 1.. -> warpgroup 0)
    float* mg = reinterpret_cast<float*>(smem + L::oMerge);
    if (wg > 0) {
      float* o = mg + (wg - 1) * kTile * 5 + row * 5;
      o[0] = st.m1;
      o[1] = st.m2;
      o[2] = st.l1;
      o[3] = st.l2;
      o[4] = st.acc;
    }
    named_bar_sync(1, 32 * L::kStatWarps);
    if (wg == 0 && !*abort_flag && grow < a.NQ) {
#pragma unroll
      for (int w = 0; w < L::kWGs - 1; ++w) {
        const float* o = mg + w * kTile * 5 + row * 5;
        const ModStats other{o[0], o[1], o[2], o[3], o[4]};
        if (other.l1 == 0.f) continue;
        if (st.l1 == 0.f) st = other;
        else merge_stats(st, other);
      }
      const size_t rows = size_t(a.B) * a.H * a.NQ;
      const size_t idx = size_t(bh + slot) * a.NQ + grow;
      if (!SKL_CHECK(a.status, idx < rows && split < a.num_splits)) {
        // (debug build) out-of-range row or split: nothing is written
      } else if (a.partial != nullptr) {
        float* p = a.partial + size_t(split) * 5 * rows + idx;
        p[0 * rows] = st.m1;
        p[1 * rows] = st.m2;
        p[2 * rows] = st.l1;
        p[3 * rows] = st.l2;
        p[4 * rows] = st.acc;
      } else {
        constexpr bool kTables = KIND == kAny;
        write_row(st, kTables ? hb[0].masked : -INFINITY, kTables ? hb[1].masked : -INFINITY, a.kl + idx, a.lse1 + idx,
                  a.lse2 + idx);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D1, int D2, bool CAP1, bool CAP2, int KIND, bool MASKED>
int launch_fwd_mod_k(const ModMaps& m, const ModFwdArgs& a, cudaStream_t st) {
  using L = ModFwdLayout<D1, D2>;
  auto kern = fwd_mod_kernel<D1, D2, CAP1, CAP2, KIND, MASKED>;
  ModFwdArgs b = a;
  const size_t near = KIND == kAny ? near_smem_bytes(a.s1, a.s2, 1 << a.pack_shift) : 0;
  b.near_smem = near > 0 && L::kAlloc + near <= 232448;
  const int bytes = int(L::kAlloc + (b.near_smem ? near : 0));
  // (always the most a block may have: threads that launch at once would set each other's size)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e != cudaSuccess) return e;
  dim3 grid((a.NQ + kTile - 1) / kTile, a.B * (a.H >> a.pack_shift), a.num_splits);
  kern<<<grid, L::kThreads, bytes, st>>>(m.q1, m.k1, m.q2, m.k2, b);
  return cudaGetLastError();
}

// One kernel for each set of modifications: what a side does not have must
// not cost the loop over full tiles registers or instructions (with 16 + 2
// warps a thread has 96).  At 8K x 32 heads, d = 128, causal, the last kernel
// that branched (64 columns a warp) took 593 us without modifications and 906
// with both sides capped, a kernel for each set 497 and 831; these take 468
// and 778 (the plain forward 460).
template <int D1, int D2, bool CAP1, bool CAP2>
int launch_fwd_mod_c(const ModMaps& m, const ModFwdArgs& a, cudaStream_t st) {
  const bool masked = a.vis.ids_q != nullptr || a.vis.prefix != nullptr;
  if (a.s1.kind == kBiasTable || a.s2.kind == kBiasTable)
    return masked ? launch_fwd_mod_k<D1, D2, CAP1, CAP2, kAny, true>(m, a, st)
                  : launch_fwd_mod_k<D1, D2, CAP1, CAP2, kAny, false>(m, a, st);
  if (a.s1.kind == kBiasSlopes || a.s2.kind == kBiasSlopes)
    return masked ? launch_fwd_mod_k<D1, D2, CAP1, CAP2, kLinear, true>(m, a, st)
                  : launch_fwd_mod_k<D1, D2, CAP1, CAP2, kLinear, false>(m, a, st);
  return masked ? launch_fwd_mod_k<D1, D2, CAP1, CAP2, kNone, true>(m, a, st)
                : launch_fwd_mod_k<D1, D2, CAP1, CAP2, kNone, false>(m, a, st);
}

template <int D1, int D2>
int launch_fwd_mod_t(const ModMaps& m, const ModFwdArgs& a, cudaStream_t st) {
  const bool c1 = a.s1.carg != 0.f, c2 = a.s2.carg != 0.f;
  if (c1) return c2 ? launch_fwd_mod_c<D1, D2, true, true>(m, a, st) : launch_fwd_mod_c<D1, D2, true, false>(m, a, st);
  return c2 ? launch_fwd_mod_c<D1, D2, false, true>(m, a, st) : launch_fwd_mod_c<D1, D2, false, false>(m, a, st);
}

}  // namespace

}  // namespace skl
