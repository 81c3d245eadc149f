// Backward over modified scores (see mod_common.cuh), head dims up to 128.
//
// With e_t = (S_t - LSE_t) log2 e rebuilt per tile from the forward's LSEs:
//   mode P2:  dS = dKL (2^e2 - 2^e1)
//   mode P1:  dS = dKL 2^e1 (ln 2 (e1 - e2) - KL)
//   dX = s dS (1 - T^2)  (T = tanh of the gradient side's capped score; no
//        cap: dX = s dS),  dQ = dX K,  dK = dX^T Q
//   d table[h][b] = sum of dS over the pairs whose relative position is in
//        bucket b
//
// The pipeline is the fused backward's (bwd.cu; the same warps, barriers and
// TMEM map): one CTA per query head and 128-key tile walks the query tiles
// that can see it, dK accumulates in TMEM, dQ leaves as fp32 reduce-adds into
// a workspace that launch_mod_finish rounds to bf16 once at the end.
// What differs: the dS warps' arithmetic; K rows whose id matches nothing and
// Q rows that saw no key are zeroed in shared memory before a product reads
// them (they may hold anything); with ids the walk is cut to the query tiles
// that share one; dK goes out as bf16 where one CTA owns it.
//
// The table's gradient (kTab): along a warp's 32 x 32 block of dS the
// relative position is constant on diagonals, so 32 steps of "shift by one
// lane, add the next column" leave every diagonal's sum in a lane (those that
// leave lane 31 early move to a second register); the sums of a bucket are
// neighbours, joined by a segmented scan (add_to_buckets).  Tiles beyond the
// table's reach add to one bucket as a whole.  Each warp has its own sums, in
// the workspace, and a last kernel adds them in a fixed order.
#pragma once

#include <climits>

#include "bwd_common.cuh"
#include "bwd_fused.cuh"
#include "mod_common.cuh"
#include "tiles.cuh"

namespace skl {

template <int D1, int D2, int MODE>
struct ModBwdLayout : BwdLayout<D1, D2, MODE> {
  using Base = BwdLayout<D1, D2, MODE>;
  static constexpr uint32_t oReady = Base::kBytes;  // barrier: K rows that match nothing are zeroed
  static constexpr uint32_t oRange = oReady + 8;    // first and last query tile with a shared id
  static constexpr uint32_t oBias = (oRange + 8 + 15) / 16 * 16;  // HeadBias of the other side and of the gradient side
  static constexpr uint32_t oNear = (oBias + 2 * sizeof(HeadBias) + 15) / 16 * 16;  // lookup rows, where they fit
  static constexpr uint32_t kAlloc = oNear + 1024;
  static_assert(oReady % 8 == 0, "barriers are 8-byte aligned");
  static_assert(kAlloc <= 232448, "over the 227 KB shared memory limit");
};

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) { st_shared_v4(addr, 0u, 0u, 0u, 0u); }

// Row `row` of an operand tile becomes zeros (a swizzle moves 16-byte pieces
// within a row only).
template <typename T>
__device__ __forceinline__ void zero_row(uint32_t base, int row) {
#pragma unroll 1
  for (int c = 0; c < T::kBlocks; ++c)
    for (int p = 0; p < int(T::kRowBytes); p += 16)
      st_shared_zero16(base + c * T::kBlockBytes + row * T::kRowBytes + p);
}

// Adds v of each lane to this warp's sum of bucket k of each lane (k < 0:
// nothing).  Equal buckets are neighbours: a segmented scan joins them, and
// the last of each adds to memory.  Only this warp adds to these sums, and
// the warp barrier orders one call's additions before the next one's, so the
// order is fixed.  (Passing each bucket to a lane that keeps it took 32 rounds
// near the diagonal: 198 us at 4096 x 16 heads, d = 64, 194 us so.)
__device__ __forceinline__ void add_to_buckets(float* sums, float v, int k, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float pv = __shfl_up_sync(0xffffffffu, v, o);
    const int pk = __shfl_up_sync(0xffffffffu, k, o);
    if (lane >= o && pk == k) v += pv;
  }
  const int nk = __shfl_down_sync(0xffffffffu, k, 1);
  __syncwarp();
  if (k >= 0 && (lane == 31 || nk != k)) atomicAdd(sums + k, v);
}

constexpr float kUnseen = -3.0e38f;

struct DsParams {
  float cmul;   // of the gradient side
  float sg;     // its softmax scale
  float capf;   // -s / cmul^2: dX = dS (s + capf Y^2); 0 without a cap
  float w, wo;  // mode P2: weights of 2^e of the gradient side and of the other side; mode P1: weight, and what
                // the difference of the two e has to be moved by (kTab only)
};

// dX of 16 columns of a row, packed to bf16 pairs.  yg: base-2 score without
// bias of the gradient side (CAP), or its product; eo: e of the other side.
// HOW, bias: the gradient side's bias, with -LSE in bias.add.  MASK: only the
// columns in bits; what the others hold does not matter.  kTab: how the
// columns' dS goes to the table: 0 not at all, 1 as a whole (total), 2 by
// diagonal (after 32 columns lane l holds in acc the sum over diagonal 31 - l
// of the 32 x 32 block and in done that of diagonal -1 - l).
template <int MODE, bool CAP, int HOW, int kTab, bool MASK>
__device__ __forceinline__ void dx_chunk(const uint64_t (&yg)[8], const uint64_t (&eo)[8], const DsParams& p,
                                         const RowBias& bias, uint32_t bits, int lane, uint32_t* out8, float& total,
                                         float& acc, float& done) {
  const uint64_t CG = f2(p.cmul, p.cmul), W = f2(p.w, p.w), WO = f2(p.wo, p.wo), SG = f2(p.sg, p.sg),
                 CF = f2(p.capf, p.capf);
  uint64_t T = f2(0.f, 0.f);
  Quad q{};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k % 2 == 0) q = bias_quad<HOW>(bias, 2 * k);
    const uint64_t B2 = k % 2 == 0 ? q.lo : q.hi;
    uint64_t Y = yg[k];
    const uint64_t EG = CAP ? f2_add(Y, B2) : f2_fma(Y, CG, B2);
    float a, b, c, d;
    f2_split(EG, a, b);
    uint64_t D;
    if (MODE == STREAMKL_GRAD_P2) {
      f2_split(eo[k], c, d);
      D = f2_fma(W, f2(ex2(a), ex2(b)), f2_mul(WO, f2(ex2(c), ex2(d))));
    } else {
      // p1 = 2^e1; the other side carries -LSE2 + KL
      const uint64_t R = f2_sub(EG, eo[k]);
      D = f2_mul(f2_mul(W, f2(ex2(a), ex2(b))), kTab != 0 ? f2_add(R, WO) : R);
    }
    float da, db;
    if (MASK) {
      const bool va = (bits >> (2 * k)) & 1u, vb = (bits >> (2 * k + 1)) & 1u;
      f2_split(D, da, db);
      D = f2(va ? da : 0.f, vb ? db : 0.f);
      if (CAP) {
        f2_split(Y, c, d);
        Y = f2(va ? c : 0.f, vb ? d : 0.f);
      }
    }
    if (kTab == 1) T = f2_add(T, D);
    if (kTab == 2) {
      f2_split(D, da, db);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float up = __shfl_sync(0xffffffffu, acc, lane + 31);
        const float dn = __shfl_sync(0xffffffffu, done, lane + 31);
        done = lane == 0 ? up : dn;
        acc = (lane == 0 ? 0.f : up) + (e == 0 ? da : db);
      }
    }
    f2_split(f2_mul(D, CAP ? f2_fma(f2_mul(Y, Y), CF, SG) : SG), da, db);
    out8[k] = pack_bf16(da, db);
  }
  if (kTab == 1) {
    float u, v;
    f2_split(T, u, v);
    total += u + v;
  }
}

// 16 columns of both sides from TMEM to what dx_chunk takes.  MASK: masked
// products become zeros first (they must not choose the path of the cap).
// HOW: the other side's bias where MASK is false (else how_o says).
template <bool CAP, bool BIASED, bool MASK, int HOW>
__device__ __forceinline__ void load_scores(uint32_t tg, uint32_t to, uint64_t (&yg)[8], uint64_t (&eo)[8],
                                            const ModSide& sg, const ModSide& so, const SideRegs& pg,
                                            const SideRegs& po, int how_o, const RowBias& rbo, uint32_t bits) {
  uint32_t xg[16], xo[16];
  const RowBias none{0.f, 0.f, 0.f, 0.f, nullptr};
  auto load = [&]() {
    tmem_ld2x16(tg, to, xg, xo);
    if (MASK && CAP) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (!((bits >> k) & 1u)) xg[k] = xo[k] = 0u;
    }
  };
  load();
  float zo;
  if (MASK) zo = scores<CAP, BIASED>(xo, eo, po, how_o, rbo);
  else zo = scores_how<CAP, HOW>(xo, eo, po, rbo);
  if (CAP) {
    const float zg = scores_how<true, kZero>(xg, yg, pg, none);
    if (__any_sync(0xffffffffu, zo > so.zmax || zg > sg.zmax)) {  // a score beyond half of its cap
      load();
      scores_any<true, BIASED>(xo, eo, so, how_o, rbo);
      scores_any<true, false>(xg, yg, sg, kZero, none);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) yg[k] = f2(__uint_as_float(xg[2 * k]), __uint_as_float(xg[2 * k + 1]));
  }
}

// What the rounding of x log2 e to fp32 (y) loses.
__device__ __forceinline__ float log2e_lost(float x, float y) { return fmaf(x, kLog2e, -y) + x * kLog2eLo; }
// 2^x for a small x.
__device__ __forceinline__ float exp2_small(float x) { return fmaf(x, kLn2, 1.f); }

template <int V>
struct Int {
  static constexpr int value = V;
};

// What a launch needs of the dX arithmetic: no bias, some bias, the gradient
// of the gradient side's table.
enum { kNoBias = 0, kBias = 1, kTable = 2 };

// CAP: some side is capped (the other then has a polynomial of degree 0).
template <int D1, int D2, int MODE, bool CAP, int BIAS>
__global__ void __launch_bounds__(BwdLayout<D1, D2, MODE>::kThreads, 1)
    bwd_mod_kernel(const __grid_constant__ CUtensorMap tq1, const __grid_constant__ CUtensorMap tk1,
                   const __grid_constant__ CUtensorMap tq2, const __grid_constant__ CUtensorMap tk2,
                   const __grid_constant__ CUtensorMap tdq, const __grid_constant__ CUtensorMap tdk,
                   const __grid_constant__ ModBwdArgs a) {
  using L = ModBwdLayout<D1, D2, MODE>;
  constexpr int DG = L::DG, DO = L::DO;
  constexpr bool kP2 = MODE == STREAMKL_GRAD_P2;
  using T1 = OpTile<D1>;
  using T2 = OpTile<D2>;
  using TO = OpTile<DO>;
  using TG = OpTile<DG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gg = kP2 ? a.g2 : a.g1;  // query heads per gradient-side key head

  auto bar = [&](int id) { return sb + L::oBar + 8u * id; };
  const uint32_t bar_ready = sb + L::oReady;
  const CUtensorMap* tqo = kP2 ? &tq1 : &tq2;
  const CUtensorMap* tqg = kP2 ? &tq2 : &tq1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oMisc + 4);
  volatile int* s_queued = reinterpret_cast<volatile int*>(smem + L::oMisc + 8);
  int* unit_slot = reinterpret_cast<int*>(smem + L::oMisc + 12);
  volatile int* turn_ok = reinterpret_cast<volatile int*>(smem + L::oMisc + 16);
  int* range = reinterpret_cast<int*>(smem + L::oRange);
  const Ctl ctl{abort_flag, a.status};

  if (threadIdx.x == 0) {
    // ordered dK of grouped key heads: units in the order CTAs start, so a
    // head waits only for CTAs that run
    *unit_slot = a.ticket ? atomicAdd(a.ticket, 1) : int(blockIdx.y * gridDim.x + blockIdx.x);
    *s_queued = 0;
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t count = 1;
      if (i == L::B_SFREE || i == L::B_DSFULL) count = 8;     // one per dS warp
      if (i == L::B_DQEMPTY) count = 4;                       // one per epilogue warp
      if (i == L::B_DSEMPTY) count = L::kSplitIssue ? 2 : 1;  // dK (and dQ) issuers
      if (i == L::B_DONE) count = L::kSplitIssue ? 3 : 2;     // one per MMA issuer
      mbar_init(bar(i), count);
    }
    mbar_init(bar_ready, 8);
    *abort_flag = 0;
    range[0] = INT_MAX;
    range[1] = -1;
    fence_barrier_init();
    // K at once: it does not wait for the rest of the block's start
    int u_bh, u_kt;
    grouped_unit(*unit_slot, a.B * a.H, int(gridDim.x), a.head_group, u_bh, u_kt);
    const int u_b = u_bh / a.H, u_h = u_bh - u_b * a.H;
    mbar_arrive_expect_tx(bar(L::B_KFULL), L::kK1 + L::kK2);
    load_tile<T1>(sb + L::oK1, &tk1, bar(L::B_KFULL), u_kt * kTile, u_h / a.g1, u_b);
    load_tile<T2>(sb + L::oK2, &tk2, bar(L::B_KFULL), u_kt * kTile, u_h / a.g2, u_b);
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_s1 = tmem, t_s2 = tmem + 128, t_dk = tmem + 256, t_dq = tmem + 384;

  const int nkt = int(gridDim.x), nqt = (a.NQ + kTile - 1) / kTile;
  int bh, kt;
  grouped_unit(*unit_slot, a.B * a.H, nkt, a.head_group, bh, kt);
  const int b = bh / a.H, h = bh - b * a.H;
  const int k0 = kt * kTile;
  const int off = a.NK - a.NQ;
  const int prefix = a.vis.prefix != nullptr ? min(max(a.vis.prefix[b], 0), a.NK) : 0;
  // causal: query i sees key j iff i >= j - off, or j < prefix
  int qt_lo = a.vis.causal && k0 >= prefix ? max(0, k0 - off) / kTile : 0;
  int qt_hi = nqt;
  const bool ids = a.vis.ids_q != nullptr;
  int4 tk{0, 0, 1, 0};
  if (BIAS != kNoBias) {
    HeadBias* hb = reinterpret_cast<HeadBias*>(smem + L::oBias);
    if (threadIdx.x == 0) hb[0] = head_bias(kP2 ? a.s1 : a.s2, h);
    if (threadIdx.x == 32) hb[1] = head_bias(kP2 ? a.s2 : a.s1, h);
    if (a.near_smem) {
      float* rows = reinterpret_cast<float*>(smem + L::oNear);
      __syncthreads();
      near_to_smem(hb, 2, rows);
      __syncthreads();
      if (threadIdx.x == 0) near_in_smem(hb, 2, rows);
    }
    if (!ids) __syncthreads();
  }
  if (ids) {
    tk = a.vis.tiles_k[size_t(b) * nkt + kt];
    int lo = INT_MAX, hi = -1;
    for (int j = qt_lo + int(threadIdx.x); j < nqt; j += int(blockDim.x))
      if (tiles_meet(tk, a.vis.tiles_q[size_t(b) * nqt + j])) {
        lo = min(lo, j);
        hi = max(hi, j);
      }
    if (hi >= 0) {
      atomicMin(range, lo);
      atomicMax(range + 1, hi);
    }
    __syncthreads();
    qt_hi = range[1] + 1;
    qt_lo = qt_hi > 0 ? range[0] : 0;
  }
  const int n = max(0, qt_hi - qt_lo);
  // K may be read by the products once its rows that match nothing are zeroed
  const uint32_t bar_k = ids ? bar_ready : bar(L::B_KFULL);

  if (warp == 12) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int q0 = (qt_lo + i) * kTile;
        if (!mbar_wait_polled(bar(L::B_QOEMPTY), (i & 1) ^ 1, ctl)) break;
        mbar_arrive_expect_tx(bar(L::B_QOFULL), L::kQo);
        load_tile<TO>(sb + L::oQo, tqo, bar(L::B_QOFULL), q0, h, b);
        const int g = i % L::kQgBufs;
        if (!mbar_wait_polled(bar(L::B_QGEMPTY0 + g), ((i / L::kQgBufs) & 1) ^ 1, ctl)) {
          mbar_drain(bar(L::B_QOFULL), i & 1, 200000000ull);
          break;
        }
        mbar_arrive_expect_tx(bar(L::B_QGFULL0 + g), L::kQg);
        load_tile<TG>(sb + L::oQg + g * L::kQg, tqg, bar(L::B_QGFULL0 + g), q0, h, b);
        issued = i + 1;
      }
      if (*abort_flag) {  // let the copies already started land before the CTA exits
        const uint64_t lim = 200000000ull;
        mbar_drain(bar(L::B_KFULL), 0, lim);
        if (issued > 0) mbar_drain(bar(L::B_QOFULL), (issued - 1) & 1, lim);
        for (int i = issued > L::kQgBufs ? issued - L::kQgBufs : 0; i < issued; ++i)
          mbar_drain(bar(L::B_QGFULL0 + i % L::kQgBufs), (i / L::kQgBufs) & 1, lim);
      }
    }
    if (lane == 0 && n <= 0) mbar_drain(bar(L::B_KFULL), 0, 200000000ull);  // no product to wait for it
  } else if (warp == 13) {
    // ---------------------------------------------------------------- S issuer
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);
      auto s_product = [&](auto tile, uint32_t d, uint32_t qs, uint32_t ks) {
        using T = decltype(tile);
        const uint64_t qd = T::desc_k(qs), kd = T::desc_k(ks);
#pragma unroll
        for (int kk = 0; kk < T::kD / 16; ++kk) {
          const uint32_t o = T::off_k(kk);
          mma_bf16_ss(1u, d, sdesc_add(qd, o), sdesc_add(kd, o), id_s, kk > 0);
        }
      };
      bool ok = n > 0 && mbar_wait_polled(bar_k, 0, ctl);
      for (int i = 0; ok && i < n; ++i) {
        if (!mbar_wait_polled(bar(L::B_SFREE), (i & 1) ^ 1, ctl)) break;
        if (!mbar_wait_polled(bar(L::B_QOFULL), i & 1, ctl)) break;
        tc_fence_after();
        // the other side first: its single Q buffer is released as early as possible
        if constexpr (kP2) s_product(T1{}, t_s1, sb + L::oQo, sb + L::oK1);
        else s_product(T2{}, t_s2, sb + L::oQo, sb + L::oK2);
        mma_commit(1u, bar(L::B_QOEMPTY));
        if (!mbar_wait_polled(bar(L::B_QGFULL0 + i % L::kQgBufs), (i / L::kQgBufs) & 1, ctl)) break;
        tc_fence_after();
        if constexpr (kP2) s_product(T2{}, t_s2, sb + L::oQg + (i % L::kQgBufs) * L::kQg, sb + L::oK2);
        else s_product(T1{}, t_s1, sb + L::oQg + (i % L::kQgBufs) * L::kQg, sb + L::oK1);
        mma_commit(1u, bar(L::B_SFULL));
        *s_queued = i + 1;
      }
      // every MMA of every issuer has finished before TMEM is released
      mma_commit(1u, bar(L::B_DONE));
      mbar_drain(bar(L::B_DONE), 0, 1000000000ull);
    }
  } else if (warp == 14 || warp == 15) {
    // ---------------------------------------------------------------- gradient issuers
    // warp 14: dK, and dQ too in mode P2; warp 15 (mode P1): dQ
    if (lane == 0) {
      const bool do_dk = warp == 14, do_dq = L::kSplitIssue ? warp == 15 : true;
      constexpr uint32_t id_dk = idesc_bf16(128, DG, 1, 1);  // A = dX^T M-major, B = Q_g N-major
      constexpr uint32_t id_dq = idesc_bf16(128, DG, 0, 1);  // A = dX K-major,   B = K_g N-major
      const uint64_t dsm = sdesc_sw128(sb + L::oDS, kTile * 128, 1024);
      const uint64_t dsk = sdesc_sw128(sb + L::oDS, 16, 1024);
      const uint64_t kgn = TG::desc_n(sb + (kP2 ? L::oK2 : L::oK1));
      int t = 0;
      if (n > 0 && mbar_wait_polled(bar_k, 0, ctl)) {
        for (; t < n; ++t) {
          if (!mbar_wait_polled(bar(L::B_DSFULL), t & 1, ctl)) break;
          wait_s_queued(s_queued, t + 1 < n ? t + 2 : 0);
          tc_fence_after();
          if (do_dk) {
            const uint64_t qgn = TG::desc_n(sb + L::oQg + (t % L::kQgBufs) * L::kQg);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_bf16_ss(1u, t_dk, sdesc_add(dsm, kk * 2048), sdesc_add(qgn, TG::off_n(kk)), id_dk,
                          (t > 0 || kk > 0) ? 1u : 0u);
            mma_commit(1u, bar(L::B_QGEMPTY0 + t % L::kQgBufs));  // Q_g(t) may be reloaded
          }
          if (do_dq) {
            if (!mbar_wait_polled(bar(L::B_DQEMPTY), (t & 1) ^ 1, ctl)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_bf16_ss(1u, t_dq, sdesc_add(dsk, (kk >> 2) * (kTile * 128) + (kk & 3) * 32),
                          sdesc_add(kgn, TG::off_n(kk)), id_dq, kk > 0 ? 1u : 0u);
          }
          mma_commit(1u, bar(L::B_DSEMPTY));
          if (do_dq) mma_commit(1u, bar(L::B_DQFULL));
        }
      }
      if (do_dk && n > 0 && t == n && !*abort_flag) mma_commit(1u, bar(L::B_DKFULL));
      mma_commit(1u, bar(L::B_DONE));  // the TMEM owner drains it before releasing TMEM
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- dX (thread = query row)
    // warpgroup wg takes key columns [64 wg, 64 wg + 64) of every tile
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const ModSide& so = kP2 ? a.s1 : a.s2;  // the other side
    const ModSide& sg = kP2 ? a.s2 : a.s1;  // the gradient side
    constexpr bool TAB = BIAS == kTable;
    HeadBias* hb = reinterpret_cast<HeadBias*>(smem + L::oBias);  // the other side's, then the gradient side's
    const SideRegs po = side_regs<CAP>(so), pg = side_regs<CAP>(sg);
    if (ids && n > 0) {
      // keys that match nothing: their K may hold anything and must not reach a product
      const bool pad = (tk.z == 0) && a.vis.ids_k[size_t(b) * nkt * kTile + k0 + row] < 0;
      bool ok = mbar_wait_warp(bar(L::B_KFULL), 0, ctl);
      if (ok) {
        if (pad && wg == 0) zero_row<T1>(sb + L::oK1, row);
        if (pad && wg == 1) zero_row<T2>(sb + L::oK2, row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ready);
      }
    }
    // the row's -LSE of both sides in base 2 (mode P1: KL with the other
    // side's) and its weights; a row that saw no key (ng = kUnseen, finite, so
    // that nothing below is a NaN) contributes exact zeros.
    // The table's gradient is a sum of differences of nearly equal sums, so
    // there (TAB) what the rounding of these and of a far tile's bias loses,
    // errors common to a whole row, goes back in: into the weights of the
    // exponentials, and in mode P1 into the difference of the two e
    auto params = [&](int i, float& ng, float& no, float& w, float& wo) {
      const int qi = (qt_lo + i) * kTile + row;
      ng = kUnseen;
      no = kP2 ? kUnseen : 0.f;
      w = wo = 0.f;
      if (qi < a.NQ && SKL_CHECK(a.status, bh < a.B * a.H)) {
        const size_t idx = size_t(bh) * a.NQ + qi;
        const float l1 = a.lse1[idx], l2 = a.lse2[idx];
        if (l1 != -INFINITY) {
          w = a.dkl[idx];
          if (kP2) {
            ng = -l2 * kLog2e;
            no = -l1 * kLog2e;
            wo = -w;
            if (TAB) {
              w *= exp2_small(log2e_lost(-l2, ng));
              wo *= exp2_small(log2e_lost(-l1, no));
            }
          } else {
            const float kl = a.kl[idx], d = kl - l2;
            ng = -l1 * kLog2e;
            no = d * kLog2e;
            w *= kLn2;
            if (TAB) {
              const float back = d + l2, lost = (kl - back) + (back - d - l2);  // of the subtraction
              const float g = log2e_lost(-l1, ng);
              w *= exp2_small(g);
              wo = g - (log2e_lost(d, no) + lost * kLog2e);
            }
          }
        }
      }
    };
    const float capf = sg.carg != 0.f ? -sg.scale / (sg.cmul * sg.cmul) : 0.f;
    float* sums = TAB ? a.dtab + ((size_t(bh) * nkt + kt) * 8 + warp) * kMaxBuckets : nullptr;
    float left = 0.f, right = 0.f;  // this thread's dS beyond the table's reach
    float ng, no, w, wo;
    if (n > 0) params(0, ng, no, w, wo);
    for (int i = 0; i < n; ++i) {
      const int q0 = (qt_lo + i) * kTile;
      const int qi = q0 + row;
      DsParams p{sg.cmul, sg.scale, capf, w, wo};
      const float cng = ng, cno = no;
      if (i + 1 < n) params(i + 1, ng, no, w, wo);  // used next tile: the loads overlap this one
      const int rmin = k0 - (q0 + kTile - 1 + off), rmax = rmin + 2 * kTile - 2;
      const bool same = !ids || tiles_same(tk, a.vis.tiles_q[size_t(b) * nqt + qt_lo + i]);
      // a warp with a row that saw no key masks it: 0 times what such a row
      // holds need not be 0
      const bool need_mask = (k0 + kTile > a.NK) || (q0 + kTile > a.NQ) || !same ||
                             (a.vis.causal && rmax > 0 && k0 + kTile > prefix) ||
                             __any_sync(0xffffffffu, cng == kUnseen);
      const int r0 = k0 + wg * 64 - (qi + off);
      TileBias tbo{kZero, 0.f, 0.f}, tbg = tbo;
      RowBias rbo{0.f, 0.f, cno, cno, nullptr}, rbg{0.f, 0.f, cng, cng, nullptr};
      if (BIAS != kNoBias) {
        tbo = tile_bias(hb[0], rmin, rmax);
        tbg = tile_bias(hb[1], rmin, rmax);
        rbo = row_bias(hb[0], tbo, r0, cno);
        rbg = row_bias(hb[1], tbg, r0, cng);
        if (TAB) {
          const float lg = flat_lost(hb[1], tbg, rbg, rmax), lo = flat_lost(hb[0], tbo, rbo, rmax);
          p.w *= exp2_small(lg);
          if (kP2) p.wo *= exp2_small(lo);
          else p.wo += lg - lo;
        }
      }
      const uint32_t tg = (kP2 ? t_s2 : t_s1) + lane_off + wg * 64, to = (kP2 ? t_s1 : t_s2) + lane_off + wg * 64;
      const uint32_t row_addr = sb + L::oDS + wg * (kTile * 128) + (row >> 3) * 1024 + (row & 7) * 128;
      if (!mbar_wait_warp(bar(L::B_SFULL), i & 1, ctl)) break;
      tc_fence_after();
      auto release_s = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_SFREE));
      };
      // the sums over diagonals of a 32 x 32 block that begins at this row
      // group's column col: lane l holds diagonal 31 - l in acc, -1 - l in
      // done; diagonal d is relative position d + rd
      auto diagonals = [&](int col, float acc, float done) {
        const int rd = k0 + wg * 64 + col - (q0 + (warp & 3) * 32 + off);
        const int* bm = a.bmap + a.reach + kNearPad + rd;
        add_to_buckets(sums, acc, __ldg(bm + 31 - lane), lane);
        add_to_buckets(sums, done, lane < 31 ? __ldg(bm - 1 - lane) : -1, lane);
      };
      if (!need_mask && tbo.how != kFold && tbg.how != kFold) {
        // every column visible: dX in registers, so that the products of the
        // previous tile may still read its dX
        uint32_t dsr[32];
        float total = 0.f, acc = 0.f, done = 0.f;
        auto tile = [&](auto how_o, auto how_g) {
          constexpr int kHowO = decltype(how_o)::value, kHowG = decltype(how_g)::value;
          constexpr int kTab = TAB ? (kHowG == kLook ? 2 : 1) : 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint64_t yg[8], eo[8];
            load_scores<CAP, BIAS != kNoBias, false, kHowO>(tg + 16 * c, to + 16 * c, yg, eo, sg, so, pg, po, kHowO,
                                                            rbo, 0u);
            if (c == 3) release_s();
            dx_chunk<MODE, CAP, kHowG, kTab, false>(yg, eo, p, rbg, 0u, lane, dsr + 8 * c, total, acc, done);
            if (kTab == 2 && (c & 1)) {
              diagonals(16 * (c - 1), acc, done);
              acc = done = 0.f;
            }
            if (BIAS != kNoBias) {
              rbo = further(rbo, 16);
              rbg = further(rbg, 16);
            }
          }
        };
        if constexpr (BIAS == kNoBias) {
          tile(Int<kZero>{}, Int<kZero>{});
        } else {
          if (tbg.how == kLook) {
            if (tbo.how == kLook) tile(Int<kLook>{}, Int<kLook>{});
            else tile(Int<kFlat>{}, Int<kLook>{});
          } else {
            if (tbo.how == kLook) tile(Int<kLook>{}, Int<kFlat>{});
            else tile(Int<kFlat>{}, Int<kFlat>{});
          }
        }
        if (TAB && tbg.how != kLook) (rmax <= -a.reach ? left : right) += total;
        if (!mbar_wait_warp(bar(L::B_DSEMPTY), (i & 1) ^ 1, ctl)) break;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(row_addr + ((c ^ (row & 7)) << 4), dsr[4 * c], dsr[4 * c + 1], dsr[4 * c + 2], dsr[4 * c + 3]);
      } else {
        // the others go to shared memory as they come, behind the products
        // of the previous tile
        if (!mbar_wait_warp(bar(L::B_DSEMPTY), (i & 1) ^ 1, ctl)) break;
        const int id = same ? 0 : a.vis.ids_q[size_t(b) * nqt * kTile + qi];
        float total = 0.f, acc = 0.f, done = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t bits = 0xffffu;
          if (need_mask)
            bits = cng == kUnseen
                       ? 0u
                       : visible_bits<16>(qi, k0 + wg * 64 + 16 * c, off, a.NK, a.vis.causal, prefix, id,
                                          same ? nullptr : a.vis.ids_k + size_t(b) * nkt * kTile + k0 + wg * 64 + 16 * c);
          uint64_t yg[8], eo[8];
          load_scores<CAP, BIAS != kNoBias, true, kZero>(tg + 16 * c, to + 16 * c, yg, eo, sg, so, pg, po, tbo.how, rbo, bits);
          if (c == 3) release_s();
          uint32_t o[8];
          if constexpr (BIAS == kNoBias) {
            dx_chunk<MODE, CAP, kZero, 0, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
          } else if constexpr (TAB) {
            if (tbg.how == kLook) dx_chunk<MODE, CAP, kLook, 2, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
            else dx_chunk<MODE, CAP, kFlat, 1, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
            if (tbg.how == kLook && (c & 1)) {
              diagonals(16 * (c - 1), acc, done);
              acc = done = 0.f;
            }
          } else {
            if (tbg.how == kZero) dx_chunk<MODE, CAP, kZero, 0, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
            else if (tbg.how == kFlat) dx_chunk<MODE, CAP, kFlat, 0, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
            else if (tbg.how == kFold) dx_chunk<MODE, CAP, kFold, 0, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
            else dx_chunk<MODE, CAP, kLook, 0, true>(yg, eo, p, rbg, bits, lane, o, total, acc, done);
          }
          st_shared_v4(row_addr + (((2 * c) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          st_shared_v4(row_addr + (((2 * c + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
          if (BIAS != kNoBias) {
            rbo = further(rbo, 16);
            rbg = further(rbg, 16);
          }
        }
        if (TAB && tbg.how != kLook) (rmax <= -a.reach ? left : right) += total;
        // queries that saw no key or match nothing: their Q_g may hold anything
        // (its S product is done, its dK product waits for this tile's dX)
        if (wg == 0 && (cng == kUnseen || (!same && id < 0))) zero_row<TG>(sb + L::oQg + (i % L::kQgBufs) * L::kQg, row);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::B_DSFULL));
    }
    if constexpr (TAB) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        left += __shfl_xor_sync(0xffffffffu, left, o);
        right += __shfl_xor_sync(0xffffffffu, right, o);
      }
      __syncwarp();
      if (lane == 0) atomicAdd(sums + a.bmap[0], left);
      __syncwarp();
      if (lane == 0) atomicAdd(sums + a.bmap[near_len(a.reach) - 1], right);
    }
  } else {
    // ---------------------------------------------------------------- dQ / dK epilogue
    const int w4 = warp - 8;
    const int row = w4 * 32 + lane;
    const uint32_t lane_off = uint32_t(w4 * 32) << 16;
    {
      // the dQ tile leaves in boxes of 32 rows x 32 fp32 (128-byte swizzle)
      // through kDqBoxes staging boxes per warp, each a bulk reduce-add; in
      // the deterministic mode every value is first rounded to its row's grid
      constexpr int kChunks = DG / 32;
      const uint32_t stage = sb + L::oStage + w4 * (kDqBoxes * kDqBoxBytes);
      int nred = 0;
      if (lane == 0) tma_prefetch_desc(&tdq);
      const bool fixed = a.dq_fixed != 0;
      const float sgs = kP2 ? a.s2.scale : a.s1.scale;
      const float kmax = fixed ? __uint_as_float(a.kmax[bh / gg] << 16) : 0.f;
      float dkl_nx = 0.f, kl_nx = 0.f;
      // row `lane` of 32 rows x 32 columns, reduce-added at (x, y, z)
      auto push_box = [&](const CUtensorMap* map, const uint32_t (&v)[32], int x, int y, int z) {
        const uint32_t box = stage + (nred % kDqBoxes) * kDqBoxBytes;
        if (!SKL_CHECK(a.status, box + kDqBoxBytes <= sb + L::oBar)) return;
        if (lane == 0) bulk_wait_read_le<kDqBoxes - 1>();  // the box used kDqBoxes reduces ago has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_reduce_add_3d(map, box, x, y, z);
          bulk_commit();
        }
        ++nred;
      };
      auto load_row = [&](int i) {
        const int qi = (qt_lo + i) * kTile + row;
        dkl_nx = kl_nx = 0.f;
        if (fixed && qi < a.NQ && SKL_CHECK(a.status, bh < a.B * a.H)) {
          const size_t idx = size_t(bh) * a.NQ + qi;
          dkl_nx = a.dkl[idx];
          kl_nx = a.kl[idx];
        }
      };
      auto to_fixed = [&](uint32_t (&x)[32], uint64_t ME) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float v0, v1;
          f2_split(f2_sub(f2_add(f2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), ME), ME), v0, v1);
          x[j] = __float_as_uint(v0);
          x[j + 1] = __float_as_uint(v1);
        }
      };
      if (n > 0) load_row(0);
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait_warp(bar(L::B_DQFULL), i & 1, ctl)) break;
        tc_fence_after();
        const int r0 = (qt_lo + i) * kTile + w4 * 32;  // first query row of this warp
        const float me = fixed ? 1.5f * exp2_int(23 - dq_fixed_exp(MODE, sgs, dkl_nx, kl_nx, kmax)) : 0.f;
        const uint64_t ME = f2(me, me);
        if (i + 1 < n) load_row(i + 1);
        uint32_t v[kChunks][32];
        // nothing to add past the row length or past NQ, and then no box is
        // touched (the box count must match the committed reduce groups)
        auto put_box = [&](int c0) {
          if (c0 * 32 < a.pitch && r0 < a.NQ) push_box(&tdq, v[c0], c0 * 32, r0, bh);
        };
        if constexpr (kChunks == 4) {
          tmem_ld2x32(t_dq + lane_off, t_dq + lane_off + 32, v[0], v[1]);
          tmem_ld32(t_dq + lane_off + 64, v[2]);
          if (fixed) to_fixed(v[0], ME);
          put_box(0);
          tmem_ld32(t_dq + lane_off + 96, v[3]);
        } else {
          tmem_ld2x32(t_dq + lane_off, t_dq + lane_off + 32, v[0], v[1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_DQEMPTY));
#pragma unroll
        for (int c = kChunks == 4 ? 1 : 0; c < kChunks; ++c) {
          if (fixed) to_fixed(v[c], ME);
          put_box(c);
        }
      }
      // dK of a key head that other CTAs add to as well, any order: the same boxes
      if (a.dk32 != nullptr && a.dk_turns == nullptr && n > 0 && mbar_wait_warp(bar(L::B_DKFULL), 0, ctl)) {
        tc_fence_after();
        const int r0 = k0 + w4 * 32;
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
          if (ch * 32 >= a.pitch || r0 >= a.NK) break;
          uint32_t v[32];
          tmem_ld32(t_dk + lane_off + ch * 32, v);
          push_box(&tdk, v, ch * 32, r0, bh / gg);
        }
      }
      if (lane == 0) bulk_wait_all();  // every reduce has landed before the CTA exits
    }
    // dK otherwise: bf16 where this CTA owns it, or, deterministic with
    // shared key heads, fp32 into the workspace in head order
    const int kj = k0 + row;
    const int hk = bh / gg;
    float* dst32 = a.dk32 + (size_t(hk) * a.NK + kj) * a.pitch;
    __nv_bfloat16* dst16 = static_cast<__nv_bfloat16*>(a.dk) + (long long)b * a.dk_sb +
                           (long long)(h / gg) * a.dk_sh + (long long)kj * a.dk_sn;
    auto write_dk = [&](int how, bool zero) {
#pragma unroll 1
      for (int ch = 0; ch < DG / 32; ++ch) {
        uint32_t v[32];
        if (zero) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        } else {
          tmem_ld32(t_dk + lane_off + ch * 32, v);
        }
        if (kj >= a.NK || ch * 32 >= a.dg || !SKL_CHECK(a.status, hk < a.B * (a.H / gg))) continue;
        if (a.dk32 != nullptr) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            put_dk4(dst32 + ch * 32 + e,
                    make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]),
                                __uint_as_float(v[e + 3])),
                    how);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (ch * 32 + e < a.dg) {
              uint4 o;
              o.x = pack_bf16(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              o.y = pack_bf16(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
              o.z = pack_bf16(__uint_as_float(v[e + 4]), __uint_as_float(v[e + 5]));
              o.w = pack_bf16(__uint_as_float(v[e + 6]), __uint_as_float(v[e + 7]));
              *reinterpret_cast<uint4*>(dst16 + ch * 32 + e) = o;
            }
          }
        }
      }
    };
    if (a.dk32 == nullptr) {
      if (n > 0 && mbar_wait_warp(bar(L::B_DKFULL), 0, ctl)) {
        tc_fence_after();
        write_dk(kDkStore, false);
      } else if (n == 0) {
        write_dk(kDkStore, true);  // no query row sees this key tile
      }
    } else if (a.dk_turns != nullptr) {
      // deterministic, grouped key heads: head m of a group waits until the
      // (key head, key tile) count reads m, then stores (m = 0) or adds
      const int member = bh % gg;
      int* turn = a.dk_turns + size_t(hk) * nkt + kt;
      const bool have = n > 0 && mbar_wait_warp(bar(L::B_DKFULL), 0, ctl);
      if (warp == 8 && lane == 0) *turn_ok = wait_turn(turn, member, a.dk_abort, ctl) ? 1 : 0;
      named_bar_sync(1, 128);
      if (*turn_ok) {
        if (have) {
          tc_fence_after();
          write_dk(member == 0 ? kDkStore : kDkAdd, false);
        } else if (n == 0 && member == 0) {
          write_dk(kDkStore, true);
        }
      }
      named_bar_sync(1, 128);
      if (warp == 8 && lane == 0) {
        if (*turn_ok && !*abort_flag) {
          __threadfence();
          st_release_gpu(turn, member + 1);
        } else {
          atomicExch(a.dk_abort, 1);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D1, int D2, int MODE, bool CAP, int BIAS>
int launch_bwd_mod_k(const ModMaps& m, const ModBwdArgs& a, cudaStream_t st) {
  using L = ModBwdLayout<D1, D2, MODE>;
  auto kern = bwd_mod_kernel<D1, D2, MODE, CAP, BIAS>;
  ModBwdArgs b = a;
  const size_t near = BIAS != kNoBias ? near_smem_bytes(a.s1, a.s2, 1) : 0;
  b.near_smem = near > 0 && L::kAlloc + near <= 232448;
  const int bytes = int(L::kAlloc + (b.near_smem ? near : 0));
  // (always the most a block may have: threads that launch at once would set each other's size)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e != cudaSuccess) return e;
  dim3 grid((a.NK + kTile - 1) / kTile, a.B * a.H);
  kern<<<grid, L::kThreads, bytes, st>>>(m.q1, m.k1, m.q2, m.k2, m.dq, m.dk, b);
  return cudaGetLastError();
}

template <int D1, int D2, int MODE>
int launch_bwd_mod_t(const ModMaps& m, const ModBwdArgs& a, cudaStream_t st) {
  const bool cap = a.s1.carg != 0.f || a.s2.carg != 0.f;
  if (a.dtab != nullptr)
    return cap ? launch_bwd_mod_k<D1, D2, MODE, true, kTable>(m, a, st)
               : launch_bwd_mod_k<D1, D2, MODE, false, kTable>(m, a, st);
  if (a.s1.kind != kBiasNone || a.s2.kind != kBiasNone)
    return cap ? launch_bwd_mod_k<D1, D2, MODE, true, kBias>(m, a, st)
               : launch_bwd_mod_k<D1, D2, MODE, false, kBias>(m, a, st);
  return cap ? launch_bwd_mod_k<D1, D2, MODE, true, kNoBias>(m, a, st)
             : launch_bwd_mod_k<D1, D2, MODE, false, kNoBias>(m, a, st);
}

template <int MODE>
int launch_bwd_mod_mode(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st) {
  if (d1 == 64) return d2 == 64 ? launch_bwd_mod_t<64, 64, MODE>(m, a, st) : launch_bwd_mod_t<64, 128, MODE>(m, a, st);
  return d2 == 64 ? launch_bwd_mod_t<128, 64, MODE>(m, a, st) : launch_bwd_mod_t<128, 128, MODE>(m, a, st);
}

}  // namespace skl
