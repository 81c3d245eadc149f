// Forward over selected blocks (sel_common.cuh): the sums of every (row, block)
// pair, then their merge into KL, LSE1 and LSE2.
//
// Persistent CTAs walk their lists: K1, K2 of the list's block once, then tiles
// of 128 gathered rows, a side's tile at a time, through a ring of slots.  19 warps:
//   warps 0-11  statistics: a warpgroup takes every third tile; thread = row
//   warps 12-15 gather 32 rows each, 16 bytes a lane (cp.async).  TMA takes
//               some 50 clocks for a copy of few rows, whatever its form: at
//               rows of 256 bytes out of L2 its gather of four reached 2.5
//               TB/s, cp.async 19.5 (64 bytes of 8 rows at a time, as here;
//               20.5 with whole rows; of 4 and 8 warps alike).
//   warp 16     S1 = Q1 K1^T, S2 = Q2 K2^T into one of 4 TMEM buffers (2 for blocks of 128)
//   warp 17     K by TMA
//   warp 18     tells the others what to take (SelShare)
// A row's keys in one block are few, so its references are its own largest
// scores there (one more read of TMEM), and nothing is rescaled:
//   e_t = S_t log2 e - m_t,  l_t = sum 2^e_t,  acc = sum 2^e1 (e1 - e2).
// The merge adds the parts of a row's slots in their order (as merge_stats of
// the dense forward does for splits), so results do not depend on which CTA
// took which list.
#include "fwd_mod.cuh"
#include "sel_common.cuh"

namespace skl {

namespace {

struct SelFwdLayout {
  static constexpr int kWGs = 3;  // of statistics
  static constexpr int kGatherWarp = 4 * kWGs, kGatherWarps = 4;
  static constexpr int kMmaWarp = kGatherWarp + kGatherWarps, kLoadWarp = kMmaWarp + 1, kWalkWarp = kMmaWarp + 2;
  static constexpr int kThreads = 32 * (kWalkWarp + 1);
  static constexpr int kMaxSlots = 8;
  // k_full[2], k_empty[2], q_full[8], q_empty[8], s_full[12], s_empty[4], done, shares.  (A warpgroup waits for every
  // phase of the barriers that it waits for: each belongs to one warpgroup and one buffer of S.)
  static constexpr int kTurns = 12;
  static_assert(kTurns % kWGs == 0 && kTurns % 4 == 0, "a turn is of one warpgroup and one buffer");
  static constexpr int kKFull = 0, kKEmpty = 2, kQFull = 4, kQEmpty = 12, kSFull = 20, kSEmpty = kSFull + kTurns,
                       kDone = kSEmpty + 4, kTold = kDone + 1;
  static constexpr int kNumBars = (kTold + 2 * kShares + 1) / 2 * 2;  // (16-byte words behind them)
  static_assert(kNumBars % 2 == 0, "shares are aligned");
  static constexpr uint32_t kTail = kNumBars * 8 + kShares * sizeof(SelShare) + 16;
  static constexpr uint32_t kMost = 232448;
  static constexpr uint32_t slot_bytes(int d1, int d2) { return uint32_t(d1 > d2 ? d1 : d2) * 2u * kTile; }
  static uint32_t bytes(int slots, int k_bufs, int d1, int d2, int bs) {
    return 1024u + slots * slot_bytes(d1, d2) + uint32_t(d1 + d2) * 2u * uint32_t(k_bufs * bs) + kTail;
  }
};

// One row's sums over its block: n visible of the bs columns at ts, ts + bs.
template <bool MASK>
__device__ __forceinline__ void block_sums(uint32_t ts, int bs, float c1, float c2, int i, int k0, const SelFwdArgs& a,
                                           int prefix, int id, const int* kids, ModStats& st) {
  const int off = a.p.NK - a.p.NQ;
  float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < bs; c += 16) {
    uint32_t x1[16], x2[16];
    tmem_ld2x16(ts + c, ts + bs + c, x1, x2);
    uint32_t on = 0xffffffffu;
    if (MASK) on = visible_bits<16>(i, k0 + c, off, a.p.NK, a.p.causal, prefix, id, kids == nullptr ? nullptr : kids + c);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      float u = __uint_as_float(x1[k]), v = __uint_as_float(x1[k + 1]);
      float w = __uint_as_float(x2[k]), z = __uint_as_float(x2[k + 1]);
      if (MASK) {
        if (!((on >> k) & 1u)) u = w = -INFINITY;
        if (!((on >> (k + 1)) & 1u)) v = z = -INFINITY;
      }
      t1 = max3(t1, u, v);
      t2 = max3(t2, w, z);
    }
  }
  const float m1 = rintf(t1 * c1), m2 = rintf(t2 * c2);
  const uint64_t C1 = f2(c1, c1), C2 = f2(c2, c2), M1 = f2(-m1, -m1), M2 = f2(-m2, -m2);
  ChunkSums s{};
#pragma unroll 1
  for (int c = 0; c < bs; c += 16) {
    uint32_t x1[16], x2[16];
    uint64_t e1[8], e2[8];
    tmem_ld2x16(ts + c, ts + bs + c, x1, x2);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      e1[k / 2] = f2_fma(f2(__uint_as_float(x1[k]), __uint_as_float(x1[k + 1])), C1, M1);
      e2[k / 2] = f2_fma(f2(__uint_as_float(x2[k]), __uint_as_float(x2[k + 1])), C2, M2);
    }
    if (MASK)
      mask_scores(e1, e2, visible_bits<16>(i, k0 + c, off, a.p.NK, a.p.causal, prefix, id, kids == nullptr ? nullptr : kids + c));
    sums_all(e1, e2, s);
  }
  st = ModStats{m1, m2, sum2(s.l1a, s.l1b), sum2(s.l2a, s.l2b), sum2(s.aa, s.ab)};
}

template <int D1, int D2>
__global__ void __launch_bounds__(SelFwdLayout::kThreads, 1)
    sel_fwd_kernel(const __grid_constant__ CUtensorMap tk1, const __grid_constant__ CUtensorMap tk2,
                   const __grid_constant__ SelFwdArgs a) {
  using L = SelFwdLayout;
  constexpr uint32_t kSlot = L::slot_bytes(D1, D2);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = a.p.bs;
  const uint32_t kK1 = uint32_t(bs) * D1 * 2, kK = uint32_t(bs) * (D1 + D2) * 2;
  const uint32_t oQ = a.k_bufs * kK, oBar = oQ + a.slots * kSlot;
  auto bar = [&](int id) { return sb + oBar + 8u * id; };
  SelShare* shares = reinterpret_cast<SelShare*>(smem + oBar + L::kNumBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shares + kShares);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const Ctl ctl{abort_flag, a.status};
  const int bufs = bs == 128 ? 2 : 4;  // of S1, S2 in TMEM, bs columns each
  const uint32_t told = sb + oBar + 8u * L::kTold;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      int count = 1;
      if (i >= L::kQFull && i < L::kQEmpty) count = 32 * L::kGatherWarps;
      if (i >= L::kSEmpty && i < L::kDone) count = 4;  // the warps of a warpgroup
      if (i >= L::kTold + kShares) count = L::kWalkWarp;  // the warps before it
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // columns past the head dim (K's are zeros, and no product may meet a NaN there; slots_of_sides keeps them so)
  if (a.r1.chunks < D1 / 8 || a.r2.chunks < D2 / 8)
    for (uint32_t o = threadIdx.x * 16; o < a.slots * kSlot; o += L::kThreads * 16) st_shared_v4(sb + oQ + o, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int per_tile = a.p.queries_per_tile, G = a.p.G;

  if (warp >= L::kGatherWarp && warp < L::kMmaWarp) {
    // ---------------------------------------------------------------- gather: rows [first, first + 32)
    const int first = (warp - L::kGatherWarp) * 32;
    const int r = first + lane, ql = r / G, hl = r - ql * G;
    const bool place = ql < per_tile;
    int s = 0, m = 0;  // the slot, and how often the ring has been round
    bool ok = true;
    SelReader share(shares, told);
    const uint8_t *b1 = nullptr, *b2 = nullptr;  // the lane's row 0 of both sides
    auto enter = [&]() {
      if (!share.next(ctl)) return false;
      b1 = a.r1.at(share.b, share.head0 + hl, 0);
      b2 = a.r2.at(share.b, share.head0 + hl, 0);
      return true;
    };
    bool more = enter();
    int e0 = 0;
    unsigned ent = entry_of(a.p, share, ql, place);
    while (ok && more) {
      // (rows past the last are not read: what the slot holds there gives scores that nobody takes)
      const int i = int(ent >> kSlotBits);
      const unsigned long long p1 = ent != kNoEntry ? reinterpret_cast<unsigned long long>(b1 + i * a.r1.sn) : 0ull;
      const unsigned long long p2 = ent != kNoEntry ? reinterpret_cast<unsigned long long>(b2 + i * a.r2.sn) : 0ull;
      e0 += per_tile;
      if (e0 >= share.count) {
        more = enter();
        e0 = 0;
      }
      ent = entry_of(a.p, share, e0 + ql, place);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        ok = mbar_wait_warp(bar(L::kQEmpty + s), (m & 1) ^ 1, ctl);
        if (!ok) break;
        if (side == 0) gather_rows<D1, false>(sb + oQ + s * kSlot, first, p1, a.r1);
        else gather_rows<D2, false>(sb + oQ + s * kSlot, first, p2, a.r2);
        cp_async_arrive(bar(L::kQFull + s));
        if (++s == a.slots) s = 0, ++m;
      }
    }
    cp_async_wait_all();
  } else if (warp >= L::kMmaWarp) {
    if (warp == L::kWalkWarp) {
      tell_shares(a.p, shares, told, ctl);
    } else if (warp == L::kLoadWarp) {
      // -------------------------------------------------------------- K
      int kept = 0;
      for (SelReader share(shares, told); share.next(ctl); ++kept) {
        const int kb = kept % a.k_bufs, hu = share.head0 / G;
        if (!mbar_wait_warp(bar(L::kKEmpty + kb), ((kept / a.k_bufs) & 1) ^ 1, ctl)) break;
        if (lane != 0) continue;
        const uint32_t full = bar(L::kKFull + kb);
        mbar_arrive_expect_tx(full, kK);
#pragma unroll
        for (int c = 0; c < D1 / 64; ++c)
          tma_load_4d(sb + kb * kK + c * (bs * 128), &tk1, full, c * 64, share.block * bs, hu / a.u1, share.b);
#pragma unroll
        for (int c = 0; c < D2 / 64; ++c)
          tma_load_4d(sb + kb * kK + kK1 + c * (bs * 128), &tk2, full, c * 64, share.block * bs, hu / a.u2, share.b);
      }
      if (*abort_flag && lane == 0)  // let the copies already started land before the CTA exits
        for (int j = kept > a.k_bufs ? kept - a.k_bufs : 0; j < kept; ++j)
          mbar_drain(bar(L::kKFull + j % a.k_bufs), (j / a.k_bufs) & 1, 200000000ull);
    } else if (warp == L::kMmaWarp) {
      // -------------------------------------------------------------- MMA issuer
      const uint32_t leader = elect_one();
      const uint32_t idesc = idesc_bf16(128, bs, 0, 0);
      const uint32_t dhi = uint32_t(sdesc_sw128(0, 16, 1024) >> 32), dlo = uint32_t(sdesc_sw128(0, 16, 1024));
      int n = 0, s = 0, m = 0, kept = 0;
      bool ok = true;
      // S of one side: the tile in slot s by K at ks
      auto product = [&](auto width, uint32_t d, uint32_t ks) {
        constexpr int D = decltype(width)::value;
        ok = mbar_wait_warp(bar(L::kQFull + s), m & 1, ctl);
        if (!ok) return;
        fence_proxy_async_smem();  // (copies of cp.async)
        tc_fence_after();
        const uint32_t q = dlo + ((sb + oQ + s * kSlot) >> 4), kd = dlo + (ks >> 4), half = bs * 8;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_step(leader, d, q + (kk >> 2) * (kTile * 8) + (kk & 3) * 2, dhi, kd + (kk >> 2) * half + (kk & 3) * 2, dhi, idesc,
                   kk > 0);
        mma_commit(leader, bar(L::kQEmpty + s));
        if (++s == a.slots) s = 0, ++m;
      };
      for (SelReader share(shares, told); ok && share.next(ctl); ++kept) {
        const int kb = kept % a.k_bufs;
        ok = mbar_wait_warp(bar(L::kKFull + kb), (kept / a.k_bufs) & 1, ctl);
        for (int e0 = 0; ok && e0 < share.count; e0 += per_tile, ++n) {
          const int i = n & (bufs - 1);
          const uint32_t d1 = tmem + uint32_t(i * 2 * bs);
          ok = mbar_wait_warp(bar(L::kSEmpty + i), ((n / bufs) & 1) ^ 1, ctl);
          if (ok) product(std::integral_constant<int, D1>{}, d1, sb + kb * kK);
          if (ok) product(std::integral_constant<int, D2>{}, d1 + uint32_t(bs), sb + kb * kK + kK1);
          if (ok) mma_commit(leader, bar(L::kSFull + n % L::kTurns));
        }
        if (ok) mma_commit(leader, bar(L::kKEmpty + kb));
      }
      mma_commit(leader, bar(L::kDone));  // every MMA has finished before TMEM is released
      mbar_drain(bar(L::kDone), 0, 1000000000ull);
    }
  } else {
    // ---------------------------------------------------------------- statistics
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const int ql = row / G, hl = row - ql * G;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const float c1 = a.scale1 * kLog2e, c2 = a.scale2 * kLog2e;
    const int nqt = (a.p.NQ + kTile - 1) / kTile, nkt = (a.p.NK + kTile - 1) / kTile;
    const int off = a.p.NK - a.p.NQ;
    const bool place = ql < per_tile;
    SelReader share(shares, told);
    int e0 = 0, n = wg;
    bool more = share.next(ctl);
    // to this warpgroup's next tile; whether that is of another share
    auto skip = [&](int tiles) {
      bool other = false;
      for (e0 += tiles * per_tile; more && e0 >= share.count; other = true) {
        e0 -= (share.count + per_tile - 1) / per_tile * per_tile;
        more = share.next(ctl);
      }
      return other;
    };
    skip(wg);
    unsigned ent = entry_of(a.p, share, e0 + ql, place);
    size_t first = 0;  // record of the row's query 0
    int prefix = 0, b = 0, k0 = 0;
    for (bool other = true, here = more; here; here = more) {
      if (other) {
        b = share.b;
        k0 = share.block * bs;
        first = size_t(b * a.p.H + share.head0 + hl) * a.p.NQ * a.p.T;
        if (a.p.prefix != nullptr) prefix = min(max(a.p.prefix[b], 0), a.p.NK);
      }
      const int buf = n & (bufs - 1);
      const bool on = ent != kNoEntry;
      const int i = on ? int(ent >> kSlotBits) : 0, t = int(ent & ((1u << kSlotBits) - 1u));
      other = skip(L::kWGs);
      ent = entry_of(a.p, share, e0 + ql, place);
      int id = 0;
      const int* kids = nullptr;
      if (a.vis.ids_q != nullptr) {
        id = a.vis.ids_q[size_t(b) * nqt * kTile + i];
        kids = a.vis.ids_k + size_t(b) * nkt * kTile + k0;
      }
      const int last = a.p.causal ? min(max(i + off + 1, prefix), a.p.NK) : a.p.NK;
      const bool whole = __all_sync(0xffffffffu, !on || last >= k0 + bs) && kids == nullptr;
      const bool idle = __all_sync(0xffffffffu, !on);
      if (!mbar_wait_warp(bar(L::kSFull + n % L::kTurns), (n / L::kTurns) & 1, ctl)) break;
      tc_fence_after();
      ModStats st{0.f, 0.f, 0.f, 0.f, 0.f};
      if (!idle) {
        const uint32_t ts = tmem + lane_off + uint32_t(buf * 2 * bs);
        if (whole) block_sums<false>(ts, bs, c1, c2, i, k0, a, prefix, id, kids, st);
        else block_sums<true>(ts, bs, c1, c2, i, k0, a, prefix, id, kids, st);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kSEmpty + buf));
      const size_t at = first + size_t(i) * a.p.T + t;
      if (on && SKL_CHECK(a.status, i < a.p.NQ && t < a.p.T && b < a.p.B)) {
        // a row that ids hide the whole block from has sums of 2^(-3e38 - ...) = 0, relative to nothing
        const bool none = st.m1 == -INFINITY && st.l1 == 0.f;
        a.rec[at] = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(st.m1, st.m2, st.l1, st.l2);
        a.acc[at] = none ? 0.f : st.acc;
      }
      n += L::kWGs;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kMergeThreads = 256, kMergeLanes = 4;

// Four lanes a row, each with every fourth slot, joined pairwise.
__global__ void __launch_bounds__(kMergeThreads) sel_merge_kernel(const __grid_constant__ SelFwdArgs a) {
  const long long rows = (long long)a.p.B * a.p.H * a.p.NQ;
  const long long r = ((long long)blockIdx.x * kMergeThreads + threadIdx.x) / kMergeLanes;
  const int part = threadIdx.x % kMergeLanes;
  const long long row = r < rows ? r : rows - 1;  // (whole warps take part)
  const int bh = int(row / a.p.NQ), i = int(row - (long long)bh * a.p.NQ), b = bh / a.p.H, h = bh - b * a.p.H;
  const int sel = b * a.p.HS + h / (a.p.H / a.p.HS);
  const unsigned* slots = a.p.slots + (size_t(sel) * a.p.NQ + i) * a.p.words;
  ModStats st{0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 4;
  for (int t0 = part; t0 < a.p.T; t0 += kAhead * kMergeLanes) {
    // (slots that do not count were not written: read, but not looked at)
    float4 v[kAhead];
    float acc[kAhead];
    bool on[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int t = t0 + x * kMergeLanes;
      on[x] = t < a.p.T && ((slots[t >> 5] >> (t & 31)) & 1u);
      if (t < a.p.T) {
        v[x] = __ldcs(a.rec + row * a.p.T + t);
        acc[x] = __ldcs(a.acc + row * a.p.T + t);
      }
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const ModStats o{v[x].x, v[x].y, v[x].z, v[x].w, acc[x]};
      if (!on[x] || o.l1 == 0.f) continue;
      if (st.l1 == 0.f) st = o;
      else merge_stats(st, o);
    }
  }
#pragma unroll
  for (int d = 1; d < kMergeLanes; d *= 2) {
    ModStats o;
    o.m1 = __shfl_xor_sync(0xffffffffu, st.m1, d);
    o.m2 = __shfl_xor_sync(0xffffffffu, st.m2, d);
    o.l1 = __shfl_xor_sync(0xffffffffu, st.l1, d);
    o.l2 = __shfl_xor_sync(0xffffffffu, st.l2, d);
    o.acc = __shfl_xor_sync(0xffffffffu, st.acc, d);
    if (part & d) {  // the same sums in both lanes of a pair
      const ModStats x = st;
      st = o;
      o = x;
    }
    if (o.l1 == 0.f) continue;
    if (st.l1 == 0.f) st = o;
    else merge_stats(st, o);
  }
  if (part == 0 && r < rows) write_row(st, -INFINITY, -INFINITY, a.kl + row, a.lse1 + row, a.lse2 + row);
}

template <int D1, int D2>
int launch_sel_fwd_t(const SelMaps& m, const SelFwdArgs& args, cudaStream_t st) {
  using L = SelFwdLayout;
  SelFwdArgs a = args;
  // two buffers of K (the next list's loads) where they leave five slots, then as many slots as fit
  a.k_bufs = L::bytes(5, 2, D1, D2, a.p.bs) <= L::kMost ? 2 : 1;
  a.slots = 5;
  while (a.slots < L::kMaxSlots && L::bytes(a.slots + 1, a.k_bufs, D1, D2, a.p.bs) <= L::kMost) ++a.slots;
  a.slots = slots_of_sides(a.slots, a.r1, D1, a.r2, D2);
  auto kern = sel_fwd_kernel<D1, D2>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kMost);
  if (e != cudaSuccess) return e;
  kern<<<a.p.ctas, L::kThreads, L::bytes(a.slots, a.k_bufs, D1, D2, a.p.bs), st>>>(m.k1, m.k2, a);
  return cudaGetLastError();
}

}  // namespace

int launch_sel_fwd(const SelMaps& m, int d1, int d2, const SelFwdArgs& a, cudaStream_t st) {
  if (d1 == 64) return d2 == 64 ? launch_sel_fwd_t<64, 64>(m, a, st) : launch_sel_fwd_t<64, 128>(m, a, st);
  return d2 == 64 ? launch_sel_fwd_t<128, 64>(m, a, st) : launch_sel_fwd_t<128, 128>(m, a, st);
}

int launch_sel_merge(const SelFwdArgs& a, cudaStream_t st) {
  const long long threads = (long long)a.p.B * a.p.H * a.p.NQ * kMergeLanes;
  sel_merge_kernel<<<unsigned((threads + kMergeThreads - 1) / kMergeThreads), kMergeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace skl
