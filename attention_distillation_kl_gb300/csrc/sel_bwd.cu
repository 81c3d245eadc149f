// Backward over selected blocks (sel_common.cuh): both distributions rebuilt
// per (tile of gathered rows, block) from the forward's LSEs,
//   mode P2:  dS = s2 dKL (P2 - P1),   mode P1:  dS = s1 dKL P1 (ln(P1 / P2) - KL),
//   dQ = dS K,  dK = dS^T Q.
//
// Persistent CTAs walk their lists.  dK of a list's block accumulates in TMEM
// and leaves as one fp32 tile for each CTA that had a share of the list, which
// sel_finish_kernel adds in order.
// A row of dQ gets a contribution from each of its blocks, out of different
// CTAs: fp32 vector reductions, each value rounded to its row's grid first
// (dq_fixed_exp), so that the sums are exact in any order and the result is
// bitwise repeatable.  24 warps:
//   warps 0-7   dS (thread = row; a warpgroup takes half of the columns)
//   warps 8-15  dQ (a warpgroup takes half of the columns): TMEM -> registers ->
//               shared memory, 8 rows x 32 values at a time, so that 8 lanes
//               reduce a whole line of 128 bytes; after a list, dK alike
//   warps 16-19 gather 32 rows each of both sides, and the rows' parameters
//               (row_params)
//   warp 20     S1, S2      warp 21     dK, dQ      warp 22     K by TMA
//   warp 23     tells the others what to take (SelShare)
// TMEM: S1, S2 of bs columns (two buffers with blocks up to 64), dK [256, 384),
// dQ [384, 512).
//
// Bound by the reductions: a row and block bring 4 dg bytes to L2, which takes
// some 6.4 TB/s of them (measured alone, rows of 512 bytes over 32 MB: 6.4 with 8
// or 32 lanes to a line, 3.8 with lanes to sectors of several lines, 3.1 with a
// row a lane; as bulk reductions 5.4 in pieces of 256 bytes and 2.8 in 128),
// where rows that are read come at 19.5.
#include "sel_common.cuh"

namespace skl {

namespace {

template <int D1, int D2>
struct SelBwdLayout {
  static constexpr int kDsWarps = 8, kEpiWarp = 8, kEpiWGs = 2, kGatherWarp = 16, kGatherWarps = 4;
  static constexpr int kSWarp = 20, kGradWarp = 21, kLoadWarp = 22, kWalkWarp = 23;
  static constexpr int kThreads = 32 * (kWalkWarp + 1);
  static constexpr int kMaxRing = 6;  // slots of gathered tiles
  // Tiles whose rows' parameters and numbers are kept.  Those of tile n are replaced with the copies of tile n + that,
  // which wait for the dK of tile n + that - 1 - slots / 2 at least: behind the dS of n, which reads the parameters, and
  // of n + 2, whose dS was stored behind the dQ of n + 1, which waits until the warps of dQ have read the numbers of n.
  __host__ __device__ static int params(int slots) { return 1 + slots / 2; }
  __host__ __device__ static int numbers(int slots) { return 3 + slots / 2; }
  enum {
    kKFull = 0, kKEmpty = 2, kReady = 4, kQFull = 6, kQEmpty = kQFull + kMaxRing, kSFull = kQEmpty + kMaxRing,
    kSFree = kSFull + 2, kDsFull = kSFree + 2, kDsEmpty, kDqFull, kDqEmpty, kDkFull, kDkEmpty, kDone, kTold,
    kNumBars = (kTold + 2 * kShares + 1) / 2 * 2  // (16-byte words behind them)
  };
  static constexpr uint32_t kSlot = kTile * 2u * (D1 > D2 ? D1 : D2);
  __host__ __device__ static uint32_t param_bytes(int slots) { return uint32_t(params(slots)) * kTile * 12u; }
  __host__ __device__ static uint32_t number_bytes(int slots) { return uint32_t(numbers(slots)) * kTile * 5u; }
  static constexpr uint32_t kPitch = 144, kStage = 4 * kEpiWGs * 8 * kPitch;  // staged rows of 32 values, padded
  // operands, dS (64-key blocks of 128 rows), staged rows, parameters, numbers, barriers
  static uint32_t bytes(int slots, int k_bufs, int bs) {
    return 1024u + slots * kSlot + uint32_t(k_bufs * bs) * (D1 + D2) * 2u + ds_bytes(bs) + kStage + param_bytes(slots) +
           number_bytes(slots) + kNumBars * 8 + kShares * sizeof(SelShare) + 16;
  }
  __host__ __device__ static uint32_t ds_bytes(int bs) { return bs == 128 ? 32768u : 16384u; }
  static constexpr uint32_t kMost = 232448;
};

__device__ __forceinline__ void red_add4(float* p, float4 v) {
  asm volatile("red.global.add.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// 32 columns of 16 rows, and the wait for them: lane l holds, for every 8
// columns e, v[4 e] and v[4 e + 1]: row l / 4, columns 8 e + 2 (l % 4) and the
// next; v[4 e + 2], v[4 e + 3]: the same of row l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t t, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SKL_R8(v, 0), SKL_R8(v, 8)
      : "r"(t)
      : "memory");
}

// dS of 16 columns of a row, as pairs of bf16 (ds_chunk_row without its mask).
template <int MODE>
__device__ __forceinline__ void ds_columns(const uint32_t (&x1)[16], const uint32_t (&x2)[16], uint64_t C1, uint64_t C2,
                                           uint64_t S1, uint64_t NR, uint64_t NA, uint64_t NB, uint64_t WW, uint32_t (&out)[8]) {
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const uint64_t X1 = f2(__uint_as_float(x1[k]), __uint_as_float(x1[k + 1]));
    const uint64_t X2 = f2(__uint_as_float(x2[k]), __uint_as_float(x2[k + 1]));
    float a, b;
    f2_split(f2_fma(X1, C1, NA), a, b);
    const uint64_t P1 = f2(ex2(a), ex2(b));
    uint64_t D;
    if (MODE == STREAMKL_GRAD_P2) {
      f2_split(f2_fma(X2, C2, NB), a, b);
      D = f2_mul(WW, f2_sub(f2(ex2(a), ex2(b)), P1));
    } else {
      D = f2_mul(f2_mul(WW, P1), f2_fma(f2_fma(X2, NR, X1), S1, NB));
    }
    f2_split(D, a, b);
    out[k / 2] = pack_bf16(a, b);
  }
}

template <int D1, int D2, int MODE>
__global__ void __launch_bounds__(SelBwdLayout<D1, D2>::kThreads, 1)
    sel_bwd_kernel(const __grid_constant__ CUtensorMap tk1, const __grid_constant__ CUtensorMap tk2,
                   const __grid_constant__ SelBwdArgs a) {
  using L = SelBwdLayout<D1, D2>;
  constexpr bool kP2 = MODE == STREAMKL_GRAD_P2;
  constexpr int DG = kP2 ? D2 : D1, DO = kP2 ? D1 : D2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = a.p.bs;
  const uint32_t kK1 = uint32_t(bs) * D1 * 2, kK = uint32_t(bs) * (D1 + D2) * 2;
  const uint32_t oDS = a.k_bufs * kK, oQ = oDS + L::ds_bytes(bs), oStage = oQ + a.slots * L::kSlot;
  const uint32_t oParam = oStage + L::kStage, oNumber = oParam + L::param_bytes(a.slots),
                 oBar = oNumber + L::number_bytes(a.slots);
  const int n_params = L::params(a.slots), n_numbers = L::numbers(a.slots);
  auto bar = [&](int id) { return sb + oBar + 8u * id; };
  float* params = reinterpret_cast<float*>(smem + oParam);                     // na, nb, ws: [tile][3][128]
  int* row_of = reinterpret_cast<int*>(smem + oNumber);                        // row of dq32, or -1
  int8_t* grid_of = reinterpret_cast<int8_t*>(row_of + n_numbers * kTile);   // the exponent of its grid
  SelShare* shares = reinterpret_cast<SelShare*>(smem + oBar + L::kNumBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shares + kShares);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t told = sb + oBar + 8u * L::kTold;
  const Ctl ctl{abort_flag, a.status};

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      int count = 1;
      if (i >= L::kQFull && i < L::kQEmpty) count = 33 * L::kGatherWarps;
      if (i == L::kReady || i == L::kReady + 1 || i == L::kSFree || i == L::kSFree + 1 ||
          i == L::kDsFull)
        count = L::kDsWarps;
      if (i == L::kDqEmpty || i == L::kDkEmpty) count = 4 * L::kEpiWGs;
      if (i >= L::kTold + kShares) count = L::kWalkWarp;  // the warps before it
      if (i == L::kDone) count = 2;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == L::kGradWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // columns past the head dim (K's are zeros, and no product may meet a NaN there; slots_of_sides keeps them so)
  if (a.r1.chunks < D1 / 8 || a.r2.chunks < D2 / 8)
    for (uint32_t o = threadIdx.x * 16; o < a.slots * L::kSlot; o += L::kThreads * 16) st_shared_v4(sb + oQ + o, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int s_bufs = bs == 128 ? 1 : 2;
  const uint32_t t_s1 = tmem, t_s2 = tmem + bs, t_dk = tmem + 256, t_dq = tmem + 384;  // (S buffers 128 columns apart)
  const int per_tile = a.p.queries_per_tile, G = a.p.G;
  const bool ids = a.vis.ids_q != nullptr;

  if (warp >= L::kGatherWarp && warp < L::kGatherWarp + L::kGatherWarps) {
    // ---------------------------------------------------------------- gather: rows [first, first + 32)
    const int first = (warp - L::kGatherWarp) * 32;
    const int r = first + lane, ql = r / G, hl = r - ql * G;
    const SelRows& ro = kP2 ? a.r1 : a.r2;
    const SelRows& rg = kP2 ? a.r2 : a.r1;
    const bool place = ql < per_tile;
    SelReader share(shares, told);
    int e0 = 0;
    // the lane's row 0 of both sides and its number, in the current share
    const uint8_t *bo = nullptr, *bg = nullptr;
    int row0 = 0;
    auto enter = [&]() {
      if (!share.next(ctl)) return false;
      bo = ro.at(share.b, share.head0 + hl, 0);
      bg = rg.at(share.b, share.head0 + hl, 0);
      row0 = (share.b * a.p.H + share.head0 + hl) * a.p.NQ;
      return true;
    };
    bool ahead = enter();  // `ent` is of a tile
    // A row's parameters are read a tile ahead of its copies, its entry two tiles.
    unsigned ent = entry_of(a.p, share, ql, place);
    unsigned long long po = 0, pg = 0;  // of the tile to copy
    float4 par;
    int row = -1;
    auto look = [&]() {  // at the row of `ent`
      po = pg = 0;
      par = make_float4(-INFINITY, kP2 ? -INFINITY : 0.f, 0.f, 0.f);
      row = -1;
      if (ent == kNoEntry) return;
      const int i = int(ent >> kSlotBits);
      if (!SKL_CHECK(a.status, i < a.p.NQ)) return;
      row = row0 + i;
      par = __ldg(a.rows + row);
      po = reinterpret_cast<unsigned long long>(bo + i * ro.sn);
      pg = reinterpret_cast<unsigned long long>(bg + i * rg.sn);
    };
    auto step = [&]() {  // to the next tile's entry
      e0 += per_tile;
      if (ahead && e0 >= share.count) {
        ahead = enter();
        e0 = 0;
      }
      ent = entry_of(a.p, share, e0 + ql, place);
    };
    int s = 0, m = 0, at_p = 0, at_n = 0;  // slot, rounds of the ring, places of parameters and numbers
    bool ok = true, more = ahead;
    look();
    step();
    while (ok && more) {
      more = ahead;
      const unsigned long long xo = po, xg = pg;
      const float4 x = par;
      const int of = row;
      look();
      step();
      // rows that saw nothing (they may hold anything) and rows past the last
      // are zeros, and contribute zeros
      const bool on = of >= 0 && x.x != -INFINITY;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        ok = mbar_wait_warp(bar(L::kQEmpty + s), (m & 1) ^ 1, ctl);
        if (!ok) break;
        if (side == 0) {
          float* to = params + at_p * (3 * kTile) + r;
          to[0] = on ? x.x : -INFINITY;
          to[kTile] = on ? x.y : (kP2 ? -INFINITY : 0.f);
          to[2 * kTile] = on ? x.z : 0.f;
          row_of[at_n * kTile + r] = on ? of : -1;
          grid_of[at_n * kTile + r] = int8_t(int(x.w));
          if (++at_p == n_params) at_p = 0;
          if (++at_n == n_numbers) at_n = 0;
          gather_rows<DO, true>(sb + oQ + s * L::kSlot, first, on ? xo : 0ull, ro);
        } else {
          gather_rows<DG, true>(sb + oQ + s * L::kSlot, first, on ? xg : 0ull, rg);
        }
        cp_async_arrive(bar(L::kQFull + s));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kQFull + s));  // parameters and zeros, which are plain stores
        if (++s == a.slots) s = 0, ++m;
      }
    }
    cp_async_wait_all();
  } else if (warp == L::kLoadWarp) {
    // ---------------------------------------------------------------- K
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
  } else if (warp == L::kWalkWarp) {
    tell_shares(a.p, shares, told, ctl);
  } else if (warp == L::kSWarp) {
    // ---------------------------------------------------------------- S issuer
    const uint32_t leader = elect_one();
    const uint32_t idesc = idesc_bf16(128, bs, 0, 0);
    const uint32_t dhi = uint32_t(sdesc_sw128(0, 16, 1024) >> 32), dlo = uint32_t(sdesc_sw128(0, 16, 1024));
    int n = 0, s = 0, m = 0, kept = 0;
    bool ok = true;
    auto product = [&](auto width, uint32_t d, uint32_t ks) {  // the tile in slot s by K at ks
      constexpr int D = decltype(width)::value;
      ok = mbar_wait_warp(bar(L::kQFull + s), m & 1, ctl);
      if (!ok) return;
      fence_proxy_async_smem();  // (copies of cp.async)
      tc_fence_after();
      const uint32_t q = dlo + ((sb + oQ + s * L::kSlot) >> 4), kd = dlo + (ks >> 4), half = bs * 8;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_step(leader, d, q + (kk >> 2) * (kTile * 8) + (kk & 3) * 2, dhi, kd + (kk >> 2) * half + (kk & 3) * 2, dhi, idesc,
                 kk > 0);
    };
    for (SelReader share(shares, told); ok && share.next(ctl); ++kept) {
      const int kb = kept % a.k_bufs;
      const uint32_t k1s = sb + kb * kK, k2s = k1s + kK1;
      ok = mbar_wait_warp(bar((ids ? L::kReady : L::kKFull) + kb), (kept / a.k_bufs) & 1, ctl);
      for (int e0 = 0; ok && e0 < share.count; e0 += per_tile, ++n) {
        const int sbuf = n & (s_bufs - 1);
        ok = mbar_wait_warp(bar(L::kSFree + sbuf), ((n / s_bufs) & 1) ^ 1, ctl);
        if (!ok) break;
        // the other side first: its slot is released as early as possible
        product(std::integral_constant<int, DO>{}, (kP2 ? t_s1 : t_s2) + 128 * sbuf, kP2 ? k1s : k2s);
        if (!ok) break;
        mma_commit(leader, bar(L::kQEmpty + s));
        if (++s == a.slots) s = 0, ++m;
        product(std::integral_constant<int, DG>{}, (kP2 ? t_s2 : t_s1) + 128 * sbuf, kP2 ? k2s : k1s);
        if (!ok) break;
        if (++s == a.slots) s = 0, ++m;  // (released by dK)
        mma_commit(leader, bar(L::kSFull + sbuf));
      }
    }
    mma_commit(leader, bar(L::kDone));
  } else if (warp == L::kGradWarp) {
    // ---------------------------------------------------------------- dK and dQ issuer
    const uint32_t leader = elect_one();
    constexpr uint32_t id_dk = idesc_bf16(128, DG, 1, 1);  // A = dS^T M-major, B = Q_g N-major
    constexpr uint32_t id_dq = idesc_bf16(128, DG, 0, 1);  // A = dS K-major,   B = K_g N-major
    // (dS^T has 128 rows whatever the block: those past it multiply what lies
    // behind dS, into rows of dK that nobody reads)
    const uint64_t m_major = sdesc_sw128(0, kTile * 128, 1024), k_major = sdesc_sw128(0, 16, 1024),
                   k_rows = sdesc_sw128(0, uint32_t(bs) * 128, 1024);
    const uint32_t dhi = uint32_t(k_major >> 32);  // (the same for all three)
    const uint32_t ds_m = uint32_t(m_major) + ((sb + oDS) >> 4), ds_k = uint32_t(k_major) + ((sb + oDS) >> 4);
    int n = 0, kept = 0;
    bool ok = true;
    for (SelReader share(shares, told); ok && share.next(ctl); ++kept) {
      const int kb = kept % a.k_bufs;
      const uint32_t kg = uint32_t(k_rows) + ((sb + kb * kK + (kP2 ? kK1 : 0u)) >> 4);
      ok = mbar_wait_warp(bar((ids ? L::kReady : L::kKFull) + kb), (kept / a.k_bufs) & 1, ctl) &&
           mbar_wait_warp(bar(L::kDkEmpty), (kept & 1) ^ 1, ctl);
      bool first = true;
      for (int e0 = 0; ok && e0 < share.count; e0 += per_tile, ++n) {
        const int s = (2 * n + 1) % a.slots;
        ok = mbar_wait_warp(bar(L::kDsFull), n & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t qg = uint32_t(m_major) + ((sb + oQ + s * L::kSlot) >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_step(leader, t_dk, ds_m + kk * 128, dhi, qg + kk * 128, dhi, id_dk, !first || kk > 0);
        first = false;
        mma_commit(leader, bar(L::kQEmpty + s));
        ok = mbar_wait_warp(bar(L::kDqEmpty), (n & 1) ^ 1, ctl);
        if (!ok) break;
        tc_fence_after();
        for (int kk = 0; kk < bs / 16; ++kk)
          mma_step(leader, t_dq, ds_k + (kk >> 2) * (kTile * 8) + (kk & 3) * 2, dhi, kg + kk * 128, dhi, id_dq, kk > 0);
        mma_commit(leader, bar(L::kDsEmpty));
        mma_commit(leader, bar(L::kDqFull));
      }
      if (ok) {
        mma_commit(leader, bar(L::kDkFull));
        mma_commit(leader, bar(L::kKEmpty + kb));
      }
    }
    mma_commit(leader, bar(L::kDone));
    mbar_drain(bar(L::kDone), 0, 1000000000ull);  // every MMA has finished before TMEM is released
  } else if (warp < L::kDsWarps) {
    // ---------------------------------------------------------------- dS (thread = row)
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const int hl = row % G;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const float c1 = a.scale1 * kLog2e, c2 = a.scale2 * kLog2e, nr = -a.scale2 / a.scale1;
    const uint64_t C1 = f2(c1, c1), C2 = f2(c2, c2), S1 = f2(a.scale1, a.scale1), NR = f2(nr, nr);
    const int half = (bs + 32) / 64 * 32;                        // columns of warpgroup 0
    const int col0 = wg == 0 ? 0 : half, col1 = wg == 0 ? half : bs;
    const int nqt = (a.p.NQ + kTile - 1) / kTile, nkt = (a.p.NK + kTile - 1) / kTile, off = a.p.NK - a.p.NQ;
    int n = 0, kept = 0, at_p = 0, at_n = 0;
    bool ok = true;
    for (SelReader share(shares, told); ok && share.next(ctl); ++kept) {
      const int k0 = share.block * bs;
      const int prefix = a.p.prefix != nullptr ? min(max(a.p.prefix[share.b], 0), a.p.NK) : 0;
      const int* kids = ids ? a.vis.ids_k + size_t(share.b) * nkt * kTile + k0 : nullptr;
      if (ids) {
        // keys that match nothing may hold anything: zeros before a product reads them
        const int kb = kept % a.k_bufs;
        ok = mbar_wait_warp(bar(L::kKFull + kb), (kept / a.k_bufs) & 1, ctl);
        if (!ok) break;
        if (row < bs && kids[row] < 0) {
          const uint32_t base = sb + kb * kK + (wg == 0 ? 0u : kK1) + row * 128;
          for (int c = 0; c < (wg == 0 ? D1 : D2) / 64; ++c)
#pragma unroll
            for (int o = 0; o < 128; o += 16) st_shared_v4(base + c * (bs * 128) + o, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kReady + kb));
      }
      const int row0 = (share.b * a.p.H + share.head0 + hl) * a.p.NQ;  // of query 0
      for (int e0 = 0; ok && e0 < share.count; e0 += per_tile, ++n) {
        const int sbuf = n & (s_bufs - 1);
        const uint32_t ts = tmem + lane_off + 128 * sbuf;
        ok = mbar_wait_warp(bar(L::kSFull + sbuf), (n / s_bufs) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const float* par = params + at_p * (3 * kTile) + row;
        if (++at_p == n_params) at_p = 0;
        const int of = row_of[at_n * kTile + row];
        if (++at_n == n_numbers) at_n = 0;
        const int i = of < 0 ? 0 : of - row0;
        const float na = par[0], nb = par[kTile], ws = par[2 * kTile];
        const uint64_t NA = f2(na, na), NB = f2(nb, nb), WW = f2(ws, ws);
        const int last = a.p.causal ? min(max(i + off + 1, prefix), a.p.NK) : a.p.NK;
        const bool whole = kids == nullptr && __all_sync(0xffffffffu, of < 0 || last >= k0 + bs);
        const int id = kids != nullptr ? a.vis.ids_q[size_t(share.b) * nqt * kTile + i] : 0;
        bool waited = false;
#pragma unroll 1
        for (int c = col0; c < col1; c += 16) {
          uint32_t x1[16], x2[16], out[8];
          tmem_ld2x16(ts + c, ts + bs + c, x1, x2);
          if (c + 16 >= col1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kSFree + sbuf));
          }
          ds_columns<MODE>(x1, x2, C1, C2, S1, NR, NA, NB, WW, out);
          if (!whole) {
            const uint32_t on = visible_bits<16>(i, k0 + c, off, a.p.NK, a.p.causal, prefix, id, kids == nullptr ? nullptr : kids + c);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              out[x] &= ((on >> (2 * x)) & 1u ? 0xffffu : 0u) | ((on >> (2 * x + 1)) & 1u ? 0xffff0000u : 0u);
          }
          if (!waited) {  // the previous tile's products must be done reading dS
            ok = mbar_wait_warp(bar(L::kDsEmpty), (n & 1) ^ 1, ctl);
            if (!ok) break;
            waited = true;
          }
          // into 64-key blocks of 128-byte rows, swizzled
          const uint32_t to = sb + oDS + (c >> 6) * (kTile * 128) + row * 128, piece = (c & 63) >> 3;
          st_shared_v4(to + ((piece ^ (row & 7)) << 4), out[0], out[1], out[2], out[3]);
          st_shared_v4(to + (((piece + 1) ^ (row & 7)) << 4), out[4], out[5], out[6], out[7]);
        }
        if (!ok) break;
        if (col0 == col1) {  // blocks of 32: nothing for this warpgroup, which may not run ahead of the other
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kSFree + sbuf));
          ok = mbar_wait_warp(bar(L::kDsEmpty), (n & 1) ^ 1, ctl);
          if (!ok) break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kDsFull));
      }
    }
  } else {
    // ---------------------------------------------------------------- dQ, and dK after a list
    const int wg = (warp - L::kEpiWarp) >> 2, w4 = warp & 3;
    const uint32_t lane_off = uint32_t(w4 * 32) << 16;
    const uint32_t stage = sb + oStage + (warp - L::kEpiWarp) * (8 * L::kPitch);
    // staged by row lane / 4, read by rows lane / 8 and + 4
    const uint32_t to = stage + (lane >> 2) * L::kPitch + (lane & 3) * 8, from = stage + (lane >> 3) * L::kPitch + (lane & 7) * 16;
    int n = 0, kept = 0, at_n = 0;
    bool ok = true;
    for (SelReader share(shares, told); ok && share.next(ctl); ++kept) {
      for (int e0 = 0; ok && e0 < share.count; e0 += per_tile, ++n) {
        ok = mbar_wait_warp(bar(L::kDqFull), n & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const int at = at_n * kTile + w4 * 32;
        if (++at_n == n_numbers) at_n = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float me[2];
          float* dst[4];
          bool on[4];
#pragma unroll
          for (int x = 0; x < 2; ++x) me[x] = 1.5f * exp2_int(23 - grid_of[at + 16 * half + (lane >> 2) + 8 * x]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int of = row_of[at + 16 * half + (lane >> 3) + 4 * x];
            on[x] = of >= 0;
            dst[x] = a.dq32 + size_t(on[x] ? of : 0) * a.pitch + 4 * (lane & 7);
          }
#pragma unroll
          for (int part = 0; part < DG / 64; ++part) {
            const int c = (wg * (DG / 64) + part) * 32;
            uint32_t v[16];
            tmem_ld_16x32(t_dq + lane_off + (uint32_t(16 * half) << 16) + c, v);
            if (half == 1 && part == DG / 64 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(L::kDqEmpty));
            }
            const bool within = c + 4 * (lane & 7) < a.dg;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // on the row's grid of 2^-e: (x + 1.5 2^(23 - e)) - 1.5 2^(23 - e)
              const uint64_t ME = f2(me[x], me[x]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float q0, q1;
                f2_split(f2_sub(f2_add(f2(__uint_as_float(v[4 * e + 2 * x]), __uint_as_float(v[4 * e + 2 * x + 1])), ME), ME),
                         q0, q1);
                st_shared_v2(to + e * 32, q0, q1);
              }
              __syncwarp();
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float4 q = ld_shared_v4(from + 4 * y * L::kPitch);
                if (on[2 * x + y] && within) red_add4(dst[2 * x + y] + c, q);
              }
              __syncwarp();
            }
          }
        }
      }
      if (!ok) break;
      // dK of the list, [bs][dg]
      ok = mbar_wait_warp(bar(L::kDkFull), kept & 1, ctl);
      if (!ok) break;
      tc_fence_after();
      if (w4 * 32 < bs) {
        float* dst = a.dk_part + (size_t(share.meeting) * bs + w4 * 32 + (lane >> 3)) * a.dg + 4 * (lane & 7);
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
#pragma unroll 1
          for (int part = 0; part < DG / 64; ++part) {
            const int c = (wg * (DG / 64) + part) * 32;
            uint32_t v[16];
            tmem_ld_16x32(t_dk + lane_off + (uint32_t(16 * half) << 16) + c, v);
            const bool within = c + 4 * (lane & 7) < a.dg;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                st_shared_v2(to + e * 32, __uint_as_float(v[4 * e + 2 * x]), __uint_as_float(v[4 * e + 2 * x + 1]));
              __syncwarp();
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float4 q = ld_shared_v4(from + 4 * y * L::kPitch);
                if (within) __stcs(reinterpret_cast<float4*>(dst + (16 * half + 8 * x + 4 * y) * a.dg + c), q);
              }
              __syncwarp();
            }
          }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kDkEmpty));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kGradWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kDkThreads = 256, kDkQuads = 4;  // (four values each, of a thread)

// dK of one key head and block: the shares of its lists (a unit each), of the
// CTAs that met them, in order, rounded to bf16 once.  part_of: which of the
// block's values.
__device__ __forceinline__ void dk_of_block(const SelBwdArgs& a, int j, int head, int part_of) {
  constexpr int kUnits = 32;
  __shared__ long long first_of[kUnits];  // a unit's first share
  __shared__ int shares_of[kUnits];
  const SelPlan& p = a.p;
  const int hk = head % a.HK, b = head / a.HK;
  const int units = p.HU / a.HK, per = p.HU / p.HS;
  const int bs = p.bs, quads = a.dg / 4, rows = min(bs, p.NK - j * bs);
  const int x0 = part_of * (kDkThreads * kDkQuads) + threadIdx.x;
  float4 sum[kDkQuads] = {};
  for (int u0 = 0; u0 < units; u0 += kUnits) {
    // a warp finds what a unit's list left: its place among its group's costs, and the CTAs whose parts hold its tiles
    __syncthreads();
    for (int u = u0 + (threadIdx.x >> 5); u < min(units, u0 + kUnits); u += kDkThreads / 32) {
      const int unit = hk * units + u, s = b * p.HS + unit / per, sub = unit % per;
      const int i = __ldg(p.place + size_t(s) * p.blocks + j);
      long long first = 0;
      int n = 0;
      if (i >= 0) {
        const int g = s / p.group;
        long long total;
        const int4 l = __ldg(p.lists + size_t(s) * p.cap + i);
        const int tiles = (l.z + p.queries_per_tile - 1) / p.queries_per_tile;
        const long long at = group_cost(p, g, s, total) + (long long)(l.w + i) * per + (long long)sub * (tiles + 1) + 1;
        const long long parts = sel_parts(p, total), c0 = ((at + 1) * parts - 1) / total;
        n = int(((at + tiles) * parts - 1) / total - c0) + 1;
        first = ((long long)s * p.cap + i) * per + sub + (long long)g * p.ctas + c0;
      }
      if ((threadIdx.x & 31) == 0) {
        first_of[u - u0] = first;
        shares_of[u - u0] = n;
      }
    }
    __syncthreads();
    for (int u = 0; u < min(units - u0, kUnits); ++u) {
      const float* part = a.dk_part + size_t(first_of[u]) * bs * a.dg + 4 * x0;  // (a share is [bs][quads])
#pragma unroll 2
      for (int k = 0; k < shares_of[u]; ++k, part += size_t(bs) * a.dg) {
        float4 v[kDkQuads];
#pragma unroll
        for (int e = 0; e < kDkQuads; ++e)
          if (x0 + e * kDkThreads < rows * quads) v[e] = __ldcs(reinterpret_cast<const float4*>(part + 4 * e * kDkThreads));
#pragma unroll
        for (int e = 0; e < kDkQuads; ++e)
          if (x0 + e * kDkThreads < rows * quads) {
            sum[e].x += v[e].x;
            sum[e].y += v[e].y;
            sum[e].z += v[e].z;
            sum[e].w += v[e].w;
          }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kDkQuads; ++e) {
    const int x = x0 + e * kDkThreads;
    if (x >= rows * quads) return;
    const int key = x / quads, c = (x - key * quads) * 4;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dk) + b * a.dk_sb + hk * a.dk_sh + (j * bs + key) * a.dk_sn + c;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(sum[e].x, sum[e].y), pack_bf16(sum[e].z, sum[e].w));
  }
}

// The blocks' dK by the first CTAs, dQ's rows by the others.
__global__ void __launch_bounds__(kDkThreads, 4) sel_finish_kernel(const __grid_constant__ SelBwdArgs a,
                                                                const __grid_constant__ ModFinishArgs::Rows dq, int dk,
                                                                int rows) {
  const int blk = blockIdx.x;
  if (blk >= dk) {
    finish_rows(dq, blk - dk, rows);
    return;
  }
  const int heads = a.p.B * a.HK, x = blk / a.p.blocks;
  dk_of_block(a, blk - x * a.p.blocks, x % heads, x / heads);
}

template <int D1, int D2, int MODE>
int launch_sel_bwd_t(const SelMaps& m, const SelBwdArgs& args, cudaStream_t st) {
  using L = SelBwdLayout<D1, D2>;
  SelBwdArgs a = args;
  const int bs = a.p.bs;
  // Two tiles' slots, then a second K, then more slots.  (Two slots are enough for the walk: a tile at a time.)
  auto fits = [&](int slots, int bufs) { return L::bytes(slots, bufs, bs) <= L::kMost; };
  a.k_bufs = 1;
  a.slots = fits(4, 1) ? 4 : 3;
  if (fits(a.slots, 2)) a.k_bufs = 2;
  while (a.slots < L::kMaxRing && fits(a.slots + 1, a.k_bufs)) ++a.slots;
  if (!fits(a.slots, a.k_bufs)) return cudaErrorInvalidValue;
  a.slots = slots_of_sides(a.slots, a.r1, D1, a.r2, D2);
  auto kern = sel_bwd_kernel<D1, D2, MODE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kMost);
  if (e != cudaSuccess) return e;
  kern<<<a.p.ctas, L::kThreads, L::bytes(a.slots, a.k_bufs, bs), st>>>(m.k1, m.k2, a);
  return cudaGetLastError();
}

template <int D1, int D2>
int launch_sel_bwd_m(const SelMaps& m, const SelBwdArgs& a, cudaStream_t st) {
  return a.mode == STREAMKL_GRAD_P2 ? launch_sel_bwd_t<D1, D2, STREAMKL_GRAD_P2>(m, a, st)
                                  : launch_sel_bwd_t<D1, D2, STREAMKL_GRAD_P1>(m, a, st);
}

}  // namespace

int launch_sel_bwd(const SelMaps& m, int d1, int d2, const SelBwdArgs& a, cudaStream_t st) {
  if (d1 == 64)
    return d2 == 64 ? launch_sel_bwd_m<64, 64>(m, a, st) : launch_sel_bwd_m<64, 128>(m, a, st);
  return d2 == 64 ? launch_sel_bwd_m<128, 64>(m, a, st) : launch_sel_bwd_m<128, 128>(m, a, st);
}

int launch_sel_finish(const SelBwdArgs& a, const ModFinishArgs::Rows& dq, cudaStream_t st) {
  constexpr int kEach = kDkThreads * kDkQuads;
  const int parts = (a.p.bs * (a.dg / 4) + kEach - 1) / kEach;
  const int dk = a.p.blocks * a.p.B * a.HK * parts, rows = loop_blocks((long long)dq.heads * dq.n * (dq.d / 8));
  sel_finish_kernel<<<unsigned(dk + rows), kDkThreads, 0, st>>>(a, dq, dk, rows);
  return cudaGetLastError();
}

}  // namespace skl
