// The blocks that score best for each query (see streamkl_select_blocks):
//   score(i, hs, j) = sum over the query heads h of hs of q_h(i) . kb_hs(j).
//
// Three steps: norms of the blocks' keys and their id ranges; scores of 128
// queries x 256 blocks by the tensor core, the heads' products added up in
// TMEM; then the count-th best score of each row is found by guesses and counts
// and the blocks written in ascending order: by a thread a row, out of TMEM, where
// queries are many and blocks at most 256, else by a warp a row with the scores
// through L2, in strips that stay there.  Bound by these passes' instructions.
//
// The list has to be that of the exact scores, ties to the lowest block, while
// the tensor core's are fp32 sums.  Their error is at most
//   eps = x (1 + 2 x) sum_h |q_h| max |kb|,  x = (heads d + 64) 2^-23:
// heads d additions in any order, each off by a unit of the sum so far at most (the
// tensor core cuts off what does not fit), which stays below (1 + x) of the terms'
// sizes, and these below sum_h |q_h| |kb|.  (The root of all heads' squares would be
// short by up to the root of heads: 65535 equal heads then gave wrong lists.)  Where a block
// lies within 2 eps of the border, those that do are scored again, with
// products that are exact in fp32 and a sum kept in two floats, and the border is
// drawn by these.  The high ones' sums lose nothing, the low ones' (n 2^-24 of the
// terms' sizes at most, for n products a lane) as much as 2^-24 of themselves each
// time: n^2 / 2 2^-48 in a lane, and 10 n 2^-48 where the lanes' are joined.
#include <algorithm>
#include <cfloat>

#include "bwd_common.cuh"
#include "mod_host.cuh"
#include "sel_common.cuh"

namespace skl {

namespace {

struct SelectArgs {
  int B, H, HS, NQ, NK, d, bs, blocks, T, sink, local;
  int heads;           // query heads of a selection head
  int pitch;           // of a score row
  int tiles_q;         // query tiles of a selection head
  int tile0, tiles;    // the strip: query tiles of all selection heads
  int causal;
  const int* prefix;
  const int* doc_q;
  const int* doc_k;
  SelRows q, kb;
  float* scores;       // [tiles * 128][pitch]
  float* norms;        // [tiles * 128]: the heads' |q|, summed
  unsigned* kb_norm;   // [B HS], zeroed: max |kb|, as bits
  int2* ranges;        // [B][blocks]: smallest and largest id of a block, with ids
  int* selected;
  int* status;
};

constexpr int kPrepThreads = 256;

// At least the root of a sum of squares that was rounded (and of squares that
// vanished); 0 for nothing but zeros.
__device__ __forceinline__ float norm_above(float sum, bool some) { return some ? sqrtf(sum) * 1.0001f + 1.0e-17f : 0.f; }

// A warp a block and head: max |kb|; the first head's warps find with ids the
// range of the block's keys' ids too.
__global__ void __launch_bounds__(kPrepThreads) select_prep_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ unsigned most[kPrepThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = blockIdx.x * (kPrepThreads / 32) + warp;
  const int b = blockIdx.y / a.HS, h = blockIdx.y - b * a.HS;
  float s = 0.f;
  uint32_t any = 0;
  if (j < a.blocks && lane < a.kb.chunks) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.kb.at(b, h, j)) + lane);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(v[e] << 16), y = __uint_as_float(v[e] & 0xffff0000u);
      s = fmaf(x, x, fmaf(y, y, s));
      any |= v[e] & 0x7fff7fffu;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const bool some = __any_sync(0xffffffffu, any != 0u);
  // (a NaN compares above every number, as bits do)
  if (lane == 0) most[warp] = __float_as_uint(norm_above(s, some)) & 0x7fffffffu;
  __syncthreads();
  if (warp == 0) {
    const unsigned m = __reduce_max_sync(0xffffffffu, lane < kPrepThreads / 32 ? most[lane] : 0u);
    if (lane == 0) atomicMax(a.kb_norm + b * a.HS + h, m);
  }
  if (a.doc_k == nullptr || h != 0 || j >= a.blocks) return;
  int lo = INT_MAX, hi = -1;
  for (int e = lane; e < a.bs; e += 32) {
    const int k = j * a.bs + e;
    const int id = k < a.NK ? a.doc_k[(long long)b * a.NK + k] : -1;
    if (id >= 0) lo = min(lo, id), hi = max(hi, id);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) a.ranges[b * a.blocks + j] = make_int2(lo, hi);
}

constexpr int kN = 256;  // blocks of a tile's part

// ---------------------------------------------------------------- the best of a row

constexpr int kTopThreads = 256;

// Floats in order as integers, and back.
__device__ __forceinline__ int float_key(float x) {
  const int f = __float_as_int(x);
  return f >= 0 ? f : -(f & 0x7fffffff);
}
__device__ __forceinline__ float key_float(int k) { return k >= 0 ? __int_as_float(k) : -__int_as_float(-k); }
__device__ __forceinline__ float warp_min(float x) { return key_float(__reduce_min_sync(0xffffffffu, float_key(x))); }

struct Wide {  // hi + lo
  float hi, lo;
};
__device__ __forceinline__ Wide wide_add(Wide a, float x) {  // hi and x exactly, what they lose into lo
  const float s = __fadd_rn(a.hi, x), t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(x, t));
  return Wide{s, __fadd_rn(a.lo, e)};
}

// The scores of N blocks, by the whole warp, as the same doubles in all lanes (finite).
template <int N>
__device__ __forceinline__ void exact_scores(const SelectArgs& a, int b, int hs, int i, const int (&j)[N], double (&out)[N]) {
  const int lane = threadIdx.x & 31;
  Wide s[N] = {};
  for (int u = lane; u < a.heads * a.q.chunks; u += 32) {
    const int h = u / a.q.chunks, c = u - h * a.q.chunks;
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.q.at(b, hs * a.heads + h, i)) + c);
    const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(a.kb.at(b, hs, j[n])) + c);
      const uint32_t r[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n] = wide_add(s[n], __fmul_rn(__uint_as_float(p[e] << 16), __uint_as_float(r[e] << 16)));
        s[n] = wide_add(s[n], __fmul_rn(__uint_as_float(p[e] & 0xffff0000u), __uint_as_float(r[e] & 0xffff0000u)));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float hi = __shfl_xor_sync(0xffffffffu, s[n].hi, o), lo = __shfl_xor_sync(0xffffffffu, s[n].lo, o);
      // (the lower lane's first: the same sum in both)
      Wide t = lane & o ? Wide{hi, lo} : s[n];
      const Wide other = lane & o ? s[n] : Wide{hi, lo};
      t = wide_add(t, other.hi);
      t.lo = __fadd_rn(t.lo, other.lo);
      s[n] = t;
    }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const double d = double(s[n].hi) + double(s[n].lo);
    out[n] = d == d ? fmin(fmax(d, -DBL_MAX), DBL_MAX) : -DBL_MAX;
  }
}
__device__ __forceinline__ double exact_score(const SelectArgs& a, int b, int hs, int i, int j) {
  const int of[1] = {j};
  double s[1];
  exact_scores(a, b, hs, i, of, s);
  return s[0];
}

// Blocks that may be candidates of row i: the first of them, up to the mask's border.
__device__ __forceinline__ int reach(const SelectArgs& a, int b, int i) {
  if (!a.causal) return a.blocks;
  const int prefix = a.prefix != nullptr ? min(max(a.prefix[b], 0), a.NK) : 0;
  const int keys = min(max(i + a.NK - a.NQ + 1, prefix), a.NK);
  return keys <= 0 ? 0 : (keys - 1) / a.bs + 1;
}
__device__ __forceinline__ float finite(float x) { return x == x ? fminf(fmaxf(x, -FLT_MAX), FLT_MAX) : -FLT_MAX; }

// The next guess of a border between lo, with `T` scores or more at or above it, and hi with fewer: where the count's
// logarithm (up, down), taken as straight between the two, passes T; every fourth halves the distance, and from the 24th on
// the number of floats between the two, which ends.  False: there is none between them.
__device__ __forceinline__ bool guess(int step, float lo, float hi, float up, float down, float wanted, float& mid) {
  const float f = (step & 3) == 3 ? 0.5f : fminf(fmaxf(__fdividef(up - wanted, up - down), 0.02f), 0.98f);
  mid = fmaf(f, hi - lo, lo);
  if (step >= 24 || !(mid > lo && mid < hi)) {
    const long long m = (float_key(lo) + (long long)float_key(hi)) >> 1;
    mid = key_float(int(m));
    if (!(mid > lo && mid < hi)) return false;  // neighbours
  }
  return true;
}

// What fp32 sums of a row's products may be off by.  (The other half of 2 x is more than the norms' own sum loses.)
__device__ __forceinline__ float error_of(const SelectArgs& a, int b, int hs, float norm) {
  const float x = float(a.heads * a.d + 64) * 1.1920929e-7f;
  return x * fmaf(2.f, x, 1.f) * norm * __uint_as_float(a.kb_norm[b * a.HS + hs]);
}

// The list of row i from its scores as they compete, in shared memory (block 32 k
// + lane at mine[32 k]): `total` candidates, more than T or behind gaps; least
// and best of those not forced, each lane's or the row's.  The whole warp.
__device__ __forceinline__ void select_row(const SelectArgs& a, int b, int hs, int i, int rounds, int total, float least,
                                           float best, float norm, float* mine, int* out) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  auto each = [&](auto f) {
#pragma unroll 4
    for (int k = 0; k < rounds; ++k) f(k, mine[32 * k]);
  };
  // The T-th best score, and how those next to it are told apart.
  enum { kEvery, kForced, kAbove, kFirst, kChosen, kDeep };
  int how = kEvery, need = 0;
  float cut = 0.f, window = 0.f;
  unsigned chosen = 0;
  double deep[kMaxSelBlocks / 32];  // (of kDeep)
  auto sum_over = [&](auto f) {
    int n = 0;
    each([&](int, float x) { n += f(x) ? 1 : 0; });
    return __reduce_add_sync(0xffffffffu, n);
  };
  auto sure = [&](float x) { return x > cut + window || x == INFINITY; };
  auto near = [&](float x) { return !sure(x) && x >= cut - window && x > -INFINITY; };
  if (total > a.T) {
    least = warp_min(least);
    best = -warp_min(-best);
    // At least T scores are lo or above; fewer are hi or above (or lo is the best).
    float lo = least, hi = best;
    int n_lo = total, n_hi = sum_over([&](float x) { return x >= hi; });
    if (n_hi >= a.T) lo = hi, n_lo = n_hi;
    const float wanted = __log2f(float(a.T) + 0.5f);
    float up = __log2f(float(n_lo)), down = __log2f(n_hi > 0 ? float(n_hi) : 0.5f);
    for (int step = 0; n_lo != a.T && lo < hi; ++step) {
      float mid;
      if (!guess(step, lo, hi, up, down, wanted, mid)) break;
      const int n = sum_over([&](float x) { return x >= mid; });
      const float log_n = __log2f(n > 0 ? float(n) : 0.5f);
      if (n >= a.T) lo = mid, n_lo = n, up = log_n;
      else hi = mid, down = log_n;
    }
    float a_min = INFINITY, b_max = -INFINITY;  // the T-th best, the best behind it
    each([&](int, float x) {
      if (x >= lo) a_min = fminf(a_min, x);
      else b_max = fmaxf(b_max, x);
    });
    a_min = warp_min(a_min);
    b_max = -warp_min(-b_max);
    const float eps = error_of(a, b, hs, norm);
    cut = a_min;
    if (a_min == INFINITY) {
      how = kForced;
    } else if (n_lo == a.T && a_min - b_max > 2.f * eps) {
      how = kAbove;
    } else {
      window = eps == eps ? 2.f * eps : INFINITY;
      need = a.T - sum_over(sure);
      const int n = sum_over(near);
      if (n == need || window == 0.f) {  // all of them; or scores of 0, all equal
        how = kFirst;
      } else if (n <= 32) {
        how = kChosen;
        double mine = 0.0;
        int at = 0;
        each([&](int k, float x) {
          for (unsigned who = __ballot_sync(0xffffffffu, near(x)); who != 0u; who &= who - 1u, ++at) {
            const double s = exact_score(a, b, hs, i, 32 * k + __ffs(who) - 1);
            if (lane == at) mine = s;
          }
        });
        int better = 0;
        for (int o = 0; o < n; ++o) {
          const double s = __shfl_sync(0xffffffffu, mine, o);
          better += s > mine || (s == mine && o < lane) ? 1 : 0;
        }
        chosen = __ballot_sync(0xffffffffu, lane < n && better < need);
      } else {
        // many (equal keys, say): a lane keeps the scores of its blocks, and the best are taken one by one
        how = kDeep;
        each([&](int k, float x) {
          double mine = -INFINITY;
          for (unsigned who = __ballot_sync(0xffffffffu, near(x)); who != 0u; who &= who - 1u) {
            const int l = __ffs(who) - 1;
            const double s = exact_score(a, b, hs, i, 32 * k + l);
            if (lane == l) mine = s;
          }
          deep[k] = mine;
        });
        for (int left = need; left > 0; --left) {
          double s = -INFINITY;
          int j = INT_MAX;
          each([&](int k, float) {
            if (deep[k] > s && deep[k] != INFINITY) s = deep[k], j = 32 * k + lane;
          });
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const double t = __shfl_xor_sync(0xffffffffu, s, o);
            const int u = __shfl_xor_sync(0xffffffffu, j, o);
            if (t > s || (t == s && u < j)) s = t, j = u;
          }
          each([&](int k, float) {
            if (32 * k + lane == j) deep[k] = INFINITY;  // taken
          });
        }
      }
    }
  }
  // in ascending order
  int place = 0, ord = 0;
  each([&](int k, float x) {
    bool take = x > -INFINITY;
    if (how == kForced) take = x == INFINITY;
    if (how == kAbove) take = x >= cut;
    if (how >= kFirst) {
      const bool in = near(x);
      const unsigned who = __ballot_sync(0xffffffffu, in);
      const int o = ord + __popc(who & below);
      ord += __popc(who);
      take = sure(x);
      if (in) take = how == kFirst ? o < need : (how == kChosen ? ((chosen >> o) & 1u) != 0u : deep[k] == INFINITY);
    }
    const unsigned who = __ballot_sync(0xffffffffu, take);
    const int at = place + __popc(who & below);
    if (take && at < a.T) out[at] = 32 * k + lane;
    place += __popc(who);
  });
  for (int t = place + lane; t < a.T; t += 32) out[t] = -1;
}

// The same for rows whose scores stay in TMEM, a row a thread: a pass over them
// costs two instructions a score instead of a warp's whole sum, and no score
// goes to memory.  Borders that need exact scores are settled by the whole warp,
// row after row, and rows with more than kListed blocks at the border as above.
// There are no ids here: candidates are the first `most` blocks.
constexpr int kListed = 8;

__device__ __noinline__ void select_hard_row(const SelectArgs& a, int b, int hs, int i, int total, float least, float best,
                                             float norm, float* row, int* out) {
  select_row(a, b, hs, i, (total + 31) / 32, total, least, best, norm, row + (threadIdx.x & 31), out);
}

// tmem: the scores of the warp's 32 rows.  buffer: memory of the warp, for kListed shorts a row and the scores of one;
// lists: room for the CTA's lists of T | 1 entries a row, or null.
__device__ __forceinline__ void select_rows(const SelectArgs& a, uint32_t tmem, int b, int hs, int q0, float norm,
                                            uint8_t* buffer, int* lists) {
  constexpr unsigned kAll = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, T = a.T;
  const int first = q0 + warp * 32, i = first + lane;  // the warp's rows
  if (first >= a.NQ) return;
  uint16_t* listed = reinterpret_cast<uint16_t*>(buffer);  // [kListed][32]
  float* held = reinterpret_cast<float*>(buffer + kListed * 32 * sizeof(uint16_t));
  const int most = i < a.NQ ? reach(a, b, i) : 0;
  const int rounds = (__reduce_max_sync(kAll, most) + 31) / 32;
  const bool choose = most > T && a.sink + a.local < T;
  float least = FLT_MAX, best = -FLT_MAX;
  uint32_t v[32];
  // as they compete: the first `sink` and last `local` at the top, what is no candidate below everything
#pragma unroll 1
  for (int c = 0; c < rounds; ++c) {
    __syncwarp();
    tmem_ld32(tmem + 32 * c, v);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int j = 32 * c + e;
      float y = finite(__uint_as_float(v[e]));
      if (j < a.sink || j >= most - a.local) {
        y = j < most ? INFINITY : -INFINITY;
      } else {
        least = fminf(least, y);
        best = fmaxf(best, y);
      }
      v[e] = __float_as_uint(y);
    }
    __syncwarp();
    tmem_st32(tmem + 32 * c, v);
  }
  auto each = [&](auto f) {  // 32 scores at a time, in v
#pragma unroll 1
    for (int c = 0; c < rounds; ++c) {
      __syncwarp();
      tmem_ld32(tmem + 32 * c, v);
      f(32 * c);
    }
  };
  auto above = [&](float x) {
    int n[4] = {};
    each([&](int) {
#pragma unroll
      for (int e = 0; e < 32; ++e) n[e & 3] += __uint_as_float(v[e]) >= x ? 1 : 0;
    });
    return (n[0] + n[1]) + (n[2] + n[3]);
  };
  auto which = [&](float x) {  // of the 32: those at or above x
    unsigned m[4] = {};
#pragma unroll
    for (int e = 0; e < 32; ++e) m[e & 3] |= __uint_as_float(v[e]) >= x ? 1u << e : 0u;
    return (m[0] | m[1]) | (m[2] | m[3]);
  };
  // taken: what is `sure` or above; of those from `near` up to there, in order, the first `firsts` and chosen's bits
  float sure = most > T ? INFINITY : -FLT_MAX, near = INFINITY;
  int firsts = 0;
  unsigned chosen = 0;
  bool hard = false;
  if (__any_sync(kAll, choose)) {
    float lo = least, hi = key_float(float_key(best) + 1);  // all are lo or above; the forced ones alone are above hi
    int n_lo = most;
    const float wanted = __log2f(float(T) + 0.5f);
    float up = __log2f(float(most)), down = __log2f(fmaxf(float(a.sink + a.local), 0.5f));
    bool busy = choose;
    for (int step = 0; __any_sync(kAll, busy); ++step) {
      float mid = 0.f;
      busy = busy && guess(step, lo, hi, up, down, wanted, mid);
      const int n = above(mid);
      if (busy) {
        const float log_n = __log2f(n > 0 ? float(n) : 0.5f);
        if (n >= T) lo = mid, n_lo = n, up = log_n;
        else hi = mid, down = log_n;
        busy = n_lo != T && lo < hi;
      }
    }
    float cuts[2] = {INFINITY, INFINITY}, unders[2] = {-INFINITY, -INFINITY};
    each([&](int) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float x = __uint_as_float(v[e]);
        cuts[e & 1] = fminf(cuts[e & 1], x >= lo ? x : INFINITY);
        unders[e & 1] = fmaxf(unders[e & 1], x >= lo ? -INFINITY : x);
      }
    });
    const float cut = fminf(cuts[0], cuts[1]), under = fmaxf(unders[0], unders[1]);  // the T-th best, the best behind it
    const float eps = error_of(a, b, hs, norm);
    const float window = eps == eps ? 2.f * eps : INFINITY;
    const bool close = choose && !(n_lo == T && cut - under > window);
    if (choose) sure = cut;
    if (close) {  // (from the next float above the window)
      sure = cut + window < INFINITY ? key_float(float_key(cut + window) + 1) : INFINITY;
      near = fmaxf(cut - window, -FLT_MAX);
    }
    if (__any_sync(kAll, close)) {
      int need = T, n = 0;
      each([&](int j) {
        const unsigned in = which(sure);
        need -= __popc(in);
        for (unsigned m = which(near) & ~in; m != 0u; m &= m - 1u, ++n)
          if (n < kListed) listed[n * 32 + lane] = uint16_t(j + __ffs(m) - 1);
      });
      __syncwarp();
      const bool plain = n == need || window == 0.f;  // all of them; or scores of 0, all equal
      if (close && plain) firsts = need;
      hard = close && !plain && n > kListed;
      for (unsigned who = __ballot_sync(kAll, close && !plain && n <= kListed); who != 0u; who &= who - 1u) {
        const int r = __ffs(who) - 1, n_r = __shfl_sync(kAll, n, r), need_r = __shfl_sync(kAll, need, r);
        double mine = 0.0;
        for (int o = 0; o < n_r; o += 2) {  // (two at a time: the sums are chains)
          const int j[2] = {listed[o * 32 + r], listed[min(o + 1, n_r - 1) * 32 + r]};
          double s[2];
          exact_scores(a, b, hs, first + r, j, s);
          if (lane == o) mine = s[0];
          if (lane == o + 1) mine = s[1];
        }
        int better = 0;
        for (int o = 0; o < n_r; ++o) {
          const double s = __shfl_sync(kAll, mine, o);
          better += s > mine || (s == mine && o < lane) ? 1 : 0;
        }
        const unsigned bits = __ballot_sync(kAll, lane < n_r && better < need_r);
        if (lane == r) chosen = bits;
      }
    }
  }
  // in ascending order
  const int pitch = T | 1;  // (odd: the lanes' entries in different banks)
  int* all = a.selected + (size_t(b * a.HS + hs) * a.NQ + first) * T;
  int* mine = lists != nullptr ? lists + (warp * 32 + lane) * pitch : all + size_t(lane) * T;
  int t = 0, ord = 0;
  each([&](int j) {
    unsigned in = which(sure);
    for (unsigned m = which(near) & ~in; m != 0u; m &= m - 1u, ++ord)
      if (ord < firsts || (ord < 32 && ((chosen >> ord) & 1u) != 0u)) in |= m & -m;
    for (; in != 0u && t < T; in &= in - 1u) mine[t++] = j + __ffs(in) - 1;
  });
  if (i < a.NQ)
    for (; t < T; ++t) mine[t] = -1;
  __syncwarp();
  if (lists != nullptr)
    for (int x = lane; x < min(32, a.NQ - first) * T; x += 32) {
      const int r = x / T;
      all[x] = lists[(warp * 32 + r) * pitch + x - r * T];
    }
  __syncwarp();
  for (unsigned who = __ballot_sync(kAll, hard); who != 0u; who &= who - 1u) {
    const int r = __ffs(who) - 1;
    each([&](int j) {
      if (lane == r)
#pragma unroll
        for (int e = 0; e < 32; ++e) held[j + e] = __uint_as_float(v[e]);
    });
    __syncwarp();
    select_hard_row(a, b, hs, first + r, __shfl_sync(kAll, most, r), __shfl_sync(kAll, least, r), __shfl_sync(kAll, best, r),
                    __shfl_sync(kAll, norm, r), held, all + size_t(r) * T);
    __syncwarp();
  }
}

// A warp a row, its scores in shared memory (block 32 k + lane at a time).
// (Scores in registers, a loop unrolled for each, took 29 us instead of 21 for
// the latency alone with 1024 blocks, most of it code fetched.)
__global__ void __launch_bounds__(kTopThreads, 6) select_top_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ float held[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (blockDim.x >> 5) + warp;
  const unsigned below = (1u << lane) - 1u;
  if (unit >= a.tiles * kTile) return;
  float* mine = held + warp * ((a.blocks + 31) / 32 * 32) + lane;
  const int tile = a.tile0 + unit / kTile;
  const int sel = tile / a.tiles_q, i = (tile - sel * a.tiles_q) * kTile + unit % kTile;
  if (i >= a.NQ) return;
  const int b = sel / a.HS, hs = sel - b * a.HS;
  const float* row = a.scores + size_t(unit) * a.pitch;
  int* out = a.selected + (size_t(sel) * a.NQ + i) * a.T;
  const int id = a.doc_q != nullptr ? a.doc_q[(long long)b * a.NQ + i] : 0;
  const int most = id < 0 ? 0 : reach(a, b, i);
  const int rounds = (most + 31) / 32;
  const int2* ranges = a.doc_q != nullptr ? a.ranges + size_t(b) * a.blocks : nullptr;
  auto candidate = [&](int j) {
    if (j >= most) return false;
    if (ranges == nullptr) return true;
    const int2 r = __ldg(ranges + j);
    return r.x <= id && id <= r.y;
  };
  int total = most;
  if (ranges != nullptr) {
    total = 0;
    for (int k = 0; k < rounds; ++k) total += __popc(__ballot_sync(0xffffffffu, candidate(32 * k + lane)));
  }
  if (ranges == nullptr && total <= a.T) {  // all of them
    for (int t = lane; t < a.T; t += 32) out[t] = t < total ? t : -1;
    return;
  }
  // Scores as they compete: the first `sink` and last `local` candidates at the
  // top, what is no candidate below everything.
  float least = FLT_MAX, best = -FLT_MAX;
  int seen = 0;
  constexpr int kAhead = 4;
  for (int k0 = 0; k0 < rounds; k0 += kAhead) {
    float x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = 32 * (k0 + k) + lane;
      x[k] = j < most ? __ldcg(row + j) : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k >= rounds) break;
      const int j = 32 * (k0 + k) + lane;
      bool can = j < most;
      int rank = j;
      if (ranges != nullptr) {
        can = candidate(j);
        const unsigned who = __ballot_sync(0xffffffffu, can);
        rank = seen + __popc(who & below);
        seen += __popc(who);
      }
      const bool forced = rank < a.sink || rank >= total - a.local;
      float y = finite(x[k]);
      if (can && !forced) {
        least = fminf(least, y);
        best = fmaxf(best, y);
      }
      y = !can ? -INFINITY : (forced ? INFINITY : y);
      mine[32 * (k0 + k)] = y;
    }
  }
  __syncwarp();
  select_row(a, b, hs, i, rounds, total, least, best, a.norms[unit], mine, out);
}

// ---------------------------------------------------------------- scores

// Scores of one tile: 128 queries x kN blocks, which with LISTS are all there are.
// Warps 0-3: the heads' |q| of a row a thread while the products run, then the accumulator
// to memory, or with LISTS the rows' lists from it; warp 4 TMA; warp 5 MMA.  The K
// loop runs over heads and 64 values of d at a time.  Two CTAs share an SM.
constexpr int kScoreThreads = 192, kScoreSlots = 2;
constexpr uint32_t kQBytes = kTile * 128;  // 64 values of 128 queries
constexpr int kSelectBuffer = kListed * 32 * 2 + kN * 4;  // of a warp of select_rows
static_assert(4 * kSelectBuffer <= kN * 128, "in the keys' memory");

__device__ __forceinline__ void st_global_v8(float* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <bool LISTS>
__global__ void __launch_bounds__(kScoreThreads, 2)
    select_score_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkb,
                        const __grid_constant__ SelectArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = (a.d + 63) / 64;  // of a row
  const uint32_t oQ = uint32_t(parts) * kN * 128, oBar = oQ + kScoreSlots * kQBytes;
  auto bar = [&](int i) { return sb + oBar + 8u * i; };  // kb, full[2], empty[2], done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + oBar + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + oBar + 52);
  const Ctl ctl{abort_flag, a.status};
  // (with lists the last queries first, which see most)
  const int tile = a.tile0 + blockIdx.x, heads = a.B * a.HS;
  const int sel = LISTS ? int(blockIdx.x) % heads : tile / a.tiles_q;
  const int q0 = (LISTS ? a.tiles_q - 1 - int(blockIdx.x) / heads : tile - sel * a.tiles_q) * kTile;
  const int b = sel / a.HS, hs = sel - b * a.HS;
  const int j0 = blockIdx.y * kN;
  int columns = min(kN, a.pitch - j0);  // that some query of the tile may look at
  if (a.causal) {
    const int prefix = a.prefix != nullptr ? min(max(a.prefix[b], 0), a.NK) : 0;
    const int keys = max(min(q0 + kTile, a.NQ) + a.NK - a.NQ, prefix);
    columns = min(columns, (max(keys, 0) + a.bs - 1) / a.bs - j0);
    if (!LISTS && columns <= 0 && blockIdx.y != 0) return;  // (the first ones find |q|)
  }
  const int steps = a.heads * parts;

  if (threadIdx.x == 0) {
    mbar_init(bar(0), 1);
    for (int i = 0; i < kScoreSlots; ++i) {
      mbar_init(bar(1 + i), 1);
      mbar_init(bar(3 + i), 5);  // the products and four warps have read the slot
    }
    mbar_init(bar(5), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(0), uint32_t(parts) * kN * 128);
      for (int c = 0; c < parts; ++c) tma_load_4d(sb + c * (kN * 128), &tkb, bar(0), c * 64, j0, hs, b);
      int s = 0;
      for (; s < steps; ++s) {
        const int i = s % kScoreSlots, h = s / parts, c = s - h * parts;
        if (!mbar_wait_polled(bar(3 + i), ((s / kScoreSlots) & 1) ^ 1, ctl)) break;
        mbar_arrive_expect_tx(bar(1 + i), kQBytes);
        tma_load_4d(sb + oQ + i * kQBytes, &tq, bar(1 + i), c * 64, q0, hs * a.heads + h, b);
      }
      if (*abort_flag) {  // let the copies already started land before the CTA exits
        mbar_drain(bar(0), 0, 200000000ull);
        for (int x = s > kScoreSlots ? s - kScoreSlots : 0; x < s; ++x)
          mbar_drain(bar(1 + x % kScoreSlots), (x / kScoreSlots) & 1, 200000000ull);
      }
    }
  } else if (warp == 5) {
    const uint32_t leader = elect_one();
    const uint32_t idesc = idesc_bf16(128, max(columns + 15, 16) / 16 * 16, 0, 0);
    bool ok = mbar_wait_warp(bar(0), 0, ctl);
    for (int s = 0; ok && s < steps; ++s) {
      const int i = s % kScoreSlots, c = s % parts;
      ok = mbar_wait_warp(bar(1 + i), (s / kScoreSlots) & 1, ctl);
      if (!ok) break;
      tc_fence_after();
      const uint64_t qd = sdesc_sw128(sb + oQ + i * kQBytes, 16, 1024), kd = sdesc_sw128(sb + c * (kN * 128), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ss(leader, tmem, sdesc_add(qd, kk * 32), sdesc_add(kd, kk * 32), idesc, s > 0 || kk > 0);
      mma_commit(leader, bar(3 + i));
    }
    mma_commit(leader, bar(5));
    mbar_drain(bar(5), 0, 1000000000ull);
  } else {
    const int row = warp * 32 + lane;
    float sum = 0.f, norm = 0.f;  // of a head; of those before it
    uint32_t any = 0;
    int left = parts;  // of the head
    bool ok = true;
    for (int s = 0; ok && s < steps; ++s) {
      const int i = s % kScoreSlots;
      ok = mbar_wait_warp(bar(1 + i), (s / kScoreSlots) & 1, ctl);
      if (!ok) break;
      if (blockIdx.y == 0) {
        const uint8_t* p = smem + oQ + i * kQBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(p + ((c ^ (row & 7)) << 4));
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(v[e] << 16), y = __uint_as_float(v[e] & 0xffff0000u);
            sum = fmaf(x, x, fmaf(y, y, sum));
            any |= v[e] & 0x7fff7fffu;
          }
        }
        if (--left == 0) {
          norm += norm_above(sum, any != 0u);
          sum = 0.f;
          any = 0;
          left = parts;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(3 + i));
    }
    const size_t at = size_t(blockIdx.x) * kTile + row;
    if (!LISTS && ok && blockIdx.y == 0) a.norms[at] = norm;
    if (LISTS) named_bar_sync(1, kTile);  // all four warps have read the last slots for |q| (on an abort too)
    ok = ok && mbar_wait_warp(bar(5), 0, ctl);
    if (ok && LISTS) {  // (the products have read the operands too: their memory is free)
      tc_fence_after();
      const bool staged = kTile * (a.T | 1) * int(sizeof(int)) <= kScoreSlots * int(kQBytes);
      select_rows(a, tmem + (uint32_t(warp * 32) << 16), b, hs, q0, norm,
                  smem + warp * kSelectBuffer, staged ? reinterpret_cast<int*>(smem + oQ) : nullptr);
    } else if (ok) {
      tc_fence_after();
      float* dst = a.scores + at * a.pitch + j0;
#pragma unroll 1
      for (int c = 0; c < columns; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + (uint32_t(warp * 32) << 16) + c, v);
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          if (c + e < columns && q0 + row < a.NQ) st_global_v8(dst + c + e, v + e);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kN);
  }
}

// Whether the lists are found where the scores are.  A row a thread takes fewer
// instructions and longer: 45 us for one tile of 256 blocks, where a warp a row
// takes 26 with the scores through L2.  16384 causal queries x 8 selection heads
// x 256 blocks (1024 tiles): 143 and 239 us; 512 tiles of 64 blocks: 65 and 103; 64 tiles
// of 256: 76 and 47.  So from a wave of CTAs on, two for each of 152 SMs.  (Of 512
// blocks, with a CTA an SM, there was no gain to speak of.)  Rows whose border needs the
// exact scores of many blocks go the other way: 4096 queries x 16 selection heads x 128
// blocks take 88 and 128 us, with equal keys in half of them 0.78 and 0.29 ms, in all 4.0
// and 2.3.  A key that is not finite does the same to every row of its head.
bool lists_at_once(const SelectArgs& a) {
  return a.doc_q == nullptr && a.blocks <= kN && (long long)a.B * a.HS * a.tiles_q >= 304;
}

int launch_select(const CUtensorMap& tq, const CUtensorMap& tkb, SelectArgs a, int strip, cudaStream_t st) {
  const int all = a.B * a.HS * a.tiles_q;
  cudaError_t e = cudaMemsetAsync(a.kb_norm, 0, size_t(a.B) * a.HS * 4, st);
  if (e != cudaSuccess) return e;
  select_prep_kernel<<<dim3(unsigned((a.blocks + kPrepThreads / 32 - 1) / (kPrepThreads / 32)), unsigned(a.B * a.HS)),
                       kPrepThreads, 0, st>>>(a);
  const int parts = (a.d + 63) / 64;
  const bool lists = lists_at_once(a);
  const int smem = 1024 + parts * kN * 128 + kScoreSlots * int(kQBytes) + 64;
  auto kern = lists ? select_score_kernel<true> : select_score_kernel<false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           1024 + 2 * kN * 128 + kScoreSlots * int(kQBytes) + 64);
  if (e != cudaSuccess) return e;
  if (lists) {
    kern<<<unsigned(all), kScoreThreads, smem, st>>>(tq, tkb, a);
    return cudaGetLastError();
  }
  for (a.tile0 = 0; a.tile0 < all; a.tile0 += strip) {
    a.tiles = std::min(strip, all - a.tile0);
    kern<<<dim3(unsigned(a.tiles), unsigned((a.blocks + kN - 1) / kN)), kScoreThreads, smem, st>>>(tq, tkb, a);
    const int bytes = (a.blocks + 31) / 32 * 32 * 4, warps = std::max(1, std::min(kTopThreads / 32, 32768 / bytes));
    select_top_kernel<<<unsigned((a.tiles * kTile + warps - 1) / warps), 32 * warps, warps * bytes, st>>>(a);
  }
  return cudaGetLastError();
}

struct SelectPlan {
  SelectArgs a{};
  int strip = 0;  // query tiles
  size_t bytes = 0;
};

int check_select(const streamkl_view* q, const streamkl_view* kb, const streamkl_visible* vis, int B, int H, int heads,
                 int NQ, int NK, int d, int block, int count, int sink, int local, const int* selected, bool data) {
  if (B < 0 || H < 0 || NQ < 0 || NK < 0 || vis == nullptr) return STREAMKL_INVALID_ARG;
  if (vis->causal != 0 && vis->causal != 1) return STREAMKL_INVALID_ARG;
  if (vis->prefix != nullptr && !vis->causal) return STREAMKL_INVALID_ARG;
  if ((vis->doc_q == nullptr) != (vis->doc_k == nullptr)) return STREAMKL_INVALID_ARG;
  if (!aligned4(vis->prefix) || !aligned4(vis->doc_q) || !aligned4(vis->doc_k)) return STREAMKL_INVALID_ARG;
  if (block != 32 && block != 64 && block != 128) return STREAMKL_INVALID_ARG;
  if (count < 1 || count > kMaxSlots || sink < 0 || local < 0 || sink > count || local > count - sink)
    return STREAMKL_INVALID_ARG;
  if (heads < 1 || heads > std::max(H, 1) || H % heads != 0) return STREAMKL_INVALID_ARG;
  if (d < 16 || d > 128 || d % 16 != 0) return STREAMKL_UNSUPPORTED;
  const long long blocks = ((long long)NK + block - 1) / block;
  if (blocks > kMaxSelBlocks) return STREAMKL_UNSUPPORTED;
  if ((long long)B * H > 65535 || (long long)B * H * std::max(NQ, NK) > (1ll << 31) - 1 - 65535 * kTile)
    return STREAMKL_INVALID_ARG;
  if ((long long)B * heads * NQ * count > (1ll << 31) - 1) return STREAMKL_INVALID_ARG;
  if (!data || B == 0 || H == 0 || NQ == 0) return STREAMKL_OK;
  if (selected == nullptr || !aligned4(selected)) return STREAMKL_INVALID_ARG;
  if (NK == 0) return STREAMKL_INVALID_ARG;
  if (q == nullptr || kb == nullptr || !view_ok(*q, B, H, NQ) || !view_ok(*kb, B, heads, int(blocks))) return STREAMKL_INVALID_ARG;
  return STREAMKL_OK;
}

SelectPlan select_plan(const streamkl_visible& vis, int B, int H, int heads, int NQ, int NK, int d, int block, int count,
                       int sink, int local, void* ws) {
  SelectPlan f;
  SelectArgs& a = f.a;
  a.B = B;
  a.H = H;
  a.HS = heads;
  a.NQ = NQ;
  a.NK = NK;
  a.d = d;
  a.bs = block;
  a.blocks = (NK + block - 1) / block;
  a.T = count;
  a.sink = sink;
  a.local = local;
  a.heads = H / heads;
  a.pitch = (a.blocks + 7) / 8 * 8;
  a.tiles_q = tiles(NQ);
  a.causal = vis.causal;
  a.prefix = vis.prefix;
  a.doc_q = vis.doc_q;
  a.doc_k = vis.doc_k;
  // strips of at most 128 MB of scores: L2's size (with causal about half of them are written)
  const long long all = (long long)B * heads * a.tiles_q;
  f.strip = int(std::max(1ll, std::min(all, (128ll << 20) / (4ll * kTile * a.pitch))));
  Carver c{static_cast<uint8_t*>(ws)};
  const size_t pad = (32 - (reinterpret_cast<uintptr_t>(ws) & 31u)) & 31u;  // score rows start at 32 bytes
  c.used = pad;
  if (!lists_at_once(a)) {
    a.scores = c.take<float>(size_t(f.strip) * kTile * a.pitch);
    a.norms = c.take<float>(size_t(f.strip) * kTile);
  }
  a.kb_norm = c.take<unsigned>(size_t(B) * heads);
  if (vis.doc_q != nullptr) a.ranges = c.take<int2>(size_t(B) * a.blocks);
  f.bytes = c.used - pad + 16;
  return f;
}

}  // namespace

}  // namespace skl

extern "C" {

size_t streamkl_select_blocks_workspace_bytes(const streamkl_visible* vis, int B, int H, int heads, int NQ, int NK, int d,
                                              int block, int count, int sink, int local) {
  using namespace skl;
  if (check_select(nullptr, nullptr, vis, B, H, heads, NQ, NK, d, block, count, sink, local, nullptr, false) != STREAMKL_OK)
    return 0;
  if (B == 0 || H == 0 || NQ == 0 || NK == 0) return 0;
  return select_plan(*vis, B, H, heads, NQ, NK, d, block, count, sink, local, nullptr).bytes;
}

int streamkl_select_blocks(const streamkl_view* q, const streamkl_view* kb, const streamkl_visible* vis, int B, int H,
                           int heads, int NQ, int NK, int d, int block, int count, int sink, int local, int* selected,
                           void* workspace, size_t workspace_bytes, streamkl_stream_t stream) {
  using namespace skl;
  int s = check_select(q, kb, vis, B, H, heads, NQ, NK, d, block, count, sink, local, selected, true);
  if (s != STREAMKL_OK) return s;
  if (B == 0 || H == 0 || NQ == 0) return STREAMKL_OK;
  SelectPlan f = select_plan(*vis, B, H, heads, NQ, NK, d, block, count, sink, local, workspace);
  if (!workspace || !aligned16(workspace) || workspace_bytes < f.bytes) return STREAMKL_INVALID_ARG;
  if ((s = check_device()) != STREAMKL_OK) return s;
  CUtensorMap tq, tkb;
  if (!map_bf16(&tq, *q, B, H, NQ, d) || !map_bf16(&tkb, *kb, B, heads, f.a.blocks, d, kN)) return STREAMKL_CUDA_ERROR;
  auto rows = [&](const streamkl_view& v, int hd, int n) {
    return SelRows{static_cast<const uint8_t*>(v.data), B > 1 ? 2 * v.stride_b : 0, hd > 1 ? 2 * v.stride_h : 0,
                   n > 1 ? 2 * v.stride_n : 0, d / 8};
  };
  f.a.q = rows(*q, H, NQ);
  f.a.kb = rows(*kb, heads, f.a.blocks);
  f.a.selected = selected;
  f.a.status = status_word();
  if (!f.a.status) return STREAMKL_CUDA_ERROR;
  return as_status(launch_select(tq, tkb, f.a, f.strip, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
