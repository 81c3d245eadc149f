// Modified scores: what the kernels of streamkl_fwd_mod and streamkl_bwd_mod
// share.  With r = j - i - (NK - NQ) (the key's position relative to the
// query's), each side's score is
//   S = Y + bias_h(r),  Y = cap tanh(s x / cap)  (x = q.k; no cap: Y = s x)
//   bias_h(r) = -slope_h |r|,  or table[h][bucket(r)]
// and key j is visible to query i iff
//   (not causal, or r <= 0, or j < prefix[b])  and  (no ids, or id_q[i] == id_k[j] >= 0).
// The kernels work in base 2: e = S log2 e.
#pragma once

#include <cuda_bf16.h>

#include "kernels.cuh"
#include "ptx.cuh"

namespace skl {

// A tile is 128 x 128, so the relative positions inside one span 255 values:
// a lookup row that reaches kNearPad past the last distance whose bucket can
// differ serves every tile that touches such a distance without a clamp.
constexpr int kNearPad = 256;
constexpr float kLog2eLo = 1.925963033500e-8f;  // log2 e beyond kLog2e
constexpr int kMaxBuckets = 64;
constexpr int kMaxDistance = 4096;

enum { kBiasNone = 0, kBiasSlopes = 1, kBiasTable = 2 };

__host__ __device__ inline int near_len(int reach) { return 2 * (reach + kNearPad) + 1; }
// A head's row in memory: those, then what the rounding of the first and the
// last of them to fp32 lost, then the score below which a row of this head
// sees only masks (half of the largest entry that is one; without one -inf).
__host__ __device__ inline int near_row(int reach) { return near_len(reach) + 3; }

// Base 2: table entries below this (-6.9e5) are masks.
constexpr float kLow = -1.0e6f;

struct ModSide {
  float scale;          // s
  float cmul;           // multiplies tanh (capped: cap log2 e) or x (s log2 e)
  float carg;           // s / cap; 0 without a cap
  float poly[5];        // Y log2 e = x poly(x^2) where x^2 <= zmax (no cap: cmul, 0, 0, 0, 0)
  float zmax;           // 1e36 without a cap; below 0: nowhere
  int kind;             // kBiasNone, kBiasSlopes, kBiasTable
  int reach;            // table: buckets do not change beyond |r| = reach
  const float* slopes;  // [H]
  const float* near;    // [H][near_row(reach)]: bias log2 e at r = index - reach - kNearPad
};

struct ModVis {
  int causal;
  const int* prefix;     // [B] or null
  // from mod_prep_kernel, null without ids: ids padded to whole tiles, and
  // per tile (min, max, uniform) of the ids that can match anything
  const int* ids_q;      // [B][nqt * 128]; a row that matches nothing holds -2
  const int* ids_k;      // [B][nkt * 128]; a key that matches nothing holds -1
  const int4* tiles_q;   // [B][nqt]
  const int4* tiles_k;   // [B][nkt]
};

struct ModMaps {
  // 4-D (d, N, heads, B) bf16, boxes of 64 x 128 x 1 x 1 (q with packed heads: 128 >> pack_shift rows), 128-byte swizzle
  CUtensorMap q1, k1, q2, k2;
  CUtensorMap dq;              // [BH][NQ][pitch] fp32, boxes of 32 x 32, 128-byte swizzle (backward)
  CUtensorMap dk;              // [B HK_g][NK][pitch] fp32, the same (shared key heads)
};

struct ModFwdArgs {
  int B, H, NQ, NK, num_splits;
  int g1, g2;  // query heads per key head
  ModSide s1, s2;
  ModVis vis;
  float* kl;
  float* lse1;
  float* lse2;
  float* partial;  // [num_splits][5][B H NQ] or null
  int* status;
  int head_group;
  int near_smem;   // lookup rows are copied to shared memory
  int pack_shift;  // 2^pack_shift query heads share a 128-row tile (few rows), 128 >> pack_shift rows each
};

struct ModBwdArgs {
  int B, H, NQ, NK;
  int g1, g2;
  ModSide s1, s2;
  ModVis vis;
  const float* kl;
  const float* lse1;
  const float* lse2;
  const float* dkl;
  int dg, pitch;       // head dim of the gradient side; row length of dq32 and dk32 (a multiple of 32)
  float* dq32;         // [BH][NQ][pitch], zeroed: the dQ reduce-adds
  float* dk32;         // [B HK_g][NK][pitch]: dK of shared key heads (zeroed), null when each has one query head
  void* dk;            // bf16 dK (element strides below), written directly when dk32 is null
  long long dk_sb, dk_sh, dk_sn;
  int near_smem;       // as ModFwdArgs
  int reach;           // of the gradient side's table (table gradient)
  const int* bmap;     // [near_len(reach)]: bucket of r = index - reach - kNearPad
  float* dtab;         // [BH][nkt][8][kMaxBuckets], zeroed: each warp's sums of dS by bucket, or null
  int* status;
  int dq_fixed;        // deterministic: dQ contributions on their row's grid (dq_fixed_exp)
  const unsigned* kmax;
  int* ticket;         // deterministic with shared key heads (see BwdArgs)
  int* dk_turns;
  int* dk_abort;
  int head_group;
};

// Work before the main launch, in one kernel: a region of the workspace
// zeroed, ids padded and their tiles' ranges found, lookup rows filled.
struct ModPrepArgs {
  int B, H, NQ, NK;
  uint4* zero;
  size_t zero_words;  // 16-byte words
  const int* doc_q;
  const int* doc_k;
  int* ids_q;
  int* ids_k;
  int4* tiles_q;
  int4* tiles_k;
  struct Table {
    const float* table;  // [H][num_buckets] or null
    int num_buckets, max_distance, both;
    int per_side;            // buckets of a direction
    int first[kMaxBuckets];  // a direction's first distance of each
    float* near;
    int* bmap;  // or null
  } t[2];
};

// Work after the backward's main launch, in one kernel: fp32 rows rounded to
// bf16 (null source: zeros), and the warps' bucket sums added up.
struct ModFinishArgs {
  struct Rows {
    const float* src;  // [B per_batch][n][pitch]
    int heads, per_batch, n, d, pitch;
    __nv_bfloat16* dst;  // strides in elements; null: nothing to do
    long long sb, sh, sn;
  } rows[2];
  const float* dtab;
  int B, H, nkt, num_buckets;
  float* dtable;  // or null
};

int launch_mod_prep(const ModPrepArgs& a, cudaStream_t st);
// d1, d2: tile widths, 64 or 128
int launch_fwd_mod_64(const ModMaps& m, int d2, const ModFwdArgs& a, cudaStream_t st);
int launch_fwd_mod_128(const ModMaps& m, int d2, const ModFwdArgs& a, cudaStream_t st);
int launch_mod_reduce(const ModFwdArgs& a, cudaStream_t st);
int launch_bwd_mod_p2(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st);
int launch_bwd_mod_p1(const ModMaps& m, int d1, int d2, const ModBwdArgs& a, cudaStream_t st);
int launch_mod_finish(const ModFinishArgs& a, cudaStream_t st);
// ids: of the keys, padded to whole tiles (ModVis::ids_k), or null
int launch_kmax_strided(const void* k, int B, int per_batch, int n, int d, long long sb, long long sh, long long sn,
                        const int* ids, unsigned* kmax, cudaStream_t st);

// ------------------------------------------------------------------ device

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y,
                                            int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Rows [row0, row0 + 128) of (batch, head) into the operand tile at base.
template <typename T>
__device__ __forceinline__ void load_tile(uint32_t base, const CUtensorMap* m, uint32_t bar, int row0, int head,
                                          int batch) {
#pragma unroll
  for (int c = 0; c < T::kBlocks; ++c) tma_load_4d(base + c * T::kBlockBytes, m, bar, c * T::kBox, row0, head, batch);
}

// 16 columns of two tiles for the warp's 32 rows, and the wait for them.
__device__ __forceinline__ void tmem_ld2x16(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SKL_R8(a, 0), SKL_R8(a, 8), SKL_R8(b, 0), SKL_R8(b, 8)
      : "r"(ta), "r"(tb)
      : "memory");
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(u) = u P(u^2) for |u| <= 1/2: P of degree 4, fitted for a small
// largest relative error there (2.9e-8; 1.1e-7 with the roundings of fp32).
// A warp whose scores all stay inside half of their cap has no MUFU operation
// beside the softmax's own; one that meets a larger score takes cap_any for
// the tile (forward at 8K x 32 heads, d = 128, both caps 50: 778 us with
// scores of standard deviation 2.6 to 4, 1132 at 6, 2520 at 8, where nearly
// every warp does; the backward at 4K: 446, 782, 953).  The scale and the
// cap are folded into the coefficients (ModSide::poly), so a pair of capped
// scores costs six packed operations: x^2, four steps, and one that also
// adds the bias.  The FMA pipe bounds it: folding the coefficients and the
// reference of the softmax took the forward at 8K x 32 heads, d = 128, both
// sides capped, from 1105 us to 788 us.
constexpr float kTanhMax = 0.5f;
__host__ __device__ constexpr float tanh_p(int k) {
  return k == 0 ? 1.0f : k == 1 ? -0.33333069f : k == 2 ? 0.13324779f : k == 3 ? -0.052986074f : 0.017135005f;
}

// What turns products into base-2 scores, held in registers by the loops:
// the coefficients as pairs (capped), or cmul in p[0].
struct SideRegs {
  uint64_t p[5];
};
template <bool CAP>
__device__ __forceinline__ SideRegs side_regs(const ModSide& s) {
  SideRegs r;
#pragma unroll
  for (int k = 0; k < (CAP ? 5 : 1); ++k) {
    const float v = CAP ? s.poly[k] : s.cmul;
    r.p[k] = f2(v, v);
    asm volatile("" : "+l"(r.p[k]));  // in registers, not taken from the arguments again at each use
  }
  return r;
}

// poly(z) for two columns.
__device__ __forceinline__ uint64_t cap_poly(const SideRegs& s, uint64_t Z) {
  uint64_t P = f2_fma(Z, s.p[4], s.p[3]);
  P = f2_fma(Z, P, s.p[2]);
  P = f2_fma(Z, P, s.p[1]);
  return f2_fma(Z, P, s.p[0]);
}

// cmul tanh(carg x) for any x: the polynomial, and beyond it
// 1 - 2 / (1 + e^(2u)), whose subtraction loses at most two bits there
// (2^126 stands for everything above: the quotient is 0).
__device__ __forceinline__ float cap_any(float x, float cmul, float carg) {
  const float u = x * carg, z = u * u;
  float t = fmaf(z, tanh_p(4), tanh_p(3));
  t = fmaf(z, t, tanh_p(2));
  t = fmaf(z, t, tanh_p(1));
  t = fmaf(z, t, tanh_p(0)) * u;
  if (!(fabsf(u) <= kTanhMax)) t = fmaf(-2.f, rcp_approx(1.f + ex2(fminf(u * (2.f * kLog2e), 126.f))), 1.f);
  if (u != u) t = u;  // (fminf drops a NaN)
  return cmul * t;
}

// A side's bias over one tile, from the tile's range of relative positions:
// kFlat: base + step r (slopes on one side of the diagonal; a table beyond
// its reach, step 0); kFold: -step |r| (slopes across the diagonal);
// kLook: near[r] (a table within its reach); kZero: none.
enum { kZero = 0, kFlat = 1, kFold = 2, kLook = 3 };

struct alignas(16) HeadBias {  // of one head, base 2
  int kind, reach;
  float slope;
  float left, right;        // the table's value far to the left and to the right
  float left_lo, right_lo;  // and what its rounding lost
  float masked;             // a row whose largest score is below this sees only masks
  const float* near;  // its lookup row (shared memory where there is room)
};

__device__ __forceinline__ HeadBias head_bias(const ModSide& s, int h) {
  HeadBias b{s.kind, s.reach, 0.f, 0.f, 0.f, 0.f, 0.f, -INFINITY, nullptr};
  if (s.kind == kBiasSlopes) b.slope = s.slopes[h] * kLog2e;
  if (s.kind == kBiasTable) {
    const int len = near_len(s.reach);
    b.near = s.near + size_t(h) * near_row(s.reach);
    b.left = b.near[0];
    b.right = b.near[len - 1];
    b.left_lo = b.near[len];
    b.right_lo = b.near[len + 1];
    b.masked = b.near[len + 2];
  }
  return b;
}

// Copies the lookup rows of `count` HeadBias into shared memory at dst, one
// after the other, by the whole block; a __syncthreads before and after.
__device__ __forceinline__ void near_to_smem(HeadBias* hb, int count, float* dst) {
  for (int i = 0; i < count; ++i) {
    if (hb[i].kind != kBiasTable) continue;
    const int len = near_len(hb[i].reach);
    for (int p = threadIdx.x; p < len; p += blockDim.x) dst[p] = hb[i].near[p];
    dst += len;
  }
}
// Then, by one thread: where they are.
__device__ __forceinline__ void near_in_smem(HeadBias* hb, int count, const float* src) {
  for (int i = 0; i < count; ++i) {
    if (hb[i].kind != kBiasTable) continue;
    hb[i].near = src;
    src += near_len(hb[i].reach);
  }
}
__host__ __device__ inline size_t near_smem_bytes(const ModSide& s1, const ModSide& s2, int heads) {
  size_t n = 0;
  if (s1.kind == kBiasTable) n += near_len(s1.reach);
  if (s2.kind == kBiasTable) n += near_len(s2.reach);
  return n * heads * 4;
}

struct TileBias {
  int how;
  float base, step;
};

// rmin, rmax: the tile's smallest and largest relative position.
__device__ __forceinline__ TileBias tile_bias(const HeadBias& b, int rmin, int rmax) {
  TileBias t{kZero, 0.f, 0.f};
  if (b.kind == kBiasSlopes) {
    t.how = kFlat;
    t.step = rmin >= 0 ? -b.slope : b.slope;
    if (rmin < 0 && rmax > 0) t.how = kFold;
  } else if (b.kind == kBiasTable) {
    t.how = kFlat;
    t.base = rmax <= -b.reach ? b.left : b.right;
    if (rmax > -b.reach && rmin < b.reach) t.how = kLook;
  }
  return t;
}

// The bias of neighbouring columns of a row, plus `add`: rf = float(r) of
// column 0; near0: column 0's entry (kLook).
struct RowBias {
  float rf, step, first, add;  // first = base + step rf + add
  const float* near0;
};
__device__ __forceinline__ RowBias row_bias(const HeadBias& b, const TileBias& t, int r0, float add) {
  const float rf = float(r0);
  return RowBias{rf, t.step, fmaf(t.step, rf, t.base) + add, add, b.near + (r0 + b.reach + kNearPad)};
}
// What `first` of a flat table's row lost to rounding, in base 2.
__device__ __forceinline__ float flat_lost(const HeadBias& b, const TileBias& t, const RowBias& r, int rmax) {
  if (b.kind != kBiasTable || t.how != kFlat) return 0.f;
  const float x = r.first - t.base;
  return (t.base - (r.first - x)) + (r.add - x) + (rmax <= -b.reach ? b.left_lo : b.right_lo);
}
// The same n columns further on.
__device__ __forceinline__ RowBias further(const RowBias& b, int n) {
  return RowBias{b.rf + float(n), b.step, fmaf(b.step, float(n), b.first), b.add, b.near0 + n};
}
// Columns k to k + 3 as two pairs.
struct Quad {
  uint64_t lo, hi;
};
template <int HOW>
__device__ __forceinline__ Quad bias_quad(const RowBias& b, int k) {
  if (HOW == kFlat) {
    const uint64_t S = f2(b.step, b.step), F = f2(b.first, b.first);
    return Quad{f2_fma(S, f2(float(k), float(k + 1)), F), f2_fma(S, f2(float(k + 2), float(k + 3)), F)};
  }
  if (HOW == kFold) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(-b.step, fabsf(b.rf + float(k + i)), b.add);
    return Quad{f2(v[0], v[1]), f2(v[2], v[3])};
  }
  if (HOW == kLook) {
    const uint64_t A = f2(b.add, b.add);
    return Quad{f2_add(f2(b.near0[k], b.near0[k + 1]), A), f2_add(f2(b.near0[k + 2], b.near0[k + 3]), A)};
  }
  return Quad{f2(b.add, b.add), f2(b.add, b.add)};
}

// Base-2 score + bias + add of N columns of a row, as pairs; returns the
// largest x^2 of a capped side (0 without a cap): beyond ModSide::zmax the
// values are wrong and scores_any has to be called instead.  (Pairs stay
// pairs from here to the sums: taken apart into an array and packed again,
// they cost a move for each score.)
template <bool CAP, int HOW, int N>
__device__ __forceinline__ float scores_how(const uint32_t (&x)[N], uint64_t (&e)[N / 2], const SideRegs& s,
                                            const RowBias& b) {
  float za = 0.f, zb = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const Quad q = bias_quad<HOW>(b, k);
    const uint64_t X = f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    const uint64_t Y = f2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
    uint64_t M = s.p[0], L = s.p[0];
    if (CAP) {
      const uint64_t Z = f2_mul(X, X), W = f2_mul(Y, Y);
      float u, v;
      f2_split(Z, u, v);
      za = max3(za, u, v);
      f2_split(W, u, v);
      zb = max3(zb, u, v);
      M = cap_poly(s, Z);
      L = cap_poly(s, W);
    }
    e[k / 2] = f2_fma(X, M, q.lo);
    e[k / 2 + 1] = f2_fma(Y, L, q.hi);
  }
  return fmaxf(za, zb);
}
// BIASED = false: how is kZero.
template <bool CAP, bool BIASED, int N>
__device__ __forceinline__ float scores(const uint32_t (&x)[N], uint64_t (&e)[N / 2], const SideRegs& s, int how,
                                        const RowBias& b) {
  if (!BIASED || how == kZero) return scores_how<CAP, kZero>(x, e, s, b);
  if (how == kFlat) return scores_how<CAP, kFlat>(x, e, s, b);
  if (how == kFold) return scores_how<CAP, kFold>(x, e, s, b);
  return scores_how<CAP, kLook>(x, e, s, b);
}

// The bias of column k alone.
__device__ __forceinline__ float bias_one(const RowBias& b, int how, int k) {
  if (how == kFlat) return fmaf(b.step, float(k), b.first);
  if (how == kFold) return fmaf(-b.step, fabsf(b.rf + float(k)), b.add);
  if (how == kLook) return b.near0[k] + b.add;
  return b.add;
}

// The same for products of any size.
template <bool CAP, bool BIASED, int N>
__device__ __forceinline__ void scores_any(const uint32_t (&x)[N], uint64_t (&e)[N / 2], const ModSide& s, int how,
                                           const RowBias& b) {
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float t = __uint_as_float(x[k + i]);
      v[i] = (CAP && s.carg != 0.f ? cap_any(t, s.cmul, s.carg) : s.cmul * t) + (BIASED ? bias_one(b, how, k + i) : b.add);
    }
    e[k / 2] = f2(v[0], v[1]);
  }
}

// Visible columns (bit k) of the N columns that begin at key j0, for query i.
// ids: the query's id; kids: the ids of the columns (16-byte aligned), or
// null when every id of the tile pair is the same.
template <int N>
__device__ __forceinline__ uint32_t visible_bits(int i, int j0, int off, int NK, int causal, int prefix, int id,
                                                 const int* kids) {
  int n = NK - j0;
  if (causal) n = min(n, max(i + off + 1, prefix) - j0);
  constexpr uint32_t kAll = 0xffffffffu >> (32 - N);
  uint32_t bits = n >= N ? kAll : (n <= 0 ? 0u : (1u << n) - 1u);
  if (kids != nullptr) {
    uint32_t same = 0;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const int4 v = *reinterpret_cast<const int4*>(kids + k);
      same |= (v.x == id ? 1u : 0u) << k;
      same |= (v.y == id ? 1u : 0u) << (k + 1);
      same |= (v.z == id ? 1u : 0u) << (k + 2);
      same |= (v.w == id ? 1u : 0u) << (k + 3);
    }
    bits &= same;
  }
  return bits;
}

// Whether tiles with these id ranges can share an id.
__device__ __forceinline__ bool tiles_meet(int4 a, int4 b) { return a.x <= b.y && b.x <= a.y; }
// Whether every pair of them shares one.
__device__ __forceinline__ bool tiles_same(int4 a, int4 b) { return a.z && b.z && a.x == b.x; }

}  // namespace skl
