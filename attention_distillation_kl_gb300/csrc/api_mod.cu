// C entry points over modified scores: argument validation, workspace layout,
// tensor maps, launches.  Every check that can fail does so before anything
// is enqueued.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host.cuh"
#include "kernels.cuh"
#include "mod_common.cuh"
#include "mod_host.cuh"
#include "streamkl.h"
#include "views.cuh"

namespace skl {

namespace {

int check_side(const streamkl_side* s, int B, int H, int NQ, int NK, bool data) {
  if (s == nullptr) return STREAMKL_INVALID_ARG;
  if (s->HK < 0 || s->HK > H || (H > 0 && (s->HK == 0 || H % s->HK != 0))) return STREAMKL_INVALID_ARG;
  if (!(std::isfinite(s->scale) && s->scale > 0.0 && s->scale <= 1.0e4)) return STREAMKL_INVALID_ARG;
  if (!(s->softcap == 0.f || (std::isfinite(s->softcap) && s->softcap >= 1.0e-3f && s->softcap <= 1.0e6f)))
    return STREAMKL_INVALID_ARG;
  if (s->slopes != nullptr && s->table != nullptr) return STREAMKL_INVALID_ARG;
  if (!aligned4(s->slopes) || !aligned4(s->table)) return STREAMKL_INVALID_ARG;
  if (s->table != nullptr) {
    if (s->bidirectional != 0 && s->bidirectional != 1) return STREAMKL_INVALID_ARG;
    const int n = s->bidirectional ? s->num_buckets / 2 : s->num_buckets;
    if (s->num_buckets < 2 || s->num_buckets > kMaxBuckets || n < 2) return STREAMKL_INVALID_ARG;
    if (s->bidirectional && s->num_buckets % 2 != 0) return STREAMKL_INVALID_ARG;
    if (s->max_distance <= n / 2 || s->max_distance > kMaxDistance) return STREAMKL_INVALID_ARG;
  }
  if (s->d < 16 || s->d > 128 || s->d % 16 != 0) return STREAMKL_UNSUPPORTED;
  if (data && (!view_ok(s->q, B, H, NQ) || !view_ok(s->k, B, s->HK, NK))) return STREAMKL_INVALID_ARG;
  return STREAMKL_OK;
}

// A direction's first distance of each bucket: one distance each up to half
// of them, then steps of the logarithm up to max_distance.  In 64 bits; a
// border that is a whole number (the logarithm's steps meet one whenever the
// ratio is a power) must not round up past itself.
void bucket_borders(ModPrepArgs::Table& t) {
  const int n = t.both ? t.num_buckets / 2 : t.num_buckets, e = n / 2;
  t.per_side = n;
  for (int i = 0; i < n; ++i)
    t.first[i] = i <= e ? i
                        : int(std::ceil(e * std::pow(double(t.max_distance) / e, double(i - e) / (n - e)) * (1.0 - 1e-12)));
}

}  // namespace

// Sizes, masks and both sides.  *empty: no query row (or head) to compute.
int check_call(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis, int B, int H, int NQ,
               int NK, bool data, bool* empty) {
  *empty = false;
  if (B < 0 || H < 0 || NQ < 0 || NK < 0 || vis == nullptr) return STREAMKL_INVALID_ARG;
  if (vis->causal != 0 && vis->causal != 1) return STREAMKL_INVALID_ARG;
  if (vis->prefix != nullptr && !vis->causal) return STREAMKL_INVALID_ARG;
  if ((vis->doc_q == nullptr) != (vis->doc_k == nullptr)) return STREAMKL_INVALID_ARG;
  if (!aligned4(vis->prefix) || !aligned4(vis->doc_q) || !aligned4(vis->doc_k)) return STREAMKL_INVALID_ARG;
  const long long BH = (long long)B * H;
  *empty = BH == 0 || NQ == 0;
  for (const streamkl_side* s : {p1, p2}) {
    const int e = check_side(s, B, H, NQ, NK, data && !*empty && NK > 0);
    if (e != STREAMKL_OK) return e;
  }
  if (*empty) return STREAMKL_OK;
  if (NK == 0) return STREAMKL_INVALID_ARG;
  if (BH > 65535 || BH * (long long)std::max(NQ, NK) > (1ll << 31) - 1 - 65535 * kTile) return STREAMKL_INVALID_ARG;
  return STREAMKL_OK;
}

// The part of the workspace that both calls use: ids and lookup rows.
void take_prep(Carver& c, ModPrepArgs& a, const streamkl_side* const p[2], const streamkl_visible& vis, int B, int H, int NQ,
               int NK, int table_grad_side) {
  a.B = B;
  a.H = H;
  a.NQ = NQ;
  a.NK = NK;
  a.doc_q = vis.doc_q;
  a.doc_k = vis.doc_k;
  if (vis.doc_q != nullptr) {
    a.ids_q = c.take<int>(size_t(B) * tiles(NQ) * kTile);
    a.ids_k = c.take<int>(size_t(B) * tiles(NK) * kTile);
    a.tiles_q = c.take<int4>(size_t(B) * tiles(NQ));
    a.tiles_k = c.take<int4>(size_t(B) * tiles(NK));
  }
  for (int i = 0; i < 2; ++i) {
    a.t[i].table = p[i]->table;
    if (p[i]->table == nullptr) continue;
    a.t[i].num_buckets = p[i]->num_buckets;
    a.t[i].max_distance = p[i]->max_distance;
    a.t[i].both = p[i]->bidirectional;
    if (c.base != nullptr) bucket_borders(a.t[i]);
    a.t[i].near = c.take<float>(size_t(H) * near_row(p[i]->max_distance));
    if (i == table_grad_side) a.t[i].bmap = c.take<int>(near_len(p[i]->max_distance));
  }
}

ModVis vis_args(const streamkl_visible& v, const ModPrepArgs& p) {
  return ModVis{v.causal, v.prefix, p.ids_q, p.ids_k, p.tiles_q, p.tiles_k};
}

}  // namespace skl

namespace {

using namespace skl;

bool make_maps(skl::ModMaps* m, const streamkl_side& p1, const streamkl_side& p2, int B, int H, int NQ, int NK,
               int q_rows = kTile) {
  return map_bf16(&m->q1, p1.q, B, H, NQ, p1.d, q_rows) && map_bf16(&m->k1, p1.k, B, p1.HK, NK, p1.d) &&
         map_bf16(&m->q2, p2.q, B, H, NQ, p2.d, q_rows) && map_bf16(&m->k2, p2.k, B, p2.HK, NK, p2.d);
}

skl::ModSide side_args(const streamkl_side& s, const float* near) {
  skl::ModSide m{};
  constexpr double kLog2e = 1.4426950408889634;
  const double scale = s.scale;  // rounded to fp32 once, in the products below
  m.scale = float(s.scale);
  // A cap so far above the scores that u falls below fp32's normal range
  // changes nothing: tanh(u x) = u x.
  const double u = s.softcap != 0.f ? scale / double(s.softcap) : 0.0;
  const bool capped = u >= double(FLT_MIN);
  m.cmul = float((capped ? double(s.softcap) : scale) * kLog2e);
  m.carg = capped ? float(u) : 0.f;
  m.poly[0] = m.cmul;
  // (beside a capped side an uncapped one is a polynomial of degree 0, of an
  // x^2 that has to be finite)
  m.zmax = 1e36f;
  if (capped) {
    // cmul tanh(carg x) = x poly(x^2): poly_k = cmul P_k carg^(2k + 1), where
    // those stay inside fp32's normal range
    const double c = double(s.softcap) * kLog2e;
    double p = c * u;
    bool fits = true;
    for (int k = 0; k < 5; ++k, p *= u * u) {
      const double v = p * skl::tanh_p(k);
      m.poly[k] = float(v);
      fits = fits && std::fabs(v) > 1e-36 && std::fabs(v) < 1e36;
    }
    const double z = double(skl::kTanhMax) * skl::kTanhMax / (u * u);
    fits = fits && z < 1e36 && z > 1e-30;
    m.zmax = fits ? float(z) : -1.f;
  }
  m.kind = s.slopes != nullptr ? skl::kBiasSlopes : (s.table != nullptr ? skl::kBiasTable : skl::kBiasNone);
  m.reach = s.table != nullptr ? s.max_distance : 0;
  m.slopes = s.slopes;
  m.near = near;
  return m;
}

struct FwdPlan {
  skl::ModPrepArgs prep{};
  float* partial = nullptr;
  size_t bytes = 0;
};

FwdPlan fwd_plan(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible& vis, int B, int H, int NQ, int NK,
                 int splits, void* ws) {
  FwdPlan f;
  Carver c{static_cast<uint8_t*>(ws)};
  const streamkl_side* const p[2] = {p1, p2};
  take_prep(c, f.prep, p, vis, B, H, NQ, NK, -1);
  if (splits > 1) f.partial = c.take<float>(size_t(5) * splits * B * H * NQ);
  f.bytes = c.used;
  return f;
}

// Query heads that share a key head on both sides also share a 128-row tile
// when their rows fit: K is then read once for all of them.  As many as a
// power of two allows; 32 heads on 8 key heads x 16 rows x 32768 keys,
// d = 128, both sides capped: 109 us without, 36 with (19 splits of 4 heads
// each), merge included.
int pack_shift(int H, int HK1, int HK2, int NQ) {
  int s = 0;
  while (s < 3 && (H / HK1) % (2 << s) == 0 && (H / HK2) % (2 << s) == 0 && NQ <= (kTile >> (s + 1))) ++s;
  return s;
}

// The library's choice of key splits for `tiles_q` query tiles in all: with s
// splits a launch takes ceil(CTAs / SMs) rounds of (key tiles / s + kFixed),
// in units of one key tile of one CTA, plus the merge.  (Ids are not looked
// at: they live on the device.)
int resolve_splits(int splits, long long tiles_q, double rows, int NK) {
  if (splits != 0) return splits;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 1;
  const double ctas = double(tiles_q);
  const int longest = tiles(NK);
  if (ctas >= 2.0 * sms || longest < 4) return 1;  // rounds of whole rows
  constexpr double kFixed = 3.0, kMerge = 4.0, kMergeRowsPerTile = 2.0e5;
  int best = 1;
  double best_t = std::ceil(ctas / sms) * (longest + kFixed);
  for (int s = 2; s <= longest / 2 && s <= 1024; ++s) {
    const double t = std::ceil(ctas * s / sms) * ((longest + s - 1) / s + kFixed) + kMerge + rows * s / kMergeRowsPerTile;
    if (t < 0.98 * best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

int fwd_splits(int splits, const streamkl_side& p1, const streamkl_side& p2, int B, int H, int NQ, int NK) {
  const int shift = pack_shift(H, p1.HK, p2.HK, NQ);
  return resolve_splits(splits, (long long)B * (H >> shift) * tiles(NQ), double(B) * H * NQ, NK);
}

struct BwdPlan {
  skl::ModPrepArgs prep{};
  float* dq32 = nullptr;
  float* dk32 = nullptr;
  float* dtab = nullptr;
  unsigned* words = nullptr;  // kmax per key head, ticket, abort, turns
  size_t bytes = 0;
  int pitch = 0;
};

BwdPlan bwd_plan(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible& vis, int B, int H, int NQ,
                 int NK, int mode, int deterministic, bool table, void* ws) {
  BwdPlan f;
  Carver c{static_cast<uint8_t*>(ws)};
  const streamkl_side* const p[2] = {p1, p2};
  const int gs = mode == STREAMKL_GRAD_P2 ? 1 : 0;
  const streamkl_side& g = *p[gs];
  f.pitch = (g.d + 31) / 32 * 32;
  // what starts at zero comes first, in one piece
  f.dq32 = c.take<float>(size_t(B) * H * NQ * f.pitch);
  const bool shared = g.HK != H;
  if (deterministic)
    f.words = c.take<unsigned>(size_t(B) * g.HK + (shared ? 2 + size_t(B) * g.HK * tiles(NK) : 0));
  const size_t dk_count = size_t(B) * g.HK * NK * f.pitch;
  if (shared && !deterministic) f.dk32 = c.take<float>(dk_count);
  if (table) f.dtab = c.take<float>(size_t(B) * H * tiles(NK) * 8 * skl::kMaxBuckets);
  f.prep.zero = static_cast<uint4*>(ws);
  f.prep.zero_words = c.used / 16;
  if (shared && deterministic) f.dk32 = c.take<float>(dk_count);
  take_prep(c, f.prep, p, vis, B, H, NQ, NK, table ? gs : -1);
  f.bytes = c.used;
  return f;
}

}  // namespace

extern "C" {

size_t streamkl_fwd_mod_workspace_bytes(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                                        int B, int H, int NQ, int NK, int num_splits) {
  bool empty = false;
  if (check_call(p1, p2, vis, B, H, NQ, NK, false, &empty) != STREAMKL_OK || empty) return 0;
  if (num_splits < 0 || num_splits > 1024) return 0;
  return fwd_plan(p1, p2, *vis, B, H, NQ, NK, fwd_splits(num_splits, *p1, *p2, B, H, NQ, NK), nullptr).bytes;
}

int streamkl_fwd_mod(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis, int B, int H, int NQ,
                     int NK, int num_splits, void* workspace, size_t workspace_bytes, float* kl, float* lse1,
                     float* lse2, streamkl_stream_t stream) {
  bool empty = false;
  int s = check_call(p1, p2, vis, B, H, NQ, NK, true, &empty);
  if (s != STREAMKL_OK) return s;
  if (num_splits < 0 || num_splits > 1024) return STREAMKL_INVALID_ARG;
  if (empty) return STREAMKL_OK;
  if (!kl || !lse1 || !lse2 || !aligned16(kl) || !aligned16(lse1) || !aligned16(lse2)) return STREAMKL_INVALID_ARG;
  const int splits = fwd_splits(num_splits, *p1, *p2, B, H, NQ, NK);
  const FwdPlan f = fwd_plan(p1, p2, *vis, B, H, NQ, NK, splits, workspace);
  if (f.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < f.bytes)) return STREAMKL_INVALID_ARG;
  if ((s = skl::check_device()) != STREAMKL_OK) return s;
  skl::ModMaps m{};
  const int shift = pack_shift(H, p1->HK, p2->HK, NQ);
  if (!make_maps(&m, *p1, *p2, B, H, NQ, NK, kTile >> shift)) return STREAMKL_CUDA_ERROR;
  int* st = skl::status_word();
  if (!st) return STREAMKL_CUDA_ERROR;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (skl::launch_mod_prep(f.prep, cs) != 0) return STREAMKL_CUDA_ERROR;
  skl::ModFwdArgs a{};
  a.B = B;
  a.H = H;
  a.NQ = NQ;
  a.NK = NK;
  a.num_splits = splits;
  a.g1 = H / p1->HK;
  a.g2 = H / p2->HK;
  a.s1 = side_args(*p1, f.prep.t[0].near);
  a.s2 = side_args(*p2, f.prep.t[1].near);
  a.vis = vis_args(*vis, f.prep);
  a.kl = kl;
  a.lse1 = lse1;
  a.lse2 = lse2;
  a.partial = f.partial;
  a.status = st;
  a.pack_shift = shift;
  a.head_group = skl::l2_head_group(B * (H >> shift), 2.0 * NK * (p1->d + p2->d));
  const int t2 = tile_width(p2->d);
  if ((tile_width(p1->d) == 64 ? skl::launch_fwd_mod_64(m, t2, a, cs) : skl::launch_fwd_mod_128(m, t2, a, cs)) != 0)
    return STREAMKL_CUDA_ERROR;
  if (splits == 1) return STREAMKL_OK;
  return as_status(skl::launch_mod_reduce(a, cs));
}

size_t streamkl_bwd_mod_workspace_bytes(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                                        int B, int H, int NQ, int NK, int mode, int deterministic, int table_grad) {
  bool empty = false;
  if (check_call(p1, p2, vis, B, H, NQ, NK, false, &empty) != STREAMKL_OK || empty) return 0;
  if (mode != STREAMKL_GRAD_P2 && mode != STREAMKL_GRAD_P1) return 0;
  if (deterministic != 0 && deterministic != 1) return 0;
  const streamkl_side* g = mode == STREAMKL_GRAD_P2 ? p2 : p1;
  return bwd_plan(p1, p2, *vis, B, H, NQ, NK, mode, deterministic, table_grad != 0 && g->table != nullptr, nullptr).bytes;
}

int streamkl_bwd_mod(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis, int B, int H, int NQ,
                     int NK, const float* kl, const float* lse1, const float* lse2, const float* dkl, int mode,
                     int deterministic, const streamkl_view* dq, const streamkl_view* dk, float* dtable,
                     void* workspace, size_t workspace_bytes, streamkl_stream_t stream) {
  bool empty = false;
  int s = check_call(p1, p2, vis, B, H, NQ, NK, true, &empty);
  if (s != STREAMKL_OK) return s;
  if (mode != STREAMKL_GRAD_P2 && mode != STREAMKL_GRAD_P1) return STREAMKL_INVALID_ARG;
  if (deterministic != 0 && deterministic != 1) return STREAMKL_INVALID_ARG;
  const streamkl_side& g = mode == STREAMKL_GRAD_P2 ? *p2 : *p1;
  if (dtable != nullptr && (g.table == nullptr || !aligned4(dtable))) return STREAMKL_INVALID_ARG;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (empty) {
    // no query rows: nothing reaches K or the table
    if (dtable != nullptr && H > 0 &&
        cudaMemsetAsync(dtable, 0, size_t(H) * g.num_buckets * 4, cs) != cudaSuccess)
      return STREAMKL_CUDA_ERROR;
    if (B == 0 || H == 0 || NK == 0) return STREAMKL_OK;
    if (dk == nullptr || !view_ok(*dk, B, g.HK, NK)) return STREAMKL_INVALID_ARG;
    skl::ModFinishArgs fin{};
    fin.rows[0] = {nullptr, B * g.HK, g.HK, NK, g.d, 0, static_cast<__nv_bfloat16*>(dk->data), B > 1 ? dk->stride_b : 0,
                   g.HK > 1 ? dk->stride_h : 0, NK > 1 ? dk->stride_n : 0};
    return as_status(skl::launch_mod_finish(fin, cs));
  }
  if (!kl || !lse1 || !lse2 || !dkl || !aligned16(kl) || !aligned16(lse1) || !aligned16(lse2) || !aligned16(dkl))
    return STREAMKL_INVALID_ARG;
  if (dq == nullptr || dk == nullptr || !view_ok(*dq, B, H, NQ) || !view_ok(*dk, B, g.HK, NK))
    return STREAMKL_INVALID_ARG;
  const BwdPlan f = bwd_plan(p1, p2, *vis, B, H, NQ, NK, mode, deterministic, dtable != nullptr, workspace);
  if (!workspace || !aligned16(workspace) || workspace_bytes < f.bytes) return STREAMKL_INVALID_ARG;
  if ((s = skl::check_device()) != STREAMKL_OK) return s;
  skl::ModMaps m{};
  if (!make_maps(&m, *p1, *p2, B, H, NQ, NK) || !map_f32(&m.dq, f.dq32, B * H, NQ, f.pitch))
    return STREAMKL_CUDA_ERROR;
  if (f.dk32 != nullptr && !map_f32(&m.dk, f.dk32, B * g.HK, NK, f.pitch)) return STREAMKL_CUDA_ERROR;
  int* st = skl::status_word();
  if (!st) return STREAMKL_CUDA_ERROR;
  skl::ModBwdArgs a{};
  a.B = B;
  a.H = H;
  a.NQ = NQ;
  a.NK = NK;
  a.g1 = H / p1->HK;
  a.g2 = H / p2->HK;
  a.s1 = side_args(*p1, f.prep.t[0].near);
  a.s2 = side_args(*p2, f.prep.t[1].near);
  a.vis = vis_args(*vis, f.prep);
  a.kl = kl;
  a.lse1 = lse1;
  a.lse2 = lse2;
  a.dkl = dkl;
  a.dg = g.d;
  a.pitch = f.pitch;
  a.dq32 = f.dq32;
  a.dk32 = f.dk32;
  a.dk = dk->data;
  a.dk_sb = B > 1 ? dk->stride_b : 0;
  a.dk_sh = g.HK > 1 ? dk->stride_h : 0;
  a.dk_sn = NK > 1 ? dk->stride_n : 0;
  a.bmap = f.prep.t[mode == STREAMKL_GRAD_P2 ? 1 : 0].bmap;
  a.reach = g.table != nullptr ? g.max_distance : 0;
  a.dtab = f.dtab;
  a.status = st;
  a.head_group = skl::l2_head_group(B * H, 2.0 * NQ * (p1->d + p2->d) + 4.0 * NQ * f.pitch);
  if (skl::launch_mod_prep(f.prep, cs) != 0) return STREAMKL_CUDA_ERROR;
  if (deterministic) {
    if (skl::launch_kmax_strided(g.k.data, B, g.HK, NK, g.d, B > 1 ? g.k.stride_b : 0, g.HK > 1 ? g.k.stride_h : 0,
                                 NK > 1 ? g.k.stride_n : 0, f.prep.ids_k, f.words, cs) != 0)
      return STREAMKL_CUDA_ERROR;
    a.dq_fixed = 1;
    a.kmax = f.words;
    if (g.HK != H) {
      int* w = reinterpret_cast<int*>(f.words) + size_t(B) * g.HK;
      a.ticket = w;
      a.dk_abort = w + 1;
      a.dk_turns = w + 2;
      a.head_group = 1;
    }
  }
  const int t1 = tile_width(p1->d), t2 = tile_width(p2->d);
  if ((mode == STREAMKL_GRAD_P2 ? skl::launch_bwd_mod_p2(m, t1, t2, a, cs) : skl::launch_bwd_mod_p1(m, t1, t2, a, cs)) != 0)
    return STREAMKL_CUDA_ERROR;
  skl::ModFinishArgs fin{};
  fin.rows[0] = {f.dq32, B * H, H, NQ, g.d, f.pitch, static_cast<__nv_bfloat16*>(dq->data), B > 1 ? dq->stride_b : 0,
                 H > 1 ? dq->stride_h : 0, NQ > 1 ? dq->stride_n : 0};
  if (f.dk32 != nullptr)
    fin.rows[1] = {f.dk32, B * g.HK, g.HK, NK, g.d, f.pitch, static_cast<__nv_bfloat16*>(dk->data), a.dk_sb, a.dk_sh,
                   a.dk_sn};
  fin.dtab = f.dtab;
  fin.B = B;
  fin.H = H;
  fin.nkt = tiles(NK);
  fin.num_buckets = g.num_buckets;
  fin.dtable = dtable;
  return as_status(skl::launch_mod_finish(fin, cs));
}

}  // extern "C"
