// C entry points over selected blocks: argument validation, workspace layout,
// tensor maps, launches.  Every check that can fail does so before anything
// is enqueued.
#include <algorithm>
#include <numeric>

#include "mod_host.cuh"
#include "sel_common.cuh"

namespace {

using namespace skl;

int num_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

int check_blocks(const streamkl_blocks* s, int B, int H, int NQ, int NK, bool data) {
  if (s == nullptr) return STREAMKL_INVALID_ARG;
  if (s->block != 32 && s->block != 64 && s->block != 128) return STREAMKL_INVALID_ARG;
  if (s->count < 1 || s->count > kMaxSlots) return STREAMKL_INVALID_ARG;
  if (s->heads < 1 || s->heads > std::max(H, 1) || H % s->heads != 0) return STREAMKL_INVALID_ARG;
  if (((long long)NK + s->block - 1) / s->block > kMaxSelBlocks) return STREAMKL_UNSUPPORTED;
  if (data && (s->selected == nullptr || !aligned4(s->selected))) return STREAMKL_INVALID_ARG;
  if (NQ >= 1 << (32 - kSlotBits) || (long long)B * s->heads * NQ * s->count > (1ll << 31) - 1) return STREAMKL_INVALID_ARG;
  return STREAMKL_OK;
}

int check_sel(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis, const streamkl_blocks* sel,
              int B, int H, int NQ, int NK, bool data, bool* empty) {
  int s = check_call(p1, p2, vis, B, H, NQ, NK, data, empty);
  if (s != STREAMKL_OK) return s;
  for (const streamkl_side* p : {p1, p2})
    if (p->softcap != 0.f || p->slopes != nullptr || p->table != nullptr) return STREAMKL_UNSUPPORTED;
  return check_blocks(sel, B, H, NQ, NK, data && !*empty);
}

SelRows rows_of(const streamkl_view& v, int B, int heads, int n, int d) {
  return SelRows{static_cast<const uint8_t*>(v.data), B > 1 ? 2 * v.stride_b : 0, heads > 1 ? 2 * v.stride_h : 0,
                 n > 1 ? 2 * v.stride_n : 0, d / 8};
}

struct Geometry {
  SelPlan p{};
  int u1 = 1, u2 = 1;
  bool one_kernel = false;  // makes the plan
};

// Heads that share keys on both sides and a selection form a unit, whose rows
// share tiles.  (A unit has at most 128 of them.)
Geometry geometry(const streamkl_side& p1, const streamkl_side& p2, const streamkl_visible& vis, const streamkl_blocks& sel,
                  int B, int H, int NQ, int NK) {
  Geometry g;
  SelPlan& p = g.p;
  p.B = B;
  p.H = H;
  p.NQ = NQ;
  p.NK = NK;
  p.HS = sel.heads;
  p.T = sel.count;
  p.bs = sel.block;
  p.blocks = (NK + sel.block - 1) / sel.block;
  const int units = std::lcm(std::lcm(p1.HK, p2.HK), sel.heads), heads = H / units;
  p.G = std::min(heads, kTile);
  while (heads % p.G != 0) --p.G;
  p.HU = H / p.G;
  p.queries_per_tile = kTile / p.G;
  g.u1 = p.HU / p1.HK;
  g.u2 = p.HU / p2.HK;
  p.causal = vis.causal;
  p.prefix = vis.prefix;
  p.doc_q = vis.doc_q;
  p.selected = sel.selected;
  p.words = (p.T + 31) / 32;
  // Up to 512 queries x slots a warp, one kernel (a CTA's 32 warps for a selection head); else chunks of a few steps of a
  // warp at least, and at most 256 (their counts are read twice).  At 16384 queries x 16 slots x 8 selection heads a walk
  // and the scan took 24 and 12 us with 128 chunks, 17 and 22 with 512.
  int span = 1;
  while (span < p.T && span < 32) span *= 2;
  const int step = 32 / span, warps = std::min(32, kPlanShared / (4 * p.blocks));
  const int few = (NQ + warps - 1) / warps;
  g.one_kernel = p.words == 1 && (long long)few * span <= 512;
  p.chunk = g.one_kernel ? few : std::max(4 * step, (NQ + 255) / 256);
  p.chunks = (NQ + p.chunk - 1) / p.chunk;
  return g;
}

// row_bytes: what a query head's rows hold in L2 while their lists run.
void take_plan(Carver& c, Geometry& g, double row_bytes, int sms, bool places) {
  SelPlan& p = g.p;
  const size_t heads = size_t(p.B) * p.HS, listed = size_t(p.NQ) * p.T;
  if (!g.one_kernel) p.counts = c.take<unsigned>(heads * p.chunks * p.blocks);
  p.entries = c.take<unsigned>(heads * listed);
  p.slots = c.take<unsigned>(heads * p.NQ * p.words);
  p.cap = int(std::min(listed, size_t(p.blocks)));
  p.lists = c.take<int4>(heads * p.cap);
  p.sizes = c.take<int2>(heads);
  if (places) p.place = c.take<int>(heads * p.blocks);
  // As many selection heads at a time as a third of L2 holds.
  const double fits = 40.0e6 / (row_bytes * (p.H / p.HS) * p.NQ);
  p.group = int(std::max(1.0, std::min(double(heads), fits)));
  p.groups = int((heads + p.group - 1) / p.group);
  const size_t most = heads * (p.HU / p.HS) * (listed / p.queries_per_tile + p.cap);  // tiles
  p.ctas = int(std::min(size_t(std::max(sms, 1)), most));
}

struct FwdPlan {
  ModPrepArgs prep{};
  Geometry g;
  float4* rec = nullptr;
  float* acc = nullptr;
  size_t bytes = 0;
};

FwdPlan fwd_plan(const streamkl_side& p1, const streamkl_side& p2, const streamkl_visible& vis, const streamkl_blocks& sel,
                 int B, int H, int NQ, int NK, int sms, void* ws) {
  FwdPlan f;
  Carver c{static_cast<uint8_t*>(ws)};
  const streamkl_side* const p[2] = {&p1, &p2};
  take_prep(c, f.prep, p, vis, B, H, NQ, NK, -1);
  f.g = geometry(p1, p2, vis, sel, B, H, NQ, NK);
  take_plan(c, f.g, 2.0 * (p1.d + p2.d), sms, false);
  const size_t pairs = size_t(B) * H * NQ * sel.count;
  f.rec = c.take<float4>(pairs);
  f.acc = c.take<float>(pairs);
  f.bytes = c.used;
  return f;
}

struct BwdPlan {
  ModPrepArgs prep{};
  Geometry g;
  float* dq32 = nullptr;
  unsigned* kmax = nullptr;
  float* dk_part = nullptr;
  float4* rows = nullptr;
  int pitch = 0;
  size_t bytes = 0;
};

BwdPlan bwd_plan(const streamkl_side& p1, const streamkl_side& p2, const streamkl_visible& vis, const streamkl_blocks& sel,
                 int B, int H, int NQ, int NK, int mode, int sms, void* ws) {
  BwdPlan f;
  Carver c{static_cast<uint8_t*>(ws)};
  const streamkl_side* const p[2] = {&p1, &p2};
  const streamkl_side& g = mode == STREAMKL_GRAD_P2 ? p2 : p1;
  f.pitch = (g.d + 31) / 32 * 32;
  // what starts at zero comes first, in one piece
  f.dq32 = c.take<float>(size_t(B) * H * NQ * f.pitch);
  f.kmax = c.take<unsigned>(size_t(B) * g.HK);
  f.prep.zero = static_cast<uint4*>(ws);
  f.prep.zero_words = c.used / 16;
  take_prep(c, f.prep, p, vis, B, H, NQ, NK, -1);
  f.g = geometry(p1, p2, vis, sel, B, H, NQ, NK);
  take_plan(c, f.g, 2.0 * (p1.d + p2.d) + 4.0 * f.pitch, sms, true);
  f.rows = c.take<float4>(size_t(B) * H * NQ);
  // (SelWalk::meeting stays below this)
  const size_t meetings = size_t(B) * sel.heads * f.g.p.cap * (f.g.p.HU / f.g.p.HS) + size_t(f.g.p.groups) * f.g.p.ctas;
  f.dk_part = c.take<float>(meetings * sel.block * g.d);
  f.bytes = c.used;
  return f;
}

bool key_maps(SelMaps* m, const streamkl_side& p1, const streamkl_side& p2, int B, int NK, int bs) {
  return map_bf16(&m->k1, p1.k, B, p1.HK, NK, p1.d, bs) && map_bf16(&m->k2, p2.k, B, p2.HK, NK, p2.d, bs);
}

}  // namespace

extern "C" {

size_t streamkl_fwd_sel_workspace_bytes(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                                        const streamkl_blocks* sel, int B, int H, int NQ, int NK) {
  bool empty = false;
  if (check_sel(p1, p2, vis, sel, B, H, NQ, NK, false, &empty) != STREAMKL_OK || empty) return 0;
  return fwd_plan(*p1, *p2, *vis, *sel, B, H, NQ, NK, num_sms(), nullptr).bytes;
}

int streamkl_fwd_sel(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                     const streamkl_blocks* sel, int B, int H, int NQ, int NK, void* workspace, size_t workspace_bytes,
                     float* kl, float* lse1, float* lse2, streamkl_stream_t stream) {
  bool empty = false;
  int s = check_sel(p1, p2, vis, sel, B, H, NQ, NK, true, &empty);
  if (s != STREAMKL_OK || empty) return s;
  if (!kl || !lse1 || !lse2 || !aligned16(kl) || !aligned16(lse1) || !aligned16(lse2)) return STREAMKL_INVALID_ARG;
  const int sms = num_sms();
  const FwdPlan f = fwd_plan(*p1, *p2, *vis, *sel, B, H, NQ, NK, sms, workspace);
  if (!workspace || !aligned16(workspace) || workspace_bytes < f.bytes) return STREAMKL_INVALID_ARG;
  if ((s = check_device()) != STREAMKL_OK) return s;
  SelMaps m{};
  SelFwdArgs a{};
  if (!key_maps(&m, *p1, *p2, B, NK, sel->block)) return STREAMKL_CUDA_ERROR;
  a.r1 = rows_of(p1->q, B, H, NQ, p1->d);
  a.r2 = rows_of(p2->q, B, H, NQ, p2->d);
  a.status = status_word();
  if (!a.status) return STREAMKL_CUDA_ERROR;
  a.p = f.g.p;
  a.u1 = f.g.u1;
  a.u2 = f.g.u2;
  a.scale1 = float(p1->scale);
  a.scale2 = float(p2->scale);
  a.vis = vis_args(*vis, f.prep);
  a.rec = f.rec;
  a.acc = f.acc;
  a.kl = kl;
  a.lse1 = lse1;
  a.lse2 = lse2;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (launch_mod_prep(f.prep, cs) != 0 || launch_sel_plan(a.p, nullptr, cs) != 0) return STREAMKL_CUDA_ERROR;
  if (launch_sel_fwd(m, tile_width(p1->d), tile_width(p2->d), a, cs) != 0) return STREAMKL_CUDA_ERROR;
  return as_status(launch_sel_merge(a, cs));
}

size_t streamkl_bwd_sel_workspace_bytes(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                                        const streamkl_blocks* sel, int B, int H, int NQ, int NK, int mode) {
  bool empty = false;
  if (check_sel(p1, p2, vis, sel, B, H, NQ, NK, false, &empty) != STREAMKL_OK || empty) return 0;
  if (mode != STREAMKL_GRAD_P2 && mode != STREAMKL_GRAD_P1) return 0;
  return bwd_plan(*p1, *p2, *vis, *sel, B, H, NQ, NK, mode, num_sms(), nullptr).bytes;
}

int streamkl_bwd_sel(const streamkl_side* p1, const streamkl_side* p2, const streamkl_visible* vis,
                     const streamkl_blocks* sel, int B, int H, int NQ, int NK, const float* kl, const float* lse1,
                     const float* lse2, const float* dkl, int mode, const streamkl_view* dq, const streamkl_view* dk,
                     void* workspace, size_t workspace_bytes, streamkl_stream_t stream) {
  bool empty = false;
  int s = check_sel(p1, p2, vis, sel, B, H, NQ, NK, true, &empty);
  if (s != STREAMKL_OK) return s;
  if (mode != STREAMKL_GRAD_P2 && mode != STREAMKL_GRAD_P1) return STREAMKL_INVALID_ARG;
  const streamkl_side& g = mode == STREAMKL_GRAD_P2 ? *p2 : *p1;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (empty) {  // no query rows: nothing reaches K
    if (B == 0 || H == 0 || NK == 0) return STREAMKL_OK;
    if (dk == nullptr || !view_ok(*dk, B, g.HK, NK)) return STREAMKL_INVALID_ARG;
    ModFinishArgs fin{};
    fin.rows[0] = {nullptr, B * g.HK, g.HK, NK, g.d, 0, static_cast<__nv_bfloat16*>(dk->data), B > 1 ? dk->stride_b : 0,
                   g.HK > 1 ? dk->stride_h : 0, NK > 1 ? dk->stride_n : 0};
    return as_status(launch_mod_finish(fin, cs));
  }
  if (!kl || !lse1 || !lse2 || !dkl || !aligned16(kl) || !aligned16(lse1) || !aligned16(lse2) || !aligned16(dkl))
    return STREAMKL_INVALID_ARG;
  if (dq == nullptr || dk == nullptr || !view_ok(*dq, B, H, NQ) || !view_ok(*dk, B, g.HK, NK)) return STREAMKL_INVALID_ARG;
  const int sms = num_sms();
  const BwdPlan f = bwd_plan(*p1, *p2, *vis, *sel, B, H, NQ, NK, mode, sms, workspace);
  if (!workspace || !aligned16(workspace) || workspace_bytes < f.bytes) return STREAMKL_INVALID_ARG;
  if ((s = check_device()) != STREAMKL_OK) return s;
  SelMaps m{};
  if (!key_maps(&m, *p1, *p2, B, NK, sel->block)) return STREAMKL_CUDA_ERROR;
  SelBwdArgs a{};
  a.status = status_word();
  if (!a.status) return STREAMKL_CUDA_ERROR;
  a.p = f.g.p;
  a.r1 = rows_of(p1->q, B, H, NQ, p1->d);
  a.r2 = rows_of(p2->q, B, H, NQ, p2->d);
  a.u1 = f.g.u1;
  a.u2 = f.g.u2;
  a.scale1 = float(p1->scale);
  a.scale2 = float(p2->scale);
  a.vis = vis_args(*vis, f.prep);
  a.kl = kl;
  a.lse1 = lse1;
  a.lse2 = lse2;
  a.dkl = dkl;
  a.dg = g.d;
  a.pitch = f.pitch;
  a.dq32 = f.dq32;
  a.dk_part = f.dk_part;
  a.rows = f.rows;
  a.kmax = f.kmax;
  a.dk = dk->data;
  a.dk_sb = B > 1 ? dk->stride_b : 0;
  a.dk_sh = g.HK > 1 ? dk->stride_h : 0;
  a.dk_sn = NK > 1 ? dk->stride_n : 0;
  a.HK = g.HK;
  a.mode = mode;
  a.k = g.k.data;
  a.k_sb = B > 1 ? g.k.stride_b : 0;
  a.k_sh = g.HK > 1 ? g.k.stride_h : 0;
  a.k_sn = NK > 1 ? g.k.stride_n : 0;
  a.doc_k = vis->doc_k;
  const ModFinishArgs::Rows rows{f.dq32, B * H, H, NQ, g.d, f.pitch, static_cast<__nv_bfloat16*>(dq->data),
                                 B > 1 ? dq->stride_b : 0, H > 1 ? dq->stride_h : 0, NQ > 1 ? dq->stride_n : 0};
  if (launch_mod_prep(f.prep, cs) != 0 || launch_sel_plan(a.p, &a, cs) != 0 ||
      launch_sel_bwd(m, tile_width(p1->d), tile_width(p2->d), a, cs) != 0)
    return STREAMKL_CUDA_ERROR;
  return as_status(launch_sel_finish(a, rows, cs));
}

}  // extern "C"
