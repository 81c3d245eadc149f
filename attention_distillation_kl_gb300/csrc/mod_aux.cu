// The small kernels around the passes over modified scores (mod_common.cuh):
// one before them, one after the backward, and max |K| for the deterministic
// backward.  All are bound by their launch or by HBM.
#include <algorithm>
#include <climits>

#include "bwd_common.cuh"
#include "mod_common.cuh"

namespace skl {

namespace {

constexpr int kAuxThreads = 256;

// The bucket of relative position r: a direction's buckets below the one
// whose first distance is beyond |r|.
__device__ __forceinline__ int bucket_of(int r, const ModPrepArgs::Table& t) {
  const int d = t.both ? abs(r) : max(-r, 0);
  int k = t.both && r > 0 ? t.per_side : 0;
  for (int i = 1; i < t.per_side; ++i) k += d >= t.first[i] ? 1 : 0;
  return k;
}

// Blocks of one launch by part: zeroing, then the tables' lookup rows (256
// positions of a head a block), then the tiles of ids (8 warps, one tile each).
struct PrepBlocks {
  int zero, table[2], q, k;
  __host__ __device__ int total() const { return zero + table[0] + table[1] + q + k; }
};

__global__ void __launch_bounds__(kAuxThreads) mod_prep_kernel(const __grid_constant__ ModPrepArgs a,
                                                               const __grid_constant__ PrepBlocks pb) {
  int blk = blockIdx.x;
  if (blk < pb.zero) {
    for (size_t i = size_t(blk) * kAuxThreads + threadIdx.x; i < a.zero_words; i += size_t(pb.zero) * kAuxThreads)
      a.zero[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  blk -= pb.zero;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (blk < pb.table[s]) {
      const ModPrepArgs::Table& t = a.t[s];
      const int len = near_len(t.max_distance), chunks = (len + kAuxThreads - 1) / kAuxThreads;
      const int h = blk / chunks, p = (blk - h * chunks) * kAuxThreads + threadIdx.x;
      if (p >= len) return;
      const float* entries = t.table + size_t(h) * t.num_buckets;
      float mask = -INFINITY;  // the largest masking entry, by a row's first warp
      if (p < 32)
#pragma unroll
        for (int e = 0; e < kMaxBuckets; e += 32) {
          const float x = p + e < t.num_buckets ? entries[p + e] * kLog2e : 0.f;
          if (x < kLow) mask = fmaxf(mask, fmaxf(x, kNegBig));
        }
      const int k = bucket_of(p - t.max_distance - kNearPad, t);
      if (t.bmap != nullptr && h == 0) t.bmap[p] = k;
      // a table's lowest values act as a mask: kept finite in base 2
      const float w = entries[k], v = w * kLog2e;
      float* row = t.near + size_t(h) * near_row(t.max_distance);
      row[p] = v < kNegBig ? kNegBig : (v > -kNegBig ? -kNegBig : v);
      if (p == 0 || p == len - 1)
        row[p == 0 ? len : len + 1] = fabsf(w) < 1.0e6f ? fmaf(w, kLog2e, -v) + w * kLog2eLo : 0.f;
      if (p < 32) {  // (a row is longer than a warp)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mask = fmaxf(mask, __shfl_xor_sync(0xffffffffu, mask, o));
        if (p == 0) row[len + 2] = 0.5f * mask;
      }
      return;
    }
    blk -= pb.table[s];
  }
  const bool q = blk < pb.q;
  if (!q) blk -= pb.q;
  const int* src = q ? a.doc_q : a.doc_k;
  const int n = q ? a.NQ : a.NK, tiles = (n + kTile - 1) / kTile;
  const int unit = blk * (kAuxThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit >= a.B * tiles) return;
  const int b = unit / tiles, tile = unit - b * tiles;
  int lo = INT_MAX, hi = -1, all = 1;
  int* dst = (q ? a.ids_q : a.ids_k) + (size_t(b) * tiles + tile) * kTile;
  for (int e = lane; e < kTile; e += 32) {
    const int i = tile * kTile + e;
    const int id = i < n ? src[size_t(b) * n + i] : -1;
    dst[e] = id >= 0 ? id : (q ? -2 : -1);
    if (id >= 0) {
      lo = min(lo, id);
      hi = max(hi, id);
    } else if (i < n) {
      all = 0;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    all &= __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) (q ? a.tiles_q : a.tiles_k)[size_t(b) * tiles + tile] = make_int4(lo, hi, all && lo == hi, 0);
}

struct FinishBlocks {
  int rows[2];
};

// Rows by finish_rows.  The table: one block per head; thread (g, k) adds every 4th of the head's
// warp sums of bucket k in order, then the four shares are added.
__global__ void __launch_bounds__(kAuxThreads) mod_finish_kernel(const __grid_constant__ ModFinishArgs a,
                                                                 const __grid_constant__ FinishBlocks fb) {
  __shared__ float part[4][kMaxBuckets];
  int blk = blockIdx.x;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (blk < fb.rows[s]) {
      finish_rows(a.rows[s], blk, fb.rows[s]);
      return;
    }
    blk -= fb.rows[s];
  }
  const int h = blk, k = threadIdx.x % kMaxBuckets, g = threadIdx.x / kMaxBuckets;
  float sum = 0.f;
  for (int b = 0; b < a.B; ++b) {
    const float* p = a.dtab + (size_t(b) * a.H + h) * a.nkt * 8 * kMaxBuckets;
#pragma unroll 8
    for (int u = g; u < a.nkt * 8; u += 4) sum += p[size_t(u) * kMaxBuckets + k];
  }
  part[g][k] = sum;
  __syncthreads();
  if (g == 0 && k < a.num_buckets)
    a.dtable[size_t(h) * a.num_buckets + k] = (part[0][k] + part[1][k]) + (part[2][k] + part[3][k]);
}

// kmax of a strided K (see kmax_kernel in dq_fixed.cu); keys whose id matches
// nothing may hold anything and do not count.
__global__ void __launch_bounds__(256) mod_kmax_kernel(const __nv_bfloat16* __restrict__ k, int per_batch, int n, int d,
                                                       long long sb, long long sh, long long sn, const int* ids, int ids_stride,
                                                       unsigned* kmax) {
  const int b = blockIdx.y / per_batch, h = blockIdx.y - b * per_batch;
  kmax_share(k + b * sb + h * sh, n, d, sn, ids != nullptr ? ids + size_t(b) * ids_stride : nullptr, blockIdx.x, gridDim.x,
             kmax + blockIdx.y);
}

}  // namespace

// At most 16 blocks per SM of a full GPU.
int loop_blocks(long long total) { return int(std::max(1ll, std::min((total + kAuxThreads - 1) / kAuxThreads, 2432ll))); }

int launch_mod_prep(const ModPrepArgs& a, cudaStream_t st) {
  PrepBlocks pb{};
  if (a.zero_words > 0) pb.zero = loop_blocks((long long)a.zero_words);
  for (int s = 0; s < 2; ++s)
    if (a.t[s].table != nullptr) pb.table[s] = a.H * ((near_len(a.t[s].max_distance) + kAuxThreads - 1) / kAuxThreads);
  if (a.doc_q != nullptr) {
    pb.q = (a.B * ((a.NQ + kTile - 1) / kTile) + 7) / 8;
    pb.k = (a.B * ((a.NK + kTile - 1) / kTile) + 7) / 8;
  }
  if (pb.total() == 0) return cudaSuccess;
  mod_prep_kernel<<<pb.total(), kAuxThreads, 0, st>>>(a, pb);
  return cudaGetLastError();
}

int launch_mod_finish(const ModFinishArgs& a, cudaStream_t st) {
  FinishBlocks fb{};
  for (int s = 0; s < 2; ++s)
    if (a.rows[s].dst != nullptr)
      fb.rows[s] = loop_blocks((long long)a.rows[s].heads * a.rows[s].n * (a.rows[s].d / 8));
  const int blocks = fb.rows[0] + fb.rows[1] + (a.dtable != nullptr ? a.H : 0);
  if (blocks == 0) return cudaSuccess;
  mod_finish_kernel<<<blocks, kAuxThreads, 0, st>>>(a, fb);
  return cudaGetLastError();
}

int launch_kmax_strided(const void* k, int B, int per_batch, int n, int d, long long sb, long long sh, long long sn,
                        const int* ids, unsigned* kmax, cudaStream_t st) {
  const int heads = B * per_batch;
  dim3 grid(unsigned((loop_blocks((long long)n * (d / 8)) + heads - 1) / heads), unsigned(heads));
  mod_kmax_kernel<<<grid, kAuxThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(k), per_batch, n, d, sb, sh, sn, ids,
                                               (n + kTile - 1) / kTile * kTile, kmax);
  return cudaGetLastError();
}

}  // namespace skl
