// Rotary positions with several axes: every pair (u, v) of a row's values
// turns by its angle, (u cos - v sin, u sin + v cos); the inverse turns back,
// which is also the gradient.
//
// Angles: position * inv_freq, of positions that may be far, needs more than
// fp32's 24 bits (at position 10^6 an fp32 product is off by 0.03 radians).
// inv_freq / 2 pi is taken once as a 64-bit fraction of a turn; position times
// it, modulo 2^64, is the angle modulo a turn without any rounding, and its
// high 32 bits go to sincospi.  What is left is the error of that fraction: up to
// inv_freq = 1 less than 2^-63, or 2^-32 turns at position 2^31 (beyond 1024 that of
// fp64's 53 bits).
//
// The kernel reads and writes every value once and is bound by that; angles
// depend on the token and pair alone, so a block computes those of its tokens
// once, for all of its heads.  32760 tokens x 32 heads x 128 take 85 us, 6.3 TB/s;
// with 256 threads a block 101, with 4 vectors of a thread in flight instead of 2
// 87, with twice or four times the tokens 85 and 86.
#include <algorithm>

#include <cuda_bf16.h>

#include "bwd_common.cuh"
#include "views.cuh"

namespace skl {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotMaxPairs = 128;

struct RotArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  long long xb, xh, xn, yb, yh, yn;
  const int* positions;
  long long pos_axis, pos_b;
  const float* inv_freq;
  int axes, end[4];  // first pair behind each axis
  int B, heads, N, d, pairs;
  int tokens;        // of a block
  int head_step;     // heads of a block
  int token_blocks;
  int inverse;
  int copy;          // the values behind the pairs are copied (0: in place)
};

struct Turn {
  float co, si;
};

__device__ __forceinline__ void turn8(uint4& u, uint4& v, const Turn* t) {
  uint32_t* a = &u.x;
  uint32_t* b = &v.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a0 = __uint_as_float(a[k] << 16), a1 = __uint_as_float(a[k] & 0xffff0000u);
    const float b0 = __uint_as_float(b[k] << 16), b1 = __uint_as_float(b[k] & 0xffff0000u);
    const Turn t0 = t[2 * k], t1 = t[2 * k + 1];
    a[k] = pack_bf16(fmaf(a0, t0.co, -b0 * t0.si), fmaf(a1, t1.co, -b1 * t1.si));
    b[k] = pack_bf16(fmaf(a0, t0.si, b0 * t0.co), fmaf(a1, t1.si, b1 * t1.co));
  }
}
__device__ __forceinline__ void turn4(uint4& u, const Turn* t) {
  uint32_t* a = &u.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a0 = __uint_as_float(a[k] << 16), a1 = __uint_as_float(a[k] & 0xffff0000u);
    a[k] = pack_bf16(fmaf(a0, t[k].co, -a1 * t[k].si), fmaf(a0, t[k].si, a1 * t[k].co));
  }
}

// frac(f / 2 pi) 2^64.  f = m 2^-s: m times the first 64 bits of 1 / 2 pi, s bits
// down; beyond 1024 (and below 0) in fp64, which is slow here (2.5 us of a small call).
__device__ __forceinline__ unsigned long long turn_step(float f) {
  const unsigned u = __float_as_uint(f), exponent = u >> 23;
  if (exponent < 137u) {
    constexpr unsigned long long kTurn = 0x28be60db9391054aull;  // 2^64 / 2 pi
    const unsigned long long m = (u & 0x7fffffu) | (exponent != 0u ? 0x800000u : 0u);
    const int s = 150 - max(int(exponent), 1);  // 14 to 149
    const unsigned long long hi = __umul64hi(m, kTurn), lo = m * kTurn;
    return s < 64 ? (hi << (64 - s)) | (lo >> s) : (s < 128 ? hi >> (s - 64) : 0ull);
  }
  const double x = double(f) * 0.15915494309189535;
  return __double2ull_rn((x - floor(x)) * 18446744073709551616.0);
}

enum { kHalves = 0, kNeighbours = 1, kSingle = 2 };

// kHalves: pairs (p, p + R), 8 at a time, R a multiple of 8; kNeighbours: pairs
// (2p, 2p + 1), 4 at a time, R a multiple of 4; kSingle: any R, a pair at a time.
template <int HOW>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const __grid_constant__ RotArgs a, int interleaved) {
  extern __shared__ Turn turns[];  // [tokens][pairs]
  const int b = blockIdx.x / a.token_blocks, n0 = (blockIdx.x - b * a.token_blocks) * a.tokens;
  const int count = min(a.tokens, a.N - n0);
  for (int u = threadIdx.x; u < count * a.pairs; u += kRotThreads) {
    const int t = u / a.pairs, p = u - t * a.pairs;
    const int axis = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
    const long long pos = a.positions[axis * a.pos_axis + b * a.pos_b + n0 + t];
    const int part = int((unsigned long long)pos * turn_step(a.inv_freq[p]) >> 32);  // of 2^32, signed
    Turn r;
    sincospif(float(part) * 4.656612873077393e-10f, &r.si, &r.co);  // 2^-31: half turns
    if (a.inverse) r.si = -r.si;
    turns[u] = r;
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.head_step, heads = min(a.head_step, a.heads - h0);
  // units of a row: the pairs' vectors, then the copied ones
  const int turned = HOW == kHalves ? a.pairs / 8 : (HOW == kNeighbours ? a.pairs / 4 : a.pairs);
  const int rest = !a.copy ? 0 : (HOW == kSingle ? a.d - 2 * a.pairs : (a.d - 2 * a.pairs) / 8);
  const int per_row = turned + rest, per_token = per_row * heads, total = per_token * count;
  auto locate = [&](int u, const __nv_bfloat16*& x, __nv_bfloat16*& y, int& c, const Turn*& t) {
    const int tok = u / per_token, w = u - tok * per_token, h = w / per_row;
    c = w - h * per_row;
    x = a.x + b * a.xb + (h0 + h) * a.xh + (n0 + tok) * a.xn;
    y = a.y + b * a.yb + (h0 + h) * a.yh + (n0 + tok) * a.yn;
    t = turns + tok * a.pairs;
  };
  if (HOW == kSingle) {
    for (int u = threadIdx.x; u < total; u += kRotThreads) {
      const __nv_bfloat16* x;
      __nv_bfloat16* y;
      const Turn* t;
      int c;
      locate(u, x, y, c, t);
      if (c >= turned) {
        y[turned + c] = x[turned + c];  // value 2 R + (c - R)
        continue;
      }
      const int i = interleaved ? 2 * c : c, j = interleaved ? 2 * c + 1 : c + a.pairs;
      const float p = __bfloat162float(x[i]), q = __bfloat162float(x[j]);
      y[i] = __float2bfloat16_rn(fmaf(p, t[c].co, -q * t[c].si));
      y[j] = __float2bfloat16_rn(fmaf(p, t[c].si, q * t[c].co));
    }
    return;
  }
  constexpr int kAtOnce = 2;
  for (int u0 = threadIdx.x; u0 < total; u0 += kAtOnce * kRotThreads) {
    uint4 lo[kAtOnce], hi[kAtOnce];
    __nv_bfloat16* y[kAtOnce];
    const Turn* t[kAtOnce];
    int c[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int u = u0 + k * kRotThreads;
      if (u >= total) continue;
      const __nv_bfloat16* x;
      locate(u, x, y[k], c[k], t[k]);
      if (HOW == kHalves) {
        const bool pair = c[k] < turned;
        lo[k] = __ldcs(reinterpret_cast<const uint4*>(x + 8 * (pair ? c[k] : turned + c[k])));
        if (pair) hi[k] = __ldcs(reinterpret_cast<const uint4*>(x + a.pairs + 8 * c[k]));
      } else {
        lo[k] = __ldcs(reinterpret_cast<const uint4*>(x + 8 * c[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (u0 + k * kRotThreads >= total) continue;
      if (HOW == kHalves) {
        const bool pair = c[k] < turned;
        if (pair) {
          turn8(lo[k], hi[k], t[k] + 8 * c[k]);
          __stcs(reinterpret_cast<uint4*>(y[k] + a.pairs + 8 * c[k]), hi[k]);
        }
        __stcs(reinterpret_cast<uint4*>(y[k] + 8 * (pair ? c[k] : turned + c[k])), lo[k]);
      } else {
        if (c[k] < turned) turn4(lo[k], t[k] + 4 * c[k]);
        __stcs(reinterpret_cast<uint4*>(y[k] + 8 * c[k]), lo[k]);
      }
    }
  }
}

}  // namespace

}  // namespace skl

extern "C" int streamkl_rotate(const streamkl_view* x, const streamkl_view* y, const streamkl_rotary* r, int B,
                               int heads, int N, int d, int inverse, streamkl_stream_t stream) {
  using namespace skl;
  if (x == nullptr || y == nullptr || r == nullptr || B < 0 || heads < 0 || N < 0) return STREAMKL_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return STREAMKL_INVALID_ARG;
  if (d < 16 || d > 256 || d % 16 != 0) return STREAMKL_UNSUPPORTED;
  if (r->axes < 1 || r->axes > 4 || (r->interleaved != 0 && r->interleaved != 1)) return STREAMKL_INVALID_ARG;
  RotArgs a{};
  for (int i = 0; i < 4; ++i) {
    if (i < r->axes) {
      if (r->section[i] < 1 || r->section[i] > d / 2) return STREAMKL_INVALID_ARG;
      a.pairs += r->section[i];
    }
    a.end[i] = a.pairs;
  }
  if (a.pairs > d / 2) return STREAMKL_INVALID_ARG;
  // (the last axis has no end that a pair could reach)
  for (int i = r->axes - 1; i < 4; ++i) a.end[i] = kRotMaxPairs + 1;
  if (B == 0 || heads == 0 || N == 0) return STREAMKL_OK;
  if (!view_ok(*x, B, heads, N) || !view_ok(*y, B, heads, N)) return STREAMKL_INVALID_ARG;
  if (!r->positions || !r->inv_freq || !aligned4(r->positions) || !aligned4(r->inv_freq)) return STREAMKL_INVALID_ARG;
  if (r->stride_axis < 0 || r->stride_b < 0) return STREAMKL_INVALID_ARG;
  if ((long long)B * heads > 65535 || (long long)B * heads * N > (1ll << 31) - 1) return STREAMKL_INVALID_ARG;
  auto stride = [](long long s, int size) { return size <= 1 ? 0ll : s; };
  a.xb = stride(x->stride_b, B), a.xh = stride(x->stride_h, heads), a.xn = stride(x->stride_n, N);
  a.yb = stride(y->stride_b, B), a.yh = stride(y->stride_h, heads), a.yn = stride(y->stride_n, N);
  // in place means value for value
  const bool same = x->data == y->data;
  if (same && (a.xb != a.yb || a.xh != a.yh || a.xn != a.yn)) return STREAMKL_INVALID_ARG;
  const int s = check_device();
  if (s != STREAMKL_OK) return s;
  a.x = static_cast<const __nv_bfloat16*>(x->data);
  a.y = static_cast<__nv_bfloat16*>(y->data);
  a.positions = r->positions;
  a.pos_axis = r->stride_axis;
  a.pos_b = r->stride_b;
  a.inv_freq = r->inv_freq;
  a.axes = r->axes;
  a.B = B;
  a.heads = heads;
  a.N = N;
  a.d = d;
  a.inverse = inverse;
  a.copy = !same;
  const int how = r->interleaved ? (a.pairs % 4 == 0 ? kNeighbours : kSingle) : (a.pairs % 8 == 0 ? kHalves : kSingle);
  // A block has 4 vectors for each thread, where there are as many: of all
  // heads of a few tokens (their angles are then computed once), and of fewer
  // heads where tokens are few.
  const int per_row = d / 16;  // vectors of a row, two at a time
  const int want = 4 * kRotThreads;
  a.tokens = std::max(1, std::min({want / std::max(1, heads * per_row), 16, N}));
  a.head_step = heads;
  while (a.head_step > 1 && (long long)B * ((N + a.tokens - 1) / a.tokens) * ((heads + a.head_step - 1) / a.head_step) < 304)
    a.head_step = (a.head_step + 1) / 2;
  a.token_blocks = (N + a.tokens - 1) / a.tokens;
  const dim3 grid(unsigned(B * a.token_blocks), unsigned((heads + a.head_step - 1) / a.head_step));
  const size_t smem = size_t(a.tokens) * a.pairs * sizeof(Turn);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (how == kHalves) rotate_kernel<kHalves><<<grid, kRotThreads, smem, cs>>>(a, r->interleaved);
  else if (how == kNeighbours) rotate_kernel<kNeighbours><<<grid, kRotThreads, smem, cs>>>(a, r->interleaved);
  else rotate_kernel<kSingle><<<grid, kRotThreads, smem, cs>>>(a, r->interleaved);
  return as_status(cudaGetLastError());
}
