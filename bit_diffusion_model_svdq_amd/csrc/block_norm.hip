// The norms before and after a transformer block, fused with the block's gate,
// residual and modulation, gfx950:
//
//   x' = a x + c gate_b post(y)
//   h  = (pre(x') w + bias) (1 + scale_b) + shift_b
//
// post and pre: nothing, v / sqrt(mean v^2 + eps) (RMS) or
// (v - mean v) / sqrt(mean (v - mean v)^2 + eps) (LayerNorm); b is the row's
// sequence.  One pass: a row of x and y is read once into registers, its
// statistics are taken there in float32 (LayerNorm's variance from the centred
// values, so that a large mean costs no bits), x' and h are written once.
// h comes from the unrounded x'.
//
// HBM bound: 2 (or 4) + 2 bytes in and as many out per element, a few
// operations each.  A row belongs to W waves, W the smallest power of two
// that leaves a thread at most kMaxVec chunks of 8 channels; with W = 1 a
// workgroup of four waves runs without barriers, and rows of up to 256 channels
// share a wave (L lanes each): 100000 x 128 19.4 us, 46 with a wave per row.
#include "svdq_internal.h"

namespace svdq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxVec = 4;       // 16-byte bf16 chunks of a row per thread
constexpr int kMaxWaves = 8;     // waves per row: 8 x 64 x 4 x 8 = 16384 channels

__device__ inline void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}

__device__ inline u32x4 pack8(const float (&f)[8]) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_bit_cast(uint16_t, (__bf16)f[2 * i]) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[2 * i + 1]) << 16);
  return v;
}

__device__ inline void load8(const uint16_t* p, float (&f)[8]) {
  unpack8(*reinterpret_cast<const u32x4*>(p), f);
}
__device__ inline void load8(const float* p, float (&f)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
// Non-temporal: x' and h stream out to HBM.  With inputs from there 4608 x 3072 bf16
// takes 25.9 us (4.4 TB/s) against 31.4 with stores that allocate in the caches,
// 29484 x 1280 float32 93.8 (4.8 TB/s) against 102.4; loads of x and y gain nothing from it.
__device__ inline void store8(uint16_t* p, const float (&f)[8]) { __builtin_nontemporal_store(pack8(f), reinterpret_cast<u32x4*>(p)); }
__device__ inline void store8(float* p, const float (&f)[8]) {
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(p + 4));
}

// The sum of v over the row's L lanes or W waves, in every thread (the same order in each).
template <int W, int L>
__device__ inline float row_sum(float v, float* lds, int wave) {
#pragma unroll
  for (int s = L / 2; s > 0; s >>= 1) v += __shfl_xor(v, s);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += lds[w];
    __syncthreads();
  }
  return v;
}

// Normalises the row in place (chunks past the row hold 0 and stay 0).
template <int W, int L, int V>
__device__ inline void normalise(float (&v)[V][8], const bool (&ok)[V], int kind, float eps, float inv_width,
                                 float* lds, int wave) {
  if (kind == kNormNone) return;
  if (kind == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];
    const float mean = row_sum<W, L>(s, lds, wave) * inv_width;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = ok[i] ? v[i][e] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) q = __builtin_fmaf(v[i][e], v[i][e], q);
  const float r = rsqrtf(__builtin_fmaf(row_sum<W, L>(q, lds, wave), inv_width, eps));
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= r;
}

// The sequence of `row`, or -1: the last b with cu[b] <= row, if row < cu[batch].
__device__ inline int sequence_of(const int32_t* cu, int batch, int64_t row) {
  if (!cu) return 0;
  if (row < cu[0] || row >= cu[batch]) return -1;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// x and x_out, y and h may be the same buffers: a thread writes only the
// chunks that it has itself read before.
template <class S, int W, int L, int V>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void block_norm_kernel(const BlockNormArgs a) {
  __shared__ float lds[W == 1 ? 1 : W];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = W > 1 ? (int64_t)blockIdx.x
                      : L == 64 ? (int64_t)blockIdx.x * 4 + wave
                                : (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= a.rows) return;
  const int b = sequence_of(a.cu, a.batch, row);
  if (b < 0) return;
  const int t = W == 1 ? threadIdx.x % L : threadIdx.x;
  const int64_t at = row * a.width;
  const float inv_width = 1.0f / (float)a.width;
  int ch[V];
  bool ok[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ch[i] = 8 * (t + i * L * W);
    ok[i] = ch[i] < a.width;
  }
  float x[V][8], y[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = y[i][e] = 0.f;
    if (ok[i]) load8(static_cast<const S*>(a.x) + at + ch[i], x[i]);
    if (ok[i] && a.y) load8(a.y + at + ch[i], y[i]);
  }
  if (a.y) {
    normalise<W, L, V>(y, ok, a.post, a.eps, inv_width, lds, wave);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!ok[i]) continue;
      float w[8];
      if (a.post_weight) {
        load8(a.post_weight + ch[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= w[e];
      }
      if (a.gate) {
        load8(a.gate + b * a.ld_gate + ch[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= w[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = __builtin_fmaf(a.branch_scale, y[i][e], a.residual_scale * x[i][e]);
  if (a.x_out)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i]) store8(static_cast<S*>(a.x_out) + at + ch[i], x[i]);
  if (!a.h) return;
  normalise<W, L, V>(x, ok, a.pre, a.eps, inv_width, lds, wave);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!ok[i]) continue;
    float w[8];
    if (a.pre_weight) {
      load8(a.pre_weight + ch[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= w[e];
    }
    if (a.pre_bias) {
      load8(a.pre_bias + ch[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] += w[e];
    }
    if (a.scale) {
      load8(a.scale + b * a.ld_scale + ch[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = __builtin_fmaf(x[i][e], w[e], x[i][e]);
    }
    if (a.shift) {
      load8(a.shift + b * a.ld_shift + ch[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] += w[e];
    }
    store8(a.h + at + ch[i], x[i]);
  }
}

template <class S, int W, int L, int V>
hipError_t launch(const BlockNormArgs& a, hipStream_t stream) {
  constexpr int kRows = W == 1 ? 256 / L : 1;      // of a workgroup
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  hipLaunchKernelGGL((block_norm_kernel<S, W, L, V>), dim3((unsigned)blocks), dim3(W == 1 ? 256 : 64 * W), 0, stream, a);
  return hipGetLastError();
}

template <class S, int W>
hipError_t with_vec(const BlockNormArgs& a, hipStream_t stream) {
  const int v = (a.width / 8 + 64 * W - 1) / (64 * W);
  if constexpr (W == 1) {      // with more waves a thread has three chunks at least
    if (v <= 1) return launch<S, W, 64, 1>(a, stream);
    if (v == 2) return launch<S, W, 64, 2>(a, stream);
  }
  if (v == 3) return launch<S, W, 64, 3>(a, stream);
  return launch<S, W, 64, 4>(a, stream);
}

template <class S>
hipError_t with_waves(const BlockNormArgs& a, hipStream_t stream) {
  const int chunks = a.width / 8;
  if (chunks <= 16) return launch<S, 1, 16, 1>(a, stream);
  if (chunks <= 32) return launch<S, 1, 32, 1>(a, stream);
  if (chunks <= 64 * kMaxVec) return with_vec<S, 1>(a, stream);
  if (chunks <= 128 * kMaxVec) return with_vec<S, 2>(a, stream);
  if (chunks <= 256 * kMaxVec) return with_vec<S, 4>(a, stream);
  return with_vec<S, kMaxWaves>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, bool fp32, hipStream_t stream) {
  return fp32 ? with_waves<float>(a, stream) : with_waves<uint16_t>(a, stream);
}

}  // namespace svdq
