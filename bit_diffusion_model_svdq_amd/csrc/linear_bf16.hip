// The linear of the layers a 4-bit model keeps in 16 bits, gfx950:
//
//   Y = act(X W^T + bias) + residual,   X [M, K], W [N, K] bf16
//
// with bias, activation and residual in the product's epilogue: float32
// accumulators, one rounding to the output's type.  The residual enters as
// Y's type.
//
// Two kernels.  linear_tile: a workgroup computes a BM x BN tile of Y on the
// 16x16x32 bf16 MFMA from a ring of NR LDS buffers, one step of 32 channels
// each, filled by direct copies (global_load_lds) NR - 1 steps ahead; where
// the tiles do not fill the chip the channels are cut into shares whose
// float32 sums linear_join brings together.  linear_rows: few rows of X;
// then the weight's bytes are the cost, and each wave streams its share of the
// channels of a few weight rows straight into registers.
//
// Both compute Y^T tiles (W rows as the MFMA's A operand, X rows as B): a
// lane's four accumulators are then neighbouring outputs of one row of Y.
#include <algorithm>

#include "gemm_tail.h"
#include "svdq_internal.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int KS = 32;            // channels per step: one MFMA deep
constexpr int ROWB = KS * 2;      // bytes of a row's step

__device__ inline float bf16_value(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// v / (1 + e^-v)
__device__ inline float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

template <int ACT>
__device__ inline float activate(float v) {
  if constexpr (ACT == kActGeluTanh) return tail::gelu_tanh(v);
  if constexpr (ACT == kActSilu) return silu(v);
  return v;
}

// Four neighbouring outputs n .. n + 3 of row m: bias, activation, residual,
// rounding, store.  `wide`: N is a multiple of 4 and the base pointers are
// 16-byte aligned, so the four are stored (and the residual read) at once.
template <class O, int ACT>
__device__ inline void finish4(f32x4 v, const LinearArgs& a, int64_t m, int n, bool wide) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = m * a.N + n;
  O* y = static_cast<O*>(a.Y) + at;
  const O* r = a.residual ? static_cast<const O*>(a.residual) + at : nullptr;
  if (wide) {
    if (a.bias) {
      const u32x2 b = *reinterpret_cast<const u32x2*>(a.bias + n);
      v[0] += __uint_as_float(b[0] << 16);
      v[1] += __uint_as_float(b[0] & 0xFFFF0000u);
      v[2] += __uint_as_float(b[1] << 16);
      v[3] += __uint_as_float(b[1] & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate<ACT>(v[i]);
    if constexpr (sizeof(O) == 4) {
      if (r) v += *reinterpret_cast<const f32x4*>(r);
      *reinterpret_cast<f32x4*>(y) = v;
    } else {
      if (r) {
        const u32x2 b = *reinterpret_cast<const u32x2*>(r);
        v[0] += __uint_as_float(b[0] << 16);
        v[1] += __uint_as_float(b[0] & 0xFFFF0000u);
        v[2] += __uint_as_float(b[1] << 16);
        v[3] += __uint_as_float(b[1] & 0xFFFF0000u);
      }
      u32x2 w;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16);
      *reinterpret_cast<u32x2*>(y) = w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    float u = activate<ACT>(v[i] + (a.bias ? bf16_value(a.bias[n + i]) : 0.f));
    if constexpr (sizeof(O) == 4) {
      y[i] = r ? u + r[i] : u;
    } else {
      if (r) u += bf16_value(r[i]);
      y[i] = __builtin_bit_cast(uint16_t, (__bf16)u);
    }
  }
}

template <int WM_, int WN_, int TM_, int TN_, int NR_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NR = NR_;
  static constexpr int BM = WM * TM * 16;      // rows of X
  static constexpr int BN = WN * TN * 16;      // rows of W
  static constexpr int WAVES = WM * WN;
  static constexpr int THREADS = WAVES * 64;
  static constexpr int BUF = (BM + BN) * ROWB;
  static constexpr int COPIES = BUF / 1024;
  static constexpr int CPW = COPIES / WAVES;
  static_assert(COPIES % WAVES == 0, "every wave copies the same number of KB");
  static_assert(NR == 4, "four ring buffers");
  static_assert(CPW * NR < 64, "vmcnt range");
};

using Big = Tile<2, 4, 8, 4, 4>;     // 256 x 256, 8 waves, 128 KB: one workgroup per CU
using Med = Tile<2, 2, 4, 4, 4>;     // 128 x 128, 4 waves, 64 KB: two
using Small = Tile<2, 2, 2, 2, 4>;   //  64 x  64, 4 waves, 32 KB

// XOR key of the 16-byte chunks of a 64-byte LDS row: a fragment read covers
// 16 consecutive rows, chunk lane / 16.
__device__ inline int swz_key(int row) { return (row >> 1) & 3; }

// vmcnt = n (later steps' copies stay in flight), lgkmcnt = 0: this wave's LDS
// reads are complete before the barrier lets another wave copy over them.
template <int n>
__device__ inline void ring_wait() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));
}

template <class C, class O, int ACT, bool SHARES>
__global__ __launch_bounds__(C::THREADS, 2) void linear_tile(const LinearArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ring0[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring2[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring3[C::BUF];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntm = (a.M + C::BM - 1) / C::BM;
  const int ntn = (a.N + C::BN - 1) / C::BN;
  const int tiles = ntm * ntn;
  const int ksteps = (a.K + KS - 1) / KS;
  int tmi, tni, sb = 0, se = ksteps, share = 0;
  if (SHARES) {
    share = blockIdx.x / tiles;
    tail::tile_of_id(ntm, ntn, blockIdx.x % tiles, tmi, tni);
    sb = (int)((int64_t)ksteps * share / a.splits);
    se = (int)((int64_t)ksteps * (share + 1) / a.splits);
  } else {
    tail::tile_of_id(ntm, ntn, tail::xcd_compact(blockIdx.x, tiles), tmi, tni);
  }
  const int nsteps = se - sb;
  const int m0 = tmi * C::BM, n0 = tni * C::BN;

  // This wave's copies of a step: 16 rows of 64 bytes each; lane j fills
  // physical chunk j % 4 of row j / 4.  Rows past the matrix read its last
  // row; chunks past K (the last step's) the row's last chunk, zeroed below.
  const int nchunks = a.K / 8;
  const uint16_t* src[C::CPW];
  int chunk[C::CPW];
#pragma unroll
  for (int i = 0; i < C::CPW; ++i) {
    const int row = (wave * C::CPW + i) * 16 + (lane >> 2);
    chunk[i] = (lane & 3) ^ swz_key(row);
    src[i] = row < C::BM ? a.X + (int64_t)min(m0 + row, a.M - 1) * a.K
                         : a.W + (int64_t)min(n0 + row - C::BM, a.N - 1) * a.K;
  }
  auto copy_step = [&](int s, uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < C::CPW; ++i) {
      const uint16_t* g = src[i] + 8 * min(4 * s + chunk[i], nchunks - 1);
      __builtin_amdgcn_global_load_lds(g, (lds_ptr)(buf + (wave * C::CPW + i) * 1024), 16, 0, 0);
    }
  };

  const int wm = wave / C::WN, wn = wave - wm * C::WN;
  const int fr = lane & 15, fk = lane >> 4;
  const int swz = (fk ^ swz_key(fr)) << 4;
  const int x_lane = (wm * C::TM * 16 + fr) * ROWB + swz;
  const int w_lane = (C::BM + wn * C::TN * 16 + fr) * ROWB + swz;
  f32x4 acc[C::TM][C::TN];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto step = [&](int j, const uint8_t* cur, uint8_t* freed) {
    ring_wait<C::CPW * 2>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    copy_step(sb + min(j + 3, nsteps - 1), freed);
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 xf[C::TM], wf[C::TN];
#pragma unroll
    for (int t = 0; t < C::TN; ++t) wf[t] = *reinterpret_cast<const bf16x8*>(cur + w_lane + t * 16 * ROWB);
#pragma unroll
    for (int t = 0; t < C::TM; ++t) xf[t] = *reinterpret_cast<const bf16x8*>(cur + x_lane + t * 16 * ROWB);
    if (4 * (sb + j) + 4 > nchunks) {      // the matrices' last step, cut short
      if (4 * (sb + j) + fk >= nchunks) {
#pragma unroll
        for (int t = 0; t < C::TN; ++t) wf[t] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
#pragma unroll
        for (int t = 0; t < C::TM; ++t) xf[t] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
      }
    }
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn)
        acc[tm][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[tn], xf[tm], acc[tm][tn], 0, 0, 0);
  };

  copy_step(sb, ring0);
  copy_step(sb + min(1, nsteps - 1), ring1);
  copy_step(sb + min(2, nsteps - 1), ring2);
  int j0 = 0;
  for (; j0 + 4 <= nsteps; j0 += 4) {
    step(j0, ring0, ring3);
    step(j0 + 1, ring1, ring0);
    step(j0 + 2, ring2, ring1);
    step(j0 + 3, ring3, ring2);
  }
  if (j0 < nsteps) step(j0, ring0, ring3);
  if (j0 + 1 < nsteps) step(j0 + 1, ring1, ring0);
  if (j0 + 2 < nsteps) step(j0 + 2, ring2, ring1);
  ring_wait<0>();     // a workgroup may not leave copies into its LDS behind

  const bool wide = a.wide;
#pragma unroll
  for (int tm = 0; tm < C::TM; ++tm) {
    const int64_t m = m0 + wm * C::TM * 16 + 16 * tm + fr;
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) {
      const int n = n0 + wn * C::TN * 16 + 16 * tn + 4 * fk;
      if constexpr (SHARES) {
        if (m < a.M && n < a.N) {
          float* p = a.part + ((int64_t)share * a.M + m) * a.part_ld + n;   // part_ld: N rounded up to 4
          *reinterpret_cast<f32x4*>(p) = acc[tm][tn];
        }
      } else {
        finish4<O, ACT>(acc[tm][tn], a, m, n, wide);
      }
    }
  }
}

// Sums the shares in order and finishes the outputs, four per thread.
template <class O, int ACT>
__global__ __launch_bounds__(256) void linear_join(const LinearArgs a) {
  const int quads = a.part_ld / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.M * quads) return;
  const int64_t m = i / quads;
  const int n = (int)(i - m * quads) * 4;
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s)
    v += *reinterpret_cast<const f32x4*>(a.part + ((int64_t)s * a.M + m) * a.part_ld + n);
  finish4<O, ACT>(v, a, m, n, a.wide);
}

// Few rows: 16 weight rows (n) and MT x 16 rows of X per workgroup; wave w takes
// every WAVES-th block of 64 channels.  Lane (fk, fr) reads 32 neighbouring
// bytes of weight row fr, so that the four lanes of a row take a whole
// 128-byte line; the MFMA's k slots are any 32 channels as long as both
// operands agree, so the two 16-byte halves are two MFMA steps.
constexpr int kRowWaves = 8;
template <class O, int ACT, int MT>
__global__ __launch_bounds__(kRowWaves * 64) void linear_rows(const LinearArgs a) {
  __shared__ f32x4 sums[kRowWaves][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fk = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const uint16_t* w = a.W + (int64_t)min(n0 + fr, a.N - 1) * a.K;
  const uint16_t* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = a.X + (int64_t)min(16 * t + fr, a.M - 1) * a.K;
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int blocks = (a.K + 63) / 64;
  const u32x4 zero = u32x4{0u, 0u, 0u, 0u};
#pragma unroll 4
  for (int kb = wave; kb < blocks; kb += kRowWaves) {
    const int k = 64 * kb + 16 * fk;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = min(k + 8 * u, a.K - 8);
      const bool in = k + 8 * u < a.K;
      u32x4 wv = *reinterpret_cast<const u32x4*>(w + at);
      wv = in ? wv : zero;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        u32x4 xv = *reinterpret_cast<const u32x4*>(x[t] + at);
        xv = in ? xv : zero;
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv),
                                                         __builtin_bit_cast(bf16x8, xv), acc[t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave >= MT) return;
  // wave t joins and finishes rows 16 t .. + 15
  f32x4 v = sums[0][wave][lane];
#pragma unroll
  for (int s = 1; s < kRowWaves; ++s) v += sums[s][wave][lane];
  finish4<O, ACT>(v, a, 16 * wave + fr, n0 + 4 * fk, a.wide);
}

constexpr int kRowsMax = 64;       // linear_rows: at most four blocks of 16 rows

enum Kind { kKindRows, kKindBig, kKindMed, kKindSmall };
struct Plan {
  Kind kind = kKindSmall;
  int splits = 1;
  int64_t blocks = 0;
  size_t bytes = 0;
};

template <class C>
int64_t tiles_of(int M, int N) {
  return (int64_t)((M + C::BM - 1) / C::BM) * ((N + C::BN - 1) / C::BN);
}

Plan plan_of(int M, int K, int N) {
  Plan p;
  const int cus = device_cu_count();
  if (M <= kRowsMax) {
    p.kind = kKindRows;
    p.blocks = (N + 15) / 16;
    return p;
  }
  if (tiles_of<Big>(M, N) >= cus) {
    p.kind = kKindBig;
    p.blocks = tiles_of<Big>(M, N);
    return p;
  }
  if (tiles_of<Med>(M, N) >= cus) {
    p.kind = kKindMed;
    p.blocks = tiles_of<Med>(M, N);
    return p;
  }
  p.kind = kKindSmall;
  p.blocks = tiles_of<Small>(M, N);
  const int ksteps = (K + KS - 1) / KS;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({2 * cus / p.blocks, ksteps / 16, 8}));
  if (p.splits > 1) {
    p.bytes = (size_t)p.splits * M * ((N + 3) / 4 * 4) * sizeof(float);
    p.blocks *= p.splits;
  }
  return p;
}

template <class O, int ACT>
hipError_t launch(const Plan& p, const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  switch (p.kind) {
    case kKindRows: {
      const dim3 threads(kRowWaves * 64);
      if (a.M <= 16)
        hipLaunchKernelGGL((linear_rows<O, ACT, 1>), grid, threads, 0, stream, a);
      else if (a.M <= 32)
        hipLaunchKernelGGL((linear_rows<O, ACT, 2>), grid, threads, 0, stream, a);
      else
        hipLaunchKernelGGL((linear_rows<O, ACT, 4>), grid, threads, 0, stream, a);
      return hipGetLastError();
    }
    case kKindBig:
      hipLaunchKernelGGL((linear_tile<Big, O, ACT, false>), grid, dim3(Big::THREADS), 0, stream, a);
      return hipGetLastError();
    case kKindMed:
      hipLaunchKernelGGL((linear_tile<Med, O, ACT, false>), grid, dim3(Med::THREADS), 0, stream, a);
      return hipGetLastError();
    case kKindSmall:
      break;
  }
  if (p.splits == 1) {
    hipLaunchKernelGGL((linear_tile<Small, O, ACT, false>), grid, dim3(Small::THREADS), 0, stream, a);
    return hipGetLastError();
  }
  // the shares do not depend on the output's type or the activation
  hipLaunchKernelGGL((linear_tile<Small, float, kActNone, true>), grid, dim3(Small::THREADS), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.M * (a.part_ld / 4);
  hipLaunchKernelGGL((linear_join<O, ACT>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <class O>
hipError_t with_act(const Plan& p, const LinearArgs& a, int act, hipStream_t stream) {
  if (act == kActGeluTanh) return launch<O, kActGeluTanh>(p, a, stream);
  if (act == kActSilu) return launch<O, kActSilu>(p, a, stream);
  return launch<O, kActNone>(p, a, stream);
}

}  // namespace

size_t linear_workspace(int M, int K, int N) { return plan_of(M, K, N).bytes; }
int64_t linear_blocks(int M, int K, int N) { return plan_of(M, K, N).blocks; }

hipError_t launch_linear_bf16(LinearArgs a, int act, bool fp32, hipStream_t stream) {
  const Plan p = plan_of(a.M, a.K, a.N);
  a.splits = p.splits;
  a.part_ld = (a.N + 3) / 4 * 4;
  a.wide = a.N % 4 == 0;
  return fp32 ? with_act<float>(p, a, act, stream) : with_act<uint16_t>(p, a, act, stream);
}

}  // namespace svdq
