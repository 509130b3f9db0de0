// The linear of the layers a 4-bit model keeps in 16 bits, gfx950:
//
//   Y = act(X W^T + bias) + residual,   X [M, K], W [N, K] bf16
//
// with bias, activation and residual in the product's epilogue: float32
// accumulators, one rounding to the output's type.  The residual enters as
// Y's type.
//
// Three kernels, all on the 16x16x32 bf16 MFMA with Y^T tiles (W rows as the
// MFMA's A operand, X rows as B): a lane's four accumulators are then
// neighbouring outputs of one row of Y.  A step is 64 channels: a row's step
// is one 128-byte line, moved whole by direct copies into LDS
// (global_load_lds).  With steps of 32 channels the half lines cost twice the
// requests: the L2 then delivers 16 TB/s instead of 28.
//
//   linear_tile   a ring of NR LDS buffers, NR - 1 steps of copies in flight,
//                 one barrier a step; 128 x 128, 128 x 64 and 64 x 64 tiles.
//                 Where tiles are few, the channels are cut into shares whose
//                 float32 sums linear_join brings together.
//   linear_turns  256 x 256, eight waves in two groups that take turns: while
//                 one group's MFMAs run, the other reads its fragments.  Large
//                 products: the tile moves the fewest bytes per operation.
//   linear_rows   up to 16 rows of X: the weight's bytes are the cost, and each
//                 wave streams its share of the channels of 16 weight rows
//                 straight into registers.
//
// Measured: 4608 x 3072 -> 12288 296 us (1175 TFLOP/s) with 256 x 256 turns (with bf16
// stored straight from the accumulators 330 us), 354 / 444 / 502 with the smaller
// tiles; 1155 x 1288 -> 1290 with a float32 residual 14.2 us with 128 x 64, 15.9 with
// 64 x 64, 27 with 128 x 128, on the same inputs each time (128 x 64 with inputs from
// HBM 18.6); 2 x 3072 -> 18432 24.7 us (4.6 TB/s) in linear_rows, 1 x 3072 -> 3072 8.5.
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

// Vectors of four at any element's alignment: rows of Y need not start on a
// 16-byte boundary, and the memory pipeline takes such accesses whole.
typedef f32x4 f32x4u __attribute__((aligned(4)));
typedef u32x2 u32x2u __attribute__((aligned(2)));
typedef u32x4 u32x4u __attribute__((aligned(2)));

__device__ inline f32x4 unpack4(u32x2 b) {
  return f32x4{__uint_as_float(b[0] << 16), __uint_as_float(b[0] & 0xFFFF0000u), __uint_as_float(b[1] << 16),
               __uint_as_float(b[1] & 0xFFFF0000u)};
}

// bias[n .. n + 3], zeros past the row and where there is none
__device__ inline f32x4 bias4(const LinearArgs& a, int n) {
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!a.bias || n >= a.N) return v;
  if (n + 4 <= a.N) return unpack4(*reinterpret_cast<const u32x2u*>(a.bias + n));
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) v[i] = bf16_value(a.bias[n + i]);
  return v;
}

// The residual at n .. n + 3 of row m as it lies in memory; zeros outside the
// matrix and where there is none.
__device__ inline f32x4 residual4(const LinearArgs& a, int64_t m, int n, float) {
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!a.residual || m >= a.M || n >= a.N) return v;
  const float* r = static_cast<const float*>(a.residual) + m * a.N + n;
  if (n + 4 <= a.N) return *reinterpret_cast<const f32x4u*>(r);
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) v[i] = r[i];
  return v;
}
__device__ inline u32x2 residual4(const LinearArgs& a, int64_t m, int n, uint16_t) {
  u32x2 v = u32x2{0u, 0u};
  if (!a.residual || m >= a.M || n >= a.N) return v;
  const uint16_t* r = static_cast<const uint16_t*>(a.residual) + m * a.N + n;
  if (n + 4 <= a.N) return *reinterpret_cast<const u32x2u*>(r);
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) v[i >> 1] |= (uint32_t)r[i] << (16 * (i & 1));
  return v;
}
__device__ inline f32x4 widen(f32x4 v) { return v; }
__device__ inline f32x4 widen(u32x2 v) { return unpack4(v); }

// Four neighbouring outputs in float32 but for the residual.
template <int ACT>
__device__ inline f32x4 value4(f32x4 v, f32x4 bias) {
  v += bias;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = activate<ACT>(v[i]);
  return v;
}

__device__ inline u32x2 pack4(f32x4 v) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16);
  return w;
}

template <class O>
__device__ inline void store4(f32x4 v, const LinearArgs& a, int64_t m, int n) {
  if (m >= a.M || n >= a.N) return;
  O* y = static_cast<O*>(a.Y) + m * a.N + n;
  if (n + 4 <= a.N) {
    if constexpr (sizeof(O) == 4)
      *reinterpret_cast<f32x4u*>(y) = v;
    else
      *reinterpret_cast<u32x2u*>(y) = pack4(v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    if constexpr (sizeof(O) == 4)
      y[i] = v[i];
    else
      y[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
  }
}

template <class O, int ACT>
__device__ inline void finish4(f32x4 v, f32x4 bias, const LinearArgs& a, int64_t m, int n) {
  store4<O>(value4<ACT>(v, bias) + widen(residual4(a, m, n, O())), a, m, n);
}

constexpr int KS = 64;            // channels per step: two MFMAs deep
constexpr int ROWB = KS * 2;      // bytes of a row's step, one line
constexpr int CHUNKS = ROWB / 16;

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
  static constexpr int PITCH = 16 * TN + 8;             // bf16 of a staged output row
  static constexpr int STAGE = WAVES * 16 * PITCH * 2;  // bytes: 16 rows per wave
  static_assert(COPIES % WAVES == 0, "every wave copies the same number of KB");
  static_assert(NR == 2 || NR == 3, "two or three ring buffers");
  static_assert(CPW * NR < 64, "vmcnt range");
};

using Big = Tile<2, 4, 8, 4, 2>;     // 256 x 256, 8 waves, 128 KB: linear_turns
using Med = Tile<2, 2, 4, 4, 2>;     // 128 x 128, 4 waves, 64 KB
using Tall = Tile<2, 2, 4, 2, 3>;    // 128 x 64, 4 waves, 72 KB
using Deep = Tile<2, 2, 2, 2, 3>;    //  64 x 64, 4 waves, 48 KB: one step more in flight
using Small = Tile<2, 2, 2, 2, 2>;   //  64 x 64, 4 waves, 32 KB

// XOR key of the 16-byte chunks of an LDS row: a fragment read covers 16
// consecutive rows at one chunk, which must fill all banks.
__device__ inline int swz_key(int row) { return (row >> 1) & (CHUNKS - 1); }

// vmcnt = n (later steps' copies stay in flight), lgkmcnt = 0: this wave's LDS
// reads are complete before the barrier lets another wave copy over them.
template <int n>
__device__ inline void ring_wait() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));
}

// lgkmcnt = 0 alone
__device__ inline void lds_wait() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// One wave's part of a tile: its copies, fragments, accumulators and outputs.
template <class C>
struct Wave {
  int m0, n0;                      // the tile
  int lane, wave, wm, wn, fr, fk;
  int nchunks;                     // 16-byte chunks of a row
  const uint16_t* src[C::CPW];
  int chunk[C::CPW];
  int key, x_lane, w_lane;
  f32x4 acc[C::TM][C::TN];

  __device__ Wave(const LinearArgs& a, int tmi, int tni) : m0(tmi * C::BM), n0(tni * C::BN) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    nchunks = a.K / 8;
    // copies of a step, 1 KB each: lane j fills physical chunk j % 8 of row j / 8.
    // Rows past the matrix read its last row; chunks past K (the last step's)
    // the row's last chunk, zeroed in read().
#pragma unroll
    for (int i = 0; i < C::CPW; ++i) {
      const int row = (wave * C::CPW + i) * (1024 / ROWB) + lane / CHUNKS;
      chunk[i] = (lane % CHUNKS) ^ swz_key(row);
      src[i] = row < C::BM ? a.X + (int64_t)min(m0 + row, a.M - 1) * a.K
                           : a.W + (int64_t)min(n0 + row - C::BM, a.N - 1) * a.K;
    }
    wm = wave / C::WN;
    wn = wave - wm * C::WN;
    fr = lane & 15;
    fk = lane >> 4;
    // tile t of a wave starts 16 rows further, where the swizzle key is the same
    key = swz_key(fr);
    x_lane = (wm * C::TM * 16 + fr) * ROWB;
    w_lane = (C::BM + wn * C::TN * 16 + fr) * ROWB;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  __device__ void copy(int step, uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < C::CPW; ++i) {
      const uint16_t* g = src[i] + 8 * min(CHUNKS * step + chunk[i], nchunks - 1);
      __builtin_amdgcn_global_load_lds(g, (lds_ptr)(buf + (wave * C::CPW + i) * 1024), 16, 0, 0);
    }
  }

  // the fragments of half u (32 channels) of a step
  __device__ void read(bf16x8 (&xf)[C::TM], bf16x8 (&wf)[C::TN], const uint8_t* buf, int step, int u) {
    const int at = ((4 * u + fk) ^ key) << 4;
#pragma unroll
    for (int t = 0; t < C::TN; ++t) wf[t] = *reinterpret_cast<const bf16x8*>(buf + w_lane + at + t * 16 * ROWB);
#pragma unroll
    for (int t = 0; t < C::TM; ++t) xf[t] = *reinterpret_cast<const bf16x8*>(buf + x_lane + at + t * 16 * ROWB);
    if (CHUNKS * (step + 1) > nchunks) {       // the matrices' last step, cut short
      if (CHUNKS * step + 4 * u + fk >= nchunks) {
#pragma unroll
        for (int t = 0; t < C::TN; ++t) wf[t] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
#pragma unroll
        for (int t = 0; t < C::TM; ++t) xf[t] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
      }
    }
  }

  __device__ void multiply(const bf16x8 (&xf)[C::TM], const bf16x8 (&wf)[C::TN]) {
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn)
        acc[tm][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[tn], xf[tm], acc[tm][tn], 0, 0, 0);
  }

  // The residual of register quad (tm, tn).
  template <class O>
  __device__ auto residual(const LinearArgs& a, int tm, int tn) const {
    return residual4(a, (int64_t)m0 + wm * C::TM * 16 + 16 * tm + fr, n0 + wn * C::TN * 16 + 16 * tn + 4 * fk, O());
  }

  // The wave's outputs.  float32 goes straight from the accumulators (64
  // neighbouring bytes of a row per instruction); bf16 through the wave's own
  // staging rows, 16 rows at a time, so that whole lines are stored, which then
  // stream out non-temporally: 4608 x 3072 -> 12288 300 us, against 306 with
  // stores that allocate in the caches and 330 with 8-byte stores straight from
  // the accumulators.
  // add(v, tm, tn): v and the residual of a register quad.
  template <class O, int ACT, class F>
  __device__ void outputs(const LinearArgs& a, uint8_t* stage, F add) {
    const int n1 = n0 + wn * C::TN * 16;
    const int64_t m1 = (int64_t)m0 + wm * C::TM * 16;
    f32x4 bias[C::TN];
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) bias[tn] = bias4(a, n1 + 16 * tn + 4 * fk);
    if constexpr (sizeof(O) == 4) {
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
        for (int tn = 0; tn < C::TN; ++tn)
          store4<O>(add(value4<ACT>(acc[tm][tn], bias[tn]), tm, tn), a, m1 + 16 * tm + fr, n1 + 16 * tn + 4 * fk);
    } else {
      uint16_t* rows = reinterpret_cast<uint16_t*>(stage) + wave * 16 * C::PITCH;
      constexpr int CPR = 2 * C::TN;      // 16-byte chunks of a row
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
#pragma unroll
        for (int tn = 0; tn < C::TN; ++tn) {
          const f32x4 v = add(value4<ACT>(acc[tm][tn], bias[tn]), tm, tn);
          *reinterpret_cast<u32x2*>(rows + fr * C::PITCH + 16 * tn + 4 * fk) = pack4(v);
        }
        // a wave's LDS accesses complete in issue order; the fences keep the
        // compiler's order of the writes, the reads and the next pass's writes
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
        for (int c = lane; c < 16 * CPR; c += 64) {
          const int row = c / CPR, ch = c - (c / CPR) * CPR;
          const int64_t m = m1 + 16 * tm + row;
          const int n = n1 + 8 * ch;
          const u32x4 v = *reinterpret_cast<const u32x4*>(rows + row * C::PITCH + 8 * ch);
          if (m < a.M && n < a.N) {
            uint16_t* y = static_cast<uint16_t*>(a.Y) + m * a.N + n;
            if (n + 8 <= a.N) {
              __builtin_nontemporal_store(v, reinterpret_cast<u32x4u*>(y));
            } else {
              for (int i = 0; i < 8; ++i)
                if (n + i < a.N) y[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
            }
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
      }
    }
  }

  // A share's sums, for linear_join; part_ld: N rounded up to 4.
  __device__ void sums(const LinearArgs& a, int share) {
#pragma unroll
    for (int tn = 0; tn < C::TN; ++tn) {
      const int n = n0 + wn * C::TN * 16 + 16 * tn + 4 * fk;
#pragma unroll
      for (int tm = 0; tm < C::TM; ++tm) {
        const int64_t m = (int64_t)m0 + wm * C::TM * 16 + 16 * tm + fr;
        if (m < a.M && n < a.N)
          *reinterpret_cast<f32x4*>(a.part + ((int64_t)share * a.M + m) * a.part_ld + n) = acc[tm][tn];
      }
    }
  }
};

template <class C, class O, int ACT, bool SHARES>
__global__ __launch_bounds__(C::THREADS, 2) void linear_tile(const LinearArgs a) {
  // each buffer its own array: reading one then does not wait for copies into another
  __shared__ __attribute__((aligned(16))) uint8_t ring0[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring2[C::NR > 2 ? C::BUF : 16];
  __shared__ __attribute__((aligned(16))) uint8_t stage[SHARES || sizeof(O) == 4 ? 16 : C::STAGE];
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
  Wave<C> w(a, tmi, tni);

  // step sb + j from `cur`; step sb + j + NR - 1 (past the last: the last
  // again, never read) is copied to the buffer that step sb + j - 1 used
  auto step = [&](int j, const uint8_t* cur, uint8_t* freed) {
    ring_wait<C::CPW * (C::NR - 2)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    w.copy(sb + min(j + C::NR - 1, nsteps - 1), freed);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8 xf[C::TM], wf[C::TN];
      w.read(xf, wf, cur, sb + j, u);
      w.multiply(xf, wf);
    }
  };
  // small tiles have registers to spare for the residual, which then arrives
  // beside the first copies
  constexpr bool kEarly = !SHARES && C::TM * C::TN <= 8;
  decltype(residual4(a, 0, 0, O())) early[kEarly ? C::TM : 1][kEarly ? C::TN : 1];
  if constexpr (kEarly) {
#pragma unroll
    for (int tm = 0; tm < C::TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < C::TN; ++tn) early[tm][tn] = w.template residual<O>(a, tm, tn);
  }
  w.copy(sb, ring0);
  if constexpr (C::NR > 2) w.copy(sb + min(1, nsteps - 1), ring1);
  // whole turns of the ring without branches, then the rest
  int j = 0;
  if constexpr (C::NR == 2) {
    for (; j + 2 <= nsteps; j += 2) {
      step(j, ring0, ring1);
      step(j + 1, ring1, ring0);
    }
    if (j < nsteps) step(j, ring0, ring1);
  } else {
    for (; j + 3 <= nsteps; j += 3) {
      step(j, ring0, ring2);
      step(j + 1, ring1, ring0);
      step(j + 2, ring2, ring1);
    }
    if (j < nsteps) step(j, ring0, ring2);
    if (j + 1 < nsteps) step(j + 1, ring1, ring0);
  }
  ring_wait<0>();     // a workgroup may not leave copies into its LDS behind

  if constexpr (SHARES)
    w.sums(a, share);
  else
    w.template outputs<O, ACT>(a, stage, [&](f32x4 v, int tm, int tn) {
      if constexpr (kEarly)
        return v + widen(early[tm][tn]);
      else
        return a.residual ? v + widen(w.template residual<O>(a, tm, tn)) : v;
    });
}

// The 256 x 256 tile: waves 0..3 and 4..7, one of each on every SIMD, are half a
// turn apart, so that one group's MFMAs run while the other's LDS reads do.
// A turn is half a step: read the fragments, barrier, multiply, barrier; the
// second group passes one barrier more at the start, the first one more at
// the end.  Buffers: step j + 1 is copied while step j runs, from the group's
// first turn of j on (by then both groups have read step j - 1 whole), and
// has landed before the barrier that ends the reading of j's second half.
// Alone, the MFMAs and LDS reads of this loop reach 2085 TFLOP/s, the copies
// 12 TB/s; together 8192 x 8192 -> 8192 takes 791 us (1389 TFLOP/s).  Halving the
// tiles of a last round that leaves most CUs idle gains nothing (305 us either
// way at 4608 x 3072 -> 12288, 3.4 rounds): the tiles of such a round run faster.
template <class O, int ACT>
__global__ __launch_bounds__(Big::THREADS, 2) void linear_turns(const LinearArgs a) {
  using C = Big;
  __shared__ __attribute__((aligned(16))) uint8_t ring0[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[C::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t stage[sizeof(O) == 4 ? 16 : C::STAGE];
  const int ntm = (a.M + C::BM - 1) / C::BM;
  const int ntn = (a.N + C::BN - 1) / C::BN;
  const int nsteps = (a.K + KS - 1) / KS;
  int tmi, tni;
  tail::tile_of_id(ntm, ntn, tail::xcd_compact(blockIdx.x, ntm * ntn), tmi, tni);
  Wave<C> w(a, tmi, tni);
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int j, const uint8_t* cur, uint8_t* other) {
    w.copy(min(j + 1, nsteps - 1), other);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8 xf[C::TM], wf[C::TN];
      w.read(xf, wf, cur, j, u);
      if (u == 1)
        ring_wait<0>();
      else
        lds_wait();
      barrier();
      __builtin_amdgcn_s_setprio(1);
      w.multiply(xf, wf);
      __builtin_amdgcn_s_setprio(0);
      barrier();
    }
  };
  w.copy(0, ring0);
  ring_wait<0>();
  barrier();
  const bool second = w.wave >= C::WAVES / 2;
  if (second) barrier();
  int j = 0;
  for (; j + 2 <= nsteps; j += 2) {
    step(j, ring0, ring1);
    step(j + 1, ring1, ring0);
  }
  if (j < nsteps) step(j, ring0, ring1);
  if (!second) barrier();
  w.template outputs<O, ACT>(a, stage, [&](f32x4 v, int tm, int tn) {
    return a.residual ? v + widen(w.template residual<O>(a, tm, tn)) : v;
  });
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
  finish4<O, ACT>(v, bias4(a, n), a, m, n);
}

// Up to 16 rows: 16 weight rows per workgroup; wave w takes every
// kRowWaves-th block of 64 channels.  Lane (fk, fr) reads 32 neighbouring
// bytes of weight row fr, so that the four lanes of a row take a whole
// 128-byte line; the MFMA's k slots are any 32 channels as long as both
// operands agree, so the two 16-byte halves are two MFMAs.  The loop is not
// unrolled: a wave has one block's loads in flight, and the waves of a CU make up
// for it where N gives it several workgroups.  (From 17 rows on the
// tiles are faster: 32 x 3072 -> 18432 31 us in 64 x 64 tiles with two shares,
// 54 us here with two blocks of rows.)
constexpr int kRowsMax = 16;
constexpr int kRowWaves = 8;
template <class O, int ACT>
__global__ __launch_bounds__(kRowWaves * 64) void linear_rows(const LinearArgs a) {
  __shared__ f32x4 sums[kRowWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fk = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const uint16_t* w = a.W + (int64_t)min(n0 + fr, a.N - 1) * a.K;
  const uint16_t* x = a.X + (int64_t)min(fr, a.M - 1) * a.K;
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  const int blocks = (a.K + 63) / 64;
  const u32x4 zero = u32x4{0u, 0u, 0u, 0u};
  for (int kb = wave; kb < blocks; kb += kRowWaves) {
    const int k = 64 * kb + 16 * fk;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = min(k + 8 * u, a.K - 8);
      const bool in = k + 8 * u < a.K;
      u32x4 wv = *reinterpret_cast<const u32x4*>(w + at);
      u32x4 xv = *reinterpret_cast<const u32x4*>(x + at);
      wv = in ? wv : zero;
      xv = in ? xv : zero;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, xv), acc,
                                                    0, 0, 0);
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  f32x4 v = sums[0][lane];
#pragma unroll
  for (int s = 1; s < kRowWaves; ++s) v += sums[s][lane];
  finish4<O, ACT>(v, bias4(a, n0 + 4 * fk), a, fr, n0 + 4 * fk);
}

enum Kind { kKindRows, kKindBig, kKindMed, kKindTall, kKindDeep, kKindSmall };
struct Plan {
  Kind kind = kKindRows;
  int splits = 1;
  int64_t blocks = 0;
  size_t bytes = 0;
};

template <class C>
int64_t tiles_of(int64_t M, int64_t N) {
  return ((M + C::BM - 1) / C::BM) * ((N + C::BN - 1) / C::BN);
}

// Tile and shares by an estimate of the time, in us: a CU that gets n tiles
// takes max(alone, n each) for a step of 64 channels of all of them (`alone`:
// what the copies' latency costs one tile; `each`: its part of the CU's
// bandwidth; 128 x 128 tiles run in pairs, so an odd one costs two), `fill` once
// for filling the ring and storing the tile, and shares cost a second launch
// and the traffic of their sums.  The table's figures are measured ones.  64 x 64
// tiles come in two forms: with two steps of copies in flight while a CU has two
// of them at most (512 x 1280 -> 1280 8.0 us, 11.5 with one step; 32 x 3072 -> 18432
// 30.9 and 39.2), else with one, since more of the smaller workgroups fit a CU
// (4096 x 640 -> 640 9.1 us, 10.8 with two steps).  Over 29 shapes from 77 x 640 -> 640
// to 4608 x 12288 -> 3072 the choice is the fastest or within 10 % of it, where always
// taking 128 x 64 loses up to 61 % and always 64 x 64 up to 83 %.
constexpr int kMaxSplits = 8;
constexpr int kMinShareSteps = 8;          // below that a share is all latency
constexpr size_t kMaxPartBytes = size_t(32) << 20;

Plan plan_of(int M, int K, int N) {
  Plan best;
  if (M <= kRowsMax) {
    best.blocks = ((int64_t)N + 15) / 16;
    return best;
  }
  const struct {
    Kind kind;
    int64_t tiles;
    double alone, each, fill;
  } tile[] = {{kKindBig, tiles_of<Big>(M, N), 1.4, 1.5, 3.5},
              {kKindMed, tiles_of<Med>(M, N), 0.8, 0.47, 0.0},
              {kKindTall, tiles_of<Tall>(M, N), 0.31, 0.36, 0.8},
              {kKindDeep, tiles_of<Deep>(M, N), 0.26, 0.28, 0.0},
              {kKindSmall, tiles_of<Small>(M, N), 0.42, 0.24, 0.0}};
  const int cus = device_cu_count();
  const int64_t steps = ((int64_t)K + KS - 1) / KS;
  double least = 0;
  for (const auto& t : tile)
    for (int s = 1; s <= (t.kind == kKindBig || t.kind == kKindSmall ? 1 : kMaxSplits); s *= 2) {
      if ((t.kind == kKindDeep && t.tiles * s > 2 * cus) || (t.kind == kKindSmall && t.tiles <= 2 * cus)) break;
      const size_t part = s > 1 ? (size_t)s * M * (((size_t)N + 3) / 4 * 4) * sizeof(float) : 0;
      if (s > 1 && (steps / s < kMinShareSteps || part > kMaxPartBytes)) break;
      int64_t n = (t.tiles * s + cus - 1) / cus;
      if (t.kind == kKindMed && n > 1) n += n & 1;
      double us = t.fill + (double)((steps + s - 1) / s) * std::max(t.alone, n * t.each);
      if (s > 1) us += 3.0 + 2.0 * part / 4e6;
      if (best.blocks == 0 || us < least) {
        least = us;
        best.kind = t.kind;
        best.splits = s;
        best.blocks = t.tiles * s;
        best.bytes = part;
      }
    }
  return best;
}

template <class C, class O, int ACT>
hipError_t launch_whole(const Plan& p, const LinearArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((linear_tile<C, O, ACT, false>), dim3((unsigned)p.blocks), dim3(C::THREADS), 0, stream, a);
  return hipGetLastError();
}

template <class C, class O, int ACT>
hipError_t launch_tile(const Plan& p, const LinearArgs& a, hipStream_t stream) {
  if (p.splits == 1) return launch_whole<C, O, ACT>(p, a, stream);
  const dim3 grid((unsigned)p.blocks);
  // the shares do not depend on the output's type or the activation
  hipLaunchKernelGGL((linear_tile<C, float, kActNone, true>), grid, dim3(C::THREADS), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.M * (a.part_ld / 4);
  hipLaunchKernelGGL((linear_join<O, ACT>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <class O, int ACT>
hipError_t launch(const Plan& p, const LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  switch (p.kind) {
    case kKindRows:
      hipLaunchKernelGGL((linear_rows<O, ACT>), grid, dim3(kRowWaves * 64), 0, stream, a);
      return hipGetLastError();
    case kKindBig:
      hipLaunchKernelGGL((linear_turns<O, ACT>), grid, dim3(Big::THREADS), 0, stream, a);
      return hipGetLastError();
    case kKindMed:
      return launch_tile<Med, O, ACT>(p, a, stream);
    case kKindTall:
      return launch_tile<Tall, O, ACT>(p, a, stream);
    case kKindDeep:
      return launch_tile<Deep, O, ACT>(p, a, stream);
    case kKindSmall:
      return launch_whole<Small, O, ACT>(p, a, stream);
  }
  return hipErrorInvalidValue;
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
  return fp32 ? with_act<float>(p, a, act, stream) : with_act<uint16_t>(p, a, act, stream);
}

}  // namespace svdq
