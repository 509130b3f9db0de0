// The norm of every head of the queries and keys and the rotation by the token's position, in one
// pass between the QKV projection and attention, gfx950:
//
//   n = norm(v) w + b            over the head's channels, float32 statistics
//   (x, y) -> (x cos - y sin, y cos + x sin)   for the pairs of the first rot channels
//
// HBM bound: 2 bytes in and 2 out per element, a few operations each; the table's rows and the
// weights are small and come from the caches.
//
// A head belongs to L lanes of 8 channels each (L the power of two that holds it), laid out so
// that both channels of a pair are in one lane: 8 t .. 8 t + 7 where neighbours are paired,
// 4 t .. 4 t + 3 and rot / 2 + the same where halves are.  So the rotation needs no exchange,
// the norm log2(L) of them, and a thread writes only what it has itself read (the outputs may be
// the inputs).  A wave takes U steps of 64 / L heads of one row (of several rows where a row has
// fewer heads), queries or keys, so that one row of the table and one of the weights serve
// U heads of a lane.
#include <algorithm>

#include "svdq_internal.h"

namespace svdq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kWaves = 4096;      // of a launch, at least, where a wave takes more than one step

struct Params {
  QkNormRopeArgs a;
  int log_rows;            // 2^log_rows rows in a wave's step
  int parts_q, parts;      // waves per row(s): those of the queries first
  int units;               // waves of the launch
  Quotient by_parts;
};

__device__ inline void unpack4(u32x2 v, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ inline u32x2 pack4(const float* f) {
  u32x2 v;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = __builtin_bit_cast(uint16_t, (__bf16)f[2 * i]) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[2 * i + 1]) << 16);
  return v;
}

// A lane's 8 channels: two pieces of 4, at ca and cb (neighbours: one piece of 8).
template <bool HALVES>
__device__ inline u32x4 load8(const uint16_t* p, int ca, int cb) {
  if constexpr (HALVES) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(p + ca), b = *reinterpret_cast<const u32x2*>(p + cb);
    return u32x4{a[0], a[1], b[0], b[1]};
  }
  return *reinterpret_cast<const u32x4*>(p + ca);
}
template <bool HALVES>
__device__ inline void store8(uint16_t* p, int ca, int cb, const float (&f)[8]) {
  const u32x2 a = pack4(f), b = pack4(f + 4);
  if constexpr (HALVES) {
    __builtin_nontemporal_store(a, reinterpret_cast<u32x2*>(p + ca));
    __builtin_nontemporal_store(b, reinterpret_cast<u32x2*>(p + cb));
  } else {
    __builtin_nontemporal_store(u32x4{a[0], a[1], b[0], b[1]}, reinterpret_cast<u32x4*>(p + ca));
  }
}
__device__ inline void unpack8(u32x4 v, float (&f)[8]) {
  unpack4(u32x2{v[0], v[1]}, f);
  unpack4(u32x2{v[2], v[3]}, f + 4);
}

// The sum of v over the head's L lanes, in all of them.  Within 16 lanes by DPP: the halves of
// a quad, then mirrored groups whose lanes already hold the same.
template <int CTRL>
__device__ inline float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int L>
__device__ inline float head_sum(float v) {
  if constexpr (L >= 2) v += dpp<0xB1>(v);       // quad_perm 1, 0, 3, 2
  if constexpr (L >= 4) v += dpp<0x4E>(v);       // quad_perm 2, 3, 0, 1
  if constexpr (L >= 8) v += dpp<0x141>(v);      // row_half_mirror
  if constexpr (L >= 16) v += dpp<0x140>(v);     // row_mirror
  if constexpr (L >= 32) v += __shfl_xor(v, 16);
  return v;
}

// The position of `row` in its sequence, and whether it has one.  The wave's first row is looked
// up among 64 offsets at a time; its other rows (ROWS) may lie in later sequences.
template <bool ROWS>
__device__ inline bool place_of(const int32_t* cu, int batch, int64_t row0, int64_t row, int lane, int64_t& at) {
  int b = -1, begin = 0, end = 0;
  for (int base = 0; base <= batch; base += 64) {
    const int c = cu[min(base + lane, batch)];
    const uint64_t m = __ballot(base + lane <= batch && c <= row0);
    const int n = __builtin_popcountll(m);
    b += n;
    if (n > 0) begin = __builtin_amdgcn_readlane(c, n - 1);
    if (n < 64) {
      end = __builtin_amdgcn_readlane(c, n);      // past the last offset: that again
      break;
    }
  }
  if constexpr (ROWS)
    while (b < batch && end <= row) {
      begin = end;
      ++b;
      if (b < batch) end = cu[b + 1];
    }
  at = row - begin;
  return b >= 0 && b < batch;
}

// ROWS: a step takes several rows, else one, whose number is the same in all lanes.
template <int L, int U, bool HALVES, bool ROWS>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(const Params p) {
  const QkNormRopeArgs& a = p.a;
  constexpr int kGroups = 64 / L, kLogGroups = __builtin_ctz(kGroups);      // heads of a wave's step
  const int lane = threadIdx.x & 63;
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= p.units) return;
  const int rest = p.by_parts.of(unit);
  const int part = unit - rest * p.parts;
  const int64_t row0 = ROWS ? (int64_t)rest << p.log_rows : rest;
  const bool is_q = part < p.parts_q;
  const int heads = is_q ? a.heads_q : a.heads_k;
  const uint16_t* in = is_q ? a.Q : a.K;
  uint16_t* out = is_q ? a.Q_out : a.K_out;
  const int64_t ldi = is_q ? a.ldq : a.ldk, ldo = is_q ? a.ldqo : a.ldko;
  const uint16_t* weight = is_q ? a.q_weight : a.k_weight;
  const uint16_t* bias = is_q ? a.q_bias : a.k_bias;

  const int t = lane % L, g = lane / L;
  const int log_step = ROWS ? kLogGroups - p.log_rows : kLogGroups;      // heads of a step in one row
  const int step = 1 << log_step;
  const int64_t row = ROWS ? row0 + (g >> log_step) : row0;
  const int head0 = (is_q ? part : part - p.parts_q) * U * step + (g & (step - 1));
  if (row0 >= a.rows) return;
  bool row_ok = row < a.rows;

  int64_t at = row;                            // the position
  if (a.cu) row_ok = place_of<ROWS>(a.cu, a.batch, row0, row, lane, at) && row_ok;
  if (!row_ok) return;
  if (a.positions) at = a.positions[row];

  // the lane's channels, and whether it has any
  const bool turned = 8 * t < a.rotary_dim;    // rotary_dim: a multiple of 8
  const int ca = HALVES && turned ? 4 * t : 8 * t;
  const int cb = HALVES && turned ? a.rotary_dim / 2 + 4 * t : 8 * t + 4;
  const bool on = 8 * t < a.head_dim;

  u32x4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = head0 + u * step;
    raw[u] = u32x4{0u, 0u, 0u, 0u};
    if (on && head < heads) raw[u] = load8<HALVES>(in + row * ldi + (int64_t)head * a.head_dim, ca, cb);
  }
  f32x4 c = {1.f, 1.f, 1.f, 1.f}, s = {0.f, 0.f, 0.f, 0.f};
  const bool turn = turned && at >= 0 && at < a.table_rows;
  if (turn) {
    c = *reinterpret_cast<const f32x4*>(a.cos + at * a.ld_table + 4 * t);
    s = *reinterpret_cast<const f32x4*>(a.sin + at * a.ld_table + 4 * t);
  }
  float w[8], bs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 1.f;
    bs[e] = 0.f;
  }
  if (weight && on) unpack8(load8<HALVES>(weight, ca, cb), w);
  if (bias && on) unpack8(load8<HALVES>(bias, ca, cb), bs);

  const float inv = 1.0f / (float)a.head_dim;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = head0 + u * step;
    float v[8];
    unpack8(raw[u], v);
    if (a.norm == kNormLayer) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e];
      const float mean = head_sum<L>(sum) * inv;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] -= mean;
    }
    if (a.norm != kNormNone) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = __builtin_fmaf(v[e], v[e], q);
      if (!on) q = 0.f;                        // lanes past the head hold -mean by now
      const float r = rsqrtf(__builtin_fmaf(head_sum<L>(q), inv, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= r;
    }
    if (!on || head >= heads) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], w[e], bs[e]);
    if (turn)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& x = v[HALVES ? i : 2 * i];
        float& y = v[HALVES ? 4 + i : 2 * i + 1];
        const float x0 = x;
        x = __builtin_fmaf(x0, c[i], -(y * s[i]));
        y = __builtin_fmaf(y, c[i], x0 * s[i]);
      }
    store8<HALVES>(out + row * ldo + (int64_t)head * a.head_dim, ca, cb, v);
  }
}

template <int L, int U, bool ROWS>
hipError_t launch(const Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)(((unsigned)p.units + 3) / 4));
  if (p.a.halves)
    hipLaunchKernelGGL((qk_norm_rope_kernel<L, U, true, ROWS>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<L, U, false, ROWS>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

int lanes_of(int head_dim) {
  int l = 1;
  while (8 * l < head_dim) l *= 2;
  return l;
}

// Steps of a wave: four, which spread what a wave does once (its row of the table and of the
// weights, the look-up of its row) over most heads, or as many as leave 4096 waves, four
// per SIMD, and then as evenly as the heads allow.  With one, two, three, four steps: 4608 rows x
// (24 + 24) x 128 25.6, 25.0, 23.9, 24.5 us; 15832 x (16 + 16) x 72 with LayerNorm 64, 45, 47, 38;
// 1024 x (24 + 24) x 128 8.7, 6.8, 7.1, 7.2; 400 4.8, 4.9, 5.2, 5.3; 16 x (32 + 8) 3.4, 3.6, 3.9, 4.2.
int64_t units_of(const QkNormRopeArgs& a, Params& p, int& lanes, int& steps) {
  lanes = lanes_of(a.head_dim);
  const int groups = 64 / lanes, most = std::max(a.heads_q, a.heads_k);
  p.log_rows = 0;
  while ((groups >> (p.log_rows + 1)) >= most) ++p.log_rows;
  const int step = groups >> p.log_rows;
  const int64_t row_steps = (a.rows + (1 << p.log_rows) - 1) >> p.log_rows;
  for (steps = p.log_rows > 0 ? 1 : 4;; --steps) {
    const int parts = (most + steps * step - 1) / (steps * step);
    const int each = (most + parts * step - 1) / (parts * step) * step;       // heads of a wave
    p.parts_q = (a.heads_q + each - 1) / each;
    p.parts = p.parts_q + (a.heads_k + each - 1) / each;
    if (steps > 1 && row_steps * p.parts < kWaves) continue;
    steps = each / step;
    return row_steps * p.parts;
  }
}

template <int L>
hipError_t with_steps(const Params& p, int steps, hipStream_t stream) {
  switch (steps) {
    case 4: return launch<L, 4, false>(p, stream);
    case 3: return launch<L, 3, false>(p, stream);
    case 2: return launch<L, 2, false>(p, stream);
  }
  return p.log_rows > 0 ? launch<L, 1, true>(p, stream) : launch<L, 1, false>(p, stream);
}

}  // namespace

int64_t qk_norm_rope_blocks(const QkNormRopeArgs& a) {
  Params p;
  int lanes, steps;
  return (units_of(a, p, lanes, steps) + 3) / 4;
}

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream) {
  Params p;
  int lanes, steps;
  p.a = a;
  p.units = (int)units_of(a, p, lanes, steps);
  p.by_parts = Quotient(p.parts);
  switch (lanes) {
    case 1: return with_steps<1>(p, steps, stream);
    case 2: return with_steps<2>(p, steps, stream);
    case 4: return with_steps<4>(p, steps, stream);
    case 8: return with_steps<8>(p, steps, stream);
    case 16: return with_steps<16>(p, steps, stream);
    default: return with_steps<32>(p, steps, stream);
  }
}

}  // namespace svdq
