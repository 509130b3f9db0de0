// Softmax attention over packed sequences (no padding, no score matrix), gfx950.
//
//   O_i = sum_j p_ij V_j,   p_ij = exp(scale q_i.k_j - m_i) / l_i
//
// over the keys j of query i's own sequence (causal: j <= i + nk - nq, so the
// last query sees the last key), in one pass over the keys with the running
// maximum m and sum l of the softmax.  A query without keys gets O = 0 and
// log-sum-exp -inf.
//
// Work split.  The `group` query heads that share a key head are rows of one
// problem: row r of (sequence, key head) is token r / group, head r % group.
// So a tile of rows reads its keys once for the whole group, and a single new
// token already brings `group` rows.  Two kernels share the arithmetic:
//   kRows   a workgroup takes 32 rows per wave; its waves share each K/V tile.
//   kKeys   a workgroup takes 32 rows in all; its waves take alternate K/V
//           tiles and join at the end.  For few rows per sequence, where the
//           keys' bytes are what counts.
// Where the tiles do not fill the chip, each tile's keys are cut into
// `splits` shares; shares write float32 partial rows and attention_join
// brings them together.
//
// Arithmetic of a wave, all in the 32x32x16 bf16 MFMA.  The scores are
// computed transposed, S^T = K Q^T: the accumulator then holds, in each lane,
// keys of ONE query (column lane % 32), so the softmax's maximum and sum are
// in-lane plus one exchange between the wave's halves, and the same registers,
// rounded to bf16, are the B operand of O^T += V^T P^T as they stand: the
// MFMA's k slots are assigned to keys in the accumulator's own order (slot
// 8 h + j of half h = lane / 32 is key 8 (j / 4) + 4 h + j % 4) and V^T is read
// in that order by ds_read_b64_tr_b16, which transposes 4 keys x 16 channels
// on the way out of LDS.  P never touches LDS.
//
// The running maximum is lazy: the accumulators are rescaled only when a
// tile's maximum exceeds the one in use by more than 8 (in the base-2 exponent),
// which leaves p <= 2^8: exact sums in float32, and the
// rounding of p to bf16 is relative.  p is rounded to bf16 because V is bf16
// and the MFMA takes both operands in one type; l sums the unrounded values.
#include <algorithm>

#include "svdq_internal.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;        // rescale when the maximum grows by more than this (base 2)
constexpr int kWaveRows = 32;        // rows (queries x heads of a group) of a wave
constexpr int kRows = 0, kKeys = 1;

struct Params {
  const uint16_t *Q, *K, *V;
  int64_t ldq, ldk, ldv, ldo;
  const int32_t *cu_q, *cu_k;
  int batch, total_q, total_k;
  int heads_q, heads_kv, group, head_dim;
  float c;               // scale * log2(e)
  int causal;
  uint16_t* O;
  float* lse;
  int splits;
  float* part;           // [unit][rows][head_dim] partial rows, unit = (tile, key head, split)
  float* part_lse;       // [unit][rows], base 2; -inf: the share saw no key
};

// One head's geometry: DP the LDS row in channels, KS the MFMA steps of 16
// channels of q.k, DB the blocks of 32 channels of the output.
template <int DP_, int KS_, int DB_>
struct Head {
  static constexpr int DP = DP_, KS = KS_, DB = DB_;
  static constexpr int ROWB = DP * 2;
  static constexpr int CHUNKS = ROWB / 16;      // 16-byte chunks per LDS row
};

template <class H, int MODE, int NW_>
struct Tile {
  static constexpr int NW = NW_;
  static constexpr int THREADS = NW * 64;
  static constexpr int ROWS = MODE == kRows ? NW * kWaveRows : kWaveRows;
  static constexpr int KT = MODE == kRows ? 64 : 32;     // keys of a tile
  static constexpr int KB = KT / 32;
  static constexpr int TILE_BYTES = KT * H::ROWB;        // K or V
  static constexpr int COPIERS = MODE == kRows ? NW : 1; // waves that fill one tile
  static constexpr int CPW = TILE_BYTES / 1024 / COPIERS;   // 1 KB copies per wave, K or V
  static constexpr int BUFS = MODE == kRows ? 1 : NW;    // K/V tiles a workgroup works on at once
  static_assert(TILE_BYTES % (1024 * COPIERS) == 0, "whole copies");
};

// LDS swizzles: the 16-byte chunk c of a row sits at chunk c ^ key(row).
// K fragments: 16 lanes read chunk c of 16 consecutive rows, which must land
// in 16 different chunks of the 256 bytes that the banks span.  V fragments:
// the transposing read takes 4 rows x 4 chunks at once.
template <class H>
__device__ inline int k_key(int row) {
  return H::DP == 128 ? row & 15 : (row >> 1) & 7;
}
template <class H>
__device__ inline int v_key(int row) {
  return H::DP == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

__device__ inline float max_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float sum_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A sequence's rows, kept inside the buffers whatever the offsets hold.
__device__ inline void span(const int32_t* cu, int b, int total, int& begin, int& len) {
  const int lo = cu ? cu[b] : 0, hi = cu ? cu[b + 1] : total;
  begin = min(max(lo, 0), total);
  len = max(min(hi, total) - begin, 0);
}

// Tile number `t` of the packed batch -> its sequence and the tile's number in
// it (rows: tile height).  False: past the last tile.  64 sequences at a time,
// one per lane.
__device__ inline bool find_tile(const Params& p, int rows, int t, int lane, int& b, int& local) {
  for (int base = 0; base < p.batch; base += 64) {
    int n = 0;
    if (base + lane < p.batch) {
      int q0, nq;
      span(p.cu_q, base + lane, p.total_q, q0, nq);
      n = (nq * p.group + rows - 1) / rows;
    }
    int end = n;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(end, s);
      if (lane >= s) end += o;
    }
    const uint64_t after = __ballot(t < end);
    if (after) {
      const int l = __builtin_ctzll(after);
      b = base + l;
      local = t - (__shfl(end, l) - __shfl(n, l));
      return true;
    }
    t -= __shfl(end, 63);
  }
  return false;
}

// s_waitcnt vmcnt(n) and lgkmcnt(0), expcnt untouched
template <int n>
__device__ inline void copies_wait() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));
}

template <class H, int MODE, int NW>
__global__ __launch_bounds__(NW * 64, 2) void attention_kernel(const Params p) {
  using T = Tile<H, MODE, NW>;
  constexpr int KT = T::KT, KB = T::KB;
  // each buffer its own array: reading one then does not wait for copies into another
  __shared__ __attribute__((aligned(16))) uint8_t k0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k1s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v1s[T::BUFS * T::TILE_BYTES];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5;
  const int col = lane & 31;

  // blocks run over key heads first, then shares, then tiles
  const int hk = blockIdx.x % p.heads_kv;
  const int rest = blockIdx.x / p.heads_kv;
  const int split = rest % p.splits;
  int b, local;
  if (!find_tile(p, T::ROWS, rest / p.splits, lane, b, local)) return;
  b = __builtin_amdgcn_readfirstlane(b);
  local = __builtin_amdgcn_readfirstlane(local);
  int q0, nq, kv0, nk;
  span(p.cu_q, b, p.total_q, q0, nq);
  span(p.cu_k, b, p.total_k, kv0, nk);
  const int nrows = nq * p.group;
  // causal tiles see more keys the later they are: start with the last
  if (p.causal) local = (nrows + T::ROWS - 1) / T::ROWS - 1 - local;
  const int row0 = local * T::ROWS;
  const int wrow0 = row0 + (MODE == kRows ? wave * kWaveRows : 0);
  const int row = wrow0 + col;                       // this lane's query
  const bool row_ok = row < nrows;
  const int rowc = min(row, nrows - 1);
  const int token = rowc / p.group;
  const int head = hk * p.group + (rowc - token * p.group);

  // keys: [0, kend) for the tile; `seen` for this lane's query
  const int shift = nk - nq;
  const int last_tok = (min(row0 + T::ROWS, nrows) - 1) / p.group;
  const int kend = p.causal ? min(max(last_tok + shift + 1, 0), nk) : nk;
  const int seen = p.causal ? min(max(token + shift + 1, 0), nk) : nk;
  // wave bounds: every query of the wave sees [0, wfull), none sees from wend on
  const int wfull = __builtin_amdgcn_readfirstlane(
      p.causal ? min(max(min(wrow0, nrows - 1) / p.group + shift + 1, 0), nk) : nk);
  const int wend = __builtin_amdgcn_readfirstlane(
      p.causal ? min(max(min(wrow0 + kWaveRows - 1, nrows - 1) / p.group + shift + 1, 0), nk) : nk);
  const int ntiles = (kend + KT - 1) / KT;
  const int t0 = (int)((int64_t)ntiles * split / p.splits);
  const int t1 = (int)((int64_t)ntiles * (split + 1) / p.splits);

  // Q as the B operand: lane's query, channels 16 ks + 8 half .. + 7
  bf16x8 qf[H::KS];
  {
    const uint16_t* q = p.Q + (int64_t)(q0 + token) * p.ldq + (int64_t)head * p.head_dim;
#pragma unroll
    for (int ks = 0; ks < H::KS; ++ks) {
      const int d = 16 * ks + 8 * half;
      u32x4 v = *reinterpret_cast<const u32x4*>(q + min(d, p.head_dim - 8));
      if (d >= p.head_dim) v = u32x4{0u, 0u, 0u, 0u};
      qf[ks] = __builtin_bit_cast(bf16x8, v);
    }
  }

  // ---- copies: 1 KB each, lane l fills chunk l of 64 consecutive chunks
  constexpr int RPC = 1024 / H::ROWB;                // rows per copy
  const int crow = lane / H::CHUNKS;                 // row within the copy
  const int cchunk = lane % H::CHUNKS;
  const int copier = MODE == kRows ? wave : 0;
  const int mybuf = MODE == kRows ? 0 : wave * T::TILE_BYTES;
  const uint16_t* kbase = p.K + (int64_t)kv0 * p.ldk + (int64_t)hk * p.head_dim;
  const uint16_t* vbase = p.V + (int64_t)kv0 * p.ldv + (int64_t)hk * p.head_dim;
  const int last_chunk = p.head_dim / 8 - 1;
  auto copy_tile = [&](int t, uint8_t* kdst, uint8_t* vdst) {
#pragma unroll
    for (int i = 0; i < T::CPW; ++i) {
      const int q = copier * T::CPW + i;
      const int r = q * RPC + crow;                  // tile row
      const int key = min(t * KT + r, nk - 1);       // past the end: the last key again, masked below
      const int kc = min(cchunk ^ k_key<H>(r), last_chunk);
      __builtin_amdgcn_global_load_lds(kbase + (int64_t)key * p.ldk + kc * 8,
                                       (lds_ptr)(kdst + mybuf + q * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < T::CPW; ++i) {
      const int q = copier * T::CPW + i;
      const int r = q * RPC + crow;
      const int key = min(t * KT + r, nk - 1);
      const int vc = min(cchunk ^ v_key<H>(r), last_chunk);
      __builtin_amdgcn_global_load_lds(vbase + (int64_t)key * p.ldv + vc * 8,
                                       (lds_ptr)(vdst + mybuf + q * 1024), 16, 0, 0);
    }
  };

  f32x16 o[H::DB];
#pragma unroll
  for (int i = 0; i < H::DB; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float m = -INFINITY;     // the maximum in use, raw scores
  float l = 0.f;           // this lane's share (its half's keys) of the sum

  auto compute = [&](int t, const uint8_t* kb_, const uint8_t* vb_) {
    const int key0 = t * KT;
    if (key0 >= wend) return;
    const uint8_t* kt = kb_ + mybuf;
    const uint8_t* vt = vb_ + mybuf;
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[kb][j] = 0.f;
      const int r = 32 * kb + col;
#pragma unroll
      for (int ks = 0; ks < H::KS; ++ks) {
        const int chunk = (2 * ks + half) ^ k_key<H>(r);
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kt + r * H::ROWB + chunk * 16);
        s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[ks], s[kb], 0, 0, 0);
      }
    }
    if (key0 + KT > wfull) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (key0 + 32 * kb + 8 * (j >> 2) + 4 * half + (j & 3) >= seen) s[kb][j] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[kb][j]);
    top = max_halves(top);
    // (top - m) c > kLazy somewhere in the wave: move to the new maximum
    if (__any(top * p.c > __builtin_fmaf(m, p.c, kLazy))) {
      const float mn = fmaxf(m, top);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * p.c);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= f;
    }
    const float mc = m == -INFINITY ? 0.f : -m * p.c;
    bf16x8 pf[2 * KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][j], p.c, mc));
        l += e;
        pf[2 * kb + (j >> 3)][j & 7] = (__bf16)e;
      }
#pragma unroll
    for (int st = 0; st < 2 * KB; ++st)
#pragma unroll
      for (int db = 0; db < H::DB; ++db) {
        s16x4 v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 16 * st + 8 * u + 4 * half + ((lane & 15) >> 2);
          const int d = 32 * db + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
          const int chunk = (d >> 3) ^ v_key<H>(r);
          v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(vt + r * H::ROWB + chunk * 16 + (d & 4) * 2));
        }
        const bf16x8 vf = __builtin_shufflevector(__builtin_bit_cast(bf16x4, v[0]),
                                                  __builtin_bit_cast(bf16x4, v[1]), 0, 1, 2, 3, 4, 5, 6, 7);
        o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[st], o[db], 0, 0, 0);
      }
  };

  // kKeys: wave w takes tiles t0 + w, t0 + w + NW, ...; kRows: every wave takes all of them
  const int step = MODE == kRows ? 1 : NW;
  int t = t0 + (MODE == kRows ? 0 : wave);
  if (t < t1) copy_tile(t, k0s, v0s);
  // kRows: the barrier tells that everyone's copies have landed and that
  // everyone is done with the other buffer; kKeys waves only wait for themselves
  auto turn = [&](const uint8_t* kc, const uint8_t* vc, uint8_t* kn, uint8_t* vn) {
    copies_wait<0>();
    if (MODE == kRows) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + step < t1) copy_tile(t + step, kn, vn);
    __builtin_amdgcn_sched_barrier(0);
    compute(t, kc, vc);
    t += step;
  };
  while (t < t1) {
    turn(k0s, v0s, k1s, v1s);
    if (t >= t1) break;
    turn(k1s, v1s, k0s, v0s);
  }
  l = sum_halves(l);

  if constexpr (MODE == kKeys) {
    // join the waves' results: maxima and sums first, then the rows, wave by wave
    __shared__ float wm[NW][kWaveRows], wl[NW][kWaveRows];
    copies_wait<0>();
    if (half == 0) {
      wm[wave][col] = m;
      wl[wave][col] = l;
    }
    __syncthreads();
    float mn = wm[0][col];
#pragma unroll
    for (int w = 1; w < NW; ++w) mn = fmaxf(mn, wm[w][col]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      sum += wl[w][col] == 0.f ? 0.f : wl[w][col] * __builtin_amdgcn_exp2f((wm[w][col] - mn) * p.c);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - mn) * p.c);
#pragma unroll
    for (int i = 0; i < H::DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] *= f;
    // wave w parks its registers in its own K and V buffers; wave 0 sums in wave order
    float* mine0 = reinterpret_cast<float*>(k0s + mybuf);   // first half of the registers
    float* mine1 = reinterpret_cast<float*>(v0s + mybuf);   // second half
    constexpr int HALF_REGS = H::DB * 8;                    // registers per buffer: 64 lanes x 4 B each
    static_assert(HALF_REGS * 256 <= T::TILE_BYTES, "half of the registers fit one buffer");
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int g = i * 16 + j;
          if (g < HALF_REGS) mine0[g * 64 + lane] = o[i][j];
          else mine1[(g - HALF_REGS) * 64 + lane] = o[i][j];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float* a = reinterpret_cast<const float*>(k0s + w * T::TILE_BYTES);
      const float* c = reinterpret_cast<const float*>(v0s + w * T::TILE_BYTES);
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int g = i * 16 + j;
          o[i][j] += g < HALF_REGS ? a[g * 64 + lane] : c[(g - HALF_REGS) * 64 + lane];
        }
    }
    m = mn;
    l = sum;
  }

  const float inv = l > 0.f ? 1.f / l : 0.f;
  const float lse2 = l > 0.f ? __builtin_fmaf(m, p.c, __builtin_amdgcn_logf(l)) : -INFINITY;
  if (!row_ok) return;
  if (p.splits > 1) {
    const int64_t unit = blockIdx.x;
    const int64_t slot = unit * T::ROWS + (row - row0);
    if (half == 0) p.part_lse[slot] = lse2;
    float* dst = p.part + slot * p.head_dim;
    if (l > 0.f) {
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int d = 32 * i + 8 * g + 4 * half;
          if (d < p.head_dim)
            *reinterpret_cast<float4*>(dst + d) =
                make_float4(o[i][4 * g] * inv, o[i][4 * g + 1] * inv, o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv);
        }
    }
    return;
  }
  if (p.lse && half == 0) p.lse[(int64_t)head * p.total_q + q0 + token] = lse2 * kLn2;
  uint16_t* dst = p.O + (int64_t)(q0 + token) * p.ldo + (int64_t)head * p.head_dim;
  // 4 channels per register group in each half; exchanged so that half h holds
  // channels 16 e + 8 h .. + 7 of each 16: 16-byte stores
#pragma unroll
  for (int i = 0; i < H::DB; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t w[2][2];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = 8 * e + 4 * g + 2 * u;
          const uint16_t a = __builtin_bit_cast(uint16_t, (__bf16)(o[i][j] * inv));
          const uint16_t c = __builtin_bit_cast(uint16_t, (__bf16)(o[i][j + 1] * inv));
          w[g][u] = a | ((uint32_t)c << 16);
        }
      const u32x2 x = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      const u32x2 y = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      const int d = 32 * i + 16 * e + 8 * half;
      if (d < p.head_dim) *reinterpret_cast<u32x4*>(dst + d) = u32x4{x[0], y[0], x[1], y[1]};
    }
}

// Joins the shares of a tile's rows: weights 2^(lse_s - max), rows summed in
// share order in float32.  One wave per row.
template <int ROWS>
__global__ __launch_bounds__(256) void attention_join(const Params p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = blockIdx.x % p.heads_kv;
  const int rest = blockIdx.x / p.heads_kv;
  const int tile = rest / (ROWS / 4);
  int b, local;
  if (!find_tile(p, ROWS, tile, lane, b, local)) return;
  b = __builtin_amdgcn_readfirstlane(b);
  local = __builtin_amdgcn_readfirstlane(local);
  int q0, nq;
  span(p.cu_q, b, p.total_q, q0, nq);
  const int nrows = nq * p.group;
  if (p.causal) local = (nrows + ROWS - 1) / ROWS - 1 - local;
  const int r = (rest % (ROWS / 4)) * 4 + wave;          // row of the tile
  const int row = local * ROWS + r;
  if (row >= nrows) return;
  const int token = row / p.group;
  const int head = hk * p.group + (row - token * p.group);
  auto slot = [&](int s) { return ((int64_t)(tile * p.splits + s) * p.heads_kv + hk) * ROWS + r; };
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_lse[slot(s)]);
  float sum = 0.f, a0 = 0.f, a1 = 0.f;
  const int d = 2 * lane;
  if (top > -INFINITY)
    for (int s = 0; s < p.splits; ++s) {
      const float e = p.part_lse[slot(s)];
      if (e == -INFINITY) continue;
      const float w = __builtin_amdgcn_exp2f(e - top);
      sum += w;
      if (d < p.head_dim) {
        const float2 v = *reinterpret_cast<const float2*>(p.part + slot(s) * p.head_dim + d);
        a0 = __builtin_fmaf(w, v.x, a0);
        a1 = __builtin_fmaf(w, v.y, a1);
      }
    }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  if (d < p.head_dim) {
    const uint16_t x = __builtin_bit_cast(uint16_t, (__bf16)(a0 * inv));
    const uint16_t y = __builtin_bit_cast(uint16_t, (__bf16)(a1 * inv));
    *reinterpret_cast<uint32_t*>(p.O + (int64_t)(q0 + token) * p.ldo + (int64_t)head * p.head_dim + d) =
        x | ((uint32_t)y << 16);
  }
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.total_q + q0 + token] =
        sum > 0.f ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
}

constexpr int kBigWaves = 4;
constexpr int kSmallWaves = 4;

struct Plan {
  bool keys = false;      // kKeys: 32 rows per workgroup
  int rows = 0, splits = 1;
  int64_t tiles = 0;      // at most, over the packed batch
  size_t part = 0, bytes = 0;
};

Plan plan_of(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim) {
  Plan pl;
  const int group = heads_q / heads_kv;
  const int64_t rows = (int64_t)total_q * group;
  pl.keys = rows <= (int64_t)batch * 64;
  pl.rows = pl.keys ? kWaveRows : kBigWaves * kWaveRows;
  // every sequence has at most one partly filled tile
  pl.tiles = std::min<int64_t>(rows / pl.rows + batch, rows);
  const int64_t units = pl.tiles * heads_kv;
  const int kt = pl.keys ? 32 * kSmallWaves : 64;
  const int64_t want = (pl.keys ? 4 : 2) * (int64_t)device_cu_count() / std::max<int64_t>(units, 1);
  const int64_t most = ((int64_t)total_k / batch + 2 * kt - 1) / (2 * kt);   // two rounds of tiles at least
  pl.splits = (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 64}));
  if (pl.splits > 1) {
    const size_t slots = (size_t)units * pl.splits * pl.rows;
    pl.part = (slots * head_dim * 4 + 255) & ~size_t(255);
    pl.bytes = pl.part + ((slots * 4 + 255) & ~size_t(255));
  }
  return pl;
}

template <class H>
hipError_t launch(const Plan& pl, const Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)(pl.tiles * p.heads_kv * pl.splits));
  if (pl.keys)
    hipLaunchKernelGGL((attention_kernel<H, kKeys, kSmallWaves>), grid, dim3(kSmallWaves * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((attention_kernel<H, kRows, kBigWaves>), grid, dim3(kBigWaves * 64), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.splits == 1) return e;
  const dim3 jgrid((unsigned)(pl.tiles * p.heads_kv * (pl.rows / 4)));
  if (pl.keys)
    hipLaunchKernelGGL((attention_join<kWaveRows>), jgrid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((attention_join<kBigWaves * kWaveRows>), jgrid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim) {
  if (total_q == 0 || total_k == 0) return 0;
  return plan_of(total_q, total_k, batch, heads_q, heads_kv, head_dim).bytes;
}

int64_t attention_blocks(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim) {
  const Plan pl = plan_of(total_q, total_k, batch, heads_q, heads_kv, head_dim);
  return pl.tiles * heads_kv * std::max(pl.splits, pl.splits > 1 ? pl.rows / 4 : 1);
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  const Plan pl = plan_of(a.total_q, a.total_k, a.batch, a.heads_q, a.heads_kv, a.head_dim);
  Params p;
  p.Q = a.Q; p.K = a.K; p.V = a.V; p.O = a.O; p.lse = a.lse;
  p.ldq = a.ldq; p.ldk = a.ldk; p.ldv = a.ldv; p.ldo = a.ldo;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k;
  p.batch = a.batch; p.total_q = a.total_q; p.total_k = a.total_k;
  p.heads_q = a.heads_q; p.heads_kv = a.heads_kv; p.group = a.heads_q / a.heads_kv;
  p.head_dim = a.head_dim;
  p.c = a.scale * kLog2e;
  p.causal = a.causal;
  p.splits = pl.splits;
  p.part = static_cast<float*>(a.workspace);
  p.part_lse = pl.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + pl.part) : nullptr;
  if (a.head_dim <= 64) return launch<Head<64, 4, 2>>(pl, p, stream);
  if (a.head_dim <= 96) return launch<Head<128, 6, 3>>(pl, p, stream);
  return launch<Head<128, 8, 4>>(pl, p, stream);
}

}  // namespace svdq
