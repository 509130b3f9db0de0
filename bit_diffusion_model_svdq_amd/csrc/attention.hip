// Softmax attention over packed sequences (no padding, no score matrix), gfx950.
//
//   O_i = sum_j p_ij V_j,   p_ij = exp(scale q_i.k_j - m_i) / l_i
//
// over the keys j of query i's own sequence (causal: j <= i + nk - nq, so the
// last query sees the last key), in one pass over the keys with the running
// maximum m and sum l of the softmax.  A query without keys gets O = 0 and
// log-sum-exp -inf; one with a NaN or +inf among its scores, or with none in
// float32's range, gets NaN in both.
//
// Work split.  The `group` query heads that share a key head are rows of one
// problem: row r of (sequence, key head) is token r / group, head r % group.
// So a tile of rows reads its keys once for the whole group, and a single new
// token already brings `group` rows.  Two kernels share the arithmetic:
//   attention_rows  a workgroup takes 32 rows per wave; its waves share each
//                   K/V tile.
//   attention_keys  a workgroup takes 32 rows in all; its waves take alternate
//                   K/V tiles and join at the end.  For few rows per
//                   sequence, where the keys' bytes are what counts, and for
//                   launches whose larger tiles would leave CUs idle.
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
// With few rows per sequence (new tokens) p goes in two bf16 parts instead, the
// upper 16 bits and the rounded rest: O is then as good as its own rounding
// (Frobenius error against float64 1.66e-3; 2.0e-3 to 2.3e-3 with one part).  There
// the keys' bytes are what counts: 16 single tokens 56.4 -> 56.8 us, 64 against 64 k keys
// 59.3 -> 59.6 (46.2 -> 48.3 and 47.8 -> 48.2 with the keys in the Infinity Cache, one
// against 32 k 34.1 -> 34.4).  Elsewhere the second MFMA of P V costs more than those digits are worth: 16384 tokens x 24 x 128 2.93 -> 4.13 ms,
// 4608 tokens 268 -> 362 us, and in attention_keys 1024 x 16 x 128 23.2 -> 26.2 us,
// 1536 x 10 x 64 15.7 -> 18.3.
#include <algorithm>
#include <cmath>

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
  int tiles;             // of the launch (at least those of the batch)
  int splits, chunk;     // a sequence's keys are cut into shares of about `chunk` keys, at most `splits`
  float* part;           // [unit][rows][head_dim] partial rows, unit = (share, tile, key head)
  float* part_lse;       // [unit][rows], base 2; -inf: the share has no weight, and no row

  __device__ int shares(int nk) const { return min(nk > 0 ? (nk - 1) / chunk + 1 : 1, splits); }
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
  static constexpr int KT = 32;                          // keys of a tile
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

__device__ inline float highest(const f32x16& s) {
  float top = s[0];
#pragma unroll
  for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
  return top;
}

// A sequence's rows, kept inside the buffers whatever the offsets hold.
__device__ inline void span(const int32_t* cu, int b, int total, int& begin, int& len) {
  const int lo = cu ? cu[b] : 0, hi = cu ? cu[b + 1] : total;
  begin = min(max(lo, 0), total);
  len = max(min(hi, total) - begin, 0);
}

// Where a tile lies: its number in its sequence, and the sequence's rows.
struct Place {
  int local, q0, nq, kv0, nk;
};

// Tile number `t` of the packed batch (rows: tile height).  False: past the
// last tile.  64 sequences at a time, one per lane, all offsets loaded at once.
__device__ inline bool find_tile(const Params& p, int rows, int t, int lane, Place& at) {
  for (int base = 0; base < p.batch; base += 64) {
    const int b = min(base + lane, p.batch - 1);
    int q0, nq, kv0, nk;
    span(p.cu_q, b, p.total_q, q0, nq);
    span(p.cu_k, b, p.total_k, kv0, nk);
    const int n = base + lane < p.batch ? (nq * p.group + rows - 1) / rows : 0;
    int end = n;
    if (p.batch > 1) {
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const int o = __shfl_up(end, s);
        if (lane >= s) end += o;
      }
    }
    const uint64_t after = __ballot(t < end);
    if (after) {
      const int l = __builtin_ctzll(after);
      at.local = t - (__builtin_amdgcn_readlane(end, l) - __builtin_amdgcn_readlane(n, l));
      at.q0 = __builtin_amdgcn_readlane(q0, l);
      at.nq = __builtin_amdgcn_readlane(nq, l);
      at.kv0 = __builtin_amdgcn_readlane(kv0, l);
      at.nk = __builtin_amdgcn_readlane(nk, l);
      return true;
    }
    t -= __builtin_amdgcn_readlane(end, 63);
    if (t < 0) return false;      // offsets that overlap so often that the count wrapped
  }
  return false;
}

// s_waitcnt vmcnt(n) and lgkmcnt(0), expcnt untouched
template <int n>
__device__ inline void copies_wait() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));
}

// One tile of rows: where it lies, which keys it sees, and the parts of the
// work that both kernels share.
template <class H, int MODE, int NW>
struct Work {
  using T = Tile<H, MODE, NW>;
  const Params& p;
  int lane, wave, half, col;
  int hk, q0, kv0, nk;
  int row0, row;             // the tile's first row, this lane's row
  bool row_ok;
  int token, head;
  int seen;                  // keys that this lane's query sees
  int wfull, wend;           // every query of the wave sees [0, wfull), none sees from wend on
  int shares;                // of the sequence's keys
  int t0, t1;                // key tiles of this share
  bf16x8 qf[H::KS];
  f32x16 o[H::DB];
  float m = -INFINITY;       // the maximum in use, raw scores
  float l = 0.f;             // this lane's share (its half's keys) of the sum
  int koff, voff[H::DB];
  int kvo[T::CPW], vvo[T::CPW];   // byte offsets of this lane's chunks in a tile of K and V
  int copier, mybuf;

  __device__ explicit Work(const Params& p_) : p(p_) {}

  // False: no such tile.
  __device__ bool locate() {
    const int tid = threadIdx.x;
    lane = tid & 63;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    half = lane >> 5;
    col = lane & 31;
    // blocks run over key heads first, then tiles, then shares (the first of
    // which every tile has)
    hk = blockIdx.x % p.heads_kv;
    const int rest = blockIdx.x / p.heads_kv;
    const int split = rest / p.tiles;
    Place at;
    if (!find_tile(p, T::ROWS, rest % p.tiles, lane, at)) return false;
    int local = at.local;
    const int nq = at.nq;
    q0 = at.q0;
    kv0 = at.kv0;
    nk = at.nk;
    shares = p.shares(nk);
    if (split >= shares) return false;
    const int nrows = nq * p.group;
    // causal tiles see more keys the later they are: start with the last
    if (p.causal) local = (nrows + T::ROWS - 1) / T::ROWS - 1 - local;
    row0 = local * T::ROWS;
    const int wrow0 = row0 + (MODE == kRows ? wave * kWaveRows : 0);
    row = wrow0 + col;
    row_ok = row < nrows;
    const int rowc = min(row, nrows - 1);
    token = rowc / p.group;
    head = hk * p.group + (rowc - token * p.group);
    const int shift = nk - nq;
    auto visible = [&](int r) { return p.causal ? min(max(min(r, nrows - 1) / p.group + shift + 1, 0), nk) : nk; };
    seen = visible(row);
    wfull = __builtin_amdgcn_readfirstlane(visible(wrow0));
    wend = __builtin_amdgcn_readfirstlane(visible(wrow0 + kWaveRows - 1));
    const int ntiles = (visible(row0 + T::ROWS - 1) + T::KT - 1) / T::KT;
    t0 = (int)((int64_t)ntiles * split / shares);
    t1 = (int)((int64_t)ntiles * (split + 1) / shares);
    return true;
  }

  __device__ void prepare() {
    // Q as the B operand: this lane's query, channels 16 ks + 8 half .. + 7
    const uint16_t* q = p.Q + (int64_t)(q0 + token) * p.ldq + (int64_t)head * p.head_dim;
#pragma unroll
    for (int ks = 0; ks < H::KS; ++ks) {
      const int d = 16 * ks + 8 * half;
      qf[ks] = *reinterpret_cast<const bf16x8*>(q + min(d, p.head_dim - 8));
    }
#pragma unroll
    for (int i = 0; i < H::DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    // fragment addresses of row `col` (K) and of the transposing read (V)
    koff = col * H::ROWB + ((half ^ k_key<H>(col)) << 4);
    const int vrow = 4 * half + ((lane & 15) >> 2);
#pragma unroll
    for (int db = 0; db < H::DB; ++db) {
      const int d = 32 * db + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      voff[db] = vrow * H::ROWB + (((d >> 3) ^ v_key<H>(vrow)) << 4) + (d & 4) * 2;
    }
    // copies, 1 KB each: lane l fills chunk l of 64 consecutive chunks
    constexpr int RPC = 1024 / H::ROWB;                // rows per copy
    copier = MODE == kRows ? wave : 0;
    mybuf = MODE == kRows ? 0 : wave * T::TILE_BYTES;
    const int last_chunk = p.head_dim / 8 - 1;
#pragma unroll
    for (int i = 0; i < T::CPW; ++i) {
      const int r = (copier * T::CPW + i) * RPC + lane / H::CHUNKS;
      const int c = lane % H::CHUNKS;
      kvo[i] = r * (int)p.ldk * 2 + min(c ^ k_key<H>(r), last_chunk) * 16;
      vvo[i] = r * (int)p.ldv * 2 + min(c ^ v_key<H>(r), last_chunk) * 16;
    }
  }

  // Zeros in Q's channels past the head.  Apart from prepare(), so that the first
  // copies leave before Q is waited for.
  __device__ void trim() {
#pragma unroll
    for (int ks = 0; ks < H::KS; ++ks)
      if (16 * ks + 8 * half >= p.head_dim) qf[ks] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
  }

  // The next tile of K or V into LDS, through a buffer descriptor that ends with
  // the sequence's last key: keys past it arrive as zeros (their scores are
  // masked, and zero times anything stays finite in P V).  kAttentionMaxLd keeps the
  // 32-bit offsets of a tile's rows below 2^31.
  struct Cursor {
    const uint16_t* at;      // the tile's first key, this head
    int left;                // keys from there on
  };
  __device__ Cursor cursor(const uint16_t* base, int64_t ld, int t) const {
    return {base + (int64_t)(kv0 + t * T::KT) * ld + (int64_t)hk * p.head_dim, nk - t * T::KT};
  }
  __device__ void copy(Cursor& c, int ld, int step, const int (&off)[T::CPW], uint8_t* dst) {
    // past the last tile: a descriptor of nothing, so that every turn issues the same copies
    const int bytes = c.left > 0 ? ((min(c.left, T::KT) - 1) * ld + p.head_dim) * 2 : 0;
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(c.at), 0, bytes, 0x00027000);
#pragma unroll
    for (int i = 0; i < T::CPW; ++i) {
      const int o_ = off[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(dst + mybuf + (copier * T::CPW + i) * 1024), 16, o_, 0, 0,
                                               0);
    }
    c.at += (int64_t)step * T::KT * ld;
    c.left -= step * T::KT;
  }
  Cursor ck, cv;
  __device__ void copy_k(uint8_t* dst, int step) { copy(ck, (int)p.ldk, step, kvo, dst); }
  __device__ void copy_v(uint8_t* dst, int step) { copy(cv, (int)p.ldv, step, vvo, dst); }
  __device__ void start(int t) {
    ck = cursor(p.K, p.ldk, t);
    cv = cursor(p.V, p.ldv, t);
  }

  __device__ bf16x8 k_frag(const uint8_t* kt, int ks) const {
    return *reinterpret_cast<const bf16x8*>(kt + mybuf + (koff ^ (ks << 5)));
  }
  __device__ bf16x8 v_frag(const uint8_t* vt, int st, int db) const {
    const uint8_t* a = vt + mybuf + voff[db] + 16 * st * H::ROWB;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(a));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(a + 8 * H::ROWB));
    return __builtin_shufflevector(__builtin_bit_cast(bf16x4, lo), __builtin_bit_cast(bf16x4, hi), 0, 1, 2, 3, 4, 5,
                                   6, 7);
  }

  // Scores of tile t past the keys that this lane's query sees: -inf.
  __device__ void mask(f32x16& s, int t) const {
    const int left = seen - t * T::KT - 4 * half;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (8 * (j >> 2) + (j & 3) >= left) s[j] = -INFINITY;
  }
  __device__ bool whole(int t) const { return t * T::KT + T::KT <= wfull; }

  // Moves to the maximum `top` of a tile to come where, somewhere in the wave,
  // it exceeds the one in use by more than kLazy.  A maximum below float32's range
  // (and a NaN) is none: m c stays above -inf.
  __device__ void follow(float top) {
    top = max_halves(top);
    if (__any(top * p.c > __builtin_fmaf(m, p.c, kLazy))) {
      const float mn = fmaxf(m, top * p.c > -INFINITY ? top : -INFINITY);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * p.c);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= f;
    }
  }

  // The rows' results: to O and lse, or to this share's slots of the workspace.
  // A sum of 0 stands for no weight at all, and only that: a NaN or infinite
  // score makes the sum NaN, which goes on into O and lse.  No weight is
  // right for a query that sees no key.  Where it does see some, their scores
  // all left float32's range (scale log2(e) times the maximum is infinite, or
  // every score is -inf), and the result is NaN; a share whose scores are all
  // -inf is like an empty one, and the join decides.
  __device__ void finish() {
    const bool none = l == 0.f;
    const bool lost = none && (shares > 1 ? m * p.c == INFINITY : seen > 0);
    const float inv = lost ? NAN : none ? 0.f : 1.f / l;
    const float lse2 = lost ? NAN : none ? -INFINITY : __builtin_fmaf(m, p.c, __builtin_amdgcn_logf(l));
    if (!row_ok) return;
    if (none)                      // V's infinities and NaN times no weight
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    if (shares > 1) {
      const int64_t slot = (int64_t)blockIdx.x * T::ROWS + (row - row0);
      if (half == 0) p.part_lse[slot] = lse2;
      float* dst = p.part + slot * p.head_dim;
      if (!none) {
#pragma unroll
        for (int i = 0; i < H::DB; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int d = 32 * i + 8 * g + 4 * half;
            if (d < p.head_dim)
              *reinterpret_cast<float4*>(dst + d) = make_float4(o[i][4 * g] * inv, o[i][4 * g + 1] * inv,
                                                                o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv);
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
            const uint16_t x = __builtin_bit_cast(uint16_t, (__bf16)(o[i][j] * inv));
            const uint16_t y = __builtin_bit_cast(uint16_t, (__bf16)(o[i][j + 1] * inv));
            w[g][u] = x | ((uint32_t)y << 16);
          }
        const u32x2 x = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const u32x2 y = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        const int d = 32 * i + 16 * e + 8 * half;
        if (d < p.head_dim) *reinterpret_cast<u32x4*>(dst + d) = u32x4{x[0], y[0], x[1], y[1]};
      }
  }
};

// Many rows: the waves share each K/V tile.  The loop is pipelined across tiles
// and laid out by hand in pieces of two or three MFMAs with a few softmax
// elements after each (VALU work issues beside a running MFMA of its own
// wave): the scores of tile t + 1 beside the weights of tile t, then P V of tile
// t beside the rest of them.  Tiles of 32 keys: with 64 the scores of two tiles
// spill.  One path for every tile, with the mask as the one thing that branches:
// variants of the tile make the compiler spill or merge their weights into one
// block away from the MFMAs.
//
// K and V each go through a ring of four LDS buffers, filled by direct copies
// three tiles ahead.  At the top of turn t the copies of K up to tile t + 2 and
// of V up to tile t + 1 have landed for everyone (vmcnt leaves the last turn's
// in flight), and everyone is done with K of tile t and V of tile t - 1, whose
// buffers are filled again.
//
// Bound by the card's power: 16384 tokens x 24 x 128 take 2.93 ms (1125 TFLOP/s)
// with 8 waves and 2.97 ms with 4, though the 4 waves' form needs 11 % fewer
// cycles (5.1 M against 5.7 M): it moves twice the bytes from L2 and the clock
// drops to 1.71 GHz (1.95).  MFMAs run in 62 % (55 %) of the cycles.
template <class H, int NW>
__global__ __launch_bounds__(NW * 64, 2) void attention_rows(const Params p) {
  using T = Tile<H, kRows, NW>;
  // each buffer its own array: reading one then does not wait for copies into another
  __shared__ __attribute__((aligned(16))) uint8_t k0s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k1s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k2s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k3s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v0s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v1s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v2s[T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v3s[T::TILE_BYTES];
  Work<H, kRows, NW> w(p);
  if (!w.locate()) return;
  w.prepare();
  const int t0 = w.t0, t1 = w.t1;
  f32x16 sa, sb;                         // scores of the tile at hand and of the next
  bf16x8 kf[2][2];                       // K fragments of two pieces
  float l2 = 0.f;                        // a second partial sum: shorter chains

  constexpr int NS = (H::KS + 1) / 2;                 // score pieces: 2 MFMAs each
  constexpr int CB = H::DB % 2 ? 3 : 2;               // P V's MFMAs per piece
  constexpr int NP = 2 * H::DB / CB;                  // P V pieces
  // elements whose weights are done after n pieces: P V's operands in time
  constexpr auto due = [](int n) { return n >= NS + NP / 2 ? 16 : 16 * n / (NS + NP / 2); };
  static_assert(due(NS) >= 8, "the first weights are ready when P V takes them");
  auto k_load = [&](const uint8_t* kt, int q) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (2 * q + c < H::KS) kf[q & 1][c] = w.k_frag(kt, 2 * q + c);
  };
  // Tile t (scores `cur`) and the scores of tile t + 1 (`nxt`).  Past the share's
  // last tile those are of whatever its buffer holds (finite: copies past the
  // sequence are zeros); they move the maximum in use at most.
  auto tile = [&](int t, f32x16& cur, f32x16& nxt, const uint8_t* kt, const uint8_t* vt, const uint8_t* kafter) {
    const float mc = w.m == -INFINITY ? 0.f : -w.m * p.c;
    bf16x8 pf[2], vf[2][CB];
    auto weights = [&](int from, int to) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < from || i >= to) continue;
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(cur[i], p.c, mc));
        if (i & 1)
          l2 += e;
        else
          w.l += e;
        pf[i >> 3][i & 7] = (__bf16)e;
      }
    };
    auto v_load = [&](int q) {
#pragma unroll
      for (int c = 0; c < CB; ++c) vf[q & 1][c] = w.v_frag(vt, (q * CB + c) / H::DB, (q * CB + c) % H::DB);
    };
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      if (q + 1 < NS) k_load(kt, q + 1);
      if (q + 1 == NS) v_load(0);
      if (q == 0)
#pragma unroll
        for (int j = 0; j < 16; ++j) nxt[j] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (2 * q + c < H::KS)
          nxt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[q & 1][c], w.qf[2 * q + c], nxt, 0, 0, 0);
      weights(due(q), due(q + 1));
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      if (q + 1 < NP)
        v_load(q + 1);
      else
        k_load(kafter, 0);
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const int i = q * CB + c;
        w.o[i % H::DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[q & 1][c], pf[i / H::DB], w.o[i % H::DB], 0, 0, 0);
      }
      weights(due(NS + q), due(NS + q + 1));
      __builtin_amdgcn_sched_barrier(0);
    }
    w.l += l2;
    l2 = 0.f;
    if (!w.whole(t + 1)) {
      asm volatile("" ::: "memory");       // keeps the comparisons out of the other tiles
      w.mask(nxt, t + 1);
    }
    w.follow(highest(nxt));
  };

  auto turn = [&](int t, f32x16& cur, f32x16& nxt, const uint8_t* kt, const uint8_t* kafter, uint8_t* kfill,
                  const uint8_t* vt, uint8_t* vfill) {
    copies_wait<2 * T::CPW>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    w.copy_v(vfill, 1);
    w.copy_k(kfill, 1);
    __builtin_amdgcn_sched_barrier(0);
    if (t * T::KT < w.wend) tile(t, cur, nxt, kt, vt, kafter);
  };
  if (t0 < t1) {
    w.start(t0);
    w.copy_k(k0s, 1);
    w.copy_v(v0s, 1);
    w.copy_k(k1s, 1);
    w.copy_v(v1s, 1);
    w.copy_k(k2s, 1);
    w.copy_v(v2s, 1);
    w.copy_k(k3s, 1);
    __builtin_amdgcn_sched_barrier(0);
    w.trim();
    copies_wait<4 * T::CPW>();           // K of the first two tiles
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j) sa[j] = 0.f;
#pragma unroll
    for (int ks = 0; ks < H::KS; ++ks)
      sa = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.k_frag(k0s, ks), w.qf[ks], sa, 0, 0, 0);
    if (!w.whole(t0)) w.mask(sa, t0);
    w.follow(highest(sa));
    k_load(k1s, 0);
    int t = t0;
    for (; t + 4 <= t1; t += 4) {
      turn(t, sa, sb, k1s, k2s, k0s, v0s, v3s);
      turn(t + 1, sb, sa, k2s, k3s, k1s, v1s, v0s);
      turn(t + 2, sa, sb, k3s, k0s, k2s, v2s, v1s);
      turn(t + 3, sb, sa, k0s, k1s, k3s, v3s, v2s);
    }
    if (t < t1) turn(t, sa, sb, k1s, k2s, k0s, v0s, v3s);
    if (t + 1 < t1) turn(t + 1, sb, sa, k2s, k3s, k1s, v1s, v0s);
    if (t + 2 < t1) turn(t + 2, sa, sb, k3s, k0s, k2s, v2s, v1s);
  }
  copies_wait<0>();
  w.l = sum_halves(w.l + l2);
  w.finish();
}

// Few rows: all waves have the same 32 rows and take every NW-th tile, each in
// buffers of its own, without barriers until they join.  PARTS: of a weight in
// the product with V.  Heads of more than 64 channels take the registers of a whole
// SIMD, and two workgroups of two waves the LDS of a CU.
template <class H, int NW, int PARTS>
__global__ __launch_bounds__(NW * 64, H::DP == 64 ? 2 : 1) void attention_keys(const Params p) {
  using T = Tile<H, kKeys, NW>;
  __shared__ __attribute__((aligned(16))) uint8_t k0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k1s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v1s[T::BUFS * T::TILE_BYTES];
  __shared__ float wm[NW][kWaveRows], wl[NW][kWaveRows];
  Work<H, kKeys, NW> w(p);
  if (!w.locate()) return;
  w.prepare();
  const int wave = w.wave, col = w.col;

  auto compute = [&](int t, const uint8_t* kt, const uint8_t* vt) {
    f32x16 s;
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
    for (int ks = 0; ks < H::KS; ++ks)
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.k_frag(kt, ks), w.qf[ks], s, 0, 0, 0);
    if (!w.whole(t)) w.mask(s, t);
    w.follow(highest(s));
    const float mc = w.m == -INFINITY ? 0.f : -w.m * p.c;
    bf16x8 pf[2], rest[2];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], p.c, mc));
      w.l += e;
      if constexpr (PARTS == 2) {
        const uint32_t upper = __float_as_uint(e) >> 16;
        pf[j >> 3][j & 7] = __builtin_bit_cast(__bf16, (uint16_t)upper);
        rest[j >> 3][j & 7] = (__bf16)(e - __uint_as_float(upper << 16));
      } else {
        pf[j >> 3][j & 7] = (__bf16)e;
      }
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      bf16x8 vf[H::DB];
#pragma unroll
      for (int db = 0; db < H::DB; ++db) {
        vf[db] = w.v_frag(vt, st, db);
        w.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[db], pf[st], w.o[db], 0, 0, 0);
      }
      if constexpr (PARTS == 2)
#pragma unroll
        for (int db = 0; db < H::DB; ++db)
          w.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[db], rest[st], w.o[db], 0, 0, 0);
    }
  };
  int t = w.t0 + wave;
  w.start(t);
  if (t < w.t1) {
    w.copy_k(k0s, NW);
    w.copy_v(v0s, NW);
  }
  __builtin_amdgcn_sched_barrier(0);
  w.trim();
  auto turn = [&](const uint8_t* kc, const uint8_t* vc, uint8_t* kn, uint8_t* vn) {
    copies_wait<0>();
    asm volatile("" ::: "memory");
    if (t + NW < w.t1) {
      w.copy_k(kn, NW);
      w.copy_v(vn, NW);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (t * T::KT < w.wend) compute(t, kc, vc);
    t += NW;
  };
  while (t < w.t1) {
    turn(k0s, v0s, k1s, v1s);
    if (t >= w.t1) break;
    turn(k1s, v1s, k0s, v0s);
  }
  w.l = sum_halves(w.l);

  // join the waves' results: maxima and sums first, then the rows, wave by wave
  copies_wait<0>();
  if (w.half == 0) {
    wm[wave][col] = w.m;
    wl[wave][col] = w.l;
  }
  __syncthreads();
  float mn = wm[0][col];
#pragma unroll
  for (int i = 1; i < NW; ++i) mn = fmaxf(mn, wm[i][col]);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i)
    sum += wl[i][col] == 0.f ? 0.f : wl[i][col] * __builtin_amdgcn_exp2f((wm[i][col] - mn) * p.c);
  const float f = w.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((w.m - mn) * p.c);
#pragma unroll
  for (int i = 0; i < H::DB; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) w.o[i][j] *= f;
  // wave w parks its registers in its own K and V buffers; wave 0 sums in wave order
  constexpr int HALF_REGS = H::DB * 8;                    // registers per buffer: 64 lanes x 4 B each
  static_assert(HALF_REGS * 256 <= T::TILE_BYTES, "half of the registers fit one buffer");
  const int lane = w.lane;
  if (wave > 0) {
    float* mine0 = reinterpret_cast<float*>(k0s + wave * T::TILE_BYTES);
    float* mine1 = reinterpret_cast<float*>(v0s + wave * T::TILE_BYTES);
#pragma unroll
    for (int i = 0; i < H::DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int g = i * 16 + j;
        if (g < HALF_REGS)
          mine0[g * 64 + lane] = w.o[i][j];
        else
          mine1[(g - HALF_REGS) * 64 + lane] = w.o[i][j];
      }
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 1; i < NW; ++i) {
    const float* x = reinterpret_cast<const float*>(k0s + i * T::TILE_BYTES);
    const float* y = reinterpret_cast<const float*>(v0s + i * T::TILE_BYTES);
#pragma unroll
    for (int k = 0; k < H::DB; ++k)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int g = k * 16 + j;
        w.o[k][j] += g < HALF_REGS ? x[g * 64 + lane] : y[(g - HALF_REGS) * 64 + lane];
      }
  }
  w.m = mn;
  w.l = sum;
  w.finish();
}

// Joins the shares of a tile's rows: weights 2^(lse_s - max), rows summed in
// share order in float32.  One wave per row: lane s holds share s's weight (at
// most 64 shares), then each lane two channels, eight shares at a time.  A NaN
// lse_s passes the maximum by and makes its weight, the sum and the row NaN.
__global__ __launch_bounds__(256) void attention_join(const Params p, int rows_per_tile) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = blockIdx.x % p.heads_kv;
  const int rest = blockIdx.x / p.heads_kv;
  const int tile = rest / (rows_per_tile / 4);
  Place at;
  if (!find_tile(p, rows_per_tile, tile, lane, at)) return;
  const int shares = p.shares(at.nk);
  if (shares == 1) return;                               // written by its one share
  const int nrows = at.nq * p.group;
  int local = at.local;
  if (p.causal) local = (nrows + rows_per_tile - 1) / rows_per_tile - 1 - local;
  const int r = (rest % (rows_per_tile / 4)) * 4 + wave;          // row of the tile
  const int row = local * rows_per_tile + r;
  if (row >= nrows) return;
  const int token = row / p.group;
  const int head = hk * p.group + (row - token * p.group);
  auto slot = [&](int s) { return (((int64_t)s * p.tiles + tile) * p.heads_kv + hk) * rows_per_tile + r; };
  const int d = 2 * lane;
  const bool on = d < p.head_dim;
  // eight shares at a time; past the last one the last again, with weight 0
  float2 v[8];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      v[u] = *reinterpret_cast<const float2*>(p.part + slot(min(s0 + u, shares - 1)) * p.head_dim + (on ? d : 0));
  };
  const float e = lane < shares ? p.part_lse[slot(lane)] : -INFINITY;
  load(0);                                               // beside the weights' loads
  float top = e;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
  const float weight = e == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(e - top);
  float sum = weight;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
  float a0 = 0.f, a1 = 0.f;
  for (int s0 = 0; s0 < shares; s0 += 8) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = __shfl(weight, (s0 + u) & 63);
      if (s0 + u < shares && w != 0.f) {                 // a share without weight has written nothing
        a0 = __builtin_fmaf(w, v[u].x, a0);
        a1 = __builtin_fmaf(w, v[u].y, a1);
      }
    }
  }
  // as in finish(): no weight at all is NaN for a query that sees keys
  const int seen = p.causal ? min(token + at.nk - at.nq + 1, at.nk) : at.nk;
  const bool none = sum == 0.f;
  const float inv = !none ? 1.f / sum : seen > 0 ? NAN : 0.f;
  if (on) {
    const uint16_t x = __builtin_bit_cast(uint16_t, (__bf16)(a0 * inv));
    const uint16_t y = __builtin_bit_cast(uint16_t, (__bf16)(a1 * inv));
    *reinterpret_cast<uint32_t*>(p.O + (int64_t)(at.q0 + token) * p.ldo + (int64_t)head * p.head_dim + d) =
        x | ((uint32_t)y << 16);
  }
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.total_q + at.q0 + token] =
        !none ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : seen > 0 ? NAN : -INFINITY;
}

// attention_keys' waves: so many that two workgroups fit a CU's LDS (a wave
// holds two K and two V tiles).  Measured with keys from HBM: 16 single tokens against
// 49.5 k keys x 8 x 128 56.8 us with 2 waves, 60.6 with 4, 32 against 64 k x 16 x 80
// 85.2 and 91.1; 64 against 64 k x 16 x 64 59.0 and 59.5.
constexpr int key_waves(int dp) { return dp == 64 ? 4 : 2; }

// Rows per sequence, on average, up to which a call counts as one of new tokens.
constexpr int kTokenRows = 64;

struct Plan {
  bool keys = false;      // attention_keys: 32 rows per workgroup
  int parts = 1;          // of a weight in P V
  int waves = 4;          // of a workgroup
  int rows = 0, splits = 1, chunk = 0;
  int64_t tiles = 0;      // at most, over the packed batch
  size_t part = 0, bytes = 0;
};

// What a tile of 32 keys costs a workgroup, in us, by the head's size (up to 64,
// 96, 128 channels): alone on its CU, where latency counts, and as its part of a
// full CU; with 8 waves a workgroup has the CU to itself.  For attention_keys it
// is a turn of all its waves.
struct Cost {
  double rows4, rows4_each, rows8, keys, keys_each;
  int keys_waves;
};
Cost cost_of(int head_dim) {
  if (head_dim <= 64) return {0.38, 0.30, 0, 0.46, 0.45, key_waves(64)};
  if (head_dim <= 96) return {0.45, 0.44, 0.76, 0.75, 0.40, key_waves(128)};
  return {0.53, 0.49, 0.90, 0.80, 0.50, key_waves(128)};
}

// The kernel, its waves and the shares of the keys by an estimate of the time for
// sequences of the average lengths (the lengths themselves are on the device):
// the longest chain of tiles, or all tiles over the CUs; shares add the
// join's launch and the traffic of their partial rows, 4.3 us per million
// channels.  The constants are measured ones.  Where the estimates differ, measured
// (attention_rows with 4 waves / 8 waves / attention_keys): 16384 tokens x 24 x 128
// 3.05 / 2.97 ms / -; 4608 tokens 279 / 264 us / -; 1024 x 24 x 128 24 / 34 / 38 us;
// 1024 x 16 x 128 23 / 33 / 21; 1536 x 10 x 64 24 / - / 16; 512 causal x 32 / 8 x 128
// 14.8 / 19.8 / 13.7.  Shares: 1024 x 24 x 128 24 us with one, 45 with two; 400
// queries x 2 x 64 against 8000 keys 35 us with one, 14 with eight (attention_keys).
Plan plan_of(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim, bool causal) {
  Plan pl;
  const int group = heads_q / heads_kv;
  const int64_t rows = (int64_t)total_q * group;
  const int64_t cus = device_cu_count();
  const Cost cost = cost_of(head_dim);
  const double mean_rows = (double)rows / batch, mean_q = (double)total_q / batch, mean_k = (double)total_k / batch;
  auto estimate = [&](bool keys, int waves, int splits, double longest = 1) {
    const double units = std::ceil(mean_rows / (keys ? kWaveRows : waves * kWaveRows)) * batch * heads_kv;
    double each_cu = std::ceil(units * splits / cus);
    if (keys && each_cu > 1) each_cu = 2 * std::ceil(each_cu / 2);       // two fit a CU
    auto turns = [&](double nk) {
      return std::ceil(std::ceil(std::ceil(nk / 32) / (keys ? cost.keys_waves : 1)) / splits);
    };
    // causal: half of the tiles, and their unequal lengths leave CUs waiting
    const double seen = causal ? 1 - 0.4 * std::min(1.0, mean_q / std::max(mean_k, 1.0)) : 1;
    const double alone = keys ? cost.keys : waves == 8 ? cost.rows8 : cost.rows4;
    const double each = keys ? cost.keys_each : waves == 8 ? cost.rows8 : cost.rows4_each;
    const double us = std::max(turns(longest * mean_k) * alone, turns(mean_k) * seen * each_cu * each);
    return splits == 1 ? us : us + 4.0 + 4.3e-6 * rows * heads_kv * splits * head_dim;
  };
  // every sequence has at most one partly filled tile
  auto tiles = [&](int height) { return std::min<int64_t>(rows / height + batch, rows); };
  double least = 0;
  auto offer = [&](bool keys, int waves, int splits, int chunk) {
    const int height = keys ? kWaveRows : waves * kWaveRows;
    // a launch with shares holds at most 4 workgroups per CU (2 of attention_rows)
    if (splits > 1 && tiles(height) * heads_kv * splits > (keys ? 4 : 2) * cus) return;
    const double us = estimate(keys, waves, splits);
    if (pl.rows && us >= least) return;
    least = us;
    pl.keys = keys;
    pl.waves = waves;
    pl.rows = height;
    pl.splits = splits;
    pl.chunk = chunk;
  };
  if (rows <= (int64_t)batch * kTokenRows) {
    pl.parts = 2;
    // New tokens, whose sequences' lengths differ most: attention_keys, whole or in
    // shares by each sequence's own length, so long that the two workgroups of a
    // CU get one share each on average, 256 keys at least.  The longest is taken to be
    // twice the average.
    const int64_t fair = ((int64_t)total_k * heads_kv / (2 * cus) + 127) / 128 * 128;
    const int chunk = (int)std::max<int64_t>(256, std::min<int64_t>(fair, total_k));     // with many key heads: one share
    const int64_t want = 4 * cus / std::max<int64_t>(tiles(kWaveRows) * heads_kv, 1);
    const int64_t most = std::min<int64_t>({want, ((int64_t)total_k + chunk - 1) / chunk, 64});
    const double longest = batch > 1 ? 2 : 1;
    offer(true, 4, 1, chunk);
    const int mean = (int)std::min<int64_t>(most, (int64_t)std::ceil(mean_k / chunk));
    if (most > 1 && estimate(true, 4, std::max(mean, 2), longest) < estimate(true, 4, 1, longest)) pl.splits = (int)most;
  } else {
    offer(false, 4, 1, 0);
    if (head_dim > 64 && !causal) offer(false, 8, 1, 0);    // causal: the finer grain balances the tiles' lengths
    offer(true, 4, 1, 0);
    for (const int s : {2, 3, 4, 6, 8, 12, 16}) {
      const int chunk = (int)std::ceil(mean_k / s);
      if (chunk < 128) break;
      offer(false, 4, s, chunk);
      offer(true, 4, s, chunk);
    }
  }
  pl.chunk = std::max(pl.chunk, 128);
  pl.tiles = tiles(pl.rows);
  if (pl.splits > 1) {
    const size_t slots = (size_t)pl.tiles * heads_kv * pl.splits * pl.rows;
    pl.part = (slots * head_dim * 4 + 255) & ~size_t(255);
    pl.bytes = pl.part + ((slots * 4 + 255) & ~size_t(255));
  }
  return pl;
}

template <class H>
hipError_t launch(const Plan& pl, const Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)(pl.tiles * p.heads_kv * pl.splits));
  if (pl.keys) {
    constexpr int kWaves = key_waves(H::DP);
    if (pl.parts == 2)
      hipLaunchKernelGGL((attention_keys<H, kWaves, 2>), grid, dim3(kWaves * 64), 0, stream, p);
    else
      hipLaunchKernelGGL((attention_keys<H, kWaves, 1>), grid, dim3(kWaves * 64), 0, stream, p);
  } else if (pl.waves == 8) {
    if constexpr (H::DP == 128)
      hipLaunchKernelGGL((attention_rows<H, 8>), grid, dim3(512), 0, stream, p);
  } else {
    hipLaunchKernelGGL((attention_rows<H, 4>), grid, dim3(256), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.splits == 1) return e;
  const dim3 jgrid((unsigned)(pl.tiles * p.heads_kv * (pl.rows / 4)));
  hipLaunchKernelGGL(attention_join, jgrid, dim3(256), 0, stream, p, pl.rows);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim) {
  if (total_q == 0 || total_k == 0) return 0;
  return std::max(plan_of(total_q, total_k, batch, heads_q, heads_kv, head_dim, false).bytes,
                  plan_of(total_q, total_k, batch, heads_q, heads_kv, head_dim, true).bytes);
}

int64_t attention_blocks(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim) {
  int64_t most = 0;
  for (const bool causal : {false, true}) {
    const Plan pl = plan_of(total_q, total_k, batch, heads_q, heads_kv, head_dim, causal);
    most = std::max(most, pl.tiles * heads_kv * std::max(pl.splits, pl.splits > 1 ? pl.rows / 4 : 1));
  }
  return most;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  const Plan pl = plan_of(a.total_q, a.total_k, a.batch, a.heads_q, a.heads_kv, a.head_dim, a.causal != 0);
  Params p;
  p.Q = a.Q; p.K = a.K; p.V = a.V; p.O = a.O; p.lse = a.lse;
  p.ldq = a.ldq; p.ldk = a.ldk; p.ldv = a.ldv; p.ldo = a.ldo;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k;
  p.batch = a.batch; p.total_q = a.total_q; p.total_k = a.total_k;
  p.heads_q = a.heads_q; p.heads_kv = a.heads_kv; p.group = a.heads_q / a.heads_kv;
  p.head_dim = a.head_dim;
  p.c = a.scale * kLog2e;
  p.causal = a.causal;
  p.tiles = (int)pl.tiles;
  p.splits = pl.splits;
  p.chunk = pl.chunk;
  p.part = static_cast<float*>(a.workspace);
  p.part_lse = pl.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + pl.part) : nullptr;
  if (a.head_dim <= 64) return launch<Head<64, 4, 2>>(pl, p, stream);
  if (a.head_dim <= 96) return launch<Head<128, 6, 3>>(pl, p, stream);
  return launch<Head<128, 8, 4>>(pl, p, stream);
}

}  // namespace svdq
