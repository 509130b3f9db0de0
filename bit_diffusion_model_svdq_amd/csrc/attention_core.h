// The attention kernels over packed sequences (no padding, no score matrix), gfx950: the plain form
// (attention.hip) and the one whose keys lie in two pieces (attention_spans.hip).
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
#pragma once

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

// Keys in two pieces.  The tiles of piece A come first, all of whose keys every query
// of the tile sees, then those of piece B, in which each query sees a range:
//   sinks    A: the sequence's first keys that stay visible; B: from the first key of
//            the tile's windows on.  Where the two meet there is no A, and B starts with
//            the sequence.
//   prefix   A: the keys that all sequences share; B: the sequence's own.
// A tile's copies begin with the first and end with the last key that one of its
// queries sees: keys in front of all windows and behind them are not read.
//
// A shared prefix against few rows of each sequence (new tokens) is cut off instead:
// pre_splits > 0.  The rows of all sequences then are one problem against the prefix, so
// that 32 of them share its bytes and the MFMA's columns, and every sequence's rows another
// against its own keys; workgroups of both kinds run in one launch, all write partial
// rows, and the join brings a row's shares of both together.
struct SpanParams : Params {
  int left, right;       // keys before and behind a query's own that it sees; -1: all
  int sinks;             // first keys that stay visible
  const uint16_t *PK, *PV;
  int64_t ldpk, ldpv;
  int prefix;            // shared keys; 0 with a window or sinks
  int reach;             // own keys that a tile sees at most (sinks and window), for the shares
  int pre_splits, pre_tiles, pre_blocks;   // shares of the cut-off prefix, tiles of all rows; the launch's first workgroups
  // The launch's tiles from tail_tile on are cut into tail_splits shares (0: none are), its workgroups
  // from tail_block on: what would be a last round of few tiles is spread over all CUs.
  int tail_tile, tail_splits, tail_block;
  Quotient by_heads, by_heads_q, by_group, by_tiles, by_pre_tiles, by_tail_tiles;

  __device__ int keys(int nk) const { return min(nk, reach) + (pre_splits > 0 ? 0 : prefix); }
  // The first partial row of share s of tail tile t and a key head.
  __device__ int64_t tail_slot(int s, int t, int hk, int rows) const {
    return ((int64_t)(s * (tiles - tail_tile) + t) * heads_kv + hk) * rows;
  }
  // The partial row of share s (a cut-off prefix's first) of a query's row: sequences that
  // fill little of their tiles take no more room for it.
  __device__ int64_t slot(int s, int hk, int query, int in_group) const {
    return ((int64_t)s * heads_kv + hk) * total_q * group + (int64_t)query * group + in_group;
  }
  // Query `token` of nq against nk own keys sees [lo, hi) and [0, first).  left and right may
  // be anything up to 2^31 - 1: the sums are ordered so that none leaves 32 bits.
  __device__ void view(int token, int nq, int nk, int& lo, int& hi, int& first) const {
    const int behind = nq - token;                     // at least 1: the query stands at key nk - behind
    const int at = max(nk - behind, -1);
    lo = left < 0 ? 0 : max(at - left, 0);
    hi = right < 0 ? nk : max(nk - max(behind - 1 - right, 0), 0);
    first = min(sinks, nk);
    if (causal) {
      hi = min(hi, at + 1);
      first = min(first, at + 1);
    }
  }
  __device__ bool sees(int token, int nq, int nk) const {
    int lo, hi, first;
    view(token, nq, nk, lo, hi, first);
    return prefix > 0 || hi > lo || first > 0;
  }
};
template <bool SPANS> struct ParamsOf { using type = Params; };
template <> struct ParamsOf<true> { using type = SpanParams; };

// Bits [0, n) of 32.
__device__ inline uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

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

// v summed over lanes 0 .. this one.
__device__ inline int sum_to_lane(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);     // 1, 2, 4, 8 lanes on in a row of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);     // a row's last lane to the next row
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);     // lane 31 to the upper half
  return v;
}

// Sequence b's rows of both kinds.  The four offsets are loaded together: one after the
// other, behind each test for NULL, they cost a memory latency each.
__device__ inline void spans_of(const SpanParams& p, int b, int& q0, int& nq, int& kv0, int& nk) {
  if (p.cu_q && p.cu_k) {
    const int qa = p.cu_q[b], qb = p.cu_q[b + 1], ka = p.cu_k[b], kb = p.cu_k[b + 1];
    q0 = min(max(qa, 0), p.total_q);
    nq = max(min(qb, p.total_q) - q0, 0);
    kv0 = min(max(ka, 0), p.total_k);
    nk = max(min(kb, p.total_k) - kv0, 0);
  } else {
    span(p.cu_q, b, p.total_q, q0, nq);
    span(p.cu_k, b, p.total_k, kv0, nk);
  }
}

// find_tile with the sum over the lanes by DPP, none for a single sequence.
__device__ inline bool find_tile_spans(const SpanParams& p, int rows, int t, int lane, Place& at) {
  if (p.batch == 1) {
    spans_of(p, 0, at.q0, at.nq, at.kv0, at.nk);
    at.local = t;
    at.q0 = __builtin_amdgcn_readfirstlane(at.q0);
    at.nq = __builtin_amdgcn_readfirstlane(at.nq);
    at.kv0 = __builtin_amdgcn_readfirstlane(at.kv0);
    at.nk = __builtin_amdgcn_readfirstlane(at.nk);
    return t < (at.nq * p.group + rows - 1) / rows;
  }
  for (int base = 0; base < p.batch; base += 64) {
    const int b = min(base + lane, p.batch - 1);
    int q0, nq, kv0, nk;
    spans_of(p, b, q0, nq, kv0, nk);
    const int n = base + lane < p.batch ? (nq * p.group + rows - 1) / rows : 0;
    const int end = sum_to_lane(n);
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
template <class H, int MODE, int NW, bool SPANS>
struct Work {
  using T = Tile<H, MODE, NW>;
  using P = typename ParamsOf<SPANS>::type;
  const P& p;
  int lane, wave, half, col;
  int hk, q0, kv0, nk;
  int row0, row;             // the tile's first row, this lane's row
  bool row_ok;
  int token, head;
  int seen;                  // keys that this lane's query sees (two pieces: whether any)
  int wfull, wend;           // every query of the wave sees [0, wfull), none sees from wend on
  // two pieces: keys and tiles of A, B's first key and its keys up to the last that the
  // tile sees, this lane's ranges, and the wave's bounds of them
  int na, ta, b0, nb;
  int lo, hi, first;
  int wlo, wfirst;           // every query of the wave sees [wlo, wfull) and [0, wfirst)
  int shares;                // of the sequence's keys
  bool partial;              // two pieces: the results go to the workspace, as this share
  int share;
  int tail;                  // number of its tile among the tail's, or -1
  int t0, t1;                // key tiles of this share
  bf16x8 qf[H::KS];
  f32x16 o[H::DB];
  float m = -INFINITY;       // the maximum in use, raw scores
  float l = 0.f;             // this lane's share (its half's keys) of the sum
  int koff, voff[H::DB];
  int kvo[T::CPW], vvo[T::CPW];   // byte offsets of this lane's chunks in a tile of K and V
  int copier, mybuf;

  __device__ explicit Work(const P& p_) : p(p_) {}

  // False: no such tile.
  __device__ bool locate() {
    const int tid = threadIdx.x;
    lane = tid & 63;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    half = lane >> 5;
    col = lane & 31;
    if constexpr (SPANS) return locate_spans();
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

  // The same for keys in two pieces.  A tile takes 10 to 20 us, so what stands before
  // its first copy counts: no division is left but those of shares.
  __device__ bool locate_spans() {
    bool pre = false;                                  // a workgroup of the cut-off prefix
    int block = blockIdx.x;
    if (p.pre_splits > 0) {
      pre = block < p.pre_blocks;
      if (!pre) block -= p.pre_blocks;
    }
    const bool in_tail = MODE == kRows && p.tail_splits > 0 && block >= p.tail_block;
    if (in_tail) block -= p.tail_block;
    const int rest = p.by_heads.of(block);
    hk = block - rest * p.heads_kv;
    int split = (pre ? p.by_pre_tiles : p.by_tiles).of(rest);
    Place at;
    at.local = rest - split * (pre ? p.pre_tiles : p.tiles);
    tail = -1;
    if (in_tail) {
      split = p.by_tail_tiles.of(rest);
      tail = rest - split * (p.tiles - p.tail_tile);
      at.local = p.tail_tile + tail;
    }
    if (pre) {
      const int begin = p.cu_q[0], end = p.cu_q[p.batch];      // batch > 1: not NULL
      at.q0 = __builtin_amdgcn_readfirstlane(min(max(begin, 0), p.total_q));
      at.nq = max(__builtin_amdgcn_readfirstlane(min(end, p.total_q)) - at.q0, 0);
      at.kv0 = at.nk = 0;
      if (at.local >= (at.nq * p.group + T::ROWS - 1) / T::ROWS) return false;
    } else if (!find_tile_spans(p, T::ROWS, at.local, lane, at)) {
      return false;
    }
    q0 = at.q0;
    kv0 = at.kv0;
    nk = at.nk;
    const int nq = at.nq;
    shares = 1;
    if (pre)
      shares = p.pre_splits;
    else if (in_tail)
      shares = p.tail_splits;
    else if (p.splits > 1)
      shares = p.shares(p.keys(nk));
    partial = shares > 1 || p.pre_splits > 0;
    share = pre ? split : p.pre_splits + split;
    if (split >= shares) return false;
    const int nrows = nq * p.group;
    int local = at.local;
    // causal tiles see more keys the later they are: start with the last
    if (p.causal && !pre) local = (nrows + T::ROWS - 1) / T::ROWS - 1 - local;
    row0 = local * T::ROWS;
    const int wrow0 = row0 + (MODE == kRows ? wave * kWaveRows : 0);
    row = wrow0 + col;
    row_ok = row < nrows;
    const int rowc = min(row, nrows - 1);
    token = p.by_group.of(rowc);
    head = hk * p.group + (rowc - token * p.group);
    p.view(token, nq, nk, lo, hi, first);
    int l0, h0, f0, l1, h1, f1;
    p.view(p.by_group.of(min(wrow0, nrows - 1)), nq, nk, l0, h0, f0);
    p.view(p.by_group.of(min(wrow0 + kWaveRows, nrows) - 1), nq, nk, l1, h1, f1);
    wlo = l1;
    wfull = h0;
    wfirst = f0;
    // a wave without rows works on nothing, one with rows on all of A
    wend = MODE == kRows && wrow0 >= nrows ? INT32_MIN : max(max(h1, f1), 0);
    if constexpr (MODE == kRows) {
      p.view(p.by_group.of(row0), nq, nk, l0, h0, f0);
      p.view(p.by_group.of(min(row0 + T::ROWS, nrows) - 1), nq, nk, l1, h1, f1);
    }
    // the windows begin behind the first keys: every query of the tile sees all of those
    const bool apart = l0 > f1;
    na = pre || (p.prefix > 0 && p.pre_splits == 0) ? p.prefix : apart ? f1 : 0;
    b0 = apart ? l0 : 0;
    nb = max(max(h1, f1) - b0, 0);
    ta = (na + T::KT - 1) / T::KT;
    const int ntiles = ta + (nb + T::KT - 1) / T::KT;
    seen = na > 0 || hi > lo || first > 0;
    t0 = 0;
    t1 = ntiles;
    if (shares > 1) {                                  // ntiles split / shares, without 64 bits
      const int q = ntiles / shares, r = ntiles - q * shares;
      t0 = q * split + r * split / shares;
      t1 = q * (split + 1) + r * (split + 1) / shares;
    }
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
    if constexpr (SPANS) __builtin_amdgcn_sched_barrier(0);      // they leave here, not behind the first copies
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
    if constexpr (SPANS) return;                       // start() knows the piece
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
    int t;                   // two pieces: the tile, and whether it is one of B
    bool own;
  };
  // Two pieces: the cursor of tile t, with this lane's offsets in tiles of its piece.
  template <bool K>
  __device__ Cursor enter(int t, int (&off)[T::CPW]) const {
    static_assert(SPANS);
    Cursor c;
    c.t = t;
    c.own = t >= ta;
    const uint16_t* base = K ? p.K : p.V;
    int64_t ld = K ? p.ldk : p.ldv;
    int64_t key;
    if (c.own) {
      key = (int64_t)kv0 + b0 + (int64_t)(t - ta) * T::KT;
      c.left = min(nb, (t1 - ta) * T::KT) - (t - ta) * T::KT;      // a share copies no tile of the next one
    } else {
      key = (int64_t)t * T::KT;
      c.left = min(na, t1 * T::KT) - t * T::KT;
      if (p.prefix > 0) {
        base = K ? p.PK : p.PV;
        ld = K ? p.ldpk : p.ldpv;
      } else {
        key += kv0;
      }
    }
    c.at = base + key * ld + (int64_t)hk * p.head_dim;
    constexpr int RPC = 1024 / H::ROWB;
    const int last_chunk = p.head_dim / 8 - 1;
#pragma unroll
    for (int i = 0; i < T::CPW; ++i) {
      const int r = (copier * T::CPW + i) * RPC + lane / H::CHUNKS;
      off[i] = r * (int)ld * 2 + min((lane % H::CHUNKS) ^ (K ? k_key<H>(r) : v_key<H>(r)), last_chunk) * 16;
    }
    return c;
  }
  __device__ Cursor cursor(const uint16_t* base, int64_t ld, int t) const {
    return {base + (int64_t)(kv0 + t * T::KT) * ld + (int64_t)hk * p.head_dim, nk - t * T::KT, 0, false};
  }
  template <bool K>
  __device__ void copy(Cursor& c, int ld, int step, int (&off)[T::CPW], uint8_t* dst) {
    if constexpr (SPANS)
      if (!c.own && p.prefix > 0) ld = (int)(K ? p.ldpk : p.ldpv);
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
    if constexpr (SPANS) {
      c.t += step;
      if (!c.own && c.t >= ta) {
        c = enter<K>(c.t, off);
        return;
      }
    }
    c.at += (int64_t)step * T::KT * ld;
    c.left -= step * T::KT;
  }
  Cursor ck, cv;
  __device__ void copy_k(uint8_t* dst, int step) { copy<true>(ck, (int)p.ldk, step, kvo, dst); }
  __device__ void copy_v(uint8_t* dst, int step) { copy<false>(cv, (int)p.ldv, step, vvo, dst); }
  __device__ void start(int t) {
    if constexpr (SPANS) {
      ck = enter<true>(t, kvo);
      cv = enter<false>(t, vvo);
    } else {
      ck = cursor(p.K, p.ldk, t);
      cv = cursor(p.V, p.ldv, t);
    }
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
    if constexpr (SPANS) {
      const int at = b0 + (t - ta) * T::KT;
      uint32_t bits = t >= t1 ? 0u : t < ta ? below(na - t * T::KT) : (below(hi - at) & ~below(lo - at)) | below(first - at);
      bits >>= 4 * half;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (!(bits >> (8 * (j >> 2) + (j & 3)) & 1)) s[j] = -INFINITY;
      return;
    }
    const int left = seen - t * T::KT - 4 * half;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (8 * (j >> 2) + (j & 3) >= left) s[j] = -INFINITY;
  }
  // Whether every query of the wave sees all of tile t.
  __device__ bool whole(int t) const {
    if constexpr (SPANS) {
      const int at = b0 + (t - ta) * T::KT, end = at + T::KT;
      if (t >= t1) return false;
      return t < ta ? (t + 1) * T::KT <= na : (at >= wlo && end <= wfull) || end <= wfirst;
    }
    return t * T::KT + T::KT <= wfull;
  }
  // Whether a query of the wave may see a key of tile t or of one after it.
  __device__ bool live(int t) const {
    if constexpr (SPANS) return b0 + (t - ta) * T::KT < wend;      // a tile of A lies in front of b0, or of 0
    return t * T::KT < wend;
  }

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
    const bool part = SPANS ? partial : shares > 1;
    const bool lost = none && (part ? m * p.c == INFINITY : seen > 0);
    const float inv = lost ? NAN : none ? 0.f : 1.f / l;
    const float lse2 = lost ? NAN : none ? -INFINITY : __builtin_fmaf(m, p.c, __builtin_amdgcn_logf(l));
    if (!row_ok) return;
    if (none)                      // V's infinities and NaN times no weight
#pragma unroll
      for (int i = 0; i < H::DB; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    if (part) {
      int64_t slot;
      if constexpr (SPANS)
        slot = MODE == kRows && tail >= 0 ? p.tail_slot(share, tail, hk, T::ROWS) + (row - row0)
                                          : p.slot(share, hk, q0 + token, head - hk * p.group);
      else
        slot = (int64_t)blockIdx.x * T::ROWS + (row - row0);
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
// t beside the rest of them.  The compiler keeps the exponentials there and sinks the
// sum's 17 additions behind the tile's last MFMA.  Tiles of 32 keys: with 64 the scores of two tiles
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
//
// With SPANS it is the loop itself that bounds them: between a turn's barrier and its first
// MFMA stand about 50 scalar instructions, five branches and eight register moves (the
// piece, its stride and the lanes' offsets, for K and for V), where the plain form has 11 to 16
// and one branch, and another chain of branches behind the MFMAs (whole()).  MFMAs run in
// 47 % of the cycles of 16384 tokens x 24 x 128 with windows of 2048 to both sides
// (824 to 838 us), in 41 % behind a prefix of 4608 keys (4 x 1024 tokens, 303 us).
template <class H, int NW, bool SPANS>
__global__ __launch_bounds__(NW * 64, 2) void attention_rows(const typename ParamsOf<SPANS>::type p) {
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
  Work<H, kRows, NW, SPANS> w(p);
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
    if (w.live(t)) tile(t, cur, nxt, kt, vt, kafter);
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
template <class H, int NW, int PARTS, bool SPANS>
__global__ __launch_bounds__(NW * 64, H::DP == 64 ? 2 : 1) void attention_keys(const typename ParamsOf<SPANS>::type p) {
  using T = Tile<H, kKeys, NW>;
  __shared__ __attribute__((aligned(16))) uint8_t k0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t k1s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v0s[T::BUFS * T::TILE_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t v1s[T::BUFS * T::TILE_BYTES];
  __shared__ float wm[NW][kWaveRows], wl[NW][kWaveRows];
  Work<H, kKeys, NW, SPANS> w(p);
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
  // Two pieces: also past the last tile (of nothing), so that Q can be waited for without
  // these copies: no branch between them.
  if (SPANS || t < w.t1) {
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
    if (w.live(t)) compute(t, kc, vc);
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

// attention_keys' waves: so many that two workgroups fit a CU's LDS (a wave
// holds two K and two V tiles).  Measured with keys from HBM: 16 single tokens against
// 49.5 k keys x 8 x 128 56.8 us with 2 waves, 60.6 with 4, 32 against 64 k x 16 x 80
// 85.2 and 91.1; 64 against 64 k x 16 x 64 59.0 and 59.5.
constexpr int key_waves(int dp) { return dp == 64 ? 4 : 2; }

// Rows per sequence, on average, up to which a call counts as one of new tokens.
constexpr int kTokenRows = 64;

using Plan = AttentionPlan;

// What a tile of 32 keys costs a workgroup, in us, by the head's size (up to 64,
// 96, 128 channels): alone on its CU, where latency counts, and as its part of a
// full CU; with 8 waves a workgroup has the CU to itself.  For attention_keys it
// is a turn of all its waves.
struct Cost {
  double rows4, rows4_each, rows8, keys, keys_each;
  int keys_waves;
};
inline Cost cost_of(int head_dim) {
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
// window: the own keys that a query sees at most, where that is limited (a tile of rows sees
// one more for each of its tokens); prefix: keys that every query sees besides.
inline Plan plan_of(int total_q, int total_k, int batch, int heads_q, int heads_kv, int head_dim, bool causal,
                    double window = INFINITY, int prefix = 0) {
  Plan pl;
  const int group = heads_q / heads_kv;
  const int64_t rows = (int64_t)total_q * group;
  const int64_t cus = device_cu_count();
  const Cost cost = cost_of(head_dim);
  const double mean_rows = (double)rows / batch, mean_q = (double)total_q / batch, mean_own = (double)total_k / batch;
  auto keys_of = [&](int height) { return std::min(mean_own, window + std::min((double)height / group, mean_q)) + prefix; };
  auto estimate = [&](bool keys, int waves, int splits, double longest = 1) {
    const double units = std::ceil(mean_rows / (keys ? kWaveRows : waves * kWaveRows)) * batch * heads_kv;
    double each_cu = std::ceil(units * splits / cus);
    if (keys && each_cu > 1) each_cu = 2 * std::ceil(each_cu / 2);       // two fit a CU
    auto turns = [&](double nk) {
      return std::ceil(std::ceil(std::ceil(nk / 32) / (keys ? cost.keys_waves : 1)) / splits);
    };
    const double mean_k = keys_of(keys ? kWaveRows : waves * kWaveRows);
    // causal: half of the tiles, and their unequal lengths leave CUs waiting
    const double seen = causal && mean_own <= window ? 1 - 0.4 * std::min(1.0, mean_q / std::max(mean_k, 1.0)) : 1;
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
    const double mean_k = keys_of(kWaveRows);
    const int64_t all_k = prefix == 0 && mean_k == mean_own ? total_k : (int64_t)(mean_k * batch);
    // with a window the sequences are alike, and the shares end where the workgroups do (16 single
    // tokens with windows of 1024 keys in 2, 3, 4, 5 shares 24.5, 21.8, 20.9, 22.2 us)
    const int64_t grain = mean_own > window ? 32 : 128;
    const int64_t fair = (all_k * heads_kv / (2 * cus) + grain - 1) / grain * grain;
    const int chunk = (int)std::max<int64_t>(256, std::min<int64_t>({fair, all_k, INT32_MAX}));     // with many key heads: one share
    const int64_t want = 4 * cus / std::max<int64_t>(tiles(kWaveRows) * heads_kv, 1);
    const int64_t most = std::min<int64_t>({want, (all_k + chunk - 1) / chunk, 64});
    const double longest = batch > 1 ? 2 : 1;
    offer(true, 4, 1, chunk);
    const int mean = (int)std::min<int64_t>(most, (int64_t)std::ceil(mean_k / chunk));
    if (most > 1 && estimate(true, 4, std::max(mean, 2), longest) < estimate(true, 4, 1, longest)) pl.splits = (int)most;
  } else {
    offer(false, 4, 1, 0);
    // causal: the finer grain balances the tiles' lengths; a window: the larger tile sees more keys
    // that most of its rows do not, and nothing runs beside its start (16384 x 24 x 128, windows of
    // 1025, 4097, 8193 keys: 453, 792, 1425 us with 4 waves, 489, 841, 1478 with 8)
    if (head_dim > 64 && !causal && mean_own <= window) offer(false, 8, 1, 0);
    offer(true, 4, 1, 0);
    for (const int s : {2, 3, 4, 6, 8, 12, 16}) {
      const int chunk = (int)std::ceil(keys_of(kWaveRows) / s);
      if (chunk < 128) break;
      offer(false, 4, s, (int)std::ceil(keys_of(4 * kWaveRows) / s));
      offer(true, 4, s, chunk);
    }
  }
  pl.us = least;
  pl.chunk = std::max(pl.chunk, 128);
  pl.tiles = tiles(pl.rows);
  if (pl.splits > 1) {
    const size_t slots = (size_t)pl.tiles * heads_kv * pl.splits * pl.rows;
    pl.part = (slots * head_dim * 4 + 255) & ~size_t(255);
    pl.bytes = pl.part + ((slots * 4 + 255) & ~size_t(255));
  }
  return pl;
}

}  // namespace
}  // namespace svdq
