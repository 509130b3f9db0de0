// svdq_attention_window_forward and svdq_attention_prefix_forward: attention over keys in
// two pieces, first keys and a window, or a shared prefix and a sequence's own keys.  The
// kernels are attention_core.h's with SPANS.
#include "attention_core.h"

namespace svdq {
namespace {

// Joins the shares of a row as attention_join does: a wave per row, lane s holding share s's
// weight.  The weights and the first sixteen rows of the `most` shares it can have are loaded before
// find() says how many it has, and whose row it is (false: nobody's, or written by its one share): 64
// tokens behind a prefix of 8192 7.4 -> 6.3 us, 16 with windows of 1024 keys 7.3 -> 4.1.
struct JoinRow {
  int shares, query, token, nq, nk;
};
template <class Slot, class Find>
__device__ inline void join_row(const SpanParams& p, int lane, int most, int head, Slot slot, Find find) {
  constexpr int kAhead = 16;
  const int d = 2 * lane;
  const bool on = d < p.head_dim;
  float2 v[kAhead];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s0 + u < most) v[u] = *reinterpret_cast<const float2*>(p.part + slot(s0 + u) * p.head_dim + (on ? d : 0));
  };
  float e = lane < most ? p.part_lse[slot(lane)] : -INFINITY;
  load(0);
  JoinRow r;
  if (!find(r)) return;
  if (lane >= r.shares) e = -INFINITY;
  float top = e;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
  const float weight = e == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(e - top);
  float sum = weight;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
  float a0 = 0.f, a1 = 0.f;
  for (int s0 = 0; s0 < r.shares; s0 += kAhead) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s0 + u >= r.shares) break;
      const float w = __shfl(weight, s0 + u);
      if (w != 0.f) {                                    // a share without weight has written nothing
        a0 = __builtin_fmaf(w, v[u].x, a0);
        a1 = __builtin_fmaf(w, v[u].y, a1);
      }
    }
  }
  // as in finish(): no weight at all is NaN for a query that sees keys
  const bool seen = p.sees(r.token, r.nq, r.nk);
  const bool none = sum == 0.f;
  const float inv = !none ? 1.f / sum : seen ? NAN : 0.f;
  if (on) {
    const uint16_t x = __builtin_bit_cast(uint16_t, (__bf16)(a0 * inv));
    const uint16_t y = __builtin_bit_cast(uint16_t, (__bf16)(a1 * inv));
    *reinterpret_cast<uint32_t*>(p.O + (int64_t)r.query * p.ldo + (int64_t)head * p.head_dim + d) = x | ((uint32_t)y << 16);
  }
  if (p.lse && lane == 0)
    p.lse[(int64_t)head * p.total_q + r.query] =
        !none ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : seen ? NAN : -INFINITY;
}

// Every query and head, with partial rows at SpanParams::slot.
__global__ __launch_bounds__(256) void attention_join_spans(const SpanParams p) {
  const int lane = threadIdx.x & 63;
  const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int query = p.by_heads_q.of(id), head = id - query * p.heads_q;
  if (query >= p.total_q) return;
  const int hk = p.by_group.of(head);
  auto slot = [&](int s) { return p.slot(s, hk, query, head - hk * p.group); };
  join_row(p, lane, p.pre_splits + p.splits, head, slot, [&](JoinRow& r) {
    // the last sequence that begins at or before the query, 64 at a time
    int b = p.cu_q ? -1 : 0;
    for (int base = 0; base < p.batch && p.cu_q; base += 64) {
      const uint64_t m = __ballot(base + lane < p.batch && p.cu_q[min(base + lane, p.batch - 1)] <= query);
      b += __builtin_popcountll(m);
      if (m != ~uint64_t(0)) break;
    }
    if (b < 0) return false;
    int q0, kv0;
    spans_of(p, b, q0, r.nq, kv0, r.nk);
    r.query = query;
    r.token = query - q0;
    r.shares = p.shares(p.keys(r.nk)) + p.pre_splits;
    return r.token >= 0 && r.token < r.nq && r.shares > 1;
  });
}

// The rows of the tail's tiles, with partial rows at SpanParams::tail_slot.
__global__ __launch_bounds__(256) void attention_join_tail(const SpanParams p) {
  constexpr int kRowsPerTile = 4 * kWaveRows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rest = p.by_heads.of(blockIdx.x), hk = blockIdx.x - rest * p.heads_kv;
  const int t = rest / (kRowsPerTile / 4), in_tile = rest % (kRowsPerTile / 4) * 4 + wave;
  Place at;
  if (!find_tile_spans(p, kRowsPerTile, p.tail_tile + t, lane, at)) return;
  const int nrows = at.nq * p.group;
  int local = at.local;
  if (p.causal) local = (nrows + kRowsPerTile - 1) / kRowsPerTile - 1 - local;
  const int row = local * kRowsPerTile + in_tile;
  if (row >= nrows) return;
  const int token = p.by_group.of(row), head = hk * p.group + row - token * p.group;
  auto slot = [&](int s) { return p.tail_slot(s, t, hk, kRowsPerTile) + in_tile; };
  join_row(p, lane, p.tail_splits, head, slot, [&](JoinRow& r) {
    r = {p.tail_splits, at.q0 + token, token, at.nq, at.nk};
    return true;
  });
}

// Partial rows of a cut-off prefix that a call may ask its caller to hold: those of 8128 new tokens x 32 x 128,
// with one share of the prefix and one of the own keys.
constexpr int64_t kMaxSplitBytes = int64_t(256) << 20;

// Workgroups of the join.
int64_t join_blocks(int64_t total_q, int heads_q) { return (total_q * heads_q + 3) / 4; }

// Own keys that a query sees at most.
double window_of(const SpanArgs& a) {
  const int right = a.causal ? 0 : a.right;
  return a.left < 0 || right < 0 ? INFINITY : (double)a.sinks + a.left + right + 1;
}

// Cuts the prefix off where that is less than the plan at hand: shares so long that the two
// workgroups of a CU get one each on average.  attention_rows, whose four waves share a
// tile of the prefix, where there are rows for them, and where the sequences' own tiles fill
// the chip anyway; else attention_keys, more of whose waves work for each sequence.  Measured
// (attention_keys / attention_rows / not cut off): prefix of 8192, 200 tokens x 32 / 8 x 128 135 / 72 /
// 702 us, 64 45 / 35 / 181, 16 24 / 24 / 58; with 1000 keys of its own each 237 / 184 / 826, 77 / 78 / 221,
// 31 / 40 / 64; 64 x 10 x 64 26 / 22 / 113, 16 17 / 18 / 42.  Prefix of 100, 16 tokens x 32 / 8 x 128
// 12.7 / 12.6 / 10.5.
void offer_cut(const SpanArgs& a, int64_t rows, SpanPlan& sp) {
  const int64_t cus = device_cu_count();
  const Cost cost = cost_of(a.head_dim);
  const bool keys = rows < 4 * kWaveRows && std::min<int64_t>(a.batch, rows) * a.heads_kv < 2 * cus;
  const int height = keys ? kWaveRows : 4 * kWaveRows;
  const double turn = keys ? 32.0 * cost.keys_waves : 32.0, alone = keys ? cost.keys : cost.rows4;
  const double each = keys ? cost.keys_each : cost.rows4_each;
  const int64_t pre_tiles = (rows + height - 1) / height;
  const int64_t tiles = std::min<int64_t>(rows / height + a.batch, rows);
  const double mean_own = (double)a.total_k / a.batch;
  // keys of all tiles; those of attention_rows against a sequence's own occupy one wave of four
  const double pre_work = (double)pre_tiles * a.prefix * a.heads_kv, own_work = (double)tiles * mean_own * a.heads_kv;
  const int64_t fair = (int64_t)std::min(std::ceil((pre_work + own_work) / (2.0 * cus) / 128) * 128, (double)INT32_MAX);
  const int chunk = (int)std::max<int64_t>(256, fair);
  const int pre_splits = (int)std::min<int64_t>((a.prefix + (int64_t)chunk - 1) / chunk, 32);
  const int64_t want = std::max<int64_t>(4 * cus / std::max<int64_t>(tiles * a.heads_kv, 1), 1);
  const int splits = (int)std::max<int64_t>(std::min<int64_t>({want, (a.total_k + (int64_t)chunk - 1) / chunk, 32}), 1);
  const double longest = std::max((double)a.prefix / pre_splits, std::min(mean_own, (double)chunk));
  const double us = std::max(std::ceil(longest / turn) * alone, (pre_work + (keys ? 1.0 : 0.6) * own_work) / turn / cus * each) + 3.0 +
                    2e-6 * rows * a.heads_kv * (pre_splits + std::ceil(mean_own / chunk)) * a.head_dim;
  const int64_t slots = rows * a.heads_kv * (pre_splits + splits);
  if (us >= sp.own.us || slots * (a.head_dim + 1) * 4 > kMaxSplitBytes) return;
  sp.own.us = us;
  sp.pre_splits = pre_splits;
  sp.pre_tiles = (int)pre_tiles;
  sp.own.keys = keys;
  sp.own.parts = keys ? 2 : 1;
  sp.own.waves = 4;
  sp.own.rows = height;
  sp.own.splits = splits;
  sp.own.chunk = chunk;
  sp.own.tiles = tiles;
}

// attention_rows with four waves and shares for the tiles of a last, partly filled round, if that
// is less than the plan at hand.  A CU takes one tile of rows in 0.58 of the time of two at once, so
// with k whole rounds of one per CU and a part of the next the launch lasts nearly as long as
// with k + 1; cut into so many shares that they fill it, the rest lasts that much less.  Counted
// for as much of the tiles' keys as is alike in all of them: where they differ (causal, the
// ends of windows) the tiles fill the gaps themselves.  Measured, before and with shares: prefix of 3000
// and 1408 tokens x 24 x 128 135 / 112 us, 1792 147 / 128, 2816 294 / 212; prefix of 800 and 2816 tokens 188 / 143;
// ragged continuations of 4001 keys, 1076 tokens x 32 / 8 x 128, 119 / 106.  Windows of 1500 to both sides of
// 2816 and 3328 tokens, whose tiles differ, would gain 106 / 100 and 120 / 121: not taken.
void offer_tail(const SpanArgs& a, int64_t rows, SpanPlan& sp) {
  const int64_t cus = device_cu_count();
  constexpr int kHeight = 4 * kWaveRows;
  const int64_t tiles = std::min<int64_t>(rows / kHeight + a.batch, rows);
  const double units = std::min(std::ceil((double)rows / a.batch / kHeight) * a.batch, (double)tiles) * a.heads_kv;
  const int64_t whole = (int64_t)(units / cus), first = whole * cus / a.heads_kv, tail = tiles - first;
  const double rest = (units - first * a.heads_kv) / cus;
  if (whole < 1 || whole > 6 || rest < 0.02 || rest > 0.5 || tail < 1) return;
  const int shares = (int)std::min(8.0, 1 / rest);
  const double window = window_of(a), mean_own = (double)a.total_k / a.batch, mean_q = (double)a.total_q / a.batch;
  double own = std::min(mean_own, window + std::min(mean_q, (double)kHeight * a.heads_kv / a.heads_q));
  if (a.causal && mean_own <= window) own *= 1 - 0.4 * std::min(1.0, mean_q / std::max(mean_own, 1.0));
  const bool alike = window == INFINITY ? !a.causal : mean_own > 2 * window;
  const double keys = own + a.prefix, cost = 2 * cost_of(a.head_dim).rows4_each / 32;      // us of a key for two workgroups
  const double gain = (whole % 2 ? 0.42 : 0.58) * (1 - 1.0 / shares) * cost * (alike ? keys : a.prefix);
  const int64_t slots = tail * a.heads_kv * shares * kHeight;
  const double us = cost * keys * (whole / 2 + (whole % 2 ? 1.0 : 0.58)) - gain + 6.0 + 2e-6 * slots * a.head_dim;
  if (us >= sp.own.us || gain < 6.0 + 2e-6 * slots * a.head_dim || slots * (a.head_dim + 1) * 4 > int64_t(64) << 20) return;
  sp.own = Plan();
  sp.own.rows = kHeight;
  sp.own.tiles = tiles;
  sp.own.chunk = 128;
  sp.own.us = us;
  sp.tail_tile = (int)first;
  sp.tail_splits = shares;
}

// attention_keys with four waves for heads of more than 64 channels where a CU has one workgroup at
// most, so that nothing runs beside it anyway, and for new tokens that instead of shares and a
// second launch as long as the longest sequence, taken to be twice the average, has five turns
// of their four tiles.  It is no gain for two turns of two waves.  Measured, two / four waves: 8 single
// tokens x 16 / 4 x 128 with 64 keys, 128, 256 6.7 / 7.7 us, 8.4 / 8.0, 10.9 / 9.5, and with one of 544 among
// 1 to 160 18.8 / 13.3; 7 of up to 848 keys x 8 x 72 22.9 / 15.7; prompts of 77, 160, 320 tokens x 8 / 4 x 128
// 6.9 / 6.9, 9.0 / 9.2, 11.7 / 10.8; in shares / four waves: 384 keys 14.0 / 10.8, with windows of 516 13.9 / 13.6,
// 8 x 16 / 4 x 96 with up to 1280 keys, on average 500, 14.6 / 17.8.  Eight waves for 64 channels: 128 keys 5.4 / 6.5,
// 512 7.7 / 8.5, 1024 11.2 / 10.2: not taken.
constexpr int kWideWaves = 4;
void offer_wide(const SpanArgs& a, int64_t rows, SpanPlan& sp) {
  const int64_t cus = device_cu_count();
  const int group = a.heads_q / a.heads_kv;
  const double mean_own = (double)a.total_k / a.batch, mean_q = (double)a.total_q / a.batch;
  const double longest = std::min(mean_own * (a.batch > 1 ? 2 : 1), window_of(a) + std::min(mean_q, (double)kWaveRows / group)) + a.prefix;
  const double key_tiles = std::ceil(longest / 32);
  const int64_t tiles = std::min<int64_t>(rows / kWaveRows + a.batch, rows);
  const bool shares = sp.own.splits > 1 || sp.pre_splits > 0;
  if (shares && rows <= (int64_t)a.batch * kTokenRows && tiles * a.heads_kv <= cus && key_tiles <= 5 * kWideWaves) {
    sp = SpanPlan();
    sp.own.keys = true;
    sp.own.parts = 2;
    sp.own.rows = kWaveRows;
    sp.own.tiles = tiles;
    sp.own.chunk = 128;
  }
  const int64_t blocks = (sp.own.tiles * sp.own.splits + (int64_t)sp.pre_tiles * sp.pre_splits) * a.heads_kv;
  sp.wide = sp.own.keys && blocks <= cus && (sp.own.splits > 1 || sp.pre_splits > 0 || key_tiles > 2 * key_waves(128));
}

// A prefix is cut off where that is less work by the same estimate as in plan_of: new
// tokens of several sequences, each of which would otherwise read it for itself, with most
// of the MFMA's 32 columns idle.
SpanPlan plan_spans(const SpanArgs& a) {
  SpanPlan sp;
  const int group = a.heads_q / a.heads_kv;
  const int64_t rows = (int64_t)a.total_q * group;
  sp.own = plan_of(a.total_q, a.total_k, a.batch, a.heads_q, a.heads_kv, a.head_dim, a.causal != 0, window_of(a),
                   a.prefix);
  if (rows > (int64_t)a.batch * kTokenRows)
    offer_tail(a, rows, sp);
  else if (a.prefix > 0 && a.batch > 1)
    offer_cut(a, rows, sp);
  if (a.head_dim > 64) offer_wide(a, rows, sp);
  sp.blocks = (sp.own.tiles * sp.own.splits + (int64_t)sp.pre_tiles * sp.pre_splits) * a.heads_kv;
  sp.most_blocks = sp.blocks;
  if (sp.tail_splits > 0) {
    const int64_t tail = sp.own.tiles - sp.tail_tile;
    sp.blocks += tail * (sp.tail_splits - 1) * a.heads_kv;
    const size_t slots = (size_t)tail * a.heads_kv * sp.tail_splits * sp.own.rows;
    sp.part = (slots * a.head_dim * 4 + 255) & ~size_t(255);
    sp.bytes = sp.part + ((slots * 4 + 255) & ~size_t(255));
    sp.most_blocks = std::max(sp.blocks, tail * a.heads_kv * (sp.own.rows / 4));
  } else if (sp.own.splits > 1 || sp.pre_splits > 0) {
    const size_t slots = (size_t)rows * a.heads_kv * (sp.pre_splits + sp.own.splits);
    sp.part = (slots * a.head_dim * 4 + 255) & ~size_t(255);
    sp.bytes = sp.part + ((slots * 4 + 255) & ~size_t(255));
    sp.most_blocks = std::max(sp.blocks, join_blocks(a.total_q, a.heads_q));
  }
  return sp;
}

template <class H>
hipError_t launch(const SpanPlan& sp, const SpanParams& p, hipStream_t stream) {
  const Plan& pl = sp.own;
  const dim3 grid((unsigned)sp.blocks);
  if (pl.keys) {
    auto go = [&](auto waves) {
      constexpr int kWaves = decltype(waves)::value;
      if (pl.parts == 2)
        hipLaunchKernelGGL((attention_keys<H, kWaves, 2, true>), grid, dim3(kWaves * 64), 0, stream, p);
      else
        hipLaunchKernelGGL((attention_keys<H, kWaves, 1, true>), grid, dim3(kWaves * 64), 0, stream, p);
    };
    if (sp.wide)
      go(std::integral_constant<int, kWideWaves>());
    else
      go(std::integral_constant<int, key_waves(H::DP)>());
  } else if (pl.waves == 8) {
    if constexpr (H::DP == 128)
      hipLaunchKernelGGL((attention_rows<H, 8, true>), grid, dim3(512), 0, stream, p);
  } else {
    hipLaunchKernelGGL((attention_rows<H, 4, true>), grid, dim3(256), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.bytes == 0) return e;
  if (sp.tail_splits > 0) {
    const int64_t blocks = (pl.tiles - sp.tail_tile) * p.heads_kv * (pl.rows / 4);
    hipLaunchKernelGGL(attention_join_tail, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(attention_join_spans, dim3((unsigned)join_blocks(p.total_q, p.heads_q)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

SpanPlan plan_attention_spans(const SpanArgs& a) { return plan_spans(a); }

hipError_t launch_attention_spans(const SpanArgs& a, const SpanPlan& sp, hipStream_t stream) {
  SpanParams p;
  p.Q = a.Q; p.K = a.K; p.V = a.V; p.O = a.O; p.lse = a.lse;
  p.ldq = a.ldq; p.ldk = a.ldk; p.ldv = a.ldv; p.ldo = a.ldo;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k;
  p.batch = a.batch; p.total_q = a.total_q; p.total_k = a.total_k;
  p.heads_q = a.heads_q; p.heads_kv = a.heads_kv; p.group = a.heads_q / a.heads_kv;
  p.head_dim = a.head_dim;
  p.c = a.scale * kLog2e;
  p.causal = a.causal;
  p.tiles = (int)sp.own.tiles;
  p.splits = sp.own.splits;
  p.chunk = sp.own.chunk;
  p.part = static_cast<float*>(a.workspace);
  p.part_lse = sp.bytes > 0 ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + sp.part) : nullptr;
  p.left = a.left; p.right = a.right; p.sinks = a.sinks;
  p.PK = a.PK; p.PV = a.PV; p.ldpk = a.ldpk; p.ldpv = a.ldpv; p.prefix = a.prefix;
  p.reach = (int)std::min(window_of(a) + sp.own.rows / p.group + 1, (double)INT32_MAX);
  p.pre_splits = sp.pre_splits;
  p.pre_tiles = sp.pre_tiles;
  p.pre_blocks = sp.pre_splits * sp.pre_tiles * a.heads_kv;
  p.tail_tile = sp.tail_tile;
  p.tail_splits = sp.tail_splits;
  p.tail_block = sp.tail_tile * a.heads_kv;
  p.by_tail_tiles = Quotient((int)std::max<int64_t>(sp.own.tiles - sp.tail_tile, 1));
  p.by_heads = Quotient(a.heads_kv);
  p.by_heads_q = Quotient(a.heads_q);
  p.by_group = Quotient(p.group);
  p.by_tiles = Quotient(p.tiles);
  p.by_pre_tiles = Quotient(std::max(p.pre_tiles, 1));
  if (a.head_dim <= 64) return launch<Head<64, 4, 2>>(sp, p, stream);
  if (a.head_dim <= 96) return launch<Head<128, 6, 3>>(sp, p, stream);
  return launch<Head<128, 8, 4>>(sp, p, stream);
}

}  // namespace svdq
