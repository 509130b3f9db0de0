// svdq_attention_forward: softmax attention of packed sequences over their keys.  The kernels, their
// arithmetic and the choice between them are in attention_core.h.
#include "attention_core.h"

namespace svdq {
namespace {

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

template <class H>
hipError_t launch(const Plan& pl, const Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)(pl.tiles * p.heads_kv * pl.splits));
  if (pl.keys) {
    constexpr int kWaves = key_waves(H::DP);
    if (pl.parts == 2)
      hipLaunchKernelGGL((attention_keys<H, kWaves, 2, false>), grid, dim3(kWaves * 64), 0, stream, p);
    else
      hipLaunchKernelGGL((attention_keys<H, kWaves, 1, false>), grid, dim3(kWaves * 64), 0, stream, p);
  } else if (pl.waves == 8) {
    if constexpr (H::DP == 128)
      hipLaunchKernelGGL((attention_rows<H, 8, false>), grid, dim3(512), 0, stream, p);
  } else {
    hipLaunchKernelGGL((attention_rows<H, 4, false>), grid, dim3(256), 0, stream, p);
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
