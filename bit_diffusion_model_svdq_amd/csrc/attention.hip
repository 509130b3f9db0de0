// svdq_attention_forward: softmax attention of packed sequences over their keys.  The kernels, their
// arithmetic and the choice between them are in attention_core.h.
#include "attention_core.h"

namespace svdq {
namespace {

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
  hipLaunchKernelGGL((attention_join<false>), jgrid, dim3(256), 0, stream, p, pl.rows);
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
