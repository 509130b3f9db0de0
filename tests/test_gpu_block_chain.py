"""A whole transformer block on the GPU, as a denoiser runs it: the conditioning
vectors through a SiLU linear and the modulation linear, then norm + modulation ->
QKV (SVDQuant) -> attention on the QKV output's column slices -> out (SVDQuant) ->
gate, residual, norm and modulation in one call -> up + GELU -> down (SVDQuant) ->
gate and residual, over packed images of unequal size, one of them empty.

4-bit codes jump where a value crosses the border between two of them, so the ends
of two chains say little about each other.  Every link is checked instead: each
operator's output against the float64 oracle on what the GPU chain fed it, within
the operator's own derived tolerance (the SVDQuant linears: relative Frobenius error
5e-3 and 1e-2 of the maximum, as everywhere).  Equal inputs give equal bits, so the
graph's replays must equal the eager chain.
"""
import numpy as np
import pytest

import synth
from oracle import svdq_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import check as check_attention, cu_dev, draw, f64, offsets  # noqa: E402
from test_gpu_block import layer_to_device, oracle_linear  # noqa: E402
from test_gpu_block_norm import check as check_norm  # noqa: E402
from test_gpu_linear_bf16 import check as check_linear  # noqa: E402
from test_gpu_parity import DEV, check_y, host  # noqa: E402

GELU, NONE, LAYER = S.SVDQ_ACT_GELU_TANH, S.SVDQ_NORM_NONE, S.SVDQ_NORM_LAYER
C, HEADS, D, RANK, EPS = 384, 6, 64, 32, 1e-6
LENS = [77, 0, 180]


def bf16_tensor(t):
    """The int16 tensor that the SVDQuant calls take, over the same memory."""
    return t.view(torch.int16)


class Svdq:
    """An SVDQuant linear with its output and workspace."""

    def __init__(self, M, K, N, seed, act, mx):
        g = synth.rng_for("tiny", seed)
        W = (g.standard_normal((N, K)) * K**-0.5).astype(np.float32)
        s = np.exp(g.uniform(-0.5, 0.5, K)).astype(np.float32)
        L1 = O.bf16_from_f64(g.standard_normal((RANK, K)) * 0.05)
        L2 = O.bf16_from_f64(g.standard_normal((N, RANK)) * 0.05)
        b = O.bf16_from_f64(g.standard_normal(N) * 0.1)
        Wq, ws = (O.quantize_residual_mx if mx else O.quantize_residual)(W, s, L1, L2)
        self.p = dict(s=s, L1=L1, L2=L2, Wq=Wq, w_scales=ws, b=b)
        self.d, self.act, self.mx = layer_to_device(self.p), act, mx
        self.Y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        n = (S.svdq_forward_workspace_bytes_mxfp4 if mx else S.svdq_forward_workspace_bytes)(M, K, N, RANK)
        self.ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def __call__(self, X):
        d = self.d
        f = S.svdq_linear_forward_act_mxfp4 if self.mx else S.svdq_linear_forward_act
        f(bf16_tensor(X), d["s"], d["L1"], d["L2"], d["Wq"], d["ws"], d["b"], self.act, bf16_tensor(self.Y), self.ws)
        return self.Y

    def check(self, X, label):
        want = oracle_linear(host(bf16_tensor(X), np.uint16), self.p, self.act, self.mx)
        check_y(f64(self.Y), want, label)


class Block:
    def __init__(self, mx, fp32):
        self.cu = offsets(LENS)
        T, B = int(self.cu[-1]), len(LENS)
        self.cud, self.fp32 = cu_dev(self.cu), fp32
        self.stream = torch.float32 if fp32 else torch.bfloat16
        self.x, self.t = draw((T, C), 1, 2.0).to(self.stream), draw((B, 64), 2)
        self.W1, self.b1 = draw((C, 64), 3, 0.125), draw((C,), 4, 0.1)
        self.W2, self.b2 = draw((6 * C, C), 5, C**-0.5), draw((6 * C,), 6, 0.1)
        self.qkv, self.out = Svdq(T, C, 3 * C, 61, S.SVDQ_ACT_NONE, mx), Svdq(T, C, C, 62, S.SVDQ_ACT_NONE, mx)
        self.up, self.down = Svdq(T, C, 4 * C, 63, GELU, mx), Svdq(T, 4 * C, C, 64, S.SVDQ_ACT_NONE, mx)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.full(shape, float("nan"), dtype=dtype, device=DEV)

        self.e, self.mod = empty(B, C), empty(B, 6 * C)
        self.h1, self.h2, self.a = empty(T, C), empty(T, C), empty(T, HEADS, D)
        self.x1, self.x2 = empty(T, C, dtype=self.stream), empty(T, C, dtype=self.stream)
        self.lse = empty(HEADS, T, dtype=torch.float32)
        # one workspace for all of the block's calls, which follow each other on the stream
        n = max(S.svdq_attention_workspace_bytes(T, T, B, HEADS, HEADS, D),
                S.svdq_linear_bf16_workspace_bytes(B, 64, C), S.svdq_linear_bf16_workspace_bytes(B, C, 6 * C))
        self.ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def heads(self):
        v = self.qkv.Y.unflatten(1, (3 * HEADS, D))
        return v[:, :HEADS], v[:, HEADS:2 * HEADS], v[:, 2 * HEADS:]

    def vectors(self):
        """shift, scale and gate of the attention, then of the MLP."""
        return self.mod.split(C, dim=1)

    def run(self):
        S.svdq_linear_bf16_forward(self.t, self.W1, self.b1, S.SVDQ_ACT_SILU, None, self.e, self.ws)
        S.svdq_linear_bf16_forward(self.e, self.W2, self.b2, S.SVDQ_ACT_NONE, None, self.mod, self.ws)
        sh1, sc1, g1, sh2, sc2, g2 = self.vectors()
        S.svdq_block_norm_forward(self.x, None, self.cud, NONE, None, None, 1.0, 1.0, LAYER, None, None, sc1, sh1,
                                  EPS, None, self.h1)
        self.qkv(self.h1)
        S.svdq_attention_forward(*self.heads(), self.cud, self.cud, D**-0.5, False, self.a, self.lse, self.ws)
        self.out(self.a.flatten(1))
        S.svdq_block_norm_forward(self.x, self.out.Y, self.cud, NONE, None, g1, 1.0, 1.0, LAYER, None, None, sc2, sh2,
                                  EPS, self.x1, self.h2)
        self.down(self.up(self.h2))
        S.svdq_block_norm_forward(self.x1, self.down.Y, self.cud, NONE, None, g2, 1.0, 1.0, NONE, None, None, None,
                                  None, EPS, self.x2, None)

    def check(self):
        torch.cuda.synchronize()
        check_linear(self.e, self.t, self.W1, self.b1, "silu", None, False)
        check_linear(self.mod, self.e, self.W2, self.b2, "none", None, False)
        sh1, sc1, g1, sh2, sc2, g2 = (f64(v) for v in self.vectors())
        x, x1, cu, fp32 = f64(self.x), f64(self.x1), self.cu, self.fp32
        check_norm(None, f64(self.h1), x, None, cu, "none", None, None, 1.0, 1.0, "layer", None, None, sc1, sh1, EPS, fp32)
        self.qkv.check(self.h1, "qkv")
        check_attention(self.a, self.lse, *self.heads(), cu, cu, D**-0.5, False)
        self.out.check(self.a.flatten(1), "out")
        check_norm(x1, f64(self.h2), x, f64(self.out.Y), cu, "none", None, g1, 1.0, 1.0, "layer", None, None, sc2, sh2,
                   EPS, fp32)
        self.up.check(self.h2, "up")
        self.down.check(self.up.Y, "down")
        check_norm(f64(self.x2), None, x1, f64(self.down.Y), cu, "none", None, g2, 1.0, 1.0, "none", None, None, None,
                   None, EPS, fp32)


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("mx", [False, True], ids=["int4", "mxfp4"])
def test_every_link_of_a_block(mx, fp32):
    b = Block(mx, fp32)
    b.run()
    b.check()


@pytest.mark.parametrize("mx", [False, True], ids=["int4", "mxfp4"])
def test_a_block_captured_and_replayed(mx):
    """New inputs and other lengths of the images between the replays, with eager work."""
    b = Block(mx, True)
    b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for i in range(3):
        b.x.copy_(draw(b.x.shape, 20 + i, 2.0))
        b.t.copy_(draw(b.t.shape, 30 + i))
        b.cud[1] = 77 - 20 * i
        b.run()
        torch.cuda.synchronize()
        want = [v.clone() for v in (b.mod, b.h1, b.a, b.lse, b.x1, b.h2, b.x2)]
        for v in (b.mod, b.h1, b.a, b.lse, b.x1, b.h2, b.x2):
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for v, w in zip((b.mod, b.h1, b.a, b.lse, b.x1, b.h2, b.x2), want):
            assert torch.equal(v, w) and not torch.any(torch.isnan(v))
