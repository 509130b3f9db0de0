"""Refusals of the operators around the linears: by the C ABI (status codes, nothing is
launched) and by the binding (tensors that do not match); CPU only."""
import ctypes

import numpy as np
import pytest

from oracle import block_oracle as B

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_binding_checks import g  # noqa: E402  host tensors that claim a GPU device

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
P = 1 << 20          # a plausible device address; never dereferenced on a refusal


def attention(**over):
    a = dict(Q=P, ldq=512, K=P, ldk=128, V=P, ldv=128, cu_q=P, cu_k=P, batch=2, total_q=100, total_k=4000, heads_q=8,
             heads_kv=2, head_dim=64, scale=0.125, causal=1, O=P, ldo=512, lse=None, workspace=P, bytes=1 << 30)
    a.update(over)
    return S._lib.svdq_attention_forward(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID),
    (dict(total_q=1 << 31), INVALID), (dict(total_k=1 << 31), INVALID),
    (dict(total_q=1 << 29), INVALID),                          # x 4 heads of a group: beyond 31 bits
    (dict(heads_kv=0), INVALID), (dict(heads_q=7), INVALID), (dict(heads_q=0), INVALID),
    (dict(heads_q=1), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), INVALID),
    (dict(head_dim=136, ldq=2048, ldk=512, ldv=512, ldo=2048), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=2.0**127), INVALID), (dict(causal=2), INVALID),
    (dict(ldq=504), INVALID), (dict(ldq=516), INVALID), (dict(ldk=120), INVALID), (dict(ldv=129), INVALID),
    (dict(ldo=256), INVALID), (dict(ldk=(1 << 24) + 8), UNSUPPORTED), (dict(ldv=1 << 30), UNSUPPORTED),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(O=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID),
    (dict(Q=P + 2), ALIGNMENT), (dict(K=P + 8), ALIGNMENT), (dict(V=P + 8), ALIGNMENT), (dict(O=P + 4), ALIGNMENT),
    (dict(cu_q=P + 2), ALIGNMENT), (dict(lse=P + 1), ALIGNMENT),
    (dict(workspace=None), INVALID), (dict(workspace=P + 8), ALIGNMENT), (dict(bytes=16), WORKSPACE),
])
def test_attention_refusals(over, status):
    assert attention(**over) == status
    assert S.svdq_last_error()


def test_attention_of_no_rows_does_nothing():
    assert attention(total_q=0, Q=None, O=None, workspace=None, bytes=0) == 0


def test_attention_workspace():
    assert S.svdq_attention_workspace_bytes(100, 4000, 2, 8, 2, 64) > 0
    assert S.svdq_attention_workspace_bytes(100000, 100000, 2, 8, 2, 64) == 0     # tiles enough
    assert S.svdq_attention_workspace_bytes(100, 4000, 2, 8, 3, 64) == 0          # rejected
    for batch in (1, 2, 7, 64, 1000):
        for tq in (1, 64, 1000, 20000):
            for tk in (1, 1000, 200000):
                for hq, hkv in ((1, 1), (32, 8), (24, 24), (64, 1)):
                    n = S.svdq_attention_workspace_bytes(max(tq, batch), tk, batch, hq, hkv, 128)
                    assert n <= 64 << 20, (batch, tq, tk, hq, hkv)


def heads(T, H, D, device="cuda:0", dtype=torch.bfloat16):
    return g((T, H, D), dtype, device)


@pytest.mark.parametrize("over,err", [
    (dict(Q=heads(10, 4, 64, "cpu")), "must live on the GPU"),
    (dict(Q=heads(10, 4, 64, dtype=torch.float16)), "Q must have dtype"),
    (dict(Q=g((10, 256), torch.bfloat16)), "Q must have shape"),
    (dict(K=heads(10, 2, 32)), "K must have shape"),
    (dict(V=heads(11, 2, 64)), "V must have shape"),
    (dict(O=heads(10, 2, 64)), "O must have shape"),
    (dict(cu_q=g((3,), torch.int64)), "cu_q must have dtype"),
    (dict(cu_q=g((1,), torch.int32)), "cu_q must hold"),
    (dict(cu_k=g((4,), torch.int32)), "cu_k must hold"),
    (dict(cu_k=None), "must both be given"),
    (dict(lse=g((10, 4), torch.float32)), "lse must have shape"),
    (dict(O=heads(10, 4, 64, "cuda:1")), "different devices"),
])
def test_attention_binding_checks(over, err):
    a = dict(Q=heads(10, 4, 64), K=heads(10, 2, 64), V=heads(10, 2, 64), cu_q=g((3,), torch.int32),
             cu_k=g((3,), torch.int32), scale=0.125, causal=False, O=heads(10, 4, 64), lse=None, workspace=None)
    a.update(over)
    with pytest.raises(ValueError, match=err):
        S.svdq_attention_forward(*a.values())


def test_attention_binding_wants_contiguous_heads():
    from tests.test_binding_checks import OnGpu
    q = OnGpu(torch.zeros(4, 10, 64, dtype=torch.bfloat16).transpose(0, 1))
    with pytest.raises(ValueError, match="heads of a row"):
        S.svdq_attention_forward(q, heads(10, 2, 64), heads(10, 2, 64), None, None, 0.125, False, heads(10, 4, 64))


# ------------------------------------------------------------------ the oracle against torch
@pytest.mark.parametrize("causal", [False, True])
def test_oracle_attention_against_torch(causal):
    rng = np.random.default_rng(1)
    Q, K, V = rng.normal(size=(5, 4, 8)), rng.normal(size=(7, 2, 8)), rng.normal(size=(7, 2, 8))
    O, lse, _ = B.attention(Q, K, V, [0, 5], [0, 7], 0.3, causal)
    q = torch.from_numpy(Q).transpose(0, 1)
    k = torch.from_numpy(K).repeat_interleave(2, 1).transpose(0, 1)
    v = torch.from_numpy(V).repeat_interleave(2, 1).transpose(0, 1)
    mask = torch.ones(5, 7, dtype=torch.bool).tril(2) if causal else None
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask, scale=0.3)[0]
    np.testing.assert_allclose(O, want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    s = 0.3 * q @ k.transpose(1, 2)
    if causal:
        s = s.masked_fill(~mask, -np.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), rtol=1e-12)


# ------------------------------------------------------------------ block norm
def norm(**over):
    a = dict(x=P, dtype=0, y=P, rows=10, width=64, cu=P, batch=2, post=1, post_weight=P, gate=P, ld_gate=64,
             residual_scale=1.0, branch_scale=1.0, pre=2, pre_weight=P, pre_bias=P, scale=P, ld_scale=64, shift=P,
             ld_shift=64, eps=1e-6, x_out=P, h=P)
    a.update(over)
    return S._lib.svdq_block_norm_forward(*a.values(), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 24), INVALID), (dict(width=0), INVALID), (dict(width=60), INVALID),
    (dict(width=16392, ld_gate=16392, ld_scale=16392, ld_shift=16392), INVALID),
    (dict(batch=0), INVALID), (dict(cu=None), INVALID), (dict(cu=P + 2), ALIGNMENT), (dict(dtype=2), INVALID),
    (dict(post=3), INVALID), (dict(pre=-1), INVALID), (dict(y=None), INVALID),
    (dict(y=None, post=0), INVALID), (dict(y=None, post=0, post_weight=None), INVALID),
    (dict(h=None), INVALID), (dict(h=None, pre=0, pre_weight=None, pre_bias=None, scale=None), INVALID),
    (dict(x_out=None, h=None, pre=0, pre_weight=None, pre_bias=None, scale=None, shift=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(residual_scale=NAN), INVALID), (dict(branch_scale=INF), INVALID),
    (dict(ld_gate=56), INVALID), (dict(ld_scale=68), INVALID), (dict(ld_shift=0), INVALID),
    (dict(x=None), INVALID), (dict(x=P + 8), ALIGNMENT), (dict(y=P + 8), ALIGNMENT), (dict(gate=P + 2), ALIGNMENT),
    (dict(pre_weight=P + 4), ALIGNMENT), (dict(x_out=P + 8), ALIGNMENT), (dict(h=P + 8), ALIGNMENT),
])
def test_norm_refusals(over, status):
    assert norm(**over) == status


def test_norm_of_no_rows_does_nothing():
    assert norm(rows=0) == 0


@pytest.mark.parametrize("over,err", [
    (dict(x=g((10, 64), torch.float16)), "x must have dtype"), (dict(x=g((640,), torch.bfloat16)), "x must be a"),
    (dict(y=g((10, 72), torch.bfloat16)), "y must have shape"), (dict(y=g((10, 64), torch.float32)), "y must have dtype"),
    (dict(x_out=g((10, 64), torch.float32)), "x_out must have dtype"), (dict(h=g((9, 64), torch.bfloat16)), "h must have"),
    (dict(gate=g((3, 64), torch.bfloat16)), "gate must have shape"), (dict(scale=g((64,), torch.bfloat16)), "scale must"),
    (dict(pre_weight=g((2, 64), torch.bfloat16)), "pre_weight must have shape"),
    (dict(cu=g((3,), torch.int64)), "cu must have dtype"), (dict(h=g((10, 64), torch.bfloat16, "cuda:1")), "different"),
])
def test_norm_binding_checks(over, err):
    bf = torch.bfloat16
    a = dict(x=g((10, 64), bf), y=g((10, 64), bf), cu=g((3,), torch.int32), post=1, post_weight=g((64,), bf),
             gate=g((2, 64), bf), rs=1.0, bs=1.0, pre=2, pre_weight=g((64,), bf), pre_bias=None, scale=g((2, 64), bf),
             shift=g((2, 64), bf), eps=1e-6, x_out=g((10, 64), bf), h=g((10, 64), bf))
    a.update(over)
    with pytest.raises(ValueError, match=err):
        S.svdq_block_norm_forward(*a.values())


# ------------------------------------------------------------------ 16-bit linear
def linear(**over):
    a = dict(X=P, M=100, K=2048, N=64, W=P, bias=P, act=2, residual=P, Y=P, dtype=0, workspace=P, bytes=1 << 30)
    a.update(over)
    return S._lib.svdq_linear_bf16_forward(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(M=1 << 31), INVALID), (dict(K=0), INVALID), (dict(K=12), INVALID), (dict(N=0), INVALID),
    (dict(M=(1 << 31) - 1024, N=(1 << 31) - 1024), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID),
    (dict(X=P + 8), ALIGNMENT), (dict(W=P + 8), ALIGNMENT), (dict(bias=P + 2), ALIGNMENT), (dict(Y=P + 2), ALIGNMENT),
    (dict(residual=P + 8), ALIGNMENT), (dict(workspace=None), INVALID), (dict(bytes=100), WORKSPACE),
])
def test_linear_refusals(over, status):
    assert S.svdq_linear_bf16_workspace_bytes(100, 2048, 64) > 100
    assert linear(**over) == status


def test_linear_of_no_rows_does_nothing():
    assert linear(M=0, X=None, Y=None, workspace=None) == 0


def test_linear_workspace_is_bounded():
    for M in (1, 65, 500, 1155, 3000, 20000):
        for K in (8, 1288, 16384):
            for N in (1, 640, 1290, 4096, 20000):
                assert S.svdq_linear_bf16_workspace_bytes(M, K, N) <= 64 << 20


def test_silu_is_not_an_activation_of_the_quantized_forward():
    assert S._lib.svdq_linear_forward_act(P, 32, 64, 16, 0, P, None, None, P, P, None, 2, P, P, 1 << 30, None) == INVALID


@pytest.mark.parametrize("over,err", [
    (dict(W=g((64, 120), torch.bfloat16)), "W must have shape"), (dict(bias=g((10,), torch.bfloat16)), "bias must have"),
    (dict(Y=g((10, 32), torch.bfloat16)), "Y must have shape"), (dict(X=g((10, 128), torch.float32)), "X must have dtype"),
    (dict(residual=g((10, 64), torch.float32)), "residual must have dtype"),
    (dict(Y=g((10, 64), torch.bfloat16, "cuda:1")), "different"),
])
def test_linear_binding_checks(over, err):
    bf = torch.bfloat16
    a = dict(X=g((10, 128), bf), W=g((64, 128), bf), bias=g((64,), bf), act=0, residual=g((10, 64), bf), Y=g((10, 64), bf))
    a.update(over)
    with pytest.raises(ValueError, match=err):
        S.svdq_linear_bf16_forward(*a.values())


def test_operands_that_are_no_tensors_are_named():
    bf = torch.bfloat16
    q, x, cu = heads(10, 4, 64), g((10, 64), bf), [0, 10]
    with pytest.raises(TypeError, match="cu_q must be a torch tensor"):
        S.svdq_attention_forward(q, q, q, cu, cu, 0.125, False, q)
    with pytest.raises(TypeError, match="Q must be a torch tensor"):
        S.svdq_attention_forward(np.zeros((10, 4, 64)), q, q, None, None, 0.125, False, q)
    with pytest.raises(TypeError, match="workspace must be a torch tensor"):
        S.svdq_attention_forward(q, q, q, None, None, 0.125, False, q, None, 1 << 20)
    for over, name in ((dict(x=1.0), "x"), (dict(cu=cu), "cu"), (dict(gate=1.0), "gate"), (dict(h=np.zeros((10, 64))), "h")):
        a = dict(x=x, y=x, cu=None, post=0, w=None, gate=None, rs=1.0, bs=1.0, pre=2, pw=None, pb=None, scale=None,
                 shift=None, eps=1e-6, x_out=x, h=x)
        a.update(over)
        with pytest.raises(TypeError, match=f"{name} must be a torch tensor"):
            S.svdq_block_norm_forward(*a.values())
    for i, name in ((0, "X"), (2, "bias"), (5, "Y")):
        a = [x, g((16, 64), bf), None, 0, None, g((10, 16), bf)]
        a[i] = np.zeros((10, 64))
        with pytest.raises(TypeError, match=f"{name} must be a torch tensor"):
            S.svdq_linear_bf16_forward(*a)


# ------------------------------------------------------------------ oracles against torch
def test_oracle_norm_and_linear_against_torch():
    rng = np.random.default_rng(2)
    x, y, w, b = rng.normal(size=(6, 16)), rng.normal(size=(6, 16)), rng.normal(size=16), rng.normal(size=16)
    gate, scale, shift = (rng.normal(size=(2, 16)) for _ in range(3))
    T = torch.from_numpy
    for pre in ("layer", "rms"):
        xo, h = B.block_norm(x, y, [0, 2, 6], "rms", w, gate, 0.5, 2.0, pre, w, b, scale, shift, 1e-5)
        at = [0, 0, 1, 1, 1, 1]
        want = 0.5 * T(x) + 2.0 * T(gate[at]) * torch.nn.functional.rms_norm(T(y), (16,), T(w), 1e-5)
        np.testing.assert_allclose(xo, want.numpy(), rtol=1e-12, atol=1e-12)
        n = (torch.nn.functional.layer_norm(want, (16,), None, None, 1e-5) if pre == "layer"
             else torch.nn.functional.rms_norm(want, (16,), None, 1e-5)) * T(w) + T(b)
        np.testing.assert_allclose(h, (n * (1 + T(scale[at])) + T(shift[at])).numpy(), rtol=1e-11, atol=1e-11)
    X, W = rng.normal(size=(3, 16)), rng.normal(size=(5, 16))
    z = T(X) @ T(W).t() + T(b[:5])
    np.testing.assert_allclose(B.linear(X, W, b[:5], "gelu", x[:3, :5]),
                               (torch.nn.functional.gelu(z, approximate="tanh") + T(x[:3, :5])).numpy(), rtol=1e-12)
    np.testing.assert_allclose(B.linear(X, W, b[:5], "silu", None), torch.nn.functional.silu(z).numpy(), rtol=1e-12)
