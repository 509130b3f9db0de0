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
    (dict(scale=float("nan")), INVALID), (dict(causal=2), INVALID),
    (dict(ldq=504), INVALID), (dict(ldq=516), INVALID), (dict(ldk=120), INVALID), (dict(ldv=129), INVALID),
    (dict(ldo=256), INVALID),
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
