"""Refusals of windowed attention and of attention over a shared prefix, by the C ABI and by the binding,
their workspaces, and the oracle that the GPU tests use; CPU only."""
import numpy as np
import pytest

from oracle import block_oracle as B

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_binding_checks import g  # noqa: E402  host tensors that claim a GPU device
from tests.test_block_ops_host import heads  # noqa: E402

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20          # a plausible device address; never dereferenced on a refusal
MOST = 2**31 - 1 - 512


def window(**over):
    a = dict(Q=P, ldq=512, K=P, ldk=128, V=P, ldv=128, cu_q=P, cu_k=P, batch=2, total_q=100, total_k=20000, heads_q=8,
             heads_kv=2, head_dim=64, scale=0.125, causal=1, left=9000, right=0, sinks=4, O=P, ldo=512, lse=None,
             workspace=P, bytes=1 << 30)
    a.update(over)
    return S._lib.svdq_attention_window_forward(*a.values(), None)


def prefix(**over):
    a = dict(Q=P, ldq=512, PK=P, ldpk=128, PV=P, ldpv=128, prefix=4000, K=P, ldk=128, V=P, ldv=128, cu_q=P, cu_k=P,
             batch=2, total_q=100, total_k=100, heads_q=8, heads_kv=2, head_dim=64, scale=0.125, causal=1, O=P, ldo=512,
             lse=None, workspace=P, bytes=1 << 30)
    a.update(over)
    return S._lib.svdq_attention_prefix_forward(*a.values(), None)


COMMON = [
    (dict(batch=0), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID), (dict(total_q=1 << 31), INVALID),
    (dict(total_k=MOST + 1), INVALID), (dict(total_q=1 << 29), INVALID), (dict(heads_kv=0), INVALID),
    (dict(heads_q=7), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), INVALID),
    (dict(head_dim=136, ldq=2048, ldk=512, ldv=512, ldo=2048), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=2.0**127), INVALID),
    (dict(causal=2), INVALID), (dict(causal=-1), INVALID), (dict(ldq=504), INVALID), (dict(ldk=120), INVALID),
    (dict(ldv=129), INVALID), (dict(ldo=256), INVALID), (dict(ldk=(1 << 24) + 8), UNSUPPORTED),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(O=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID), (dict(Q=P + 2), ALIGNMENT), (dict(K=P + 8), ALIGNMENT),
    (dict(V=P + 8), ALIGNMENT), (dict(O=P + 4), ALIGNMENT), (dict(cu_q=P + 2), ALIGNMENT), (dict(cu_k=P + 1), ALIGNMENT),
    (dict(lse=P + 1), ALIGNMENT), (dict(workspace=None), INVALID), (dict(workspace=P + 8), ALIGNMENT),
    (dict(bytes=16), WORKSPACE),
]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(left=-2), INVALID), (dict(right=-2), INVALID), (dict(left=-2**31), INVALID), (dict(sinks=-1), INVALID),
])
def test_window_refusals(over, status):
    assert window(**over) == status
    assert S.svdq_last_error()


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(prefix=-1), INVALID), (dict(prefix=MOST + 1), INVALID), (dict(prefix=MOST, total_k=1), INVALID),
    (dict(prefix=1 << 40), INVALID), (dict(ldpk=120), INVALID), (dict(ldpv=132), INVALID),
    (dict(ldpk=(1 << 24) + 8), UNSUPPORTED), (dict(ldpv=1 << 30), UNSUPPORTED), (dict(PK=None), INVALID),
    (dict(PV=None), INVALID), (dict(PK=P + 8), ALIGNMENT), (dict(PV=P + 2), ALIGNMENT),
])
def test_prefix_refusals(over, status):
    assert prefix(**over) == status
    assert S.svdq_last_error()


def test_calls_of_no_rows_do_nothing():
    assert window(total_q=0, Q=None, O=None, workspace=None, bytes=0) == OK
    assert prefix(total_q=0, Q=None, O=None, workspace=None, bytes=0) == OK


def test_workspaces_are_bounded_and_follow_the_sizes():
    for batch in (1, 2, 7, 64, 1000):
        for tq in (1, 64, 1000, 20000):
            for tk in (0, 1, 1000, 200000):
                for hq, hkv in ((1, 1), (32, 8), (24, 24), (64, 1)):
                    for causal in (0, 1):
                        q = max(tq, batch)
                        for left, right, sinks in ((0, 0, 0), (1000, 0, 4), (-1, -1, 0), (100000, 5, 300)):
                            n = S.svdq_attention_window_workspace_bytes(q, tk, batch, hq, hkv, 128, causal, left, right, sinks)
                            assert n <= 64 << 20, (batch, tq, tk, hq, hkv, left)
                        for pre in (0, 1, 500, 100000):
                            n = S.svdq_attention_prefix_workspace_bytes(q, pre, tk, batch, hq, hkv, 128, causal)
                            assert n <= 257 << 20, (batch, tq, tk, hq, hkv, pre)
    # rejected shapes need none
    assert S.svdq_attention_window_workspace_bytes(100, 4000, 2, 8, 3, 64, 1, 10, 0, 0) == 0
    assert S.svdq_attention_window_workspace_bytes(100, 4000, 2, 8, 2, 64, 1, -2, 0, 0) == 0
    assert S.svdq_attention_prefix_workspace_bytes(100, -1, 4000, 2, 8, 2, 64, 1) == 0
    assert S.svdq_attention_prefix_workspace_bytes(100, MOST, 4000, 2, 8, 2, 64, 1) == 0


@pytest.mark.parametrize("keys,n", [(MOST, 1), (2**28, 2**13 - 1)])
def test_the_most_keys_are_taken(keys, n):
    """As far as the workspace or the missing Q: nothing overflows on the way."""
    w = n * 8
    a = dict(heads_q=n, heads_kv=n, head_dim=8, ldq=w, ldk=w, ldv=w, ldo=w, Q=None, batch=1, cu_q=None, cu_k=None)
    assert window(total_k=keys, left=2**31 - 1, right=2**31 - 1, sinks=2**31 - 1, **a) == INVALID
    assert "Q" in S.svdq_last_error()
    assert prefix(prefix=keys, total_k=0, ldpk=w, ldpv=w, **a) == INVALID and "Q" in S.svdq_last_error()


# ------------------------------------------------------------------ binding
def call(f, **over):
    a = dict(Q=heads(10, 4, 64), PK=heads(7, 2, 64), PV=heads(7, 2, 64), K=heads(10, 2, 64), V=heads(10, 2, 64),
             cu_q=g((3,), torch.int32), cu_k=g((3,), torch.int32), O=heads(10, 4, 64), lse=None, workspace=None)
    a.update(over)
    if f == "window":
        S.svdq_attention_window_forward(a["Q"], a["K"], a["V"], a["cu_q"], a["cu_k"], 0.125, False, 3, 0, 1, a["O"],
                                        a["lse"], a["workspace"])
    else:
        S.svdq_attention_prefix_forward(a["Q"], a["PK"], a["PV"], a["K"], a["V"], a["cu_q"], a["cu_k"], 0.125, False,
                                        a["O"], a["lse"], a["workspace"])


@pytest.mark.parametrize("f", ["window", "prefix"])
@pytest.mark.parametrize("over,err", [
    (dict(Q=heads(10, 4, 64, "cpu")), "must live on the GPU"), (dict(Q=g((10, 256), torch.bfloat16)), "Q must have shape"),
    (dict(K=heads(10, 2, 32)), "K must have shape"), (dict(V=heads(11, 2, 64)), "V must have shape"),
    (dict(O=heads(10, 2, 64)), "O must have shape"), (dict(cu_q=g((3,), torch.int64)), "cu_q must have dtype"),
    (dict(cu_k=g((4,), torch.int32)), "cu_k must hold"), (dict(cu_k=None), "must both be given"),
    (dict(lse=g((10, 4), torch.float32)), "lse must have shape"), (dict(O=heads(10, 4, 64, "cuda:1")), "different devices"),
    (dict(Q=None), "Q must not be None"), (dict(K=None), "K must not be None"), (dict(cu_q=g((1,), torch.int32)), "cu_q must"),
])
def test_binding_checks(f, over, err):
    with pytest.raises(ValueError, match=err):
        call(f, **over)


@pytest.mark.parametrize("over,err", [
    (dict(PK=None), "prefix_K must not be None"), (dict(PV=None), "prefix_V must not be None"),
    (dict(PK=heads(7, 3, 64)), "prefix_K must have shape"), (dict(PV=heads(8, 2, 64)), "prefix_V must have shape"),
    (dict(PK=heads(7, 2, 64, dtype=torch.float16)), "prefix_K must have dtype"),
])
def test_prefix_binding_checks(over, err):
    with pytest.raises(ValueError, match=err):
        call("prefix", **over)


def test_operands_that_are_no_tensors_are_named():
    for f, over, name in (("window", dict(cu_q=[0, 10], cu_k=[0, 10]), "cu_q"), ("prefix", dict(PK=np.zeros((7, 2, 64))), "prefix_K"),
                          ("window", dict(workspace=1 << 20), "workspace"), ("prefix", dict(V=np.zeros((10, 2, 64))), "V")):
        with pytest.raises(TypeError, match=f"^{name} must be a torch tensor"):
            call(f, **over)


# ------------------------------------------------------------------ the oracle
def test_oracle_sees_what_the_definition_says():
    for nq, nk in ((5, 9), (9, 5), (4, 4), (3, 0)):
        for causal in (False, True):
            for left, right, sinks in ((0, 0, 0), (2, 1, 2), (-1, 0, 1), (1, -1, 100), (-1, -1, 0)):
                m = B.sees(nq, nk, causal, left, right, sinks)
                for i in range(nq):
                    for j in range(nk):
                        p = i + nk - nq
                        want = ((left < 0 or j >= p - left) and (right < 0 or j <= p + right)) or j < sinks
                        assert m[i, j] == (want and (not causal or j <= p))


@pytest.mark.parametrize("causal", [False, True])
def test_oracle_agrees_with_plain_attention(causal):
    """Without a limit it is attention; a prefix is keys in front of every sequence's own."""
    rng = np.random.default_rng(1)
    Q, K, V = rng.normal(size=(8, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    PK, PV = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8))
    cq, ck = [0, 3, 8], [0, 4, 9]
    O, lse, A, _ = B.attention_spans(Q, K, V, cq, ck, 0.3, causal)
    for got, want in zip((O, lse, A), B.attention(Q, K, V, cq, ck, 0.3, causal)):
        np.testing.assert_allclose(got, want, rtol=1e-12)
    O, lse, A, _ = B.attention_spans(Q, K, V, cq, ck, 0.3, causal, PK=PK, PV=PV)
    K2, V2 = (np.concatenate([p, t[0:4], p, t[4:9]]) for p, t in ((PK, K), (PV, V)))
    for got, want in zip((O, lse, A), B.attention(Q, K2, V2, cq, [0, 7, 15], 0.3, causal)):
        np.testing.assert_allclose(got, want, rtol=1e-12)
