"""Refusals of the norm and rotation of queries and keys, by the C ABI and by the binding, and the oracle that
the GPU tests use; CPU only."""
import numpy as np
import pytest

from oracle import block_oracle as B

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_binding_checks import g  # noqa: E402  host tensors that claim a GPU device
from tests.test_block_ops_host import heads  # noqa: E402

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
P = 1 << 20          # a plausible device address; never dereferenced on a refusal
NAN, INF = float("nan"), float("inf")


def rope(**over):
    a = dict(Q=P, ldq=512, K=P, ldk=128, rows=10, heads_q=8, heads_k=2, head_dim=64, cu=P, batch=2, positions=P, norm=1,
             qw=P, qb=P, kw=P, kb=P, eps=1e-6, cos=P, sin=P, ld_table=32, table_rows=100, rotary_dim=64, pairs=1, Qo=P,
             ldqo=512, Ko=P, ldko=128)
    a.update(over)
    return S._lib.svdq_qk_norm_rope_forward(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(heads_q=-1), INVALID), (dict(heads_k=-1), INVALID),
    (dict(heads_q=(1 << 20) + 1), INVALID), (dict(heads_q=0), INVALID), (dict(heads_k=0), INVALID),
    (dict(heads_q=0, heads_k=0, Q=None, K=None, Qo=None, Ko=None, qw=None, qb=None, kw=None, kb=None), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=60), INVALID), (dict(head_dim=264, ldq=4096, ldk=4096), UNSUPPORTED),
    (dict(batch=0), INVALID), (dict(cu=None), INVALID), (dict(norm=3), INVALID), (dict(norm=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(rotary_dim=-8), INVALID),
    (dict(rotary_dim=12), INVALID), (dict(rotary_dim=72, ld_table=36), INVALID), (dict(rotary_dim=0), INVALID),
    (dict(pairs=2), INVALID), (dict(pairs=-1), INVALID), (dict(table_rows=-1), INVALID), (dict(ld_table=28), INVALID),
    (dict(ld_table=34), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID), (dict(cos=P + 8), ALIGNMENT),
    (dict(sin=P + 4), ALIGNMENT), (dict(ldq=504), INVALID), (dict(ldq=516), INVALID), (dict(ldk=120), INVALID),
    (dict(ldqo=1024), INVALID), (dict(ldko=136), INVALID),                     # in place with other strides
    (dict(Qo=P + 4096, ldqo=256), INVALID), (dict(Ko=P + 4096, ldko=129), INVALID),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(Qo=None), INVALID), (dict(Ko=None), INVALID),
    (dict(Q=P + 8), ALIGNMENT), (dict(K=P + 2), ALIGNMENT), (dict(Qo=P + 8), ALIGNMENT), (dict(Ko=P + 8), ALIGNMENT),
    (dict(qw=P + 8), ALIGNMENT), (dict(qb=P + 2), ALIGNMENT), (dict(kw=P + 4), ALIGNMENT), (dict(kb=P + 8), ALIGNMENT),
    (dict(cu=P + 2), ALIGNMENT), (dict(positions=P + 1), ALIGNMENT),
    (dict(rows=(1 << 31) - 1, heads_q=1 << 20, ldq=1 << 26, ldqo=1 << 26), INVALID),      # more than one launch
])
def test_refusals(over, status):
    assert rope(**over) == status
    assert S.svdq_last_error()


def test_of_no_rows_does_nothing():
    assert rope(rows=0, Q=None, K=None, Qo=None, Ko=None, cos=None, sin=None, positions=None) == OK


def call(**over):
    bf = torch.bfloat16
    a = dict(Q=heads(10, 4, 64), K=heads(10, 2, 64), cu=g((3,), torch.int32), positions=None, norm=1, qw=g((64,), bf),
             qb=None, kw=g((64,), bf), kb=None, eps=1e-6, cos=g((20, 32), torch.float32), sin=g((20, 32), torch.float32),
             pairs=1, Qo=heads(10, 4, 64), Ko=heads(10, 2, 64))
    a.update(over)
    S.svdq_qk_norm_rope_forward(*a.values())


@pytest.mark.parametrize("over,err", [
    (dict(Q=None, K=None), "both None"), (dict(Q=heads(10, 4, 64, "cpu")), "must live on the GPU"),
    (dict(Q=g((10, 256), torch.bfloat16)), "Q must have shape"), (dict(K=heads(9, 2, 64)), "K must have shape"),
    (dict(K=heads(10, 2, 32)), "K must have shape"), (dict(Qo=heads(10, 2, 64)), "Q_out must have shape"),
    (dict(Ko=heads(10, 2, 64, dtype=torch.float16)), "K_out must have dtype"), (dict(Qo=None), "Q_out must not be None"),
    (dict(Ko=None), "K_out must not be None"), (dict(qw=g((32,), torch.bfloat16)), "q_weight must have shape"),
    (dict(kb=g((64,), torch.float32)), "k_bias must have dtype"), (dict(positions=g((10,), torch.int64)), "positions must have dtype"),
    (dict(positions=g((9,), torch.int32)), "positions must have shape"), (dict(cu=g((3,), torch.int64)), "cu must have dtype"),
    (dict(cu=g((1,), torch.int32)), "cu must hold"), (dict(cos=None), "must both be given"), (dict(sin=None), "must both be given"),
    (dict(cos=g((20, 32), torch.float64)), "dtype float32"), (dict(sin=g((21, 32), torch.float32)), "alike"),
    (dict(cos=g((20,), torch.float32)), "alike"),
])
def test_binding_checks(over, err):
    with pytest.raises(ValueError, match=err):
        call(**over)


@pytest.mark.parametrize("over,name", [(dict(Q=np.zeros((10, 4, 64))), "Q"), (dict(cos=np.zeros((20, 32)), sin=np.zeros((20, 32))), "cos"),
                                       (dict(cu=[0, 10]), "cu"), (dict(positions=[1] * 10), "positions")])
def test_operands_that_are_no_tensors_are_named(over, name):
    with pytest.raises(TypeError, match=f"^{name} must be a torch tensor"):
        call(**over)


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("halves", [False, True])
def test_oracle_turns_pairs_as_complex_numbers(halves):
    rng = np.random.default_rng(3)
    v, w, b = rng.normal(size=(7, 2, 16)), rng.normal(size=16), rng.normal(size=16)
    angle = rng.normal(size=(5, 4))
    out, n, _, _ = B.qk_norm_rope(v, [0, 2, 7], None, "rms", w, b, 1e-5, np.cos(angle), np.sin(angle), halves)
    want = torch.nn.functional.rms_norm(torch.from_numpy(v), (16,), torch.from_numpy(w), 1e-5).numpy() + b
    at = [0, 1, 0, 1, 2, 3, 4]
    x, y = (want[..., :4], want[..., 4:8]) if halves else (want[..., 0:8:2], want[..., 1:8:2])
    z = (x + 1j * y) * np.exp(1j * angle[at])[:, None]
    turned = np.concatenate([z.real, z.imag], -1) if halves else np.stack([z.real, z.imag], -1).reshape(7, 2, 8)
    np.testing.assert_allclose(out, np.concatenate([turned, want[..., 8:]], -1), rtol=1e-12, atol=1e-12)


def test_oracle_rotation_depends_on_the_distance_alone():
    """q at p and k at s: their product is one of p - s."""
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))
    angle = np.arange(50)[:, None] * np.array([1.0, 0.3, 0.1, 0.01])
    dots = []
    for p, s in ((3, 1), (40, 38), (49, 47)):
        t = [B.qk_norm_rope(v, [0, 1], np.array([at]), "none", None, None, 0.0, np.cos(angle), np.sin(angle), True)[0]
             for v, at in ((q, p), (k, s))]
        dots.append(float((t[0] * t[1]).sum()))
    np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
    out = B.qk_norm_rope(q, [0, 1], np.array([50]), "none", None, None, 0.0, np.cos(angle), np.sin(angle), True)[0]
    np.testing.assert_array_equal(out, q)
