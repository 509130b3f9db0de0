"""Norm and rotation of queries and keys, then attention over a window or behind a shared prefix, as a
model runs them: on a fused QKV projection of an SVDQuant linear, in place, and for new tokens against
what earlier calls left behind.  Every link is checked against the float64 oracle on what the GPU chain
fed it, within the operator's own derived tolerance; graphs replay the eager chain's bits."""
import numpy as np
import pytest

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, cu_dev, draw, f64, offsets  # noqa: E402
from test_gpu_attention_spans import check as check_spans  # noqa: E402
from test_gpu_block_chain import Svdq  # noqa: E402
from test_gpu_qk_norm_rope import check as check_rope, tables  # noqa: E402

C, HEADS, D, EPS = 384, 6, 64, 1e-6


class Layer:
    """Packed images: QKV (SVDQuant, int4 or MXFP4), norm and rotation in place, attention of each token to
    its neighbours and the first tokens."""

    def __init__(self, lens, mx):
        self.cu, self.lens = offsets(lens), lens
        T = int(self.cu[-1])
        self.cud = cu_dev(self.cu)
        self.h = draw((T, C), 1)
        self.qkv = Svdq(T, C, 3 * C, 61, S.SVDQ_ACT_NONE, mx)
        self.wq, self.wk = draw((D,), 2, 0.2) + 1, draw((D,), 3, 0.2) + 1
        self.cos, self.sin = tables(max(lens), D)
        self.a = torch.full((T, HEADS, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((HEADS, T), float("nan"), device=DEV)
        self.window = (90, 70, 5)
        n = S.svdq_attention_window_workspace_bytes(T, T, len(lens), HEADS, HEADS, D, False, *self.window)
        self.ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def heads(self):
        v = self.qkv.Y.unflatten(1, (3 * HEADS, D))
        return v[:, :HEADS], v[:, HEADS:2 * HEADS], v[:, 2 * HEADS:]

    def project(self):
        self.qkv(self.h)

    def rest(self):
        q, k, v = self.heads()
        S.svdq_qk_norm_rope_forward(q, k, self.cud, None, S.SVDQ_NORM_RMS, self.wq, None, self.wk, None, EPS, self.cos,
                                    self.sin, S.SVDQ_ROPE_HALVES, q, k)
        S.svdq_attention_window_forward(q, k, v, self.cud, self.cud, D**-0.5, False, *self.window, self.a, self.lse, self.ws)


@pytest.mark.parametrize("mx", [False, True], ids=["int4", "mxfp4"])
def test_every_link_of_a_layer(mx):
    m = Layer([77, 0, 300, 180], mx)
    m.project()
    raw = [t.clone() for t in m.heads()]
    m.qkv.check(m.h, "qkv")
    m.rest()
    torch.cuda.synchronize()
    q, k, v = m.heads()
    check_rope(q, raw[0], m.cu, None, "rms", m.wq, None, EPS, m.cos, m.sin, True)
    check_rope(k, raw[1], m.cu, None, "rms", m.wk, None, EPS, m.cos, m.sin, True)
    assert torch.equal(v, raw[2])
    check_spans(m.a, m.lse, q, k, v, m.cu, m.cu, D**-0.5, False, *m.window)


def test_a_layer_captured_and_replayed():
    """New inputs and other lengths of the images between the replays, with eager work."""
    m = Layer([77, 0, 300, 180], False)
    m.project(), m.rest()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.project(), m.rest()
    for i in range(3):
        m.h.copy_(draw(m.h.shape, 20 + i))
        m.cud[1] = 77 - 20 * i
        m.project(), m.rest()
        torch.cuda.synchronize()
        want = [t.clone() for t in (m.qkv.Y, m.a, m.lse)]
        for t in (m.a, m.lse, m.qkv.Y):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((m.qkv.Y, m.a, m.lse), want))
        assert not torch.isnan(m.a).any()


def test_new_tokens_behind_a_shared_prefix():
    """A prompt's keys are normalised and rotated once; sequences that continue it add a token each step,
    at its position, to keys of their own, and attend to both.  The steps one by one give what one call
    over each whole sequence gives, to the two calls' tolerances."""
    hq, hkv, d, P, n, steps, scale = 8, 2, 128, 1500, 6, 4, 128**-0.5
    cos, sin = tables(P + steps, d)
    raw = draw((P, 2 * hkv, d), 1)
    pk, pv = torch.empty(P, hkv, d, dtype=torch.bfloat16, device=DEV), raw[:, hkv:]
    wq, wk = draw((d,), 2, 0.2) + 1, draw((d,), 3, 0.2) + 1

    def rope(Q, K, positions, Qo, Ko):
        S.svdq_qk_norm_rope_forward(Q, K, None, positions, S.SVDQ_NORM_RMS, wq if Q is not None else None, None,
                                    wk, None, EPS, cos, sin, S.SVDQ_ROPE_NEIGHBOURS, Qo, Ko)

    rope(None, raw[:, :hkv], None, None, pk)
    check_rope(pk, raw[:, :hkv], [0, P], None, "rms", wk, None, EPS, cos, sin, False)
    # sequence b's keys are rows [b steps, b steps + t) after t steps
    K, V = (torch.empty(n * steps, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qs, outs = [], []
    for t in range(steps):
        qkv = draw((n, hq + 2 * hkv, d), 10 + t)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        at = torch.full((n,), P + t, dtype=torch.int32, device=DEV)
        before = q.clone(), k.clone()
        rope(q, k, at, q, k)
        for got, was, w in ((q, before[0], wq), (k, before[1], wk)):
            check_rope(got, was, [0, n], at, "rms", w, None, EPS, cos, sin, False)
        rows = torch.arange(n, device=DEV) * steps + t
        K[rows], V[rows] = k, v
        # the sequences' keys so far, behind each other
        have = torch.cat([torch.arange(b * steps, b * steps + t + 1) for b in range(n)]).to(DEV)
        Kt, Vt = K[have].contiguous(), V[have].contiguous()
        cu_q, cu_k = np.arange(n + 1), np.arange(n + 1) * (t + 1)
        O, lse = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(hq, n, device=DEV)
        ws = torch.full((max(S.svdq_attention_prefix_workspace_bytes(n, P, len(have), n, hq, hkv, d, True), 16),), 0xFF,
                        dtype=torch.uint8, device=DEV)
        S.svdq_attention_prefix_forward(q, pk, pv, Kt, Vt, cu_dev(cu_q), cu_dev(cu_k), scale, True, O, lse, ws)
        torch.cuda.synchronize()
        check_spans(O, lse, q, Kt, Vt, cu_q, cu_k, scale, True, PK=pk, PV=pv)
        qs.append(q)
        outs.append(O)
    # all steps at once, causal: query t of a sequence sees its keys up to its own
    Q = torch.stack(qs, 1).flatten(0, 1).contiguous()
    cu = np.arange(n + 1) * steps
    O, lse = torch.empty_like(Q), torch.empty(hq, n * steps, device=DEV)
    ws = torch.full((max(S.svdq_attention_prefix_workspace_bytes(n * steps, P, n * steps, n, hq, hkv, d, True), 16),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    S.svdq_attention_prefix_forward(Q, pk, pv, K, V, cu_dev(cu), cu_dev(cu), scale, True, O, lse, ws)
    torch.cuda.synchronize()
    check_spans(O, lse, Q, K, V, cu, cu, scale, True, PK=pk, PV=pv)
    _, _, A, M = B.attention_spans(f64(Q), f64(K), f64(V), cu, cu, scale, True, PK=f64(pk), PV=f64(pv))
    single = f64(torch.stack(outs, 1).flatten(0, 1))
    ds = (scale * (d + 8) * 2.0**-24 * M).T[..., None]
    tol = 2 * (A * (2.0**-8 + 2 * ds + 2.0**-17 + (P + steps) * 2.0**-24) + 2.0**-8 * np.abs(single) * 1.01)
    assert np.all(np.abs(single - f64(O)) <= tol)


def test_a_rolling_window_over_a_cache():
    """New tokens with a window and first tokens: a cache that has given up the keys between (they hold NaN
    by then) serves the same outputs, bit for bit, as one that still has them."""
    hq, hkv, d, n, nk, scale = 8, 2, 64, 3, 900, 0.125
    K, V = draw((n * nk, hkv, d), 1), draw((n * nk, hkv, d), 2)
    cu_q, cu_k = np.arange(n + 1), np.arange(n + 1) * nk
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    for t, last in enumerate((600, 700, 899)):
        q = draw((n, hq, d), 10 + t)
        cu = cu_k.copy()
        ends = np.minimum(cu[1:], cu[:-1] + last + 1)
        outs = []
        for gone in (False, True):
            k, v = K.clone(), V.clone()
            if gone:
                for b in range(n):
                    k[cu[b] + 4:ends[b] - 256], v[cu[b] + 4:ends[b] - 256] = float("nan"), float("nan")
            O, lse = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(hq, n, device=DEV)
            have = torch.cat([torch.arange(cu[b], ends[b]) for b in range(n)]).to(DEV)
            kk, vv, off = k[have].contiguous(), v[have].contiguous(), np.arange(n + 1) * (last + 1)
            S.svdq_attention_window_forward(q, kk, vv, cu_dev(cu_q), cu_dev(off), scale, True, 255, 0, 4, O, lse, ws)
            torch.cuda.synchronize()
            check_spans(O, lse, q, kk, vv, cu_q, off, scale, True, 255, 0, 4)
            outs.append((O, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
