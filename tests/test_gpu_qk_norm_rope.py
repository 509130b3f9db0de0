"""svdq_qk_norm_rope_forward on the GPU against the float64 oracle.

Tolerances, element by element: a head's sums run over 8 values per lane and at most 5 steps between lanes,
so the normalised value n carries test_gpu_block_norm's bound `dn` (its depth of 64 holds these); weight and
bias add 2^-22 of the terms' sizes, and so do the products and sums of the rotation, which mixes the errors
dx, dy of a pair to |cos| dx + |sin| dy; the output is rounded to bf16: half a step, 2^-8 of itself.
"""
import numpy as np
import pytest

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_block_norm import DEV, KINDS, draw, f64, norm_tol  # noqa: E402


def check(got, v, cu, positions, kind, w, bias, eps, cos, sin, halves):
    v, w, bias, cos, sin = (None if t is None else f64(t) for t in (v, w, bias, cos, sin))
    pos = None if positions is None else positions.cpu().numpy()
    want, _, c, s = B.qk_norm_rope(v, cu, pos, kind, w, bias, eps, cos, sin, halves)
    rows, H, D = v.shape
    flat = v.reshape(rows * H, D)
    n, dn = norm_tol(flat, kind, eps, np.zeros_like(flat))
    n, dn = n.reshape(v.shape), dn.reshape(v.shape)
    w = 1.0 if w is None else w
    t = n * w + (0.0 if bias is None else bias)
    dt = np.abs(w) * dn + 2.0**-22 * (np.abs(n * w) + np.abs(t))
    tol = dt.copy()
    first, second = B.pairs_of(2 * c.shape[2], halves)
    for a, b in ((first, second), (second, first)):
        tol[..., a] = (np.abs(c) * dt[..., a] + np.abs(s) * dt[..., b]
                       + 2.0**-22 * (np.abs(t[..., a] * c) + np.abs(t[..., b] * s)))
    r = slice(cu[0], cu[-1])
    err = np.abs(f64(got)[r] - want[r])
    bound = (tol + 2.0**-8 * np.abs(want) * 1.01 + 1e-38)[r]
    assert np.all(err <= bound), float(np.nanmax(err / bound))


def tables(n, r, seed=9):
    """Cosines and sines of any angles, rows 4 apart more than they are long."""
    a = torch.randn(n, r // 2, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * 3
    wide = torch.full((2, n, r // 2 + 4 + (-(r // 2)) % 4), float("nan"), device=DEV)
    wide[0, :, :r // 2], wide[1, :, :r // 2] = a.cos().to(DEV), a.sin().to(DEV)
    return wide[0, :, :r // 2], wide[1, :, :r // 2]


class Case:
    def __init__(self, lens, hq, hk, d, r, halves, kind="rms", weight=True, bias=False, given=False, table=None, first=0,
                 behind=0, eps=1e-6, mean=0.0, std=1.0, seed=1, inplace=False):
        self.cu = np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int64)
        rows = int(self.cu[-1]) + behind
        qkv = draw((rows, (hq + 2 * hk) * d + 8), seed, std, mean=mean)
        v = qkv[:, :(hq + 2 * hk) * d].unflatten(1, (hq + 2 * hk, d))
        self.Q, self.K = (v[:, :hq] if hq else None), (v[:, hq:hq + hk] if hk else None)
        table = (max(lens) if table is None else table)
        self.cos, self.sin = tables(table, r) if r else (None, None)
        g = torch.Generator().manual_seed(seed + 7)
        self.positions = (torch.randint(-2, table + 3, (rows,), generator=g, dtype=torch.int32).to(DEV) if given else None)
        vec = lambda i, on, mean: draw((d,), seed + i, 0.2, mean=mean) if on else None  # noqa: E731
        self.w = [vec(2, weight and hq, 1.0), vec(3, weight and hk, 1.0)]
        self.b = [vec(4, bias and hq, 0.0), vec(5, bias and hk, 0.0)]
        self.kind, self.eps, self.halves, self.qkv = kind, eps, halves, qkv
        self.ref = [None if t is None else t.clone() for t in (self.Q, self.K)]
        if inplace:
            self.out = [self.Q, self.K]
        else:
            self.out = [None if t is None else torch.full(t.shape, 7.0, dtype=torch.bfloat16, device=DEV) for t in (self.Q, self.K)]
        self.cud = torch.tensor(self.cu, dtype=torch.int32, device=DEV) if len(lens) > 1 or first or behind else None

    def call(self, stream=None):
        S.svdq_qk_norm_rope_forward(self.Q, self.K, self.cud, self.positions, KINDS[self.kind], self.w[0], self.b[0],
                                    self.w[1], self.b[1], self.eps, self.cos, self.sin,
                                    S.SVDQ_ROPE_HALVES if self.halves else S.SVDQ_ROPE_NEIGHBOURS, *self.out, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        for got, v, w, b in zip(self.out, self.ref, self.w, self.b):
            if v is not None:
                check(got, v, self.cu, self.positions, self.kind, w, b, self.eps, self.cos, self.sin, self.halves)
        return self


@pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])
@pytest.mark.parametrize("d,r", [(8, 8), (16, 8), (24, 24), (40, 40), (40, 16), (64, 64), (72, 40), (80, 80), (96, 32), (128, 128),
                                 (128, 0), (136, 136), (200, 104), (256, 256)])
@pytest.mark.parametrize("hq,hk", [(3, 1), (24, 24)])
def test_head_sizes(d, r, halves, hq, hk):
    Case([3, 1, 6], hq, hk, d, r, halves).call().check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (5, 3), (7, 0), (0, 9), (32, 8), (65, 1), (130, 130)])
@pytest.mark.parametrize("d", [8, 64, 128])
def test_heads(hq, hk, d):
    Case([9, 4], hq, hk, d, d, True).call().check()


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])
def test_norms_weights_and_biases(kind, weight, bias, halves):
    Case([5, 30], 4, 2, 72, 40, halves, kind, weight, bias).call().check()


@pytest.mark.parametrize("lens", [[1], [0, 1], [1] * 16, [70], [5, 0, 0, 130, 1], [2] * 200, [0] * 63 + [3, 1, 0, 4] + [1] * 70], ids=len)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("hq,hk,d", [(2, 1, 16), (10, 10, 64), (32, 8, 128)])
def test_packed_sequences(lens, given, hq, hk, d):
    """Own numbers or given positions, some of them outside of the table; empty sequences, and more than 64."""
    Case(lens, hq, hk, d, d, True, given=given).call().check()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 8), (10, 10, 64), (32, 8, 128)])
def test_rows_outside_stay(hq, hk, d, given):
    c = Case([50, 0, 13], hq, hk, d, d, False, given=given, first=3, behind=9)
    c.qkv[:3], c.qkv[c.cu[-1]:] = float("nan"), float("nan")
    c.call().check()
    for t in c.out:
        assert torch.all(t[:3] == 7) and torch.all(t[c.cu[-1]:] == 7)


@pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])
def test_in_place_leaves_the_rest(halves):
    """Queries and keys of a fused projection's output; its values and what lies behind stay."""
    c = Case([40, 25], 6, 2, 80, 40, halves, inplace=True)
    before = c.qkv.clone()
    c.call().check()
    assert torch.equal(c.qkv[:, 8 * 80:], before[:, 8 * 80:])


def test_short_tables_and_none():
    """Positions past the table's end, an empty table, and no table."""
    Case([90, 3], 4, 2, 64, 64, True, table=20).call().check()
    Case([9], 4, 2, 64, 64, True, table=1).call().check()
    c = Case([9], 4, 2, 64, 64, True, table=1)
    c.cos, c.sin = c.cos[:0], c.sin[:0]
    c.call()
    torch.cuda.synchronize()
    for got, v, w, b in zip(c.out, c.ref, c.w, c.b):
        check(got, v, c.cu, None, "rms", w, b, c.eps, None, None, True)


def test_extreme_positions_are_not_looked_up():
    c = Case([6], 2, 1, 64, 64, True, given=True, table=50)
    c.positions.copy_(torch.tensor([-2**31, 2**31 - 1, -1, 50, 49, 0], dtype=torch.int32))
    c.call().check()


@pytest.mark.parametrize("kind,mean,std,eps", [("layer", 100.0, 1.0, 1e-5), ("rms", 0.0, 1e-3, 1e-6), ("rms", 0.0, 1e4, 0.0),
                                               ("layer", 0.0, 1e-2, 1e-6)])
def test_sizes_of_values(kind, mean, std, eps):
    Case([33], 4, 2, 128, 128, True, kind, mean=mean, std=std, eps=eps).call().check()


def test_heads_of_zeros():
    c = Case([5], 4, 2, 64, 64, True, "layer", bias=True)
    c.Q.zero_(), c.K.zero_()
    c.ref = [c.Q.clone(), c.K.clone()]
    c.call().check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_head_stays_alone(bad):
    c = Case([20], 10, 10, 64, 64, False)
    c.call()
    torch.cuda.synchronize()
    clean = [t.clone() for t in c.out]
    c.Q[7, 3, 5] = bad
    c.call()
    torch.cuda.synchronize()
    assert torch.isnan(c.out[0][7, 3]).any()
    c.out[0][7, 3] = clean[0][7, 3]
    assert torch.equal(c.out[0], clean[0]) and torch.equal(c.out[1], clean[1])


def test_rows_beyond_31_bits_of_elements():
    rows, ld = 4100, 1 << 20
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)
    c = Case([rows], 2, 1, 64, 64, True)
    q, k = big.as_strided((rows, 2, 64), (ld, 64, 1)), big.as_strided((rows, 1, 64), (ld, 64, 1), 128)
    q.copy_(c.Q), k.copy_(c.K)
    c.Q, c.K, c.out = q, k, [q, k]
    c.call().check()
    del big, q, k, c
    torch.cuda.empty_cache()


def test_captured_and_replayed_on_any_stream():
    c = Case([30, 0, 55], 10, 2, 128, 128, True)
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    side = torch.cuda.Stream()
    for i in range(3):
        c.qkv.copy_(draw(c.qkv.shape, 20 + i))
        c.cud[1] = 30 - 9 * i
        torch.cuda.synchronize()
        c.call(side)
        torch.cuda.synchronize()
        want = [t.clone() for t in c.out]
        for t in c.out:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(c.out, want))
