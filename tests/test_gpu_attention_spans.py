"""svdq_attention_window_forward and svdq_attention_prefix_forward on the GPU against the float64 oracle.

Tolerances element by element, from the roundings of the kernels (as test_gpu_attention derives them):
  - a weight p is rounded to bf16 (half a step: 2^-8) and comes from a score whose float32 error is at
    most `ds` = scale (D + 8) 2^-24 max_j sum_d |q_d k_d|, from fma, exp2 and the running maximum's
    rescaling (2^-18 in all), and the normaliser carries the same error of the scores:
    sum p |v| (2^-8 + 2 ds + 2^-17)
  - the float32 sums over at most n keys: n 2^-24 sum p |v|
  - O itself is rounded to bf16: 2^-8 |O|
and of the log-sum-exp: ds + (n + 16) 2^-24 + 2^-22 (|lse| + 1).  Partial rows are joined in float32 with
weights 2^x of |x| < 2^7 where they count: within the 2^-17 above.
"""
import numpy as np
import pytest

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, cu_dev, draw, f64, offsets  # noqa: E402

CUS = torch.cuda.get_device_properties(DEV).multi_processor_count


def check(O, lse, Q, K, V, cu_q, cu_k, scale, causal, left=-1, right=-1, sinks=0, PK=None, PV=None):
    q, k, v = f64(Q), f64(K), f64(V)
    pk, pv = (None, None) if PK is None else (f64(PK), f64(PV))
    want, want_lse, A, M = B.attention_spans(q, k, v, cu_q, cu_k, scale, causal, left, right, sinks, pk, pv)
    D, got, got_lse = q.shape[2], f64(O), f64(lse)
    for b in range(len(cu_q) - 1):
        r = slice(cu_q[b], cu_q[b + 1])
        n = cu_k[b + 1] - cu_k[b] + (0 if PK is None else len(pk))
        ds = scale * (D + 8) * 2.0**-24 * M[:, r]                       # [heads, queries]
        tol = A[r] * (2.0**-8 + 2 * ds.T[..., None] + 2.0**-17 + n * 2.0**-24) + 2.0**-8 * np.abs(want[r])
        err = np.abs(got[r] - want[r])
        assert np.all(err <= tol * 1.01 + 1e-30), (b, float(np.nanmax(err / (tol + 1e-30), initial=0)), np.isnan(err).sum())
        w, g = want_lse[:, r], got_lse[:, r]
        none = np.isneginf(w)
        assert np.array_equal(none, np.isneginf(g)), b
        tl = ds + (n + 16) * 2.0**-24 + 2.0**-22 * (np.abs(np.where(none, 0, w)) + 1)
        assert np.all(np.abs(np.where(none, 0, g) - np.where(none, 0, w)) <= tl), b


class Case:
    """Inputs of a call, its outputs (NaN until written) and a workspace of NaN patterns.  prefix None:
    the windowed form."""

    def __init__(self, lq, lk, hq, hkv, d, causal, window=(-1, -1, 0), prefix=None, seed=1, std=1.4, scale=None,
                 first=0, behind=0):
        self.cu_q, self.cu_k = offsets(lq, first), offsets(lk, first + (2 if first else 0))
        Tq, Tk = int(self.cu_q[-1]) + behind, int(self.cu_k[-1]) + behind
        self.Q, self.K, self.V = draw((Tq, hq, d), seed, std), draw((Tk, hkv, d), seed + 1, std), draw((Tk, hkv, d), seed + 2)
        self.PK = self.PV = None
        if prefix is not None:
            self.PK, self.PV = draw((prefix, hkv, d), seed + 3, std), draw((prefix, hkv, d), seed + 4)
        self.O = torch.full((Tq, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((hq, Tq), float("nan"), device=DEV)
        self.scale, self.causal, self.window = d**-0.5 if scale is None else scale, causal, window
        self.cu = cu_dev(self.cu_q), cu_dev(self.cu_k)
        n = self.bytes()
        self.ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def bytes(self):
        a = (self.K.shape[0], len(self.cu_q) - 1, self.Q.shape[1], self.K.shape[1], self.Q.shape[2], self.causal)
        if self.PK is None:
            return S.svdq_attention_window_workspace_bytes(self.Q.shape[0], *a, *self.window)
        return S.svdq_attention_prefix_workspace_bytes(self.Q.shape[0], self.PK.shape[0], *a)

    def call(self, stream=None):
        if self.PK is None:
            S.svdq_attention_window_forward(self.Q, self.K, self.V, *self.cu, self.scale, self.causal, *self.window,
                                            self.O, self.lse, self.ws, stream=stream)
        else:
            S.svdq_attention_prefix_forward(self.Q, self.PK, self.PV, self.K, self.V, *self.cu, self.scale, self.causal,
                                            self.O, self.lse, self.ws, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        check(self.O, self.lse, self.Q, self.K, self.V, self.cu_q, self.cu_k, self.scale, self.causal, *self.window,
              self.PK, self.PV)
        return self


WINDOWS = [(0, 0, 0), (0, 0, 1), (5, 0, 1), (31, 2, 4), (32, 33, 40), (64, 3, 33), (-1, 2, 0), (7, -1, 3), (0, 0, 1000),
           (100, 100, 5), (-1, -1, 7), (2**31 - 1, 2**31 - 1, 0), (90, 0, 2**31 - 1)]


# ------------------------------------------------------------------ window
@pytest.mark.parametrize("window", WINDOWS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (80, 2, 2), (128, 6, 1)])
def test_windows(window, causal, d, hq, hkv):
    lens = [1, 0, 31, 130, 300]
    Case(lens, lens, hq, hkv, d, causal, window).call().check()


@pytest.mark.parametrize("d", [8, 40, 72, 96])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes(d, causal):
    Case([200, 77], [200, 77], 4, 2, d, causal, (45, 20, 3)).call().check()


@pytest.mark.parametrize("window", [(0, 0, 0), (33, 0, 4), (70, 40, 50), (-1, 0, 0), (300, -1, 2)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,heads,d", [([127, 0, 130, 5, 129], 96, 64), ([300, 1, 130], 96, 128), ([500, 333], 48, 96)])
def test_many_heads(window, causal, lens, heads, d):
    """Enough tiles that attention_rows takes them, with four and (not causal, more than 64 channels) with
    eight waves."""
    Case(lens, lens, heads, heads, d, causal, window).call().check()


@pytest.mark.parametrize("window", [(0, 0, 0), (3, 2, 0), (40, 0, 6), (20, 20, 3)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk", [([40, 200], [7, 1]), ([5, 150], [0, 0]), ([130, 0, 1], [77, 9, 77]),
                                   ([64, 128, 256], [500, 64, 31]), ([100], [1000])])
def test_lengths_of_queries_and_keys_differ(lq, lk, causal, window):
    """Queries in front of the first key, whose windows hold some keys or none."""
    Case(lq, lk, 8, 2, 128, causal, window).call().check()
    Case(lq, lk, 4, 4, 64, causal, window).call().check()


@pytest.mark.parametrize("window", [(0, 0, 0), (127, 0, 4), (1023, 0, 1), (2000, 0, 100)], ids=str)
@pytest.mark.parametrize("lk", [[1], [33], [129, 4, 5, 133], [5000], [1, 513, 0, 2047, 64], [300] * 70], ids=str)
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 5, 5), (80, 8, 1)])
def test_one_token(lk, d, hq, hkv, window):
    Case([1] * len(lk), lk, hq, hkv, d, True, window).call().check()


def test_few_tokens_against_a_history():
    Case([3, 1, 8, 5], [900, 17, 8, 2500], 12, 4, 96, True, (600, 0, 9)).call().check()


def test_a_window_cut_into_shares():
    """Few tiles, long windows: the shares join through the workspace, in both kernels."""
    for args in (([200], [4000], 2, 2, 64, False, (3000, 700, 40)), ([200], [4000], 2, 2, 128, True, (2500, 0, 40)),
                 ([100, 0, 80], [5000, 9, 1003], 24, 24, 128, True, (4000, 0, 4)), ([1], [9000], 8, 2, 128, True, (5000, 0, 4)),
                 ([100], [5000], 24, 24, 96, False, (4500, 90, 0))):
        c = Case(*args)
        if CUS == 256:
            assert c.bytes() > 0, args
        c.call().check()


def test_the_last_tiles_of_a_long_window_are_cut_into_shares():
    c = Case([6144], [6144], 6, 6, 96, True, (3000, 0, 4))
    if CUS == 256:
        assert c.bytes() > 0
    c.call().check()


@pytest.mark.parametrize("nq", [1, 3])
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 4, 4)])
def test_keys_that_a_cache_has_given_up_may_hold_anything(nq, d, hq, hkv):
    """NaN and infinities in K and V between the first keys and the earliest window, and (two-sided) past
    the last one, at every distance from a tile's border."""
    for nk in [64 + 7 * i for i in range(12)] + [900, 2500]:
        c = Case([nq], [nk], hq, hkv, d, True, (31, 0, 4))
        begin = nk - nq - 31
        c.K[4:begin], c.V[4:begin] = float("nan"), float("inf")
        c.call().check()
    c = Case([2], [3000], hq, hkv, d, False, (700, 0, 5))
    c.K[5:3000 - 2 - 700], c.V[5:3000 - 2 - 700] = float("inf"), float("nan")
    c.call().check()


@pytest.mark.parametrize("heads", [2, 96])
def test_keys_in_front_of_all_windows_of_a_sequence_are_not_read(heads):
    """As above for many rows: a long history given up in front of a prompt's windows."""
    c = Case([300, 140], [1500, 700], heads, heads, 64, True, (64, 0, 3))
    for k0, nq, nk in ((0, 300, 1500), (1500, 140, 700)):
        c.K[k0 + 3:k0 + nk - nq - 64], c.V[k0 + 3:k0 + nk - nq - 64] = float("nan"), float("nan")
    c.call().check()


# ------------------------------------------------------------------ prefix
@pytest.mark.parametrize("prefix", [0, 1, 31, 33, 100, 700])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (80, 2, 2), (128, 6, 1), (8, 1, 1)])
def test_prefixes(prefix, causal, d, hq, hkv):
    lens = [1, 0, 31, 130, 300]
    Case(lens, lens, hq, hkv, d, causal, prefix=prefix).call().check()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,heads,d,prefix", [([127, 0, 130, 5, 129], 96, 64, 77), ([300, 1, 130], 96, 128, 260),
                                                 ([500, 333], 48, 96, 95), ([100, 90], 24, 128, 4000)])
def test_prefix_of_many_heads(lens, heads, d, prefix, causal):
    Case(lens, lens, heads, heads, d, causal, prefix=prefix).call().check()


@pytest.mark.parametrize("prefix", [0, 5, 1000])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk", [([40, 200], [7, 1]), ([5, 150], [0, 0]), ([130, 0, 1], [77, 9, 77]),
                                   ([64, 128, 256], [500, 64, 31]), ([100], [0]), ([3, 2], [0, 0])])
def test_own_lengths_of_queries_and_keys_differ(lq, lk, causal, prefix):
    Case(lq, lk, 8, 2, 128, causal, prefix=prefix).call().check()
    Case(lq, lk, 4, 4, 64, causal, prefix=prefix).call().check()


@pytest.mark.parametrize("prefix", [1, 300, 4100])
@pytest.mark.parametrize("lk", [[1], [33, 1], [129, 4, 0, 133], [2000, 1, 70], [1] * 70, [5, 0, 40] * 30], ids=len)
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 5, 5), (80, 8, 1)])
def test_one_token_behind_a_prefix(lk, d, hq, hkv, prefix):
    Case([1] * len(lk), lk, hq, hkv, d, True, prefix=prefix).call().check()


def test_unequal_few_tokens_behind_a_prefix():
    """Some sequences without tokens, some with more than a tile of rows."""
    Case([3, 0, 1, 20, 2], [900, 17, 0, 25, 300], 12, 4, 96, True, prefix=2100).call().check()
    Case([9, 1, 0, 1, 1, 1, 1, 1, 1, 1], [9, 1, 5, 1, 1, 1, 1, 1, 1, 1], 16, 2, 128, False, prefix=2100).call().check()


def test_the_prefix_is_cut_off_for_new_tokens():
    """Sixteen tokens share 32-row tiles against the prefix: it needs partial rows, a single pass does not."""
    if CUS != 256:
        pytest.skip("planned for 256 compute units")
    assert S.svdq_attention_prefix_workspace_bytes(16, 8192, 16 * 100, 16, 32, 8, 128, True) > 0
    assert S.svdq_attention_prefix_workspace_bytes(4096, 512, 4096, 4, 24, 24, 128, False) == 0


# ------------------------------------------------------------------ both
FORMS = {
    "window tokens": lambda **k: Case([1, 3, 1], [5000, 700, 40], 8, 2, 128, True, (2000, 0, 4), **k),
    "window keys": lambda **k: Case([90, 200, 33], [90, 200, 33], 4, 4, 64, True, (50, 0, 4), **k),
    "window rows": lambda **k: Case([127, 0, 130, 5, 129], [127, 0, 130, 5, 129], 96, 96, 64, True, (40, 0, 2), **k),
    "window rows8": lambda **k: Case([254, 241], [254, 241], 96, 96, 128, False, (60, 70, 3), **k),
    "window shares": lambda **k: Case([200], [4000], 2, 2, 64, False, (3000, 700, 40), **k),
    "window wide": lambda **k: Case([1, 2, 1], [390, 0, 700], 8, 2, 128, True, (200, 0, 9), **k),
    "prefix wide": lambda **k: Case([1, 2, 1, 3], [50, 700, 0, 3], 6, 3, 96, True, prefix=150, **k),
    "prefix tokens": lambda **k: Case([1, 2, 1, 1], [50, 700, 0, 3], 8, 2, 128, True, prefix=3000, **k),
    "prefix keys": lambda **k: Case([90, 200, 33], [90, 200, 33], 4, 4, 64, True, prefix=70, **k),
    "prefix rows": lambda **k: Case([127, 0, 130, 5, 129], [127, 0, 130, 5, 129], 96, 96, 96, True, prefix=150, **k),
    "prefix rows8": lambda **k: Case([254, 241], [254, 241], 96, 96, 128, False, prefix=99, **k),
    "prefix tail": lambda **k: Case([300, 1, 460], [300, 1, 460], 48, 48, 128, True, prefix=4000, **k),
    "prefix tail 64": lambda **k: Case([260, 0, 700, 300], [9, 5, 700, 0], 28, 28, 64, False, prefix=5000, **k),
    "prefix shares": lambda **k: Case([100, 90], [100, 90], 4, 4, 128, True, prefix=5000, **k),
}
forms = pytest.mark.parametrize("form", FORMS, ids=lambda s: s.replace(" ", "_"))


@forms
def test_forms_that_join_shares(form):
    """By the workspace that they ask for, on the card that they are planned for."""
    if CUS != 256:
        pytest.skip("planned for 256 compute units")
    joined = any(w in form for w in ("shares", "tail")) or form in ("window tokens", "prefix tokens")
    assert (FORMS[form]().bytes() > 0) == joined


@forms
@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (0.01, 1e-3), (3.0, 20.0)])
def test_scores_of_any_size(form, std, scale):
    FORMS[form](std=std, scale=scale).call().check()


@forms
@pytest.mark.parametrize("slope", [0.02, 0.4, 8.0])
def test_a_growing_maximum_is_followed(form, slope):
    """Scores that rise along the prefix and the keys, by less and by more than the lazy threshold."""
    c = FORMS[form](scale=1.0)
    c.Q.zero_(), c.K.zero_()
    c.Q[..., 0] = torch.linspace(-1, 1, c.Q.shape[0] * c.Q.shape[1], device=DEV).view(c.Q.shape[:2])
    base = 0
    if c.PK is not None:
        c.PK.zero_()
        base = len(c.PK)
        c.PK[..., 0] = (torch.arange(base, device=DEV) * slope)[:, None]
    for b in range(len(c.cu_k) - 1):
        n = int(c.cu_k[b + 1] - c.cu_k[b])
        c.K[c.cu_k[b]:c.cu_k[b + 1], :, 0] = ((base + torch.arange(n, device=DEV)) * slope)[:, None]
    c.call().check()


@forms
def test_column_slices_and_rows_outside(form):
    """Column slices of wider tensors, a prefix of other row strides; rows of no sequence and columns
    between hold NaN, are not read, and keep what they held."""
    c = FORMS[form](first=3, behind=9)
    d = c.Q.shape[2]

    def slice_of(t, cu, extra):
        T, h, _ = t.shape
        wide = torch.full((T, h * d + extra), float("nan"), dtype=torch.bfloat16, device=DEV)
        v = wide[:, 8:8 + h * d].unflatten(1, (h, d))
        v[cu[0]:cu[-1]] = t[cu[0]:cu[-1]]
        return v

    c.Q, c.K, c.V = slice_of(c.Q, c.cu_q, 24), slice_of(c.K, c.cu_k, 24), slice_of(c.V, c.cu_k, 40)
    if c.PK is not None:
        whole = [0, len(c.PK)]
        c.PK, c.PV = slice_of(c.PK, whole, 8), slice_of(c.PV, whole, 64)
    hq, T = c.Q.shape[1], c.Q.shape[0]
    out = torch.full((T, (hq + 1) * d), 7.0, dtype=torch.bfloat16, device=DEV)
    c.O = out[:, :hq * d].unflatten(1, (hq, d))
    c.lse.fill_(5.0)
    c.call().check()
    a, z = c.cu_q[0], c.cu_q[-1]
    assert torch.all(out[:, hq * d:] == 7) and torch.all(out[:a] == 7) and torch.all(out[z:] == 7)
    assert torch.all(c.lse[:, :a] == 5) and torch.all(c.lse[:, z:] == 5)


@forms
def test_a_bad_sequence_leaves_the_others_alone(form):
    c = FORMS[form]()
    if len(c.cu_k) < 3:
        pytest.skip("one sequence")
    c.call()
    torch.cuda.synchronize()
    clean, clean_lse = c.O.clone(), c.lse.clone()
    c.K[:c.cu_k[1]], c.V[:c.cu_k[1]] = float("nan"), float("inf")
    c.call()
    torch.cuda.synchronize()
    z = c.cu_q[1]
    assert torch.equal(c.O[z:], clean[z:]) and torch.equal(c.lse[:, z:], clean_lse[:, z:])
    assert not torch.isfinite(c.O[:z]).any()


@forms
def test_bad_queries_reach_their_rows_alone(form):
    c = FORMS[form]()
    c.call()
    torch.cuda.synchronize()
    clean, clean_lse = c.O.clone(), c.lse.clone()
    row, head = int(c.cu_q[-1]) - 1, 1
    c.Q[row, head, 3] = float("nan")
    c.call()
    torch.cuda.synchronize()
    assert torch.isnan(c.O[row, head]).all() and torch.isnan(c.lse[head, row])
    c.O[row, head], c.lse[head, row] = clean[row, head], clean_lse[head, row]
    assert torch.equal(c.O, clean) and torch.equal(c.lse, clean_lse)


@forms
def test_scores_out_of_range(form):
    """A query that sees keys, all of whose scores are -inf or overflow, gets NaN; one +inf among them too; one
    that sees none is not touched by any of it."""
    c = FORMS[form](scale=1.0)
    c.K.fill_(0), c.Q.fill_(0)
    if c.PK is not None:
        c.PK.fill_(0)
        c.PK[..., 0] = 1e38
    c.K[..., 0] = 1e38
    c.Q[..., 0] = 1e38
    row = int(c.cu_q[-1]) - 1
    c.Q[row, 0, 0] = -1e38
    c.call()
    torch.cuda.synchronize()
    some = [B.sees(int(nq), int(nk), c.causal, *c.window).any(1) | (c.PK is not None)
            for nq, nk in zip(np.diff(c.cu_q), np.diff(c.cu_k))]
    some = torch.from_numpy(np.concatenate(some)).to(DEV)
    O, lse = c.O[int(c.cu_q[0]):int(c.cu_q[-1])], c.lse[:, int(c.cu_q[0]):int(c.cu_q[-1])]
    assert torch.isnan(O[some]).all() and torch.isnan(lse[:, some]).all()
    assert (O[~some] == 0).all() and (lse[:, ~some] == -float("inf")).all()      # a query that sees no key


@forms
def test_equal_calls_give_equal_bits_on_any_stream(form):
    c = FORMS[form]()
    side, ref = torch.cuda.Stream(), None
    for i in range(3):
        c.O.fill_(float("nan"))
        c.ws.fill_(17 * i)
        torch.cuda.synchronize()
        c.call(side if i == 1 else None)
        torch.cuda.synchronize()
        ref = ref if ref is not None else (c.O.clone(), c.lse.clone())
        assert torch.equal(c.O, ref[0]) and torch.equal(c.lse, ref[1])


@forms
def test_captured_and_replayed(form):
    """Inputs and the first sequence's lengths change between the replays."""
    c, other = FORMS[form](), FORMS["prefix tokens"](seed=50)
    if c.ws.numel() < other.ws.numel():
        c.ws = other.ws
    other.ws = c.ws                               # one workspace for both calls, which follow each other
    c.call(), other.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(), other.call()
    for i in range(4):
        c.Q.copy_(draw(c.Q.shape, 10 + i))
        c.K.copy_(draw(c.K.shape, 20 + i))
        if i and c.cu_k[1] > 1:
            c.cu[1][0] = i % int(c.cu_k[1])
        c.call(), other.call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (c.O, c.lse, other.O, other.lse)]
        for t in (c.O, c.lse, other.O, other.lse):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((c.O, c.lse, other.O, other.lse), want))


def test_two_calls_at_once():
    calls = [FORMS["prefix tokens"](), FORMS["window tokens"]()]
    want = []
    for c in calls:
        c.call()
        torch.cuda.synchronize()
        want.append(c.O.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for c in calls:
            c.O.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(5):
            for c, s in zip(calls, streams):
                c.call(s)
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c.O, w)


def test_offsets_past_the_rows_stay_inside():
    for c in (FORMS["window keys"](), FORMS["prefix tokens"]()):
        c.call()
        torch.cuda.synchronize()
        want = c.O.clone()
        c.cu[0][-1] = 2**31 - 1
        c.cu[1][-1] = 2**31 - 1
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.O, want)


@pytest.mark.parametrize("nq", [1, 150])
def test_rows_beyond_31_bits_of_elements(nq):
    """Key rows 2^20 elements apart, the last past 2^32: as a sequence's own keys and as a prefix."""
    n, ld = 4100, 1 << 20
    big = torch.empty(n * ld, dtype=torch.bfloat16, device=DEV)
    K = big.as_strided((n, 1, 64), (ld, 64, 1))
    V = big.as_strided((n, 1, 64), (ld, 64, 1), 64)
    K.copy_(draw((n, 1, 64), 1))
    V.copy_(draw((n, 1, 64), 2))
    c = Case([nq], [n], 2, 1, 64, True, (3000, 0, 5))
    c.K, c.V = K, V
    c.call().check()
    c = Case([nq, nq], [nq, nq], 2, 1, 64, True, prefix=n)
    c.PK, c.PV = K, V
    c.call().check()
    del big, K, V, c
    torch.cuda.empty_cache()


def test_a_thousand_sequences():
    g = np.random.default_rng(7)
    lk = g.choice([0, 1, 5, 40], 1000)
    lq = np.minimum(lk, g.choice([0, 1, 2], 1000))
    Case(lq, lk, 4, 2, 64, True, (8, 0, 2)).call().check()
    Case(lq, lk, 4, 2, 64, True, prefix=50).call().check()
    Case(lk, lk, 2, 2, 80, False, (3, 9, 1)).call().check()


def test_without_lse_and_offsets():
    c = Case([70], [300], 4, 2, 64, True, (40, 0, 3))
    c.cu, c.lse = (None, None), None
    c.call()
    d = Case([70], [300], 4, 2, 64, True, (40, 0, 3)).call()
    p = Case([70], [300], 4, 2, 64, True, prefix=90)
    p.cu, p.lse = (None, None), None
    p.call()
    e = Case([70], [300], 4, 2, 64, True, prefix=90).call()
    torch.cuda.synchronize()
    assert torch.equal(c.O, d.O) and torch.equal(p.O, e.O)
