"""svdq_attention_forward on NaN, infinity and overflow, in both kernels, whole and in shares.

What a query sees decides: a NaN or +inf among its scores, or scores that all left float32's
range, make its O and log-sum-exp NaN; a score of -inf weighs nothing; and only a query that sees
no key has O = 0 and -inf.  Rows that the bad values do not reach are held to the float64 oracle
with the tolerances of ordinary inputs.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, check, cu_dev, draw, f64, offsets, workspace  # noqa: E402

NAN, INF = float("nan"), float("inf")

# queries, keys, heads_q, heads_kv, head_dim, causal, whether the keys are cut into shares
PATHS = {
    "few rows": ([40, 9], [90, 300], 4, 2, 64, False, False),
    "few rows causal": ([40, 9], [90, 300], 4, 2, 128, True, False),
    "one token in shares": ([1], [5000], 8, 2, 128, True, True),
    "few rows in shares": ([200], [4000], 2, 2, 64, False, True),
    "many rows": ([127, 0, 130, 5, 129], [127, 0, 130, 5, 129], 96, 96, 64, False, False),
    "many rows causal": ([127, 130, 129], [127, 130, 129], 96, 96, 80, True, False),
    "many rows, 8 waves": ([300, 212], [300, 212], 96, 96, 128, False, False),
    "many rows in shares": ([100], [5000], 24, 24, 128, True, True),
    "many rows in shares, 64": ([325], [3548], 24, 24, 64, False, True),
}
paths = pytest.mark.parametrize("path", PATHS, ids=lambda s: s.replace(" ", "_"))


class Case:
    def __init__(self, path, seed=1):
        lq, lk, self.hq, self.hkv, self.d, self.causal, shares = PATHS[path]
        self.cu_q, self.cu_k = offsets(lq), offsets(lk)
        self.Q = draw((self.cu_q[-1], self.hq, self.d), seed, 1.4)
        self.K = draw((self.cu_k[-1], self.hkv, self.d), seed + 1, 1.4)
        self.V = draw((self.cu_k[-1], self.hkv, self.d), seed + 2)
        self.scale = self.d**-0.5
        self.batch, self.group = len(lq), self.hq // self.hkv
        assert (workspace(self.Q, self.K, self.batch).numel() > 16) == shares
        self.b = int(np.argmax(lk))                     # the sequence that the bad values go to
        self.nq, self.nk = lq[self.b], lk[self.b]

    def run(self):
        O = torch.full_like(self.Q, 7.0)
        lse = torch.full((self.hq, self.Q.shape[0]), 7.0, device=DEV)
        S.svdq_attention_forward(self.Q, self.K, self.V, cu_dev(self.cu_q), cu_dev(self.cu_k), self.scale, self.causal,
                                 O, lse, workspace(self.Q, self.K, self.batch))
        torch.cuda.synchronize()
        return O, lse

    def sees(self, j):
        """Whether each query of the sequence sees its key j."""
        return torch.tensor([not self.causal or j <= i + self.nk - self.nq for i in range(self.nq)], device=DEV)

    def where(self, rows, heads):
        """[tokens, heads_q]: the given rows of the bad sequence and the given heads."""
        at = torch.zeros(self.Q.shape[0], self.hq, dtype=torch.bool, device=DEV)
        q0 = self.cu_q[self.b]
        at[q0:q0 + self.nq][rows.nonzero()[:, 0][:, None], torch.tensor(heads, device=DEV)] = True
        return at


def heads_of(c, hk):
    return list(range(hk * c.group, (hk + 1) * c.group))


def check_others(c, O, lse, bad, Q, K, V):
    """Everything but the rows in `bad`, against the oracle on the clean inputs."""
    clean = Case.run(c_with(c, Q, K, V))
    O = torch.where(bad[:, :, None], clean[0], O)
    lse = torch.where(bad.t(), clean[1], lse)
    check(O, lse, Q, K, V, c.cu_q, c.cu_k, c.scale, c.causal)


def c_with(c, Q, K, V):
    n = Case.__new__(Case)
    n.__dict__.update(c.__dict__, Q=Q, K=K, V=V)
    return n


@paths
def test_a_nan_query(path):
    c = Case(path)
    clean = c.Q.clone()
    i, h = c.nq // 2, c.hq - 1
    c.Q[c.cu_q[c.b] + i, h, c.d - 1] = NAN
    O, lse = c.run()
    bad = c.where(torch.arange(c.nq, device=DEV) == i, [h])
    assert torch.isnan(O[bad]).all() and torch.isnan(lse.t()[bad]).all()
    check_others(c, O, lse, bad, clean, c.K, c.V)


@paths
@pytest.mark.parametrize("at", [0.0, 0.5, 1.0])
def test_a_nan_key(path, at):
    """In the first, a middle or the last key tile, so in any share."""
    c = Case(path)
    clean = c.K.clone()
    j, hk = int(at * (c.nk - 1)), c.hkv - 1
    c.K[c.cu_k[c.b] + j, hk, 0] = NAN
    O, lse = c.run()
    bad = c.where(c.sees(j), heads_of(c, hk))
    assert bad.any() and torch.isnan(O[bad]).all() and torch.isnan(lse.t()[bad]).all()
    # the queries that the causal mask hides the key from are left open
    check_others(c, O, lse, c.where(torch.ones(c.nq, device=DEV), heads_of(c, hk)), c.Q, clean, c.V)


@paths
def test_a_nan_value(path):
    """O of its channel is NaN; the log-sum-exp does not depend on V."""
    c = Case(path)
    clean = c.V.clone()
    want = c.run()[1]
    c.V[c.cu_k[c.b], 0, 5] = NAN
    O, lse = c.run()
    bad = c.where(c.sees(0), heads_of(c, 0))
    assert torch.isnan(O[bad][:, 5]).all() and torch.equal(lse, want)
    check_others(c, O, lse, bad, c.Q, c.K, clean)


@paths
def test_an_infinite_key(path):
    """+inf scores give NaN, -inf ones weigh nothing."""
    c = Case(path)
    j, hk = c.nk // 2, 0
    q0 = c.cu_q[c.b]
    h0 = heads_of(c, hk)
    c.Q[q0:q0 + c.nq, h0, 0] = torch.where(torch.arange(c.nq, device=DEV) % 2 == 0, 1.0, -1.0).to(c.Q.dtype)[:, None]
    if c.nq == 1:
        c.Q[q0, h0[1::2], 0] = -1.0
    c.K[c.cu_k[c.b] + j, hk, 0] = INF
    O, lse = c.run()
    bad = c.where(c.sees(j), h0) & (c.Q[:, :, 0] > 0)
    assert bad.any() and torch.isnan(O[bad]).all() and torch.isnan(lse.t()[bad]).all()
    # for the others a key whose score is at least 80 below theirs: e^-80 of their weight
    K = c.K.clone()
    K[c.cu_k[c.b] + j, hk] = 0
    K[c.cu_k[c.b] + j, hk, 0] = 1e3
    check_others(c, O, lse, bad | c.where(~c.sees(j), h0), c.Q, K, c.V)


@paths
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_all_scores_overflow(path, sign):
    """Every score of a query beyond float32's range, above or below, by the scale or by the
    product itself: NaN, never the answer of a query without keys."""
    for big, scale in ((2.0**10, 2.0**126), (2.0**70, 0.125)):
        c = Case(path)
        c.scale = scale
        c.Q.zero_()
        c.K.zero_()
        c.Q[..., 0] = big
        c.K[..., 0] = sign * big
        O, lse = c.run()
        for b in range(c.batch):
            if c.cu_k[b + 1] > c.cu_k[b]:
                r = slice(c.cu_q[b], c.cu_q[b + 1])
                assert torch.isnan(O[r]).all() and torch.isnan(lse[:, r]).all(), (big, scale)


@paths
@pytest.mark.parametrize("at", [0.0, 0.5, 1.0])
def test_one_score_overflows(path, at):
    """One key whose score leaves float32's range among ordinary ones: above, NaN; below, the key
    weighs nothing."""
    c = Case(path)
    j = int(at * (c.nk - 1))
    c.scale = 2.0**100
    q0 = c.cu_q[c.b]
    c.Q.zero_()
    c.K.zero_()
    c.Q[..., 0] = 1.0
    c.Q[q0:q0 + c.nq:2, ::2, 0] = -1.0
    c.K[c.cu_k[c.b] + j, :, 0] = 2.0**40
    O, lse = c.run()
    some = c.where(c.sees(j), range(c.hq))
    up, down = some & (c.Q[:, :, 0] > 0), some & (c.Q[:, :, 0] < 0)
    assert torch.isnan(O[up]).all() and torch.isnan(lse.t()[up]).all() and up.any()
    # below: the mean of the other values that the query sees; nothing else seen, NaN
    v, O, lse = f64(c.V[c.cu_k[c.b]:c.cu_k[c.b + 1]]), f64(O), f64(lse)
    for i, h in down.nonzero().tolist():
        n = min(i - q0 + c.nk - c.nq + 1, c.nk) if c.causal else c.nk
        keep = np.arange(n) != j
        if not keep.any():
            assert np.isnan(O[i, h]).all() and np.isnan(lse[h, i])
            continue
        w = v[:n, h // c.group][keep]
        want, size = w.mean(0), np.abs(w).mean(0)
        # equal weights of 1: float32 sums, a division, the shares' weights 2^(lse - max) with an
        # lse below 16 (off by 2^-21 and log2 and exp2 by as much), O's rounding
        tol = size * ((n + 8) * 2.0**-24 + 2.0**-19) + 2.0**-8 * np.abs(want) * 1.01
        assert np.all(np.abs(O[i, h] - want) <= tol)
        assert abs(lse[h, i] - np.log(keep.sum())) <= 2.0**-20 * (1 + np.log(n))


@paths
def test_scores_below_the_range_come_first(path):
    """Whole tiles of scores below float32's range, then ordinary ones, in a wave whose other rows
    have ordinary ones all along: the first weigh nothing."""
    c = Case(path)
    c.scale = 2.0**100
    c.Q.zero_()
    c.K.zero_()
    q0, k0 = c.cu_q[c.b], c.cu_k[c.b]
    c.Q[q0:q0 + c.nq:2, :, 0] = -1.0
    n0 = c.nk // 2
    c.K[k0:k0 + n0, :, 0] = 2.0**40
    O, lse = (f64(t) for t in c.run())
    v = f64(c.V[k0:k0 + c.nk])
    for i in range(c.nq):
        n = min(i + c.nk - c.nq + 1, c.nk) if c.causal else c.nk
        first = n0 if i % 2 == 0 else 0
        for h in range(c.hq):
            if n <= first:
                assert np.isnan(O[q0 + i, h]).all() and np.isnan(lse[h, q0 + i])
                continue
            w = v[first:n, h // c.group]
            want, size = w.mean(0), np.abs(w).mean(0)
            tol = size * ((n + 8) * 2.0**-24 + 2.0**-19) + 2.0**-8 * np.abs(want) * 1.01
            assert np.all(np.abs(O[q0 + i, h] - want) <= tol), (i, h)
            assert abs(lse[h, q0 + i] - np.log(n - first)) <= 2.0**-20 * (1 + np.log(n))


@pytest.mark.parametrize("lq,lk,hq,hkv,d,shares", [
    ([40, 200], [7, 1], 4, 4, 64, False), ([1210, 10], [1200, 8000], 2, 2, 64, True),
    ([300, 130], [290, 1], 96, 96, 128, False), ([694], [593], 1, 1, 96, True),
])
def test_queries_without_keys_beside_nans(lq, lk, hq, hkv, d, shares):
    """Causal, more queries than keys: the first queries see no key and keep O = 0 and -inf, also
    where a query, a key or a value of the sequence is not finite; the others show it."""
    cu_q, cu_k = offsets(lq), offsets(lk)
    for where in ("query", "key", "value"):
        Q, K, V = draw((cu_q[-1], hq, d), 1), draw((cu_k[-1], hkv, d), 2), draw((cu_k[-1], hkv, d), 3)
        none = lq[0] - lk[0]
        if where == "query":
            Q[0], Q[none] = NAN, NAN
        elif where == "key":
            K[0] = NAN
        else:
            V[0] = INF
        O, lse = torch.full_like(Q, 7.0), torch.full((hq, cu_q[-1]), 7.0, device=DEV)
        ws = workspace(Q, K, len(lq))
        assert (ws.numel() > 16) == shares
        S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), d**-0.5, True, O, lse, ws)
        torch.cuda.synchronize()
        assert torch.all(O[:none] == 0) and torch.all(torch.isneginf(lse[:, :none]))
        last = slice(none + 1, lq[0])
        assert not torch.isfinite(O[none]).any()
        assert torch.isnan(lse[:, none]).all() if where != "value" else torch.isfinite(lse[:, none]).all()
        assert torch.isfinite(O[last]).all() if where == "query" else not torch.isfinite(O[last]).any()
        assert torch.isnan(lse[:, last]).all() if where == "key" else torch.isfinite(lse[:, last]).all()
