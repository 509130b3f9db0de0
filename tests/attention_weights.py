"""Calls of attention whose result shows how many bits the softmax's weights have in the product with V.

Where O is about as large as sum p |v|, its own rounding to bf16 hides that of the weights.  So V's row of each
sequence's last key, whose weight is about a half, cancels the rest of one head's sum for the last query: O of
that head and query is near 0 (|O| < 2^-8 sum p |v|, by the rounding of that row), and an error of the
weights stands alone.

Q and K are multiples of 1/8 below 16 in size and the scale is 1/8: their products are multiples of 1/64 whose
sums stay below 2^18, exact in float32, so the scores carry no error and the weights only those of what
follows them.

Tolerance of O, relative to A = sum p |v| unless said:
  - a weight in two parts: its upper 16 bits leave a rest below 2^-7 of it, which is rounded by 2^-8
    of itself: 2^-15
  - its exponent s c - m c, of scores s and a maximum m up to S in size and c = scale log2(e): c is off by
    2^-24 (log2(e) and the product, 2^-25 each), m c by 2^-24 more and the fma by 2^-24 of a result of up to 2 S c:
    5 x 2^-24 S c in all, and as much in the normaliser; as a factor of the weight ln 2 times that:
    10 x 2^-24 S scale
  - exp2, the rescaling of sums, the join of waves and shares and the division: 2^-17
  - the float32 sums: every key adds its two parts, one wave adds those of `chain` keys, at most 64
    waves and shares are joined, and the normaliser adds the same once more: 3 (chain + 64) 2^-24
  - O is rounded to bf16: 2^-8 |O|
Weights rounded to bf16 once are off by up to 2^-9 each, and where the errors of some tens of weights add up at random
that leaves about 2^-12 of A; test_attention_weights_host shows that it does not pass.
"""
import numpy as np

from oracle import block_oracle as B

SCALE = 0.125


def bf16(x):
    """float64 values rounded to bf16 (to nearest, ties to even), as float64."""
    u = np.asarray(x, np.float32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)


def eighths(x):
    return np.clip(np.round(x * 8), -127, 127) / 8


class Weights:
    """Inputs in float64 (bf16 values), and the rows (token, head) whose O is near 0."""

    def __init__(self, lq, lk, hq, hkv, d, causal, keys, seed=1):
        g = np.random.default_rng(seed)
        self.window, prefix = (keys, None) if isinstance(keys, tuple) else ((-1, -1, 0), keys)
        self.causal, self.lq, self.lk = causal, lq, lk
        self.cu_q, self.cu_k = (np.concatenate([[0], np.cumsum(n)]).astype(np.int64) for n in (lq, lk))
        size = (18 / d**0.5)**0.5                       # scores of standard deviation 18 / 8
        self.Q = eighths(g.normal(size=(self.cu_q[-1], hq, d)) * size)
        self.K = eighths(g.normal(size=(self.cu_k[-1], hkv, d)) * size)
        self.V = bf16(g.normal(size=self.K.shape))
        self.PK = self.PV = None
        if prefix is not None:
            self.PK = eighths(g.normal(size=(prefix, hkv, d)) * size)
            self.PV = bf16(g.normal(size=self.PK.shape))
        self.rows = []
        for b in range(len(lq)):
            last = self.cu_k[b + 1] - 1
            if not lq[b] or not lk[b] or (lk[b] == 1 and prefix is None):
                continue
            token = self.cu_q[b + 1] - 1
            for h in range(0, hq, hq // hkv):
                hk = h // (hq // hkv)
                q = self.Q[token, h]
                s, v = self.seen(b, token, h)
                rest = np.log(np.exp(s[:-1] - s[:-1].max()).sum()) + s[:-1].max()
                self.K[last, hk] = eighths(q * (rest / SCALE / (q @ q)))      # the last key: about as much as the rest
                s, v = self.seen(b, token, h)
                e = np.exp(s - s.max())
                self.V[last, hk] = bf16(-(e[:-1] @ v[:-1]) / e[-1])
                self.rows.append((b, token, h))

    def seen(self, b, token, h):
        """Scores and values of the keys that a query sees, its own last key last."""
        k0, k1, hk = self.cu_k[b], self.cu_k[b + 1], h // (self.Q.shape[1] // self.K.shape[1])
        mask = B.sees(self.lq[b], self.lk[b], self.causal, *self.window)[token - self.cu_q[b]]
        k, v = self.K[k0:k1, hk][mask], self.V[k0:k1, hk][mask]
        if self.PK is not None:
            k, v = np.concatenate([self.PK[:, hk], k]), np.concatenate([self.PV[:, hk], v])
        return SCALE * (k @ self.Q[token, h]), v

    def off(self, O, chain):
        """The largest error of O in the rows near 0, in units of the tolerance."""
        worst = 0.0
        for b, token, h in self.rows:
            s, v = self.seen(b, token, h)
            p = np.exp(s - s.max())
            p /= p.sum()
            want, A = p @ v, p @ np.abs(v)
            assert np.all(np.abs(want) <= 2.0**-8 * A)
            tol = A * (2.0**-15 + 10 * 2.0**-24 * np.abs(s).max() + 2.0**-17 + 3 * (chain + 64) * 2.0**-24) + 2.0**-8 * np.abs(want)
            err = np.abs(O[token, h] - want)
            worst = max(worst, np.inf if np.isnan(err).any() else float((err / (tol + 1e-30)).max()))
        return worst
