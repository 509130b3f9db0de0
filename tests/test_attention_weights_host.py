"""attention_weights tells weights of two bf16 parts from weights rounded once, in every call that the GPU test
makes: the mistake is planted here, in the oracle (CPU only)."""
import numpy as np
import pytest

from tests.attention_forms import TOKENS
from tests.attention_weights import Weights, bf16


def upper(x):
    u = np.asarray(x, np.float32).view(np.uint32) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)


def result(c, weight):
    """O from weights that `weight` rounds, rounded to bf16."""
    O = np.zeros(c.Q.shape)
    for b, token, h in c.rows:
        s, v = c.seen(b, token, h)
        e = np.exp(s - s.max())
        O[token, h] = bf16(weight(e) @ v / e.sum())
    return O


@pytest.mark.parametrize("form", TOKENS)
def test_weights_rounded_once_do_not_pass(form):
    *call, _, chain = TOKENS[form]
    c = Weights(*call)
    assert len(c.rows) >= 2
    assert c.off(result(c, bf16), chain) > 2
    assert c.off(result(c, upper), chain) > 4                                   # the second part left out
    assert c.off(result(c, lambda e: upper(e) + bf16(e - upper(e))), chain) <= 1
    assert c.off(result(c, lambda e: e), chain) <= 1


def test_bf16_rounds_to_nearest_even():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).normal(size=1000).astype(np.float32)
    x[:4] = 1 + 2.0**-8, 1 + 3 * 2.0**-8, -1 - 2.0**-8, 0
    assert np.array_equal(bf16(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())
