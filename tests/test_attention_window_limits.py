"""The window's limits and first keys by the binding: any whole number means what it says, also beyond the
32 bits that the library takes (CPU only)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_binding_checks import g  # noqa: E402  host tensors that claim a GPU device
from tests.test_block_ops_host import heads  # noqa: E402

MOST = 2**31 - 1
BEYOND = [2**31, 2**32 - 1, 2**32, 2**32 + 3, 2**40 + 5, 2**63 - 1]      # their low 32 bits: -2^31, -1, 0, 3, 5, -1


def passed(monkeypatch, left, right, sinks):
    """(left, right, sinks) as the library gets them."""
    args = []
    monkeypatch.setattr(S, "_launch", lambda index, stream, f, *a: args.extend(a))
    S.svdq_attention_window_forward(heads(10, 4, 64), heads(10, 2, 64), heads(10, 2, 64), g((3,), torch.int32),
                                    g((3,), torch.int32), 0.125, False, left, right, sinks, heads(10, 4, 64))
    sig = S._sig["svdq_attention_window_forward"]
    at = 16                                       # Q, K, V, O's head sizes, scale and causal stand before them
    assert all(t is ctypes.c_int for t in sig[at:at + 3]) and sig[at - 2] is ctypes.c_float
    return tuple(ctypes.c_int(v).value for v in args[at:at + 3])


@pytest.mark.parametrize("n", BEYOND)
def test_limits_beyond_32_bits_are_no_limit(monkeypatch, n):
    """No sequence has more than 2^31 - 513 keys."""
    assert passed(monkeypatch, n, 0, 0) == (MOST, 0, 0)
    assert passed(monkeypatch, 0, n, 0) == (0, MOST, 0)
    assert passed(monkeypatch, 0, 0, n) == (0, 0, MOST)


@pytest.mark.parametrize("n", [-2, -2**31, -2**31 - 1, -2**32, -2**32 + 1, -2**40, -2**63])
def test_negative_limits_stay_negative(monkeypatch, n):
    """Below -1, which the library refuses (test_window_refusals)."""
    assert passed(monkeypatch, n, 0, 0)[0] < -1 and passed(monkeypatch, 0, n, 0)[1] < -1
    assert passed(monkeypatch, 0, 0, n)[2] < 0


@pytest.mark.parametrize("n", [0, 1, 4096, MOST - 1, MOST])
def test_limits_within_32_bits_pass_as_they_are(monkeypatch, n):
    assert passed(monkeypatch, n, n, n) == (n, n, n)
    assert passed(monkeypatch, -1, -1, n) == (-1, -1, n)


def test_the_workspace_is_that_of_the_call():
    need = lambda left, right, sinks: S.svdq_attention_window_workspace_bytes(1, 20000, 1, 8, 2, 128, True, left, right,
                                                                              sinks)  # noqa: E731
    assert need(-1, 0, 0) > need(5, 0, 0) == 0
    for n in BEYOND:
        assert need(n, 0, 0) == need(MOST, 0, 0) > 0
        assert need(5, 0, n) == need(5, 0, MOST) > 0
    assert need(-2**32, 0, 0) == 0 and need(0, 0, -2**32 + 9000) == 0       # refused
