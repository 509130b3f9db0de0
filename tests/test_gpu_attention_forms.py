"""The special situations of test_gpu_attention_spans in the forms of attention_forms, which its own list does not
reach: a cut-off prefix in attention_rows, with own keys in one share or many and heads of every class, and
the eight-wave kernel with windows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_gpu_attention_spans as spans  # noqa: E402
from test_gpu_attention_spans import CUS, Case  # noqa: E402

from tests.attention_forms import FORMS  # noqa: E402


def make(name):
    *sizes, keys, _ = FORMS[name]
    return lambda **k: Case(*sizes, **({"window": keys} if isinstance(keys, tuple) else {"prefix": keys}), **k)


@pytest.fixture(params=FORMS, ids=lambda s: s.replace(" ", "_"))
def form(request, monkeypatch):
    """The form's name, under which the tests of test_gpu_attention_spans find it."""
    monkeypatch.setitem(spans.FORMS, request.param, make(request.param))
    return request.param


def test_values(form):
    c = spans.FORMS[form]()
    if CUS == 256:
        assert (c.bytes() > 0) == (FORMS[form][-1][4] > 0)
    c.call().check()


@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (0.01, 1e-3), (3.0, 20.0)])
def test_scores_of_any_size(form, std, scale):
    spans.test_scores_of_any_size(form, std, scale)


@pytest.mark.parametrize("slope", [0.02, 0.4, 8.0])
def test_a_growing_maximum_is_followed(form, slope):
    spans.test_a_growing_maximum_is_followed(form, slope)


def test_column_slices_and_rows_outside(form):
    spans.test_column_slices_and_rows_outside(form)


def test_a_bad_sequence_leaves_the_others_alone(form):
    spans.test_a_bad_sequence_leaves_the_others_alone(form)


def test_bad_queries_reach_their_rows_alone(form):
    spans.test_bad_queries_reach_their_rows_alone(form)


def test_scores_out_of_range(form):
    spans.test_scores_out_of_range(form)


def test_equal_calls_give_equal_bits_on_any_stream(form):
    spans.test_equal_calls_give_equal_bits_on_any_stream(form)


def test_captured_and_replayed(form):
    spans.test_captured_and_replayed(form)


def test_two_calls_at_once(form):
    """Beside a second call of the same form and other inputs, each with a workspace of its own."""
    calls, want = [make(form)(), make(form)(seed=40)], []
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


def test_offsets_past_the_rows_stay_inside(form):
    c = make(form)()
    c.call()
    torch.cuda.synchronize()
    want = c.O.clone()
    c.cu[0][-1] = 2**31 - 1
    c.cu[1][-1] = 2**31 - 1
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.O, want)


@pytest.mark.parametrize("name", [n for n in FORMS if n.startswith("cut")])
def test_own_lengths_around_a_share(name):
    """Own keys that end at, before and behind the border of a share or a tile, in every sequence."""
    lq, lk, hq, hkv, d, causal, keys, _ = FORMS[name]
    around = [0, 1, 31, 32, 33, 255, 256, 257, 511, 512, 513]
    for shift in (0, 4):
        own = [around[(i + shift) % len(around)] for i in range(len(lq))]
        Case(lq, own, hq, hkv, d, causal, prefix=keys).call().check()
