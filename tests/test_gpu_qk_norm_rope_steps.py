"""svdq_qk_norm_rope_forward in calls large enough that a wave takes two, three or four steps of heads, against
the float64 oracle with the tolerances of test_gpu_qk_norm_rope."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_block_norm import KINDS, draw  # noqa: E402
from test_gpu_qk_norm_rope import Case  # noqa: E402

from tests.rope_forms import CASES  # noqa: E402

cases = pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}_{c[1]}_{c[2]}_{c[3]}_{c[4]}steps")
pairings = pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])


def rotary(d):
    """The rotated channels: all of a head, or a part."""
    return {64: 40, 72: 40}.get(d, d)


@cases
@pairings
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True)])
def test_steps(case, halves, kind, bias):
    lens, hq, hk, d, _ = case
    Case(lens, hq, hk, d, rotary(d), halves, kind, True, bias, table=max(lens) // 2 + 1).call().check()


@cases
@pairings
def test_steps_in_place_with_given_positions(case, halves):
    """Rows before and behind the sequences and the values of a fused projection stay as they were."""
    lens, hq, hk, d, _ = case
    c = Case(lens, hq, hk, d, rotary(d), halves, "layer", True, True, given=True, table=500, first=3, behind=6, inplace=True)
    before = c.qkv.clone()
    c.call().check()
    a, z = c.cu[0], c.cu[-1]
    assert torch.equal(c.qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])
    assert torch.equal(c.qkv[:a], before[:a]) and torch.equal(c.qkv[z:], before[z:])


@cases
@pairings
def test_steps_give_the_bits_of_single_ones(case, halves):
    """The same rows in calls so small that a wave takes one step: a head's arithmetic does not depend on it."""
    lens, hq, hk, d, _ = case
    c = Case([sum(lens)], hq, hk, d, rotary(d), halves, "layer", True, True, given=True, table=3000).call()
    torch.cuda.synchronize()
    parts = [torch.empty_like(t) for t in c.out]
    for r in range(0, sum(lens), 32):
        at = slice(r, min(r + 32, sum(lens)))
        S.svdq_qk_norm_rope_forward(c.Q[at], c.K[at], None, c.positions[at], KINDS[c.kind], c.w[0], c.b[0], c.w[1], c.b[1],
                                    c.eps, c.cos, c.sin, S.SVDQ_ROPE_HALVES if halves else S.SVDQ_ROPE_NEIGHBOURS, parts[0][at],
                                    parts[1][at])
    torch.cuda.synchronize()
    assert all(torch.equal(p, t) for p, t in zip(parts, c.out))


@pytest.mark.parametrize("hq,hk,rows,d", [(24, 0, 2100, 128), (0, 16, 4200, 128), (0, 13, 4100, 72)])
def test_steps_of_queries_or_keys_alone(hq, hk, rows, d):
    Case([rows], hq, hk, d, d, True, "rms").call().check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("head", [0, 5, 9, 23])
def test_a_bad_head_stays_alone(bad, head):
    """In any of a wave's steps."""
    c = Case([4608], 24, 24, 128, 128, False)
    c.call()
    torch.cuda.synchronize()
    clean = [t.clone() for t in c.out]
    c.Q[4607, head, 5] = bad
    c.call()
    torch.cuda.synchronize()
    assert torch.isnan(c.out[0][4607, head]).any()
    c.out[0][4607, head] = clean[0][4607, head]
    assert torch.equal(c.out[0], clean[0]) and torch.equal(c.out[1], clean[1])


@pytest.mark.parametrize("case", [CASES[1], CASES[5], CASES[11]], ids=["2", "3", "4"])
def test_captured_and_replayed_on_any_stream(case):
    lens, hq, hk, d, _ = case
    c = Case(lens, hq, hk, d, d, True)
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    side, end = torch.cuda.Stream(), int(c.cu[2])
    for i in range(3):
        c.qkv.copy_(draw(c.qkv.shape, 20 + i))
        c.cud[1] = min(1 + i, end)
        torch.cuda.synchronize()
        c.call(side)
        torch.cuda.synchronize()
        want = [t.clone() for t in c.out]
        for t in c.out:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(c.out, want))
