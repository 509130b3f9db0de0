"""svdq_attention_forward's special situations in every one of its forms: attention_rows with four and
with eight waves, whole and in shares, and attention_keys in shares.  (test_gpu_attention has most of
them at sizes that only attention_keys takes.)  Which form a size takes is planned for 256 compute
units; on another number the tests hold all the same."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, check, cu_dev, draw, offsets, run, workspace  # noqa: E402

CUS = torch.cuda.get_device_properties(DEV).multi_processor_count

# queries, keys, heads_q, heads_kv, head_dim, causal, whether the keys are cut into shares
FORMS = {
    "rows4": ([127, 0, 130, 5, 129], [127, 0, 130, 5, 129], 96, 96, 64, True, False),
    "rows4 96": ([127, 133, 129], [200, 3, 129], 96, 48, 72, False, False),
    "rows8": ([254, 241], [254, 241], 96, 96, 128, False, False),
    "rows4 shares": ([100], [5000], 24, 24, 128, True, True),
    "rows4 shares 96": ([67], [587], 1, 1, 96, False, True),
    "rows4 shares 64": ([325], [3548], 24, 24, 64, False, True),
    "keys shares": ([200], [4000], 2, 2, 64, False, True),
    "token shares": ([1, 3], [5000, 700], 8, 2, 128, True, True),
}
forms = pytest.mark.parametrize("form", FORMS, ids=lambda s: s.replace(" ", "_"))


def shapes(form):
    lq, lk, hq, hkv, d, causal, shares = FORMS[form]
    cu_q, cu_k = offsets(lq), offsets(lk)
    if CUS == 256:
        n = S.svdq_attention_workspace_bytes(int(cu_q[-1]), int(cu_k[-1]), len(lq), hq, hkv, d)
        assert (n > 0) == shares
    return cu_q, cu_k, hq, hkv, d, causal


@forms
@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (0.01, 1e-3), (3.0, 20.0)])
def test_scores_of_any_size(form, std, scale):
    lq, lk, hq, hkv, d, causal, _ = FORMS[form]
    run(lq, lk, hq, hkv, d, causal, std=std, scale=scale)


@forms
@pytest.mark.parametrize("slope", [0.02, 0.4, 8.0])
def test_a_growing_maximum_is_followed(form, slope):
    """Scores that rise along the keys: the running maximum moves many times, by less than the lazy
    threshold, and (8.0) from tile to tile and share to share by more than float32's exponents."""
    cu_q, cu_k, hq, hkv, d, causal = shapes(form)
    Q, K = torch.zeros(int(cu_q[-1]), hq, d), torch.zeros(int(cu_k[-1]), hkv, d)
    for b in range(len(cu_k) - 1):
        n = int(cu_k[b + 1] - cu_k[b])
        K[cu_k[b]:cu_k[b + 1], :, 0] = (torch.arange(n) * slope)[:, None]
    Q[:, :, 0] = torch.linspace(-1, 1, Q.shape[0] * hq).view(Q.shape[0], hq)
    Q, K = Q.to(torch.bfloat16).to(DEV), K.to(torch.bfloat16).to(DEV)
    V = draw(K.shape, 5)
    O, lse = torch.full_like(Q, float("nan")), torch.full((hq, Q.shape[0]), float("nan"), device=DEV)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), 1.0, causal, O, lse, workspace(Q, K, len(cu_q) - 1))
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu_q, cu_k, 1.0, causal)


@forms
def test_column_slices_and_rows_outside(form):
    """Column slices of wider tensors; rows before the first and behind the last sequence, and the
    columns between, hold NaN, are not read, and keep what they held."""
    cu_q, cu_k, hq, hkv, d, causal = shapes(form)
    first, behind = 3, 9
    cu_q, cu_k = cu_q + first, cu_k + first + 2
    Tq, Tk = int(cu_q[-1]) + behind, int(cu_k[-1]) + behind

    def slice_of(T, heads, seed, cu, std):
        wide = torch.full((T, (heads + 1) * d + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
        t = wide[:, 8:8 + heads * d].unflatten(1, (heads, d))
        t[cu[0]:cu[-1]] = draw((int(cu[-1] - cu[0]), heads, d), seed, std)
        return t

    Q, K, V = slice_of(Tq, hq, 1, cu_q, 1.4), slice_of(Tk, hkv, 2, cu_k, 1.4), slice_of(Tk, hkv, 3, cu_k, 1.0)
    out = torch.full((Tq, (hq + 1) * d), 7.0, dtype=torch.bfloat16, device=DEV)
    O = out[:, :hq * d].unflatten(1, (hq, d))
    lse = torch.full((hq, Tq), 5.0, device=DEV)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), d**-0.5, causal, O, lse, workspace(Q, K, len(cu_q) - 1))
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu_q, cu_k, d**-0.5, causal)
    assert torch.all(out[:, hq * d:] == 7) and torch.all(out[:cu_q[0]] == 7) and torch.all(out[cu_q[-1]:] == 7)
    assert torch.all(lse[:, :cu_q[0]] == 5) and torch.all(lse[:, cu_q[-1]:] == 5)


@pytest.mark.parametrize("form", ["rows4", "rows8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_sequence_leaves_the_others_alone(form, bad):
    """Neighbours whose keys and values follow directly, in other tiles of the same launch."""
    cu_q, cu_k, hq, hkv, d, causal = shapes(form)
    b = 0
    Q, K, V = draw((int(cu_q[-1]), hq, d), 1), draw((int(cu_k[-1]), hkv, d), 2), draw((int(cu_k[-1]), hkv, d), 3)
    args = (cu_dev(cu_q), cu_dev(cu_k), d**-0.5, causal)
    clean, O = torch.empty_like(Q), torch.empty_like(Q)
    ws = workspace(Q, K, len(cu_q) - 1)
    S.svdq_attention_forward(Q, K, V, *args, clean, None, ws)
    for t in (K, V):
        t[cu_k[b]:cu_k[b + 1]] = bad
    S.svdq_attention_forward(Q, K, V, *args, O, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(O[cu_q[b + 1]:], clean[cu_q[b + 1]:]) and not torch.isfinite(O[:cu_q[b + 1]]).any()


@pytest.mark.parametrize("nq,causal", [(325, False), (325, True), (2200, False)])
def test_rows_beyond_31_bits_of_elements(nq, causal):
    """Key rows 2^20 elements apart, the last past 2^32: in shares, and whole (2200 queries)."""
    n, ld, h, d = 4100, 1 << 20, 24, 64
    big = torch.empty(n * ld, dtype=torch.bfloat16, device=DEV)
    K = big.as_strided((n, h, d), (ld, d, 1))
    V = big.as_strided((n, h, d), (ld, d, 1), h * d)
    K.copy_(draw((n, h, d), 1))
    V.copy_(draw((n, h, d), 2))
    Q = draw((nq, h, d), 3)
    O, lse = torch.empty_like(Q), torch.empty(h, nq, device=DEV)
    ws = workspace(Q, K, 1)
    if CUS == 256:
        assert (ws.numel() > 16) == (nq < 1000)
    S.svdq_attention_forward(Q, K, V, None, None, 0.125, causal, O, lse, ws)
    torch.cuda.synchronize()
    keep = slice(0, 2) if nq > 1000 else slice(0, h)          # heads: the oracle's time
    check(O[:, keep], lse[keep], Q[:, keep], K[:, keep], V[:, keep], [0, nq], [0, n], 0.125, causal)
    # every head against the same call on dense copies, bit for bit
    O2 = torch.empty_like(Q)
    S.svdq_attention_forward(Q, K.contiguous(), V.contiguous(), None, None, 0.125, causal, O2, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(O, O2)
    del big, K, V
    torch.cuda.empty_cache()


@forms
def test_offsets_past_the_rows_stay_inside(form):
    """Offsets that claim more rows than there are: the last sequence ends with the rows."""
    cu_q, cu_k, hq, hkv, d, causal = shapes(form)
    Q, K, V = draw((int(cu_q[-1]), hq, d), 1), draw((int(cu_k[-1]), hkv, d), 2), draw((int(cu_k[-1]), hkv, d), 3)
    want, O = torch.empty_like(Q), torch.full_like(Q, float("nan"))
    ws = workspace(Q, K, len(cu_q) - 1)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), 0.1, causal, want, None, ws)
    far_q, far_k = cu_q.copy(), cu_k.copy()
    far_q[-1], far_k[-1] = 2**31 - 1, 2**31 - 1
    S.svdq_attention_forward(Q, K, V, cu_dev(far_q), cu_dev(far_k), 0.1, causal, O, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(O, want)


@forms
def test_equal_calls_give_equal_bits_on_any_stream(form):
    """Whatever the workspace holds before."""
    cu_q, cu_k, hq, hkv, d, causal = shapes(form)
    Q, K, V = draw((int(cu_q[-1]), hq, d), 1), draw((int(cu_k[-1]), hkv, d), 2), draw((int(cu_k[-1]), hkv, d), 3)
    cq, ck = cu_dev(cu_q), cu_dev(cu_k)
    ref = None
    side = torch.cuda.Stream()
    for i in range(4):
        O, lse = torch.full_like(Q, float("nan")), torch.full((hq, Q.shape[0]), float("nan"), device=DEV)
        ws = workspace(Q, K, len(cu_q) - 1, fill=(0, 0xFF, 0x3F, 17)[i])
        torch.cuda.synchronize()
        S.svdq_attention_forward(Q, K, V, cq, ck, 0.09, causal, O, lse, ws, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        ref = (O, lse) if ref is None else ref
        assert torch.equal(O, ref[0]) and torch.equal(lse, ref[1])


def test_captured_and_replayed():
    """One graph with a call of every form, all sharing the workspace; inputs and lengths change
    between the replays, beside eager work."""
    calls = []
    for i, form in enumerate(FORMS):
        cu_q, cu_k, hq, hkv, d, causal = shapes(form)
        Q, K, V = draw((int(cu_q[-1]), hq, d), 3 * i), draw((int(cu_k[-1]), hkv, d), 3 * i + 1), draw((int(cu_k[-1]), hkv, d), 3 * i + 2)
        calls.append([Q, K, V, cu_dev(cu_q), cu_dev(cu_k), d**-0.5, causal, torch.zeros_like(Q),
                      torch.zeros(hq, Q.shape[0], device=DEV)])
    ws = torch.empty(max(workspace(c[0], c[1], c[3].numel() - 1).numel() for c in calls), dtype=torch.uint8, device=DEV)

    def go():
        for c in calls:
            S.svdq_attention_forward(*c, ws)

    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for i in range(4):
        for c in calls:
            c[0].copy_(draw(c[0].shape, 40 + i))
            c[4][-1] -= 7
        go()
        torch.cuda.synchronize()
        want = [(c[7].clone(), c[8].clone()) for c in calls]
        for c in calls:
            c[7].fill_(float("nan"))
            c[8].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for c, (O, lse), form in zip(calls, want, FORMS):
            assert torch.equal(c[7], O) and torch.equal(c[8], lse), form
            assert not torch.isnan(c[7]).any(), form


@pytest.mark.parametrize("pair", [("rows4 shares", "keys shares"), ("rows4 shares 64", "token shares"), ("rows8", "rows4 shares")])
def test_two_calls_at_once(pair):
    """Two streams, each call with a workspace of its own."""
    calls = []
    for i, form in enumerate(pair):
        cu_q, cu_k, hq, hkv, d, causal = shapes(form)
        Q, K, V = draw((int(cu_q[-1]), hq, d), 3 * i), draw((int(cu_k[-1]), hkv, d), 3 * i + 1), draw((int(cu_k[-1]), hkv, d), 3 * i + 2)
        ws = workspace(Q, K, len(cu_q) - 1)
        assert CUS != 256 or (ws.numel() > 16) == FORMS[form][6]
        calls.append((Q, K, V, cu_dev(cu_q), cu_dev(cu_k), 0.09, causal, torch.empty_like(Q), None, ws))
    want = []
    for c in calls:
        S.svdq_attention_forward(*c)
        torch.cuda.synchronize()
        want.append(c[7].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for c in calls:
            c[7].fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(5):
            for c, s in zip(calls, streams):
                S.svdq_attention_forward(*c, stream=s)
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c[7], w)


def test_many_sequences():
    """More than one look-up of 64 sequences in attention_rows: empty, single and ragged ones."""
    lens = np.random.default_rng(7).choice([0, 1, 70, 130], 200)
    run(lens, lens, 16, 4, 80, True)
    run(lens, np.roll(lens, 1), 16, 4, 80, False)
