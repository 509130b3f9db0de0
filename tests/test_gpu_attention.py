"""svdq_attention_forward on the GPU against the float64 oracle.

Tolerance of O, element by element, from the roundings of the kernel:
  - a weight p is rounded to bf16 (half a step: 2^-8) and comes from a score
    whose float32 error is at most `ds` = scale (D + 8) 2^-24 max_j sum_d |q_d k_d|
    (every product exact, D additions), from fma, exp2 and the running maximum's
    rescaling (2^-18 in all: the exponent in base 2 is below 2^7 for every weight
    that counts, and is rounded to 2^-24 of itself twice; exp2 1 ulp); the
    normaliser carries the same error of the scores: sum p |v| (2^-8 + 2 ds + 2^-17)
  - the float32 sums over at most n keys: n 2^-24 sum p |v|
  - O itself is rounded to bf16: 2^-8 |O|
Tolerance of the log-sum-exp: ds + (n + 16) 2^-24 + 2^-22 (|lse| + 1).
"""
import numpy as np
import pytest

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda:0")


def offsets(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int64)


def cu_dev(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def draw(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def workspace(Q, K, batch, fill=0xFF):
    """Filled with NaN patterns, so that reading an unwritten part shows."""
    n = S.svdq_attention_workspace_bytes(Q.shape[0], K.shape[0], batch, Q.shape[1], K.shape[1], Q.shape[2])
    return torch.full((max(n, 16),), fill, dtype=torch.uint8, device=DEV)


def check(O, lse, Q, K, V, cu_q, cu_k, scale, causal):
    q, k, v = f64(Q), f64(K), f64(V)
    want, want_lse, A = B.attention(q, k, v, cu_q, cu_k, scale, causal)
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    got, got_lse = f64(O), f64(lse)
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n = cu_k[b + 1] - cu_k[b]
        for h in range(q.shape[1]):
            mag = np.abs(q[rq, h]) @ np.abs(k[rk, h // G]).T
            ds = scale * (D + 8) * 2.0**-24 * mag.max(axis=1, initial=0.0)[:, None]
            tol = A[rq, h] * (2.0**-8 + 2 * ds + 2.0**-17 + n * 2.0**-24) + 2.0**-8 * np.abs(want[rq, h])
            err = np.abs(got[rq, h] - want[rq, h])
            assert np.all(err <= tol * 1.01 + 1e-30), (b, h, float(np.max(err / (tol + 1e-30))))
            w, g = want_lse[h, rq], got_lse[h, rq]
            none = np.isneginf(w)
            assert np.array_equal(none, np.isneginf(g)), (b, h)
            tl = ds[:, 0] + (n + 16) * 2.0**-24 + 2.0**-22 * (np.abs(np.where(none, 0, w)) + 1)
            assert np.all(np.abs(np.where(none, 0, g) - np.where(none, 0, w)) <= tl), (b, h)


def run(lq, lk, hq, hkv, d, causal, seed=1, std=1.4, scale=None):
    cu_q, cu_k = offsets(lq), offsets(lk)
    Q, K, V = draw((cu_q[-1], hq, d), seed, std), draw((cu_k[-1], hkv, d), seed + 1, std), draw((cu_k[-1], hkv, d), seed + 2)
    O = torch.full((cu_q[-1], hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((hq, cu_q[-1]), float("nan"), device=DEV)
    scale = d**-0.5 if scale is None else scale
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), scale, causal, O, lse, workspace(Q, K, len(lq)))
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu_q, cu_k, scale, causal)
    return Q, K, V, O, lse


@pytest.mark.parametrize("d", [8, 40, 64, 72, 80, 96, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1], [2, 1], [31, 33, 0, 32], [63, 64, 65], [127, 130, 5, 129], [300]])
def test_self_attention(lens, causal, d):
    run(lens, lens, 4, 2, d, causal)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (16, 16), (40, 1), (96, 2)])
def test_head_groups(hq, hkv):
    run([70, 3, 129], [70, 3, 129], hq, hkv, 64, True)


@pytest.mark.parametrize("d", [8, 40, 64, 72, 96, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,hkv", [([127, 0, 130, 5, 129], 96), ([300, 1, 130], 96), ([257, 255], 96),
                                      ([65, 200, 31], 24), ([500, 333, 0, 129], 48)])
def test_many_heads(lens, hkv, causal, d):
    """Enough tiles that attention_rows takes them, with 4 and with 8 waves."""
    run(lens, lens, 96, hkv, d, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk", [
    ([40, 200], [7, 1]),            # causal: the first queries see no key
    ([5, 150], [0, 0]),             # no keys at all
    ([130, 0, 1], [77, 9, 77]),     # no queries
    ([64, 128, 256], [500, 64, 31]),
    ([100], [1000]),
])
def test_lengths_of_queries_and_keys_differ(lq, lk, causal):
    run(lq, lk, 4, 4, 64, causal)
    run(lq, lk, 8, 2, 128, causal)


@pytest.mark.parametrize("lk", [[1], [31], [32], [33], [129], [4000], [1, 513, 0, 2047, 64], [300] * 70])
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 5, 5), (80, 8, 1)])
def test_one_token(lk, d, hq, hkv):
    run([1] * len(lk), lk, hq, hkv, d, True)


def test_few_tokens_against_a_history():
    run([3, 1, 8, 5], [900, 17, 8, 2500], 12, 4, 96, True)


def test_a_long_sequence_is_cut_into_shares():
    """Few tiles, many keys: the keys' shares join through the workspace, in both kernels."""
    assert S.svdq_attention_workspace_bytes(200, 4000, 1, 2, 2, 64) > 0
    run([200], [4000], 2, 2, 64, False)
    run([200], [4000], 2, 2, 128, True)
    for d in (64, 96, 128):
        run([100, 0, 80], [5000, 9, 1003], 24, 24, d, d == 96)
        run([100], [5000], 24, 24, d, d == 128)
    assert S.svdq_attention_workspace_bytes(1, 5000, 1, 8, 2, 128) > 0
    run([1], [5000], 8, 2, 128, True)


@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (0.01, 1e-3), (3.0, 20.0)])
def test_scores_of_any_size(std, scale):
    """Scores of thousands (one key takes all) down to none at all (all keys alike)."""
    run([130, 1], [300, 300], 2, 2, 64, False, std=std, scale=scale)


def test_a_growing_maximum_is_followed():
    """Keys whose scores rise steadily: the running maximum moves many times, also by less
    than the lazy threshold."""
    for slope in (0.02, 0.4, 3.0):
        n, d = 512, 64
        K = torch.zeros(n, 1, d)
        K[:, 0, 0] = torch.arange(n) * slope
        Q = torch.zeros(40, 1, d)
        Q[:, 0, 0] = torch.linspace(-1, 1, 40)
        K, Q = K.to(torch.bfloat16).to(DEV), Q.to(torch.bfloat16).to(DEV)
        V = draw((n, 1, d), 5)
        O = torch.empty(40, 1, d, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(1, 40, device=DEV)
        S.svdq_attention_forward(Q, K, V, None, None, 1.0, False, O, lse, workspace(Q, K, 1))
        check(O, lse, Q, K, V, [0, 40], [0, n], 1.0, False)


def test_slices_of_a_fused_projection_and_rows_outside():
    """Q, K, V and O as column slices; rows before the first and behind the last sequence hold
    NaN, are not read, and keep what they held."""
    hq, hkv, d = 6, 2, 64
    lens, first, behind = [50, 0, 131], 3, 9
    cu = offsets(lens, first)
    T = cu[-1] + behind
    qkv = draw((T, (hq + 2 * hkv) * d + 24), 3)
    qkv[:first] = float("nan")
    qkv[cu[-1]:] = float("nan")
    v = qkv[:, :(hq + 2 * hkv) * d].unflatten(1, (hq + 2 * hkv, d))
    Q, K, V = v[:, :hq], v[:, hq:hq + hkv], v[:, hq + hkv:]
    out = torch.full((T, (hq + 1) * d), 7.0, dtype=torch.bfloat16, device=DEV)
    O = out[:, :hq * d].unflatten(1, (hq, d))
    lse = torch.full((hq, T), 5.0, device=DEV)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu), cu_dev(cu), 0.125, True, O, lse, workspace(Q, K, len(lens)))
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu, cu, 0.125, True)
    assert torch.all(out[:, hq * d:] == 7) and torch.all(out[:first] == 7) and torch.all(out[cu[-1]:] == 7)
    assert torch.all(lse[:, :first] == 5) and torch.all(lse[:, cu[-1]:] == 5)


def test_rows_outside_stay_when_shares_join():
    cu_q, cu_k = [2, 3], [10, 3010]
    Q, K, V = draw((5, 4, 128), 1), draw((3020, 1, 128), 2), draw((3020, 1, 128), 3)
    O = torch.full((5, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 5), 5.0, device=DEV)
    ws = workspace(Q, K, 1)
    assert ws.numel() > 16
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), 0.1, True, O, lse, ws)
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu_q, cu_k, 0.1, True)
    assert torch.all(O[:2] == 7) and torch.all(O[3:] == 7) and torch.all(lse[:, :2] == 5) and torch.all(lse[:, 3:] == 5)


@pytest.mark.parametrize("lens", [[90, 200, 33], [1, 1, 1]])
def test_a_sequence_of_nans_leaves_the_others_alone(lens):
    cu = offsets(lens)
    Q, K, V = draw((cu[-1], 4, 64), 1), draw((cu[-1], 4, 64), 2), draw((cu[-1], 4, 64), 3)
    clean = torch.empty_like(Q)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu), cu_dev(cu), 0.125, False, clean, None, workspace(Q, K, 3))
    for t, bad in ((K, float("nan")), (V, float("inf"))):
        t[cu[1]:cu[2]] = bad
    O = torch.empty_like(Q)
    S.svdq_attention_forward(Q, K, V, cu_dev(cu), cu_dev(cu), 0.125, False, O, None, workspace(Q, K, 3))
    torch.cuda.synchronize()
    for b in (0, 2):
        assert torch.equal(O[cu[b]:cu[b + 1]], clean[cu[b]:cu[b + 1]])


def test_rows_beyond_31_bits_of_elements():
    n, ld = 4100, 1 << 20                       # the last key starts past 2^32 elements
    big = torch.empty(n * ld, dtype=torch.bfloat16, device=DEV)
    K = big.as_strided((n, 1, 64), (ld, 64, 1))
    V = big.as_strided((n, 1, 64), (ld, 64, 1), 64)
    K.copy_(draw((n, 1, 64), 1))
    V.copy_(draw((n, 1, 64), 2))
    for nq in (1, 150):
        Q = draw((nq, 2, 64), 3)
        O = torch.empty_like(Q)
        lse = torch.empty(2, nq, device=DEV)
        S.svdq_attention_forward(Q, K, V, None, None, 0.125, True, O, lse, workspace(Q, K, 1))
        check(O, lse, Q, K, V, [0, nq], [0, n], 0.125, True)
    del big, K, V
    torch.cuda.empty_cache()


def test_equal_calls_give_equal_bits_on_any_stream():
    lens = [77, 1, 300, 1200]
    cu = offsets(lens)
    Q, K, V = draw((cu[-1], 8, 128), 1), draw((cu[-1], 2, 128), 2), draw((cu[-1], 2, 128), 3)
    ref = None
    side = torch.cuda.Stream()
    for i in range(3):
        O = torch.empty_like(Q)
        ws = workspace(Q, K, 4, fill=17 * i)
        torch.cuda.synchronize()
        S.svdq_attention_forward(Q, K, V, cu_dev(cu), cu_dev(cu), 0.09, True, O, None, ws, stream=side if i == 1 else None)
        torch.cuda.synchronize()
        ref = O if ref is None else ref
        assert torch.equal(O, ref)


def test_captured_and_replayed():
    """One graph of two calls that share the workspace; offsets and inputs change between replays."""
    Q, K, V = draw((4, 8, 128), 1), draw((6000, 2, 128), 2), draw((6000, 2, 128), 3)
    Q2 = draw((150, 2, 128), 4)
    cu_q, cu_k = cu_dev([0, 1, 2, 3, 4]), cu_dev([0, 1500, 1501, 4000, 6000])
    O, O2 = torch.empty_like(Q), torch.empty_like(Q2)
    ws = torch.empty(max(S.svdq_attention_workspace_bytes(4, 6000, 4, 8, 2, 128),
                         S.svdq_attention_workspace_bytes(150, 6000, 1, 2, 2, 128)), dtype=torch.uint8, device=DEV)

    def calls():
        S.svdq_attention_forward(Q, K, V, cu_q, cu_k, 0.1, True, O, None, ws)
        S.svdq_attention_forward(Q2, K, V, None, None, 0.1, False, O2, None, ws)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for i in range(4):
        Q.copy_(draw(Q.shape, 10 + i))
        K.copy_(draw(K.shape, 20 + i))
        cu_k[2] = 1501 + 100 * i
        calls()
        torch.cuda.synchronize()
        want, want2 = O.clone(), O2.clone()
        O.fill_(float("nan"))
        O2.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.equal(O2, want2)


def test_offsets_past_the_rows_stay_inside():
    """Offsets that claim more rows than there are: the sequence ends with the rows."""
    Q, K, V = draw((40, 2, 64), 1), draw((100, 2, 64), 2), draw((100, 2, 64), 3)
    want, O = torch.empty_like(Q), torch.empty_like(Q)
    S.svdq_attention_forward(Q, K, V, None, None, 0.1, False, want, None, workspace(Q, K, 1))
    S.svdq_attention_forward(Q, K, V, cu_dev([0, 1000]), cu_dev([0, 2**31 - 1]), 0.1, False, O, None, workspace(Q, K, 1))
    torch.cuda.synchronize()
    assert torch.equal(O, want)


def test_a_thousand_sequences():
    """Empty, single and short sequences in no order, more than one look-up of 64 at a time."""
    g = np.random.default_rng(7)
    lk = g.choice([0, 1, 5, 40], 1000)
    lq = np.minimum(lk, g.choice([0, 1, 2], 1000))
    run(lq, lk, 4, 2, 64, True)
    run(lk, lk, 2, 2, 80, False)


def test_two_calls_at_once():
    """Two streams, each call with a workspace of its own."""
    lens = [[700, 9, 1500], [1, 1, 1]]
    keys = [[700, 9, 1500], [3000, 70, 4500]]
    calls = []
    for i in range(2):
        cu_q, cu_k = offsets(lens[i]), offsets(keys[i])
        Q, K, V = draw((cu_q[-1], 8, 128), 3 * i), draw((cu_k[-1], 2, 128), 3 * i + 1), draw((cu_k[-1], 2, 128), 3 * i + 2)
        calls.append((Q, K, V, cu_dev(cu_q), cu_dev(cu_k), 0.09, True, torch.empty_like(Q), None, workspace(Q, K, 3)))
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
