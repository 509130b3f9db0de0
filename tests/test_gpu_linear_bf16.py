"""svdq_linear_bf16_forward on the GPU against the float64 oracle.

Tolerance, element by element: the products are exact in float32 and their sum
takes K additions (in any order) and the bias: (K + 2) 2^-24 (sum |x w| + |b|),
times 1.13, the steepest slope of the activations; the activations' own error
is below 2^-15 |y| (three roundings of an exponent below 128 in base 2, exp2, a
reciprocal; zero where there is none) plus the smallest normal number; the
residual's sum and the output's rounding: 2^-24 or, in bf16, 2^-8 of the result.
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
ACTS = {"none": S.SVDQ_ACT_NONE, "gelu": S.SVDQ_ACT_GELU_TANH, "silu": S.SVDQ_ACT_SILU}


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def draw(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def workspace(M, K, N):
    return torch.full((max(S.svdq_linear_bf16_workspace_bytes(M, K, N), 16),), 0xFF, dtype=torch.uint8, device=DEV)


def check(Y, X, W, b, act, R, fp32):
    x, w, bias, res = f64(X), f64(W), f64(b), f64(R)
    want = B.linear(x, w, bias, act, res)
    y = B.linear(x, w, bias, act, None)
    size = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    tol = 1.13 * (x.shape[1] + 2) * 2.0**-24 * size + (0 if act == "none" else 2.0**-15) * np.abs(y)
    tol = tol + (2.0**-23 if fp32 else 2.0**-8 * 1.01) * np.abs(want) + 1.2e-38
    err = np.abs(f64(Y) - want)
    assert np.all(err <= tol), (float((err / tol).max()), np.unravel_index(np.argmax(err / tol), err.shape))


def run(M, K, N, act="none", bias=True, residual=False, fp32=False, seed=1, inplace=False):
    dt = torch.float32 if fp32 else torch.bfloat16
    X, W = draw((M, K), seed), draw((N, K), seed + 1, K**-0.5)
    b = draw((N,), seed + 2) if bias else None
    R = draw((M, N), seed + 3, dtype=dt) if residual else None
    Y = R.clone() if inplace else torch.full((M, N), float("nan"), dtype=dt, device=DEV)
    S.svdq_linear_bf16_forward(X, W, b, ACTS[act], Y if inplace else R, Y, workspace(M, K, N))
    torch.cuda.synchronize()
    check(Y, X, W, b, act, R, fp32)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("K,N", [(8, 1), (64, 16), (72, 17), (1288, 130), (2048, 63), (520, 1000)])
def test_few_rows(M, K, N):
    run(M, K, N, residual=M % 2 == 0, fp32=N % 2 == 1)


@pytest.mark.parametrize("M,K,N", [
    (65, 8, 1), (65, 64, 15), (129, 40, 130), (200, 1024, 64), (333, 1160, 1003),     # 64 x 64 tiles, shares
    (1155, 1288, 1290), (128, 4096, 640), (70, 5000, 6),
    (2048, 200, 2100), (2100, 32, 2052),                                               # 128 x 128
    (4100, 72, 4096), (4608, 136, 3850), (4096, 24, 4099),
    (4100, 72, 643), (9000, 64, 300), (2500, 520, 1101),                               # 64 x 64, many
    (1155, 520, 1290), (2000, 968, 514),                                               # 128 x 64
    (2050, 808, 4099), (2305, 712, 3833),                                              # 256 x 256
])
@pytest.mark.parametrize("fp32", [False, True])
def test_tiles(M, K, N, fp32):
    run(M, K, N, "gelu" if N % 2 else "none", residual=True, fp32=fp32)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("M,K,N", [(2, 512, 96), (100, 768, 72), (300, 64, 60), (2050, 96, 2080), (4352, 64, 4096),
                                   (4100, 72, 643), (1155, 520, 1290), (2000, 808, 4100)])
@pytest.mark.parametrize("bias,residual,fp32", [(True, False, False), (False, True, True), (True, True, False),
                                                (False, False, True)])
def test_epilogues(act, M, K, N, bias, residual, fp32):
    run(M, K, N, act, bias, residual, fp32)


@pytest.mark.parametrize("M,K,N", [(3, 512, 96), (130, 1024, 77), (2050, 96, 2080)])
def test_residual_in_place(M, K, N):
    run(M, K, N, "gelu", True, True, True, inplace=True)
    run(M, K, N, "silu", True, True, False, inplace=True)


def test_activations_at_their_ends():
    """Arguments far from zero: no NaN from an overflowing exponential."""
    X = torch.zeros(70, 8, dtype=torch.bfloat16, device=DEV)
    X[:, 0] = 1
    W = torch.zeros(64, 8, dtype=torch.bfloat16, device=DEV)
    W[:, 0] = torch.cat([torch.linspace(-300, 300, 60), torch.tensor([-1e30, 1e30, 0.0, -0.0])]).to(DEV)
    for act in ("gelu", "silu"):
        for rows in (3, 70):
            Y = torch.empty(rows, 64, device=DEV)
            S.svdq_linear_bf16_forward(X[:rows], W, None, ACTS[act], None, Y, workspace(rows, 8, 64))
            w = f64(W[:, 0])
            with np.errstate(over="ignore"):
                want = B.activation(w, act)
            got = f64(Y)
            assert np.all(np.isfinite(got))
            assert np.all(np.abs(got - want) <= 2.0**-15 * np.abs(want) + 1.2e-38)


def test_outputs_beyond_31_bits_of_elements():
    M, K, N = 1_050_000, 8, 2056
    X, W = draw((M, K), 1), draw((N, K), 2)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    S.svdq_linear_bf16_forward(X, W, None, S.SVDQ_ACT_NONE, None, Y, workspace(M, K, N))
    for r in (slice(0, 4), slice(M - 300, M)):
        check(Y[r], X[r], W, None, "none", None, False)
    del Y
    torch.cuda.empty_cache()


def test_no_rows():
    S.svdq_linear_bf16_forward(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), draw((5, 64), 1), None,
                               S.SVDQ_ACT_NONE, None, torch.empty(0, 5, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("M,K,N", [(2, 512, 96), (130, 2048, 100), (4352, 64, 4096)])
def test_captured_and_replayed(M, K, N):
    X, W = draw((M, K), 1), draw((N, K), 2)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    ws = workspace(M, K, N)

    def call():
        S.svdq_linear_bf16_forward(X, W, None, S.SVDQ_ACT_SILU, None, Y, ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        X.copy_(draw(X.shape, 10 + i))
        call()
        torch.cuda.synchronize()
        want = Y.clone()
        Y.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_two_calls_at_once():
    """Two streams, each call with a workspace of its own (channels in shares)."""
    calls = []
    for i, (M, K, N) in enumerate([(130, 2048, 100), (70, 5000, 60)]):
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        calls.append((draw((M, K), 2 * i), draw((N, K), 2 * i + 1, K**-0.5), None, ACTS["silu"], None, Y, workspace(M, K, N)))
        assert calls[-1][6].numel() > 16
    want = []
    for c in calls:
        S.svdq_linear_bf16_forward(*c)
        torch.cuda.synchronize()
        want.append(c[5].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, s in zip(calls, streams):
            S.svdq_linear_bf16_forward(*c, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c[5], w)
