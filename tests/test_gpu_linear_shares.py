"""svdq_linear_bf16_forward where the channels are cut into shares: every tile that takes shares, at
ragged sizes, with each epilogue, in place, captured, and two calls at once.  Tolerances as in
test_gpu_linear_bf16 (the order of the sums does not enter them)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_linear_bf16 import ACTS, DEV, draw, run, workspace  # noqa: E402

# M, K, N, shares on 256 compute units: 128 x 128 tiles, 128 x 64, 64 x 64
SHARES = [(145, 2568, 10994, 2), (21, 7320, 8653, 4), (21, 4488, 4221, 8),
          (69, 3368, 4378, 2), (75, 2072, 2113, 4), (71, 4104, 1067, 8), (2149, 4280, 9, 8), (671, 5976, 237, 8),
          (101, 1368, 61, 2), (131, 2056, 99, 4), (71, 4424, 61, 8)]


def shares_of(M, K, N):
    return S.svdq_linear_bf16_workspace_bytes(M, K, N) / (4 * M * ((N + 3) // 4 * 4))


@pytest.mark.parametrize("M,K,N,shares", SHARES)
@pytest.mark.parametrize("fp32", [False, True])
def test_tiles_with_shares(M, K, N, shares, fp32):
    if torch.cuda.get_device_properties(DEV).multi_processor_count == 256:
        assert shares_of(M, K, N) == shares
    run(M, K, N, "gelu" if fp32 else "none", residual=True, fp32=fp32)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("M,K,N", [(21, 4488, 4221), (75, 2072, 2113), (671, 5976, 237), (131, 2056, 99), (71, 4424, 61)])
@pytest.mark.parametrize("bias,residual,fp32", [(True, False, False), (False, True, True), (True, True, False),
                                                (False, False, True)])
def test_epilogues_of_the_join(act, M, K, N, bias, residual, fp32):
    assert shares_of(M, K, N) >= 2
    run(M, K, N, act, bias, residual, fp32)


@pytest.mark.parametrize("M,K,N", [(21, 4488, 4221), (75, 2072, 2113), (131, 2056, 99), (70, 5000, 61)])
def test_residual_in_place_of_the_join(M, K, N):
    assert shares_of(M, K, N) >= 2
    run(M, K, N, "gelu", True, True, True, inplace=True)
    run(M, K, N, "silu", True, True, False, inplace=True)


@pytest.mark.parametrize("M,K,N", [(21, 4488, 4221), (75, 2072, 2113)])
def test_captured_and_replayed(M, K, N):
    assert shares_of(M, K, N) >= 2
    X, W, b, R = draw((M, K), 1), draw((N, K), 2, K**-0.5), draw((N,), 3), draw((M, N), 4)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    ws = workspace(M, K, N)

    def call():
        S.svdq_linear_bf16_forward(X, W, b, ACTS["gelu"], R, Y, ws)

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
    """Two streams, each call with a workspace of its own, in tiles of different sizes."""
    calls = []
    for i, (M, K, N) in enumerate([(21, 4488, 4221), (75, 2072, 2113)]):
        Y = torch.empty(M, N, device=DEV)
        calls.append((draw((M, K), 2 * i), draw((N, K), 2 * i + 1, K**-0.5), None, ACTS["none"], None, Y, workspace(M, K, N)))
        assert calls[-1][6].numel() > 16
    want = []
    for c in calls:
        S.svdq_linear_bf16_forward(*c)
        torch.cuda.synchronize()
        want.append(c[5].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c in calls:
            c[5].fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for c, s in zip(calls, streams):
                S.svdq_linear_bf16_forward(*c, stream=s)
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c[5], w)
