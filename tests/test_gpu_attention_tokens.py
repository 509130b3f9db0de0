"""svdq_attention_forward for new tokens, at most 64 rows (tokens x heads of a group) per sequence:
the softmax's weights go into the product with V in two bf16 parts, so O is held to more
than the rounding of the weights to bf16.

Tolerance of O: as for every attention, but for the weights: their upper 16 bits leave a rest
below 2^-7 of a weight, which is rounded by at most 2^-8 of itself: 2^-15 in place of 2^-8.
The rest's float32 products and sums double the number of additions: 2 n 2^-24.
"""
import numpy as np
import pytest

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, check, cu_dev, draw, f64, offsets, workspace  # noqa: E402


@pytest.mark.parametrize("lq,lk,hq,hkv,d,causal,shares", [
    ([1], [1], 8, 2, 128, True, False), ([1, 1, 1], [31, 200, 64], 4, 4, 64, True, False),
    ([1], [5000], 8, 2, 128, True, True), ([1] * 7, [4000, 1, 0, 513, 2047, 64, 3000], 32, 8, 128, True, True),
    ([1, 1], [3000, 77], 5, 5, 64, False, True), ([3, 1, 8, 5], [900, 17, 8, 2500], 12, 4, 96, True, True),
    ([64], [333], 6, 6, 72, False, False), ([20], [2000], 8, 8, 40, True, True), ([2, 0], [700, 5], 40, 2, 80, True, True),
    ([1], [9000], 64, 1, 8, True, True),
])
def test_weights_keep_their_bits(lq, lk, hq, hkv, d, causal, shares):
    cu_q, cu_k = offsets(lq), offsets(lk)
    G = hq // hkv
    assert cu_q[-1] * G <= 64 * len(lq)
    Q, K, V = draw((cu_q[-1], hq, d), 1, 1.4), draw((cu_k[-1], hkv, d), 2, 1.4), draw((cu_k[-1], hkv, d), 3)
    O, lse = torch.full_like(Q, float("nan")), torch.full((hq, cu_q[-1]), float("nan"), device=DEV)
    ws = workspace(Q, K, len(lq))
    assert (ws.numel() > 16) == shares
    S.svdq_attention_forward(Q, K, V, cu_dev(cu_q), cu_dev(cu_k), d**-0.5, causal, O, lse, ws)
    torch.cuda.synchronize()
    check(O, lse, Q, K, V, cu_q, cu_k, d**-0.5, causal)
    q, k, v = f64(Q), f64(K), f64(V)
    want, _, A = B.attention(q, k, v, cu_q, cu_k, d**-0.5, causal)
    got = f64(O)
    for b in range(len(lq)):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(hq):
            mag = np.abs(q[rq, h]) @ np.abs(k[rk, h // G]).T
            ds = d**-0.5 * (d + 8) * 2.0**-24 * mag.max(axis=1, initial=0.0)[:, None]
            w = want[rq, h]
            tol = A[rq, h] * (2.0**-15 + 2 * ds + 2.0**-17 + 2 * lk[b] * 2.0**-24) + 2.0**-8 * np.abs(w)
            err = np.abs(got[rq, h] - w)
            assert np.all(err <= tol * 1.01 + 1e-30), (b, h, float(np.max(err / (tol + 1e-30))))
