"""The softmax's weights of new tokens (at most 64 rows per sequence) keep 15 bits in the product with V: where a
query's sum cancels, weights that were rounded to bf16 once would show (attention_weights)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_attention import DEV, cu_dev, f64  # noqa: E402
from test_gpu_attention_spans import CUS  # noqa: E402

from tests.attention_forms import TOKENS  # noqa: E402
from tests.attention_weights import SCALE, Weights  # noqa: E402

if CUS != 256:
    pytest.skip("planned for 256 compute units", allow_module_level=True)


def results(c, plain=False):
    to = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)  # noqa: E731
    Q, K, V = to(c.Q), to(c.K), to(c.V)
    assert (f64(Q) == c.Q).all() and (f64(K) == c.K).all() and (f64(V) == c.V).all()
    O = torch.full_like(Q, float("nan"))
    cu = cu_dev(c.cu_q), cu_dev(c.cu_k)
    shape = (K.shape[0], len(c.lq), Q.shape[1], K.shape[1], Q.shape[2])
    space = lambda n: torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)  # noqa: E731
    if plain:
        ws = space(S.svdq_attention_workspace_bytes(Q.shape[0], *shape))
        S.svdq_attention_forward(Q, K, V, *cu, SCALE, c.causal, O, None, ws)
    elif c.PK is None:
        ws = space(S.svdq_attention_window_workspace_bytes(Q.shape[0], *shape, c.causal, *c.window))
        S.svdq_attention_window_forward(Q, K, V, *cu, SCALE, c.causal, *c.window, O, None, ws)
    else:
        PK, PV = to(c.PK), to(c.PV)
        ws = space(S.svdq_attention_prefix_workspace_bytes(Q.shape[0], PK.shape[0], *shape, c.causal))
        S.svdq_attention_prefix_forward(Q, PK, PV, K, V, *cu, SCALE, c.causal, O, None, ws)
    torch.cuda.synchronize()
    return f64(O), ws.numel() > 16


@pytest.mark.parametrize("form", TOKENS, ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("seed", [1, 2])
def test_weights_keep_their_bits(form, seed):
    *call, plan, chain = TOKENS[form]
    c = Weights(*call, seed=seed)
    O, joined = results(c)
    assert joined == (plan[3] > 1 or plan[4] > 0)
    assert c.off(O, chain) <= 1


@pytest.mark.parametrize("lq,lk,hq,hkv,d,chain", [([1, 3, 1, 2], [300, 131, 31, 512], 8, 2, 128, 512),
                                                  ([1, 3, 1], [5000, 700, 40], 8, 2, 128, 256),
                                                  ([2, 1], [77, 400], 5, 5, 64, 400)])
def test_weights_of_plain_attention_keep_their_bits(lq, lk, hq, hkv, d, chain):
    c = Weights(lq, lk, hq, hkv, d, True, (-1, -1, 0))
    O, _ = results(c, plain=True)
    assert c.off(O, chain) <= 1
