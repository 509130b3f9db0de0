"""The binding of the block operators names an operand that is missing or has no such shape, as the
SVDQuant calls do (CPU only)."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_binding_checks import g  # noqa: E402  host tensors that claim a GPU device

BF = torch.bfloat16


def attention():
    return dict(Q=g((10, 4, 64), BF), K=g((10, 2, 64), BF), V=g((10, 2, 64), BF), cu_q=g((3,), torch.int32),
                cu_k=g((3,), torch.int32), scale=0.125, causal=False, O=g((10, 4, 64), BF))


def norm():
    x = g((10, 64), BF)
    return dict(x=x, y=x, cu=g((3,), torch.int32), post=0, w=None, gate=None, rs=1.0, bs=1.0, pre=2, pw=None, pb=None,
                scale=None, shift=None, eps=1e-6, x_out=x, h=x)


def linear():
    return dict(X=g((10, 128), BF), W=g((64, 128), BF), bias=None, act=0, residual=None, Y=g((10, 64), BF))


CALLS = {"attention": (S.svdq_attention_forward, attention), "norm": (S.svdq_block_norm_forward, norm),
         "linear": (S.svdq_linear_bf16_forward, linear)}


@pytest.mark.parametrize("call,name", [("attention", "Q"), ("attention", "K"), ("attention", "V"), ("attention", "O"),
                                       ("norm", "x"), ("linear", "X"), ("linear", "W"), ("linear", "Y")])
def test_none_for_a_required_operand(call, name):
    f, args = CALLS[call]
    with pytest.raises(ValueError, match=f"^{name} must not be None$"):
        f(*dict(args(), **{name: None}).values())


@pytest.mark.parametrize("call,name", [("attention", "cu_q"), ("attention", "cu_k"), ("norm", "cu")])
@pytest.mark.parametrize("shape", [(), (0,), (1,), (3, 1)])
def test_offsets_of_no_such_shape(call, name, shape):
    f, args = CALLS[call]
    with pytest.raises(ValueError, match=f"^{name} must"):
        f(*dict(args(), **{name: g(shape, torch.int32)}).values())
