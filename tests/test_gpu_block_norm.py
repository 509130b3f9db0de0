"""svdq_block_norm_forward on the GPU against the float64 oracle.

Tolerances, element by element.  A row's sums run over at most 32 values per
thread, 6 steps in the wave and 8 waves: depth below 64, so a sum of values of
one sign has a relative error below e = 64 2^-24, the mean an absolute one below
e mean|v|; rsqrt and the products add 2^-22.  A normalised value n then is off by
  |n| (e + 2^-22) + r (e mean|v| + 2^-23 |v|)        (r: the reciprocal deviation)
and, where its input is off by dx, by r (dx + mean dx) + |n| r^2 mean(|v| dx) more.
Sums and products of the formula add 2^-22 of their terms' sizes; a bf16
output is off by half a step, 2^-8 of itself, a float32 one by 2^-24.
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
KINDS = {"none": S.SVDQ_NORM_NONE, "rms": S.SVDQ_NORM_RMS, "layer": S.SVDQ_NORM_LAYER}
E = 64 * 2.0**-24


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def draw(shape, seed, std=1.0, dtype=torch.bfloat16, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)


def norm_tol(v, kind, eps, dv):
    """(n, bound of the error of the normalised values) for an input v known to dv."""
    n = B._norm(v, kind, eps)
    if kind == "none":
        return n, dv
    c = v - v.mean(1, keepdims=True) if kind == "layer" else v
    r = 1 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    own = np.abs(n) * (E + 2.0**-22) + r * 2.0**-23 * np.abs(v)
    if kind == "layer":
        own = own + r * E * np.abs(v).mean(1, keepdims=True)
    return n, own + r * (dv + dv.mean(1, keepdims=True)) + np.abs(n) * r * r * (np.abs(c) * dv).mean(1, keepdims=True)


def check(x_out, h, x, y, cu, post, w_post, gate, a, c, pre, w_pre, b_pre, scale, shift, eps, fp32):
    for b in range(len(cu) - 1):
        r = slice(cu[b], cu[b + 1])
        if cu[b] == cu[b + 1]:
            continue
        v = a * x[r]
        dv = 2.0**-22 * np.abs(v)
        if y is not None:
            u, du = norm_tol(y[r], post, eps, np.zeros_like(y[r]))
            f = c * (w_post if w_post is not None else 1.0) * (gate[b] if gate is not None else 1.0) * np.ones_like(u)
            v = v + f * u
            dv = dv + np.abs(f) * du + 2.0**-22 * (np.abs(f * u) + np.abs(v))
        if x_out is not None:
            err = np.abs(x_out[r] - v)
            assert np.all(err <= dv + (2.0**-24 if fp32 else 2.0**-8) * np.abs(v) * 1.01 + 1e-38), (b, float(err.max()))
        if h is not None:
            n, dn = norm_tol(v, pre, eps, dv)
            w = w_pre if w_pre is not None else 1.0
            m = 1 + scale[b] if scale is not None else 1.0
            t = n * w + (b_pre if b_pre is not None else 0.0)
            want = t * m + (shift[b] if shift is not None else 0.0)
            tol = np.abs(w * m) * dn + 2.0**-21 * ((np.abs(n * w) + np.abs(t)) * np.abs(m) + np.abs(want))
            err = np.abs(h[r] - want)
            assert np.all(err <= tol + 2.0**-8 * np.abs(want) * 1.01 + 1e-38), (b, float(err.max()))


def case(lens, width, post, pre, fp32=False, affine=False, y=True, gate=True, mod=True, x_out=True, h=True, first=0,
         behind=0, a=1.0, c=1.0, eps=1e-6, mean=0.0, seed=1, inplace=False):
    cu = np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int64)
    rows, batch = int(cu[-1]) + behind, len(lens)
    dt = torch.float32 if fp32 else torch.bfloat16
    X = draw((rows, width), seed, 2.0, dt, mean)
    Y = draw((rows, width), seed + 1, mean=mean) if y else None
    mods = draw((batch, 3 * width + 8), seed + 2, 0.3)
    g = mods[:, :width] if y and gate else None
    sc, sh = (mods[:, width:2 * width], mods[:, 2 * width:3 * width]) if mod and h else (None, None)
    wp = draw((width,), seed + 3, 0.1, mean=1.0) if y and post != "none" else None
    wn = draw((width,), seed + 4, 0.1, mean=1.0) if affine and h else None
    bn = draw((width,), seed + 5, 0.1) if affine and h else None
    x64, y64 = f64(X), f64(Y)
    if inplace:
        xo, ho = X, Y
    else:
        xo = torch.full((rows, width), 7.0, dtype=dt, device=DEV) if x_out else None
        ho = torch.full((rows, width), 5.0, dtype=torch.bfloat16, device=DEV) if h else None
    args = (KINDS[post], wp, g, a, c, KINDS[pre] if h else S.SVDQ_NORM_NONE, wn, bn, sc, sh, eps)
    S.svdq_block_norm_forward(X, Y, torch.tensor(cu, dtype=torch.int32, device=DEV), *args, xo, ho)
    torch.cuda.synchronize()
    check(f64(xo), f64(ho), x64, y64, cu, post, f64(wp), f64(g), a, c, pre, f64(wn), f64(bn), f64(sc), f64(sh), eps, fp32)
    for r in (slice(0, first), slice(int(cu[-1]), rows)):
        if not inplace:
            assert xo is None or torch.all(xo[r] == 7)
            assert ho is None or torch.all(ho[r] == 5)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("width", [8, 64, 504, 512, 520, 640, 1280, 2048, 2056, 4096, 4104, 8192, 8200, 16384])
def test_widths(width, fp32):
    case([3, 1, 2], width, "none", "layer", fp32)
    case([5], width, "rms", "rms", fp32, affine=True)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("affine", [False, True])
def test_norm_kinds(post, pre, affine):
    case([1, 0, 33, 7], 640, post, pre, False, affine, a=0.7, c=-1.3)
    case([9, 40], 2568, post, pre, True, affine)


@pytest.mark.parametrize("over", [dict(y=False), dict(gate=False), dict(mod=False), dict(x_out=False), dict(h=False),
                                  dict(y=False, mod=False, x_out=False), dict(gate=False, mod=False)])
def test_absent_operands(over):
    for width in (640, 5120):
        case([4, 11], width, "none", "layer", **over)
        case([4, 11], width, "none", "rms", fp32=True, affine=True, **over)


def test_rows_outside_the_sequences_stay():
    case([10, 0, 5], 640, "rms", "layer", first=3, behind=6)
    case([10, 0, 5], 2560, "rms", "layer", first=1, behind=9)


@pytest.mark.parametrize("width", [640, 4608])
@pytest.mark.parametrize("fp32", [False, True])
def test_in_place(width, fp32):
    case([17, 30], width, "rms", "layer", fp32, affine=True, inplace=True)


def test_a_large_mean_costs_no_bits_of_the_variance():
    case([20], 1280, "layer", "layer", True, mean=1000.0)


def test_rows_of_zeros():
    z = torch.zeros(4, 640, dtype=torch.bfloat16, device=DEV)
    xo, h = torch.full_like(z, 7), torch.full_like(z, 7)
    for kind in ("rms", "layer"):
        S.svdq_block_norm_forward(z, z, None, KINDS[kind], None, None, 1.0, 1.0, KINDS[kind], None, None, None, None, 1e-6,
                                  xo, h)
        assert torch.all(xo == 0) and torch.all(h == 0)


def test_many_sequences():
    case([1] * 130 + [0] * 5 + [3, 2], 512, "none", "layer")


def test_a_nan_stays_in_its_row():
    x, y = draw((9, 640), 1), draw((9, 640), 2)
    out = [torch.empty_like(x) for _ in range(4)]
    args = (None, KINDS["rms"], None, None, 1.0, 1.0, KINDS["layer"], None, None, None, None, 1e-6)
    S.svdq_block_norm_forward(x, y, *args, out[0], out[1])
    y[4, 3] = float("nan")
    x[6, 600] = float("inf")
    S.svdq_block_norm_forward(x, y, *args, out[2], out[3])
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(out[0][keep], out[2][keep]) and torch.equal(out[1][keep], out[3][keep])
    assert torch.isnan(out[3][4]).all() and torch.isnan(out[3][6]).any()


def test_rows_beyond_31_bits_of_elements():
    rows, width = 265000, 8192
    x = torch.empty(rows, width, dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(x)
    x[-3:], y[-3:] = draw((3, width), 1), draw((3, width), 2)
    x_out, h = torch.empty_like(x), torch.empty_like(x)
    a64, b64 = f64(x[-3:]), f64(y[-3:])
    S.svdq_block_norm_forward(x, y, None, KINDS["rms"], None, None, 1.0, 1.0, KINDS["layer"], None, None, None, None, 1e-6,
                              x_out, h)
    check(f64(x_out[-3:]), f64(h[-3:]), a64, b64, [0, 3], "rms", None, None, 1.0, 1.0, "layer", None, None, None, None,
          1e-6, False)
    del x, y, x_out, h
    torch.cuda.empty_cache()


def test_captured_and_replayed_on_another_stream():
    x, y = draw((300, 1280), 1), draw((300, 1280), 2)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    mod = draw((2, 1280), 3)
    x_out, h = torch.empty_like(x), torch.empty_like(x)

    def call():
        S.svdq_block_norm_forward(x, y, cu, KINDS["none"], None, mod, 1.0, 1.0, KINDS["layer"], None, None, mod, mod, 1e-6,
                                  x_out, h)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        x.copy_(draw(x.shape, 10 + i))
        cu[1] = 50 * i
        call()
        torch.cuda.synchronize()
        want = x_out.clone(), h.clone()
        x_out.zero_(), h.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x_out, want[0]) and torch.equal(h, want[1])


def test_a_thousand_sequences():
    lens = np.random.default_rng(7).choice([0, 0, 1, 2, 9], 1000)
    case(list(lens), 512, "rms", "layer", True, affine=True, first=2, behind=3)


@pytest.mark.parametrize("width", [8, 64, 120, 128, 136, 200, 256, 264])
@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "rms"), ("layer", "none")])
def test_narrow_rows_share_a_wave(width, post, pre):
    """Rows of up to 256 channels: several to a wave, of different sequences, some outside them."""
    case([3, 0, 1, 30, 2, 5], width, post, pre, affine=True, first=3, behind=5)
    case([1, 1, 1, 1, 1], width, post, pre, fp32=True, first=1, behind=70)
