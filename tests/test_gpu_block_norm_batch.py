"""svdq_block_norm_forward with more than 2^30 packed sequences, all but the last ones empty: a row's sequence is
found, and its gate, scale and shift read, by numbers whose sums pass 31 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_block_norm import DEV, draw  # noqa: E402


def test_a_row_finds_its_sequence_among_more_than_2_30():
    batch, width = 2**30 + 9, 8
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
    cu[-4:] = torch.arange(1, 5, dtype=torch.int32, device=DEV)             # rows 0 to 3: the last four
    gate = torch.zeros(batch, width, dtype=torch.bfloat16, device=DEV)
    gate[-4:] = torch.tensor([1.0, 2.0, 4.0, 8.0], device=DEV).to(torch.bfloat16)[:, None]
    x, y = torch.zeros(6, width, dtype=torch.bfloat16, device=DEV), draw((6, width), 1)
    out = torch.full_like(x, 7.0)
    S.svdq_block_norm_forward(x, y, cu, S.SVDQ_NORM_NONE, None, gate, 1.0, 1.0, S.SVDQ_NORM_NONE, None, None, None, None,
                              1e-6, out, None)
    torch.cuda.synchronize()
    assert torch.equal(out[:4], y[:4] * gate[-4:])                          # exact: powers of two
    assert torch.all(out[4:] == 7)
    del cu, gate
    torch.cuda.empty_cache()
