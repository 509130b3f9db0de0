"""The largest numbers of packed sequences: the kernels look offsets up 64 at a time, in 32 bits, so the last
512 numbers of 31 bits are refused; CPU only.  Every call has a misaligned operand, which is looked at
later, so that none is ever launched."""
import pytest

pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

from tests.test_attention_limits_host import attention  # noqa: E402
from tests.test_attention_spans_host import prefix, window  # noqa: E402
from tests.test_qk_norm_rope_host import rope  # noqa: E402

INVALID, ALIGNMENT = 1, 3
P = 1 << 20
MOST = 2**31 - 1 - 512
CALLS = {
    "attention": lambda batch: attention(batch=batch, cu_q=P, cu_k=P, lse=P + 1),
    "window": lambda batch: window(batch=batch, lse=P + 1),
    "prefix": lambda batch: prefix(batch=batch, lse=P + 1),
    "rope": lambda batch: rope(batch=batch, positions=P + 1),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("batch", [MOST + 1, 2**31 - 64, 2**31 - 1])
def test_batches_whose_last_offsets_32_bits_do_not_reach(call, batch):
    assert CALLS[call](batch) == INVALID
    assert "batch" in S.svdq_last_error()


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("batch", [2, 1000, 2**30, MOST])
def test_batches_up_to_there_are_taken(call, batch):
    assert CALLS[call](batch) == ALIGNMENT


def test_workspaces_of_refused_batches():
    for batch in (MOST + 1, 2**31 - 1):
        assert S.svdq_attention_workspace_bytes(1, 20000, batch, 8, 2, 128) == 0
        assert S.svdq_attention_window_workspace_bytes(1, 20000, batch, 8, 2, 128, True, 9000, 0, 0) == 0
        assert S.svdq_attention_prefix_workspace_bytes(1, 20000, 0, batch, 8, 2, 128, True) == 0
