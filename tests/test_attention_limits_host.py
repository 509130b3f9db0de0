"""svdq_attention_forward at the largest numbers of keys: refused where the kernels' 32-bit counts
would not hold them, before anything is launched; CPU only."""
import pytest

pytest.importorskip("torch")
S = pytest.importorskip("bit_diffusion_model_svdq_amd")

OK, INVALID, WORKSPACE = 0, 1, 4
P = 1 << 20          # a plausible device address; never dereferenced on a refusal
MOST = 2**31 - 1 - 512


def attention(**over):
    a = dict(Q=P, ldq=8, K=P, ldk=8, V=P, ldv=8, cu_q=None, cu_k=None, batch=1, total_q=1, total_k=4000, heads_q=1,
             heads_kv=1, head_dim=8, scale=0.125, causal=1, O=P, ldo=8, lse=None, workspace=P, bytes=16)
    a.update(over)
    return S._lib.svdq_attention_forward(*a.values(), None)


@pytest.mark.parametrize("total_k", [MOST + 1, 2**31 - 31, 2**31 - 1])
@pytest.mark.parametrize("total_q", [1, 500])
def test_keys_that_32_bit_counts_do_not_hold_are_refused(total_q, total_k):
    assert attention(total_q=total_q, total_k=total_k) == INVALID
    assert S.svdq_last_error()
    assert S.svdq_attention_workspace_bytes(total_q, total_k, 1, 1, 1, 8) == 0


def test_the_most_keys_are_taken():
    """As far as the workspace, which is too small here."""
    assert S.svdq_attention_workspace_bytes(1, MOST, 1, 1, 1, 8) > 16
    assert attention(total_k=MOST) == WORKSPACE


@pytest.mark.parametrize("total_k,heads", [(2**22, 2**19), (2**20, 2**20), (MOST, 2**9), (2**28, 2**13 - 1), (300, 2**20)])
def test_many_keys_of_many_heads_make_one_share(total_k, heads):
    """Keys x heads beyond 32 bits: the plan is made in 64."""
    assert S.svdq_attention_workspace_bytes(1, total_k, 1, heads, heads, 8) == 0
    wide = heads * 8
    assert attention(total_k=total_k, heads_q=heads, heads_kv=heads, ldq=wide, ldk=wide, ldv=wide, ldo=wide, Q=None) == INVALID
