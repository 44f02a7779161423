"""Arguments that the token operators' binding refuses itself; none of them reaches a kernel."""
import pytest
import torch

from tests.test_gpu_tokens import DEV, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def test_workspace_in_host_memory():
    q = randn(gen(91), 64, 2, 64, dtype=torch.bfloat16).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    f = sc.rope_frequencies(64, device=DEV)
    out, lse = sc.window_attention(q, q, q, left=3, right=0, return_lse=True)
    ws = sc.Workspace(1 << 22, "cpu")
    for call in (lambda: sc.window_attention(q[:1], q, q, workspace=ws),
                 lambda: sc.window_attention_backward(q, q, q, q, out, lse, left=3, right=0, workspace=ws),
                 lambda: sc.qk_norm_rope_backward(q, q, q, q, pos, f, workspace=ws)):
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call()


@pytest.mark.parametrize("how", [dict(left=1 << 64), dict(right=(1 << 64) + 3), dict(sinks=1 << 32),
                                 dict(sinks=(1 << 32) + 4), dict(left=-(1 << 64) + 5), dict(sinks=-(1 << 32))])
def test_window_numbers_past_their_fields(how):
    """Refused, not taken modulo the C type's range."""
    q = randn(gen(92), 64, 2, 64, dtype=torch.bfloat16).to(DEV)
    out, lse = sc.window_attention(q, q, q, left=3, right=0, return_lse=True)
    how = {**dict(left=3, right=0, sinks=1), **how}
    with pytest.raises((ValueError, sc.TrSparseConvError)):
        sc.window_attention(q, q, q, **how)
    with pytest.raises((ValueError, sc.TrSparseConvError)):
        sc.window_attention_backward(q, q, q, q, out, lse, **how)


@pytest.mark.parametrize("sections", [[1 << 32], [(1 << 32) + 32], [-(1 << 32) + 3]])
def test_sections_past_their_field(sections):
    q = randn(gen(93), 64, 2, 64, dtype=torch.bfloat16).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    f = sc.rope_frequencies(64, device=DEV)
    with pytest.raises((ValueError, sc.TrSparseConvError)):
        sc.qk_norm_rope(q, q, pos, f, sections=sections)
