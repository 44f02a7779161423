"""Counts of heads and elements past the C ABI's 32-bit fields: refused by the binding, not taken modulo their range.
None of the calls reaches a kernel: they have no tokens, or their heads are one row repeated."""
import pytest
import torch

from tests.test_gpu_tokens import DEV

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")

FAR = 1 << 32


def rows(tokens, heads, dim=64):
    one = torch.zeros(tokens, 1, dim, dtype=torch.bfloat16, device=DEV)
    return one.expand(tokens, heads, dim)


def cache(dim=64, heads=2):
    kp, vp = (torch.zeros(0, 8, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return dict(k_pages=kp, v_pages=vp, page_table=torch.zeros(1, 0, dtype=torch.int32, device=DEV),
                k_len=torch.zeros(1, dtype=torch.int32, device=DEV))


def turn(tokens, dim=64):
    return dict(pos=torch.zeros(tokens, dtype=torch.int32, device=DEV), freqs=sc.rope_frequencies(dim, device=DEV))


@pytest.mark.parametrize("heads", [FAR + 4, FAR, (1 << 31) + 4, FAR - 4])
def test_paged_query_heads(heads):
    with pytest.raises(ValueError, match="q has"):
        sc.paged_window_attention(rows(0, heads), **cache())
    with pytest.raises(ValueError, match="q has"):
        sc.shared_prefix_attention(rows(0, heads), **cache(), prefix_pages=torch.zeros(0, dtype=torch.int32, device=DEV),
                                   prefix_len=0)
    with pytest.raises(ValueError, match="q has"):
        sc.qk_norm_rope_append(rows(0, heads), rows(0, 2), rows(0, 2), **turn(0), **cache())


@pytest.mark.parametrize("tokens", [0, 1])
def test_paged_key_heads(tokens):
    q, k = rows(tokens, 4), rows(tokens, FAR + 2)
    with pytest.raises(ValueError, match="k has"):
        sc.qk_norm_rope_append(q, k, k, **turn(tokens), **cache())


def test_paged_elements():
    dim = FAR + 64
    q = torch.zeros(0, 4, dim, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="q has"):
        sc.paged_window_attention(q, **cache(dim))


@pytest.mark.parametrize("far,tokens", [("q", 0), ("k", 0), ("both", 0), ("k", 1)])
def test_token_operators_heads(far, tokens):
    q, k = rows(tokens, FAR + 4 if far != "k" else 4), rows(tokens, FAR + 2 if far != "q" else 2)
    name = "k has" if far == "k" else "q has"
    with pytest.raises(ValueError, match=name):
        sc.qk_norm_rope(q, k, **turn(tokens), k_out=rows(tokens, 2))
    with pytest.raises(ValueError, match=name):
        sc.qk_norm_rope_backward(q, k, q, k, **turn(tokens), dk=rows(tokens, 2))
    with pytest.raises(ValueError, match=name):
        sc.window_attention(q, k, k)
    with pytest.raises(ValueError, match=name):
        sc.window_attention_backward(q, q, k, k, q, torch.zeros(4, tokens, device=DEV))


def test_token_operators_elements():
    q = torch.zeros(0, 4, FAR + 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="q has"):
        sc.window_attention(q, q, q)
