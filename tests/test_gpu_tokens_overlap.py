"""Outputs that lie between their inputs, or are their inputs where that is allowed; other overlaps are refused
(tests/test_tokens_overlap.py has more of those)."""
import pytest
import torch

from tests.test_gpu_tokens import DEV, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


@pytest.mark.parametrize("n", [1, 33, 400])
def test_attention_out_beside_its_inputs(n):
    """Queries, keys, values and the result as slices of the same rows, and of one buffer after another."""
    rows = randn(gen(81), n, 12, 64, dtype=torch.bfloat16).to(DEV)
    q, k, v, out = rows[:, :4], rows[:, 4:6], rows[:, 6:8], rows[:, 8:]
    how = dict(left=20, right=0, sinks=2)
    want, lse = sc.window_attention(q, k, v, return_lse=True, **how)
    assert torch.equal(sc.window_attention(q, k, v, out=out, **how), want) and torch.equal(out, want)
    for bad in (q, rows[:, 2:6], rows[:, 5:9], rows[:, 7:11]):
        with pytest.raises(sc.TrSparseConvError, match="overlaps"):
            sc.window_attention(q, k, v, out=bad, **how)
    flat = rows[:, 4:].reshape(-1)
    tail = torch.cat([flat, flat])[flat.numel():].view(n, 8, 64)[:, :4]
    assert torch.equal(sc.window_attention(q, k, v, out=tail, **how), want)


def test_norm_gradient_in_place():
    n, hq, hk, dim = 300, 6, 2, 72
    g = gen(82)
    rows = randn(g, n, hq + hk, dim, dtype=torch.bfloat16).to(DEV)
    grads = randn(g, n, hq + hk, dim, dtype=torch.bfloat16).to(DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    f = sc.rope_frequencies(dim, device=DEV)
    gain = torch.ones(dim, device=DEV)

    def split(x):
        return x[:, :hq], x[:, hq:]

    want = sc.qk_norm_rope_backward(*split(grads), *split(rows), pos, f, gain, gain)
    for target in ("dout", "input"):
        r, d = rows.clone(), grads.clone()
        dq, dk = split(d if target == "dout" else r)
        got = sc.qk_norm_rope_backward(*split(d), *split(r), pos, f, gain, gain, dq=dq, dk=dk)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), target
    with pytest.raises(sc.TrSparseConvError, match="overlaps"):
        sc.qk_norm_rope_backward(*split(grads), *split(rows), pos, f, gain, gain, dq=rows[:, 1:7], dk=rows[:, 6:])
    with pytest.raises(sc.TrSparseConvError, match="overlaps"):
        sc.qk_norm_rope(*split(rows), pos, f, q_out=rows[:, 2:], k_out=rows[:, :2])
