"""Layouts other than slices of one row: heads before tokens, gaps, broadcast tokens and heads; no keys, no queries."""
import pytest
import torch

from tests.test_gpu_tokens import DEV, TD, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def heads_first(t):
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def gaps(t):
    n, h, d = t.shape
    room = t.new_full((n + 1, 2 * h + 1, d + 8), float("nan"))
    room[1:, 1::2, :d] = t
    return room[1:, 1::2, :d]


def alternating(t):
    return torch.stack([t, torch.full_like(t, float("nan"))], 2).view(t.shape[0], -1, t.shape[2])[:, ::2]


LAYOUTS = dict(heads_first=heads_first, gaps=gaps, alternating=alternating)


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("f32", 40)])
@pytest.mark.parametrize("n,m,left,right,sinks", [(300, 300, 40, 40, 3), (2, 900, -1, 0, 0), (70, 200, 30, 0, 40)])
def test_attention_layouts(layout, dtype, dim, n, m, left, right, sinks):
    """The same bits whatever the strides."""
    g = gen(101)
    q, do = (randn(g, n, 6, dim, dtype=TD[dtype]).to(DEV) for _ in range(2))
    k, v = (randn(g, m, 2, dim, dtype=TD[dtype]).to(DEV) for _ in range(2))
    how = dict(left=left, right=right, sinks=sinks)
    out, lse = sc.window_attention(q, k, v, return_lse=True, **how)
    want = sc.window_attention_backward(do, q, k, v, out, lse, **how)
    f = LAYOUTS[layout]
    into = f(torch.zeros_like(q))
    got, lse2 = sc.window_attention(f(q), f(k), v, return_lse=True, out=into, **how)
    assert torch.equal(got, out) and torch.equal(lse, lse2)
    assert torch.equal(sc.window_attention(q, k, f(v), **how), out)
    grads = sc.window_attention_backward(f(do), f(q), k, f(v), f(out), lse, **how)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_norm_layouts(layout):
    f = LAYOUTS[layout]
    g = gen(102)
    n, dim = 123, 72
    q, k, dq, dk = (randn(g, n, h, dim, dtype=torch.bfloat16).to(DEV) for h in (5, 2, 5, 2))
    pos = torch.randint(0, 999, (n, 3), generator=g, dtype=torch.int32).to(DEV)
    freqs = sc.rope_frequencies(dim, 3, device=DEV)
    gains = [(1 + 0.2 * torch.randn(h, dim, generator=g)).to(DEV) for h in (5, 2)]
    want = sc.qk_norm_rope(q, k, pos, freqs, *gains)
    got = sc.qk_norm_rope(f(q), f(k), pos, freqs, *gains, q_out=f(torch.zeros_like(q)), k_out=f(torch.zeros_like(k)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = sc.qk_norm_rope_backward(dq, dk, q, k, pos, freqs, *gains)
    got = sc.qk_norm_rope_backward(f(dq), f(dk), f(q), f(k), pos, freqs, *gains, dq=f(torch.zeros_like(q)),
                                   dk=f(torch.zeros_like(k)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_broadcast_inputs(dtype):
    """One query, key, value or output gradient for all tokens or heads, as strides of zero."""
    g = gen(103)
    n, dim = 200, 64
    how = dict(left=30, right=30, sinks=2)
    t = {x: randn(g, n, 4, dim, dtype=TD[dtype]).to(DEV) for x in ("q", "k", "v", "do")}

    def both(q, k, v, do):
        out, lse = sc.window_attention(q, k, v, return_lse=True, **how)
        return [out, lse, *sc.window_attention_backward(do, q, k, v, out, lse, **how)]

    for name in t:
        for one in (t[name][:1].expand(n, 4, dim), t[name][:, :1].expand(n, 4, dim)):
            got, want = both(**{**t, name: one}), both(**{**t, name: one.contiguous()})
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,m", [(0, 0), (0, 37), (37, 0), (1, 0), (300, 0)])
@pytest.mark.parametrize("packed", [False, True])
def test_no_keys_or_queries(dtype, n, m, packed):
    q, k = (torch.ones(x, 4, 32, dtype=TD[dtype], device=DEV) for x in (n, m))
    how = dict(left=5, right=5, sinks=3)
    if packed:  # two sequences
        how.update(cu_q=torch.tensor([0, n // 2, n], dtype=torch.int32, device=DEV),
                   cu_k=torch.tensor([0, m // 3, m], dtype=torch.int32, device=DEV))
    out, lse = sc.window_attention(q, k, k, return_lse=True, **how)
    assert out.shape == (n, 4, 32) and lse.shape == (4, n)
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())
    dq, dk, dv = sc.window_attention_backward(q, q, k, k, out, lse, **how)
    assert dq.shape == q.shape and dk.shape == dv.shape == k.shape
    assert not bool(dq.any()) and not bool(dk.any()) and not bool(dv.any())
