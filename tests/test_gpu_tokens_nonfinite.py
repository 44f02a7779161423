"""Attention where some elements are not finite: each result is what the elements it sees make of it, element by
element, against a 64-bit form that touches nothing else."""
import math

import pytest
import torch

from tests import tokens_ref as R
from tests.helpers import say
from tests.test_gpu_tokens import DEV, TD, check, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def seen_only(q, k, v, dout, see, scale):
    """out, dq, dk, dv of one head in float64, row by row over the keys that the row sees."""
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(q.shape[0]):
        j = see[i].nonzero().flatten()
        if len(j) == 0:
            continue
        p = torch.softmax(k[j] @ q[i] * scale, 0)
        out[i] = (p[:, None] * v[j]).sum(0)
        dp = v[j] @ dout[i]
        ds = p * (dp - (p * dp).sum()) * scale
        dq[i] = (ds[:, None] * k[j]).sum(0)
        dk[j] += ds[:, None] * q[i]
        dv[j] += p[:, None] * dout[i]
    return dict(out=out, dq=dq, dk=dk, dv=dv)


def case(n_q, n_k, heads, dim, dtype, left, right, sinks, spoil, seed):
    """One key-value head, `heads` query heads. spoil: tensor -> [(row, element or None for all, value)]."""
    g = gen(seed)
    dt = TD[dtype]
    t = dict(q=randn(g, n_q, heads, dim, dtype=dt, scale=1.3), k=randn(g, n_k, 1, dim, dtype=dt, scale=1.3),
             v=randn(g, n_k, 1, dim, dtype=dt), do=randn(g, n_q, heads, dim, dtype=dt))
    clean = {n: x.clone() for n, x in t.items()}
    for name, places in spoil.items():
        for row, col, value in places:
            t[name][row, 0, slice(None) if col is None else col] = value
            clean[name][row, 0, slice(None) if col is None else col] = 0
    see = R.visible(n_q, n_k, left, right, sinks)
    on = {n: x.to(DEV) for n, x in t.items()}
    how = dict(left=left, right=right, sinks=sinks)
    out, lse = sc.window_attention(on["q"], on["k"], on["v"], return_lse=True, **how)
    dq, dk, dv = sc.window_attention_backward(on["do"], on["q"], on["k"], on["v"], out, lse, **how)
    want = {n: [] for n in ("out", "dq")}
    tol = {n: [] for n in ("out", "dq")}
    want.update(dk=0, dv=0)
    tol.update(dk=0, dv=0)
    for h in range(heads):
        r = seen_only(t["q"][:, h], t["k"][:, 0], t["v"][:, 0], t["do"][:, h], see, dim ** -0.5)
        b = R.attention(clean["q"][:, h], clean["k"][:, 0], clean["v"][:, 0], see, dim ** -0.5, clean["do"][:, h])
        for n in ("out", "dq"):
            want[n].append(r[n])
            tol[n].append(b[n + "_tol"])
        for n in ("dk", "dv"):
            want[n] = want[n] + r[n]
            tol[n] = tol[n] + b[n + "_tol"]
    for n, x in (("out", out), ("dq", dq), ("dk", dk[:, 0]), ("dv", dv[:, 0])):
        w, b = (torch.stack(y[n], 1) if isinstance(y[n], list) else y[n] for y in (want, tol))
        fine = torch.isfinite(w)
        got = x.cpu()
        assert torch.equal(torch.isfinite(got), fine), (n, "finite in other places",
                                                        (torch.isfinite(got) != fine).nonzero()[:4].tolist())
        check(got[fine], w[fine], b[fine], n)


nan, inf = math.nan, math.inf
SPOIL = {
    "value in the middle": dict(v=[(170, 3, nan)]),
    "value of a sink": dict(v=[(1, None, inf)]),
    "key in the middle": dict(k=[(150, 0, nan)]),
    "query": dict(q=[(97, 5, inf)]),
    "output gradient": dict(do=[(200, 2, nan), (31, 0, -inf)]),
    "last key and value": dict(k=[(-1, 1, inf)], v=[(-1, None, nan)]),
    "runs of values": dict(v=[(i, None, nan) for i in range(60, 140)]),
}


@pytest.mark.parametrize("spoil", list(SPOIL))
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 40), ("bf16", 128), ("f16", 96), ("f32", 24), ("f32", 128)])
@pytest.mark.parametrize("heads,left,right,sinks", [(1, 20, 0, 3), (3, 40, 40, 0), (2, 5, -1, 2)])
def test_each_result_is_of_what_it_sees(dtype, dim, heads, left, right, sinks, spoil):
    say("[not finite]", dtype, dim, heads, left, right, sinks, spoil)
    case(330, 330, heads, dim, dtype, left, right, sinks, SPOIL[spoil], 61)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("f32", 80), ("bf16", 24)])
@pytest.mark.parametrize("places", [[(900, 3)], [(0, None)], [(1400, None)], [(1100, 1), (20, 7)]])
def test_single_tokens(dtype, dim, places):
    """Two new tokens of four heads against a cache of 1500: split over waves and workgroups, values and keys in and
    out of the window, or the first row's only."""
    say("[not finite, token]", dtype, dim, places)
    for name in ("v", "k"):
        case(2, 1500, 4, dim, dtype, 1000, 0, 1, {name: [(*p, nan) for p in places]}, 62)
        case(2, 1500, 4, dim, dtype, -1, 0, 0, {name: [(1499, 2, nan)]}, 63)


def test_everything_not_finite():
    """All values NaN, all output gradients infinite: every result that sees any is not finite, and the calls take
    tens of times as long as others at most (32 sums a block in vector instructions and memory latency in place of a
    few products; a key at a time by whole waves would be hundreds)."""
    n = 4096
    g = gen(64)
    q, k, v, do = (randn(g, n, 4, 64, dtype=torch.bfloat16).to(DEV) for _ in range(4))
    how = dict(left=1000, right=0, sinks=4)

    def both():
        times, at = [], [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        for _ in range(8):
            at[0].record()
            out, lse = sc.window_attention(q, k, v, return_lse=True, **how)
            at[1].record()
            grads = sc.window_attention_backward(do, q, k, v, out, lse, **how)
            at[2].record()
            at[2].synchronize()
            times.append((at[0].elapsed_time(at[1]), at[1].elapsed_time(at[2])))
        return out, lse, grads, [min(t) for t in zip(*times)]

    usual = both()[3]
    v.fill_(nan)
    do.fill_(inf)
    out, lse, grads, slow = both()
    assert bool(torch.isnan(out).all()) and bool(torch.isfinite(lse).all())
    assert not any(bool(torch.isfinite(x).any()) for x in grads)
    assert all(s < 100 * u for s, u in zip(slow, usual)), (usual, slow)
