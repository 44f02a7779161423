"""The half types' attention where weights and gradients spread over more than
the type's range, against the 64-bit forms of tests/tokens_ref.py."""
import math

import pytest
import torch

from tests import tokens_ref as R
from tests.helpers import say
from tests.test_gpu_tokens import DEV, TD, check, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def led(n, nq, heads, dim, dtype, lead, seed, at=0, value=0.0):
    """q [nq, heads, dim], k, v [n, heads, dim]: key `at` leads the scaled scores of every row by about `lead`
    nats and has the value `value`; the others' scores spread by half a nat, their values around one."""
    g = gen(seed)
    dt = TD[dtype]
    q = randn(g, nq, heads, dim, dtype=dt, scale=0.7)
    k = randn(g, n, heads, dim, dtype=dt, scale=0.7)
    v = (1 + 0.25 * torch.randn(n, heads, dim, generator=g)).to(dt)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[at] = 0
    k[at, :, 0] = lead * dim ** 0.5 / 8
    v[at] = value
    return q, k, v


LEADS = [10.0, 12.0, 14.0, 16.0, 18.0]


@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_leading_sink_of_a_cache(dtype, lead):
    """Single tokens against 8192 keys, the first of which takes most of the weight and has the value zero: the
    result is what the others add, each within the roundings of its own weight (not of the leading one)."""
    n, heads, dim = 8192, 2, 64
    say("[leading sink, token]", dtype, lead)
    q, k, v = led(n, 1, heads, dim, dtype, lead, 5)
    out, lse = sc.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), left=n, right=0, sinks=1, return_lse=True)
    for h in range(heads):
        r = R.attention(q[:, h], k[:, h], v[:, h], torch.ones(1, n, dtype=torch.bool), dim ** -0.5)
        check(out[:, h], r["out"], r["out_tol"], f"head {h}")
        check(lse[h], r["lse"], r["lse_tol"], f"lse {h}")


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("dtype,at,left", [("f16", 0, 700), ("f16", 0, -1), ("f16", 600, -1), ("bf16", 0, 700)])
def test_attention_leading_key(dtype, at, left, lead, dim):
    """The same in tiles of rows; also where the leading key comes in the middle of the walk."""
    n, heads = 1500, 1
    say("[leading key]", dtype, at, left, lead, dim)
    q, k, v = led(n, n, heads, dim, dtype, lead, 6, at)
    out, lse = sc.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), left=left, right=0, sinks=1, return_lse=True)
    r = R.attention(q[:, 0], k[:, 0], v[:, 0], R.visible(n, n, left, 0, 1), dim ** -0.5)
    check(out[:, 0], r["out"], r["out_tol"], "out")
    check(lse[0], r["lse"], r["lse_tol"], "lse")


def test_attention_scores_that_fall_and_rise():
    """Blocks of 64 keys whose scores fall by 7 nats a block or two and rise again, only the lowest (14 nats down)
    with values: the result is their small share of the weight."""
    n, dim = 640, 64
    g = gen(7)
    q, k = randn(g, 300, 1, dim, dtype=torch.float16, scale=0.3), randn(g, n, 1, dim, dtype=torch.float16, scale=0.3)
    level = torch.tensor([14.0, 14, 7, 7, 0, 0, 7, 14, 14, 7]).repeat_interleave(64)
    q[..., 0] = 4.0
    k[..., 0] = (level * dim ** 0.5 / 4).half()[:, None]
    v = (4096 * (1 + 0.25 * torch.randn(n, 1, dim, generator=g))).half()  # the share is about 3e-7
    v[level > 0] = 0
    out, lse = sc.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), return_lse=True)
    r = R.attention(q[:, 0], k[:, 0], v[:, 0], torch.ones(300, n, dtype=torch.bool), dim ** -0.5)
    check(out[:, 0], r["out"], r["out_tol"], "out")
    check(lse[0], r["lse"], r["lse_tol"], "lse")


# ---------------------------------------------------------------------------
# Gradients
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lead", [12.0, 15.0, 18.0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradient_of_values_beside_a_leading_key(dtype, lead, dim):
    """dv of the keys that a leading one leaves small weights: their sums over 1000 rows of a large dout, within
    the roundings of those weights."""
    n = 1000
    say("[leading key, dv]", dtype, lead, dim)
    q, k, v = led(n, n, 1, dim, dtype, lead, 16)
    dout = randn(gen(17), n, 1, dim, dtype=TD[dtype], scale=1000.0)
    on = [x.to(DEV) for x in (q, k, v, dout)]
    out, lse = sc.window_attention(*on[:3], return_lse=True)
    dv = sc.window_attention_backward(on[3], *on[:3], out, lse)[2]
    r = R.attention(q[:, 0], k[:, 0], v[:, 0], torch.ones(n, n, dtype=torch.bool), dim ** -0.5, dout[:, 0])
    past = r["dv"].abs() >= torch.finfo(TD[dtype]).max * (1 + R.U[TD[dtype]] / 2)  # of the leading key: infinite
    check(dv[:, 0], torch.where(past, r["dv"].sign() * math.inf, r["dv"]), r["dv_tol"], "dv")


def exact_grads(q, k, v, dout, see, scale):
    """dq, dk, dv of one head in float64."""
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    p = torch.softmax((q @ k.T * scale).masked_fill(~see, -math.inf), -1)
    dp = dout @ v.T
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    return ds @ k, ds.T @ q, p.T @ dout


def rms_of_roundings(got, want, dtype, part=slice(None)):
    """Rms error over that of rounding the exact result once."""
    once = (want.to(dtype).double() - want)[part].norm()
    return float((got.cpu().double() - want)[part].norm() / once)


# two independent roundings of the type on the way to every sum (the weights' or dS's, and the last), and a sixth
# for what they share
TWICE = math.sqrt(2) * 7 / 6


@pytest.mark.parametrize("size", [1e-4, 1e-3, 1.0, 1e3])
@pytest.mark.parametrize("dtype,dim", [("f16", 32), ("f16", 64), ("f16", 96), ("f16", 128), ("bf16", 64)])
def test_gradient_keeps_its_precision_at_any_size(dtype, dim, size):
    """Long windows and output gradients of any size that the type holds: the score gradients are a thousandth of
    them and less, and still cost a sum no more than its own last rounding."""
    n, left, sinks = 3000, 1023, 4
    say("[gradient size]", dtype, dim, size)
    g = gen(23)
    q, k, v, dout = (randn(g, n, 1, dim, dtype=TD[dtype], scale=s) for s in (1.3, 1.3, 1.0, size))
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(left=left, right=0, sinks=sinks)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    got = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    want = exact_grads(q[:, 0], k[:, 0], v[:, 0], dout[:, 0], R.visible(n, n, left, 0, sinks), dim ** -0.5)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        ratio = rms_of_roundings(a[:, 0], b, TD[dtype])
        assert ratio < TWICE, (name, ratio)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("values", [1e-3, 1e4])
def test_gradient_of_small_and_large_values(values, dim):
    """fp16 values from near its smallest normal to near its largest, which the score gradients follow."""
    n, left = 1500, 100
    say("[gradient of values]", values, dim)
    g = gen(41)
    q, k, v, dout = (randn(g, n, 1, dim, dtype=torch.float16, scale=s) for s in (1.3, 1.3, values, 1.0))
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(left=left, right=0)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    got = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    want = exact_grads(q[:, 0], k[:, 0], v[:, 0], dout[:, 0], R.visible(n, n, left, 0, 0), dim ** -0.5)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        ratio = rms_of_roundings(a[:, 0], b, torch.float16)
        assert ratio < TWICE, (name, ratio)


def test_gradient_of_rows_of_different_sizes():
    """Two sequences whose output gradients are 2^12 apart, and rows in one that are 2^10 above their neighbours:
    either sequence's, and either rows', gradients keep their precision."""
    n, dim, left = 1500, 64, 300
    g = gen(29)
    q, k, v, dout = (randn(g, 2 * n, 1, dim, dtype=torch.float16, scale=s) for s in (1.3, 1.3, 1.0, 1.0))
    dout[:n] /= 4096
    dout[n + 10::50] *= 1024
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(cu_q=cu, cu_k=cu, left=left, right=0)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    got = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    see = R.visible(n, n, left, 0, 0)
    for b in range(2):
        s = slice(b * n, (b + 1) * n)
        want = exact_grads(q[s, 0], k[s, 0], v[s, 0], dout[s, 0], see, dim ** -0.5)
        large = torch.arange(n) % 50 == 10
        for part in (large, ~large):
            ratio = rms_of_roundings(got[0][s, 0], want[0], torch.float16, part)
            assert ratio < TWICE, (b, "dq", ratio)
        for name, x, y in zip(("dk", "dv"), got[1:], want[1:]):
            assert rms_of_roundings(x[s, 0], y, torch.float16) < TWICE, (b, name)


def score_grad_bounds(q, k, v, see, scale, dout):
    """Elementwise bounds of dq and dk as tests/tokens_ref.py's, but for a delta that is the row's own sum of P dP:
    nothing in it is rounded to the type."""
    u, up, e, d = R.U[q.dtype], R.U[q.dtype], R.E, q.shape[-1]
    dtype = q.dtype
    q, k, v, g = (x.double() for x in (q, k, v, dout))
    n = max(see.shape) + 64
    z = (q @ k.T * scale).masked_fill(~see, -math.inf)
    p = torch.softmax(z, -1)
    ep = 2 * ((d + 2) * e * float((q.abs() @ k.abs().T * scale).masked_fill(~see, 0.0).max())
              + 6 * e * float(z.masked_fill(~see, 0.0).abs().max()) + 8 * e) + n * e
    dp, gv = g @ v.T, g.abs() @ v.abs().T
    delta, gw = (p * dp).sum(-1, keepdim=True), (p * gv).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eds = (up + ep + (2 + n) * e) * ds.abs() + p * (1 + ep) * (
        (d + 2) * e * gv + ((d + n) * e + ep) * gw + ep * (dp.abs() + delta.abs()))
    dq, dk = scale * ds @ k, scale * ds.T @ q
    tiny = u * R.TINY[dtype]
    return (dq, u * dq.abs() + 1.01 * scale * eds @ k.abs() + tiny,
            dk, u * dk.abs() + 1.01 * scale * eds.T @ q.abs() + tiny)


@pytest.mark.parametrize("size", [1.0, 100.0])
@pytest.mark.parametrize("lead", [0.0, 10.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
def test_gradient_of_scores_beside_a_leading_key(dtype, dim, lead, size):
    """dq and dk where one key of value zero takes most of the weight. The outputs, which give a first dout . out of
    a row, are subnormal in fp16 then; it must not spoil dq. (Past heads of 64 the rounding of ordinary outputs is
    in dq's bound.)"""
    n = 1200
    say("[leading key, dq and dk]", dtype, dim, lead, size)
    g = gen(31)
    q, k, _ = led(n, n, 1, dim, dtype, lead, 18)
    v, dout = (randn(g, n, 1, dim, dtype=TD[dtype], scale=s) for s in (1.0, size))
    v[0] = 0
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(left=-1, right=0, sinks=1)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    dq, dk, _ = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    one = [x[:, 0] for x in (q, k, v)]
    see = R.visible(n, n, -1, 0, 0)
    want_q, tol_q, want_k, tol_k = score_grad_bounds(*one, see, dim ** -0.5, dout[:, 0])
    loose = R.attention(*one, see, dim ** -0.5, dout[:, 0])["dq_tol"]
    ordinary = out[:, 0].cpu().abs().amax(-1, keepdim=True) >= R.TINY[TD[dtype]]
    check(dq[:, 0], want_q, torch.where(ordinary & (dim > 64), loose, tol_q), "dq")
    check(dk[:, 0], want_k, tol_k, "dk")


@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (64, 64, 4), (7, 0, 3), (31, 5, 33), (0, 0, 1)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("bf16", 24), ("f16", 40)])
def test_gradient_of_keys_without_the_outputs_rounding(dtype, dim, left, right, sinks):
    """dk within a bound that has no term for the rounding of the forward's result."""
    n = 333
    say("[dk]", dtype, dim, left, right, sinks)
    g = gen(37)
    q, k, v, dout = (randn(g, n, 1, dim, dtype=TD[dtype], scale=s) for s in (1.3, 1.3, 1.0, 1.0))
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(left=left, right=right, sinks=sinks)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    dk = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)[1]
    _, _, want, tol = score_grad_bounds(q[:, 0], k[:, 0], v[:, 0], R.visible(n, n, left, right, sinks), dim ** -0.5,
                                        dout[:, 0])
    check(dk[:, 0], want, tol, "dk")


@pytest.mark.parametrize("dim", [64, 128])
def test_gradient_beside_an_outlier(dim):
    """One row's output gradient 2^22 above the others': dk of the keys that it does not see, but for those that
    share a block of 32 with one that it does, is as exact as without it."""
    n, left, at = 1500, 40, 700
    g = gen(47)
    q, k, v, dout = (randn(g, n, 1, dim, dtype=torch.float16, scale=s) for s in (1.3, 1.3, 1.0, 2.0 ** -9))
    dout[at] *= 2.0 ** 22
    on = [x.to(DEV) for x in (q, k, v, dout)]
    how = dict(left=left, right=0)
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    got = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    want = exact_grads(q[:, 0], k[:, 0], v[:, 0], dout[:, 0], R.visible(n, n, left, 0, 0), dim ** -0.5)
    first, end = (at - left) // 32 * 32, at // 32 * 32 + 32
    for name, part in (("before", slice(0, first)), ("after", slice(end, None)), ("near", slice(end, end + 64))):
        ratio = rms_of_roundings(got[1][:, 0], want[1], torch.float16, part)
        assert ratio < TWICE, (name, ratio)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("spread,left,right,length", [(8.0, 512, 512, 8192), (3.0, 512, 512, 8192), (1.3, 0, 0, 8192),
                                                      (1.3, 512, 0, 32)])
def test_sharp_attention_keeps_the_usual_path(spread, left, right, length, dim):
    """Rows that give nearly all their weight to one key have score gradients of rounding noise; raising that into
    fp16's range would only overflow where the noise is another. fp16 takes no more than twice bf16's time."""
    n = 8192
    g = gen(43)
    cu = torch.arange(0, n + 1, length, dtype=torch.int32, device=DEV)
    how = dict(cu_q=cu, cu_k=cu, left=left, right=right)
    times = {}
    for dtype in (torch.bfloat16, torch.float16):
        q, k, v, dout = (randn(g, n, 8, dim, dtype=dtype, scale=s).to(DEV) for s in (spread, spread, 1.0, 1.0))
        times[dtype] = []
        for same in (False, True):  # queries of their own, or each its key
            args = (k if same else q, k, v)
            out, lse = sc.window_attention(*args, return_lse=True, **how)
            at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            best = math.inf
            for _ in range(12):
                at[0].record()
                sc.window_attention_backward(dout, *args, out, lse, **how)
                at[1].record()
                at[1].synchronize()
                best = min(best, at[0].elapsed_time(at[1]))
            times[dtype].append(best)
    assert all(a < 2 * b for a, b in zip(times[torch.float16], times[torch.bfloat16])), times
