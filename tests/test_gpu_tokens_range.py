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
