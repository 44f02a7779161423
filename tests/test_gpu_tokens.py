"""The token operators on the GPU against their 64-bit forms, with elementwise
bounds of the roundings on the way (tests/tokens_ref.py)."""
import math

import numpy as np
import pytest
import torch

from tests import tokens_ref as R
from tests.helpers import say

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")
DEV = "cuda:0"
TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def check(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    same = (got == ref) | ((got - ref).abs() <= tol) | (torch.isnan(got) & torch.isnan(ref))
    if not bool(same.all()):
        bad = (~same).nonzero()[0].tolist()
        worst = torch.where(same, torch.zeros_like(got), (got - ref).abs() / tol.clamp_min(1e-300)).nan_to_num(1e9)
        raise AssertionError(f"{what}: {int((~same).sum())} of {got.numel()} off, first at {bad}: "
                             f"{float(got[tuple(bad)])} for {float(ref[tuple(bad)])}, worst {float(worst.max()):.2f} "
                             f"times its bound")


# ---------------------------------------------------------------------------
# Norm and rotation
# ---------------------------------------------------------------------------
def norm_case(tokens, hq, hk, dim, dtype, axes, interleaved, gain, seed, span=64, left_over=0):
    g = gen(seed)
    dt = TD[dtype]
    qkv = randn(g, tokens, hq + 2 * hk, dim, dtype=dt, scale=1.7)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    coords = torch.randint(0, span, (tokens, 4), generator=g, dtype=torch.int32)
    pos = coords[:, 1:1 + axes]
    n = max(0, dim // 2 // axes - left_over)
    freqs = sc.rope_frequencies(dim, axes, device="cpu")
    shape = {"none": None, "shared": (dim,), "heads": (0, dim)}[gain]
    gains = [None if shape is None else 1 + 0.2 * torch.randn((h if shape[0] == 0 else dim,) + shape[1:], generator=g)
             for h in (hq, hk)]
    return q, k, pos, freqs, gains, [n] * axes, interleaved


def on_gpu(q, k, pos, gains, freqs, hq):
    """The same views, of parents on the GPU."""
    parent = q._base.to(DEV) if q._base is not None else q.to(DEV)
    hk = k.shape[1]
    gq, gk = parent[:, :hq], parent[:, hq:hq + hk]
    coords = pos._base.to(DEV)
    return gq, gk, coords[:, 1:1 + pos.shape[1]], [None if x is None else x.to(DEV) for x in gains], freqs.to(DEV)


NORM = [
    (1, 1, 1, 8, "f32", 1, True, "none", 0), (1, 16, 4, 128, "bf16", 1, False, "shared", 0),
    (5, 3, 1, 24, "f16", 3, False, "heads", 0), (37, 12, 12, 128, "bf16", 3, True, "heads", 0),
    (64, 6, 2, 72, "f32", 3, False, "heads", 0), (131, 2, 2, 64, "bf16", 3, True, "shared", 3),
    (300, 5, 3, 96, "f16", 2, True, "heads", 0), (77, 9, 1, 16, "f32", 1, False, "shared", 2),
    (1000, 16, 16, 64, "f16", 3, True, "none", 0), (33, 7, 5, 40, "bf16", 2, False, "heads", 1),
    (9, 70, 1, 112, "f32", 3, True, "shared", 0), (3001, 1, 1, 120, "bf16", 1, False, "heads", 0),
]


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope(case):
    tokens, hq, hk, dim, dtype, axes, il, gain, left_over = case
    say("[norm_rope]", case)
    q, k, pos, freqs, gains, sec, _ = norm_case(tokens, hq, hk, dim, dtype, axes, il, gain, 3, left_over=left_over)
    gq, gk, gpos, ggain, gfreq = on_gpu(q, k, pos, gains, freqs, hq)
    how = dict(q_gain=ggain[0], k_gain=ggain[1], sections=sec, interleaved=il, eps=1e-5)
    outs = sc.qk_norm_rope(gq, gk, gpos, gfreq, **how)
    ang = R.angles(pos, freqs, sec)
    for x, gn, out, what in ((q, gains[0], outs[0], "q"), (k, gains[1], outs[1], "k")):
        check(out, R.norm_rope(x, gn, ang, il, 1e-5), R.norm_rope_bound(x, gn, ang, il, 1e-5, TD[dtype]), what)
    # backward
    g = gen(4)
    dq, dk = randn(g, tokens, hq, dim, dtype=TD[dtype]), randn(g, tokens, hk, dim, dtype=TD[dtype])
    got = sc.qk_norm_rope_backward(dq.to(DEV), dk.to(DEV), gq, gk, gpos, gfreq, **how)
    for x, gn, dy, dx, dg, what in ((q, gains[0], dq, got[0], got[2], "q"), (k, gains[1], dk, got[1], got[3], "k")):
        ref, refg = R.norm_rope_grad(x, gn, ang, il, 1e-5, dy)
        tol, tolg = R.norm_rope_grad_bounds(x, gn, ang, il, 1e-5, dy, TD[dtype])
        check(dx, ref, tol, "d" + what)
        if gn is None:
            assert dg is None
        else:
            check(dg, refg, tolg, f"d{what}_gain")
    again = sc.qk_norm_rope_backward(dq.to(DEV), dk.to(DEV), gq, gk, gpos, gfreq, **how)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))


def test_norm_rope_in_place_and_strided_outputs():
    q, k, pos, freqs, gains, sec, il = norm_case(50, 4, 2, 64, "bf16", 3, True, "heads", 8)
    gq, gk, gpos, ggain, gfreq = on_gpu(q, k, pos, gains, freqs, 4)
    how = dict(q_gain=ggain[0], k_gain=ggain[1], interleaved=il)
    want = sc.qk_norm_rope(gq, gk, gpos, gfreq, **how)
    room = torch.full((50, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    sc.qk_norm_rope(gq, gk, gpos, gfreq, q_out=room[:, 1:5], k_out=room[:, 6:8], **how)
    assert torch.equal(room[:, 1:5], want[0]) and torch.equal(room[:, 6:8], want[1])
    assert bool((room[:, [0, 5, 8]] == 7).all())
    sc.qk_norm_rope(gq, gk, gpos, gfreq, q_out=gq, k_out=gk, **how)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])


def test_norm_rope_large_positions_and_values():
    """Angles of positions up to 2^31 - 1 stay exact; huge, tiny, zero rows and rows with NaN or infinities
    keep to themselves."""
    g = gen(5)
    q = torch.randn(6, 2, 32, generator=g)
    q[1] *= 1e15
    q[2] *= 1e-15
    q[3] = 0
    k = torch.randn(6, 1, 32, generator=g)
    pos = torch.tensor([0, 1, 65535, 1 << 20, (1 << 31) - 1, -12345], dtype=torch.int32)
    freqs = sc.rope_frequencies(32, 1, device="cpu")
    a, b = sc.qk_norm_rope(q.to(DEV), k.to(DEV), pos.to(DEV), freqs.to(DEV))
    ang = R.angles(pos, freqs, [16])
    for x, out in ((q, a), (k, b)):
        # the product of position and frequency is reduced in 64 bits: 2^31 turns of 2^-52 each
        tol = R.norm_rope_bound(x, None, ang, False, 1e-6, torch.float32) + 4e-6 * R.norm_rope(
            x, None, ang * 0, False, 1e-6).abs().amax(-1, keepdim=True)
        check(out, R.norm_rope(x, None, ang, False, 1e-6), tol, "out")
    q[4, 0, 3] = math.nan
    q[5, 1, 0] = math.inf
    a, _ = sc.qk_norm_rope(q.to(DEV), k.to(DEV), pos.to(DEV), freqs.to(DEV))
    fine = torch.isfinite(a.cpu()).all(-1)
    want = torch.ones(6, 2, dtype=torch.bool)
    want[4, 0] = want[5, 1] = False
    assert torch.equal(fine, want)


def test_norm_rope_gradient_against_differences():
    """fp32 gradients against central differences of the 64-bit form."""
    q, k, pos, freqs, gains, sec, il = norm_case(3, 2, 1, 16, "f32", 2, True, "shared", 6)
    g = gen(7)
    dq, dk = torch.randn(3, 2, 16, generator=g), torch.randn(3, 1, 16, generator=g)
    gq, gk, gpos, ggain, gfreq = on_gpu(q, k, pos, gains, freqs, 2)
    got = sc.qk_norm_rope_backward(dq.to(DEV), dk.to(DEV), gq, gk, gpos, gfreq, q_gain=ggain[0], k_gain=ggain[1],
                                   sections=sec, interleaved=il, eps=1e-5)
    ang = R.angles(pos, freqs, sec)

    def loss(x, gn):
        return float((R.norm_rope(x, gn, ang, il, 1e-5) * dq.double()).sum())

    x, gn, h = q.double().clone(), gains[0].double().clone(), 1e-5
    for i in range(0, x.numel(), 7):
        hi, lo = x.flatten().clone(), x.flatten().clone()
        hi[i] += h
        lo[i] -= h
        num = (loss(hi.view_as(x), gn) - loss(lo.view_as(x), gn)) / (2 * h)
        assert abs(num - float(got[0].flatten()[i])) <= 1e-4 * (1 + abs(num))
    for i in range(gn.numel()):
        hi, lo = gn.clone(), gn.clone()
        hi[i] += h
        lo[i] -= h
        num = (loss(x, hi) - loss(x, lo)) / (2 * h)
        assert abs(num - float(got[2][i])) <= 1e-4 * (1 + abs(num))


def test_norm_rope_empty():
    q = torch.empty(0, 3, 16, device=DEV)
    pos = torch.empty(0, 1, dtype=torch.int32, device=DEV)
    f = sc.rope_frequencies(16, device=DEV)
    gain = torch.ones(16, device=DEV)
    a, b = sc.qk_norm_rope(q, q, pos, f, q_gain=gain)
    assert a.shape == b.shape == (0, 3, 16)
    out = sc.qk_norm_rope_backward(q, q, q, q, pos, f, q_gain=gain)
    assert torch.equal(out[2], torch.zeros(16, device=DEV)) and out[3] is None


# ---------------------------------------------------------------------------
# Windowed attention
# ---------------------------------------------------------------------------
def attn_inputs(lens_q, lens_k, room, hk, group, dim, dtype, seed, scale=1.3):
    """Packed q, k, v on the CPU as slices of wider rows; room[b]: rows of k and v of a sequence."""
    g = gen(seed)
    dt = TD[dtype]
    hq = hk * group
    nq, nk = sum(lens_q), sum(room)
    q = randn(g, nq, hq + 1, dim, dtype=dt, scale=scale)
    kv = randn(g, nk, 2 * hk + 1, dim, dtype=dt, scale=scale)
    return q, kv, np.concatenate([[0], np.cumsum(lens_q)]), np.concatenate([[0], np.cumsum(room)])


def reference(q, k, v, cu_q, cu_k, lens_k, group, left, right, sinks, scale, dout=None):
    """The packed batch, sequence by sequence and head by head: dict as tokens_ref.attention's."""
    hq = q.shape[1]
    out = {n: torch.zeros(q.shape, dtype=torch.float64) for n in ("out", "out_tol", "dq", "dq_tol")}
    out.update({n: torch.zeros(k.shape, dtype=torch.float64) for n in ("dk", "dk_tol", "dv", "dv_tol")})
    out.update({n: torch.zeros(hq, q.shape[0], dtype=torch.float64) for n in ("lse", "lse_tol")})
    u = R.U[q.dtype]
    for b, lk in enumerate(lens_k):
        sq, sk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b] + lk)
        lq = int(cu_q[b + 1] - cu_q[b])
        see = R.visible(lq, lk, left, right, sinks)
        for h in range(hq):
            kh = h // group
            r = R.attention(q[sq, h], k[sk, kh], v[sk, kh], see, scale, None if dout is None else dout[sq, h])
            for n in ("out", "out_tol", "dq", "dq_tol"):
                if n in r:
                    out[n][sq, h] = r[n]
            out["lse"][h, sq], out["lse_tol"][h, sq] = r["lse"], r["lse_tol"]
            if dout is not None:
                for n in ("dk", "dv"):
                    out[n][sk, kh] += r[n]
                    # the final rounding is of the sum over the group's heads
                    out[n + "_tol"][sk, kh] += r[n + "_tol"]
    return out


def run_case(lens_q, lens_k, hk, group, dim, dtype, left, right, sinks, room=None, backward=True, seed=11, scale=None,
             broadcast=False, poison=False):
    say("[window_attention]", lens_q, lens_k, hk, group, dim, dtype, left, right, sinks, room, scale)
    room_ = room or lens_k
    q, kv, cu_q, cu_k = attn_inputs(lens_q, lens_k, room_, hk, group, dim, dtype, seed)
    hq = hk * group
    if poison:  # NaN and infinities where nobody looks
        for b, lk in enumerate(lens_k):
            lq = lens_q[b]
            see = R.visible(lq, lk, left, right, sinks)
            dead = (~see.any(0)).nonzero().flatten() + int(cu_k[b])
            kv[dead] = math.nan
            kv[dead[::2]] = math.inf
            kv[int(cu_k[b]) + lk:int(cu_k[b + 1])] = math.nan
    qd, kvd = q.to(DEV), kv.to(DEV)
    qv, kk, vv = q[:, 1:], kv[:, :hk], kv[:, hk:2 * hk]
    qg, kg, vg = qd[:, 1:], kvd[:, :hk], kvd[:, hk:2 * hk]
    if broadcast:  # one key-value head for all
        kk, vv = kk[:, :1].expand(-1, hk, -1), vv[:, :1].expand(-1, hk, -1)
        kg, vg = kg[:, :1].expand(-1, hk, -1), vg[:, :1].expand(-1, hk, -1)
    i32 = dict(dtype=torch.int32, device=DEV)
    how = dict(cu_q=torch.tensor(cu_q, **i32), cu_k=torch.tensor(cu_k, **i32), left=left, right=right, sinks=sinks,
               scale=scale)
    if room is not None:
        how["k_len"] = torch.tensor(lens_k, **i32)
    g = gen(seed + 1)
    dout = randn(g, sum(lens_q), hq, dim, dtype=TD[dtype])
    s = dim ** -0.5 if scale is None else scale
    ref = reference(qv, kk, vv, cu_q, cu_k, lens_k, group, left, right, sinks, s, dout if backward else None)
    out, lse = sc.window_attention(qg, kg, vg, return_lse=True, **how)
    check(out, ref["out"], ref["out_tol"], "out")
    check(lse, ref["lse"], ref["lse_tol"], "lse")
    assert torch.equal(sc.window_attention(qg, kg, vg, **how), out)
    if not backward:
        return
    got = sc.window_attention_backward(dout.to(DEV), qg, kg, vg, out, lse, **how)
    for x, n in zip(got, ("dq", "dk", "dv")):
        check(x, ref[n], ref[n + "_tol"], n)
    again = sc.window_attention_backward(dout.to(DEV), qg, kg, vg, out, lse, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


WINDOWS = [(-1, -1, 0), (-1, 0, 0), (7, 0, 3), (64, 64, 4), (0, 0, 0), (0, 0, 1), (31, 5, 33), (130, 0, 128), (5, -1, 2)]


@pytest.mark.parametrize("left,right,sinks", WINDOWS)
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("f32", 40)])
def test_attention_windows(dtype, dim, left, right, sinks):
    run_case([150, 1, 77], [150, 1, 77], 2, 2, dim, dtype, left, right, sinks)


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 64, 72, 80, 96, 104, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_head_sizes(dtype, dim):
    run_case([67, 130], [67, 130], 1, 3, dim, dtype, 40, 9, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]), ([2], [1]), ([0, 3], [5, 0]), ([130, 40], [5, 300]), ([1, 1, 1], [200, 1, 33]), ([33], [32]),
    ([64, 0, 128, 129], [64, 0, 128, 129]), ([3, 500], [900, 500]), ([127, 1, 128], [255, 64, 65])])
def test_attention_lengths(dtype, lens_q, lens_k):
    """Empty sequences, rows before the first key (they see nothing), keys only, one token."""
    run_case(lens_q, lens_k, 1, 2, 32, dtype, 50, 0, 3)
    run_case(lens_q, lens_k, 2, 1, 64, dtype, -1, -1, 0)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f32", 128), ("f32", 32), ("bf16", 24)])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (300, 4), (31, 0), (32, 64)])
@pytest.mark.parametrize("batch,group", [(1, 4), (5, 1), (3, 8), (2, 40)])
def test_token_form(dtype, dim, left, sinks, batch, group):
    """One new token a sequence, caches with room to grow, few keys and many (split over the keys)."""
    rng = np.random.default_rng(batch)
    lens_k = [int(x) for x in rng.integers(1, 1500, size=batch)]
    room = [n + int(x) for n, x in zip(lens_k, rng.integers(0, 100, size=batch))]
    run_case([1] * batch, lens_k, 2, group, dim, dtype, left, 0, sinks, room=room, backward=False)


def test_token_form_edge_lengths():
    """Caches that are empty, hold one token, end on and beside a tile's edge; several new tokens at once."""
    lens = [0, 1, 31, 32, 33, 63, 64, 65, 128, 129]
    for n, dtype in ((1, "bf16"), (2, "f32"), (3, "f16")):
        run_case([n] * len(lens), lens, 1, 2, 64, dtype, 40, 0, 2, room=[x + 5 for x in lens], backward=n == 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k,left,right,sinks", [
    ([1, 1], [400, 90], 20, 0, 4), ([100], [300], 10, 0, 1), ([40, 3], [40, 200], 5, 0, 0), ([200], [260], 33, 0, 3)])
def test_attention_unseen_nan(dtype, lens_q, lens_k, left, right, sinks):
    """NaN and infinities in keys and values that no row sees, and past k_len, reach nothing."""
    run_case(lens_q, lens_k, 2, 2, 64, dtype, left, right, sinks, room=[n + 30 for n in lens_k], poison=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_nan_stays_with_its_rows(dtype):
    """A key (a query, a value, an output gradient) that is not finite changes only the results that see it."""
    n, left, sinks = 200, 20, 2
    g = gen(3)
    q, k, v, do = (randn(g, n, 1, 64, dtype=TD[dtype]) for _ in range(4))
    see = R.visible(n, n, left, 0, sinks)

    def both(q, k, v, do):
        how = dict(left=left, right=0, sinks=sinks)
        q, k, v, do = (x.to(DEV) for x in (q, k, v, do))
        out, lse = sc.window_attention(q, k, v, return_lse=True, **how)
        return [x.cpu() for x in (out, *sc.window_attention_backward(do, q, k, v, out, lse, **how))]

    clean = both(q, k, v, do)
    close = 2 * R.U[TD[dtype]]
    for what, at, value in (("k", 90, math.nan), ("v", 91, math.inf), ("q", 60, math.nan), ("do", 130, -math.inf),
                            ("v", 1, math.nan)):
        t = dict(q=q.clone(), k=k.clone(), v=v.clone(), do=do.clone())
        t[what][at, 0, 5] = value
        got = both(**t)
        if what in ("k", "v"):
            rows = see[:, at]                       # rows whose output (and gradient) it enters
            keys = see[rows].any(0)                 # keys those rows' gradients enter
            dirty = dict(out=rows, dq=rows, dk=keys, dv=keys if what == "k" else torch.zeros(n, dtype=torch.bool))
        else:
            rows = torch.zeros(n, dtype=torch.bool)
            rows[at] = True
            keys = see[at]
            dirty = dict(out=rows if what == "q" else rows & False, dq=rows, dk=keys, dv=keys)
        for name, x, c in zip(("out", "dq", "dk", "dv"), got, clean):
            clean_rows = ~dirty[name]
            if not bool(clean_rows.any()):
                continue
            assert bool(torch.isfinite(x[clean_rows]).all()), (what, name)
            # a result computed again one row at a time sums in another order
            far = (x[clean_rows].double() - c[clean_rows].double()).abs()
            assert float(far.max()) <= close * float(c.double().abs().max()) + 1e-5, (what, name)
            if bool(dirty[name].any()) and name != "dv":
                assert not bool(torch.isfinite(x[dirty[name]]).all(-1).any()), (what, name)


def test_attention_broadcast_heads_and_scale():
    run_case([90, 20], [90, 20], 3, 2, 64, "bf16", 30, 30, 0, broadcast=True, backward=False)
    run_case([90, 20], [90, 20], 3, 1, 64, "f16", 30, 30, 1, scale=0.02)
    run_case([90, 20], [90, 20], 1, 1, 32, "f32", 30, 30, 1, scale=0.7)


def test_attention_large_scores():
    """Scores far apart: the weights of all but a key or two vanish, the sums stay finite."""
    g = gen(9)
    q, k, v = (randn(g, 100, 2, 64, dtype=torch.float32, scale=s) for s in (30, 30, 1))
    out, lse = sc.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), left=40, right=0, sinks=1, return_lse=True)
    see = R.visible(100, 100, 40, 0, 1)
    for h in range(2):
        r = R.attention(q[:, h], k[:, h], v[:, h], see, 0.125)
        check(out[:, h], r["out"], r["out_tol"], "out")
        check(lse[h], r["lse"], r["lse_tol"], "lse")


def test_attention_gradient_against_differences():
    """fp32 gradients against central differences of the 64-bit form, shared heads, sinks, a window."""
    n, group, d, h = 40, 2, 8, 1e-5
    g = gen(21)
    q, k, v = torch.randn(n, group, d, generator=g), torch.randn(n, 1, d, generator=g), torch.randn(n, 1, d, generator=g)
    do = torch.randn(n, group, d, generator=g)
    how = dict(left=6, right=2, sinks=2)
    out, lse = sc.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), return_lse=True, **how)
    got = sc.window_attention_backward(do.to(DEV), q.to(DEV), k.to(DEV), v.to(DEV), out, lse, **how)
    see = R.visible(n, n, 6, 2, 2)

    def loss(q, k, v):
        return sum(float((R.attention(q[:, i], k[:, 0], v[:, 0], see, d ** -0.5)["out"] * do[:, i].double()).sum())
                   for i in range(group))

    x = [t.double() for t in (q, k, v)]
    for w in range(3):
        for i in range(0, x[w].numel(), 29):
            hi, lo = [t.clone() for t in x], [t.clone() for t in x]
            hi[w].view(-1)[i] += h
            lo[w].view(-1)[i] -= h
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(num - float(got[w].flatten()[i])) <= 1e-4 * (1 + abs(num)), (w, i)


def test_attention_offsets_past_32_bits():
    """A cache whose elements do not fit 32-bit offsets: the last sequence's keys lie past 2^32 elements."""
    slots, hk, d = 1 << 16, 8, 128
    batch = 66  # 66 * 2^16 * 8 * 128 elements: past 2^32
    k = torch.zeros(batch * slots, hk, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    g = gen(31)
    q = randn(g, batch, hk, d, dtype=torch.bfloat16)
    lens = torch.full((batch,), 1, dtype=torch.int32)
    tail = 70
    lens[-1] = slots
    kt, vt = randn(g, tail, hk, d, dtype=torch.bfloat16), randn(g, tail, hk, d, dtype=torch.bfloat16)
    k[-tail:], v[-tail:] = kt.to(DEV), vt.to(DEV)
    cu = torch.arange(batch + 1, dtype=torch.int32, device=DEV)
    out = sc.window_attention(q.to(DEV), k, v, cu_q=cu, cu_k=cu * slots, k_len=lens.to(DEV), left=tail - 1, right=0)
    see = torch.ones(1, tail, dtype=torch.bool)
    for h in range(hk):
        r = R.attention(q[-1:, h], kt[:, h], vt[:, h], see, d ** -0.5)
        check(out[-1:, h], r["out"], r["out_tol"], f"head {h}")
    assert bool((out[:-1] == 0).all())


def test_attention_other_stream_and_workspace():
    """On a stream of its own, with a workspace kept by the caller, and tables that lead outside the tensors."""
    g = gen(41)
    q, k, v = (randn(g, 500, 2, 64, dtype=torch.bfloat16).to(DEV) for _ in range(3))
    want = sc.window_attention(q[:2], k, v, left=300, right=0, sinks=2)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = sc.window_attention(q[:2], k, v, left=300, right=0, sinks=2, workspace=sc.Workspace(1 << 22, DEV))
    st.synchronize()
    assert torch.equal(got, want)
    bad = torch.tensor([0, 1 << 29], dtype=torch.int32, device=DEV)
    assert torch.equal(sc.window_attention(q[:2], k, v, cu_q=bad, cu_k=bad, left=300, right=0, sinks=2), want)
    bad = torch.tensor([-5, 700, 3, 2000000000], dtype=torch.int32, device=DEV)
    n = torch.tensor([-1, 1 << 30, 5], dtype=torch.int32, device=DEV)
    out, lse = sc.window_attention(q, k, v, cu_q=bad, cu_k=bad, k_len=n, left=9, right=0, sinks=2, return_lse=True)
    sc.window_attention_backward(q, q, k, v, out, lse, cu_q=bad, cu_k=bad, k_len=n, left=9, right=0, sinks=2)
    torch.cuda.synchronize()


def test_attention_many_sequences():
    """More sequences than one search level covers, most of them empty or of a few tokens."""
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.choice([0, 0, 1, 2, 5, 40], size=300)]
    run_case(lens, lens, 1, 1, 16, "f32", 3, 3, 1)
    run_case(lens, lens, 1, 2, 32, "bf16", 3, 0, 2)


def test_graph_replay():
    """Forward and backward under graph capture: every replay equals the eager result."""
    g = gen(51)
    q, k, v = (randn(g, 300, h, 64, dtype=torch.bfloat16).to(DEV) for h in (4, 2, 2))
    how = dict(left=40, right=0, sinks=3)
    ws = sc.Workspace(1 << 24, DEV)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    f = sc.rope_frequencies(64, device=DEV)
    gain = torch.ones(64, device=DEV)

    def step():
        a, b = sc.qk_norm_rope(q, k, pos, f, gain, gain)
        o, l = sc.window_attention(a, b, v, return_lse=True, workspace=ws, **how)
        da, db, dv = sc.window_attention_backward(o, a, b, v, o, l, workspace=ws, **how)
        return [o, l, dv, *sc.qk_norm_rope_backward(da, db, q, k, pos, f, gain, gain, workspace=ws)]

    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        q.copy_(randn(gen(60 + i), 300, 4, 64, dtype=torch.bfloat16))
        want = [x.clone() for x in step()]
        for x in out:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_gradient_of_short_windows_keeps_its_precision(dtype, dim):
    """Two independent roundings of the type on the way to every sum of dq, dk and
    dv (the weights' or dS's, and the last): sqrt(2) times the rms error of
    rounding the exact gradient once, with a sixth for what they share. The
    rounding of the forward's result, a share of every dS of a row, must not add
    to them."""
    n, hk, g = 1000, 2, gen(23)
    q, k, v, dout = (randn(g, n, hk, dim, dtype=TD[dtype], scale=s) for s in (1.3, 1.3, 1.0, 1.0))
    how = dict(left=16, right=0, sinks=4)
    on = [x.to(DEV) for x in (q, k, v, dout)]
    out, lse = sc.window_attention(*on[:3], return_lse=True, **how)
    grads = sc.window_attention_backward(on[3], *on[:3], out, lse, **how)
    i = torch.arange(n)
    sees = (i[None] <= i[:, None]) & ((i[None] >= i[:, None] - 16) | (i[None] < 4))
    x = [t.double().transpose(0, 1).contiguous().requires_grad_() for t in (q, k, v)]
    z = (x[0] @ x[1].transpose(1, 2).contiguous() * dim ** -0.5).masked_fill(~sees, -math.inf)
    exact = torch.autograd.grad((torch.softmax(z, -1) @ x[2] * dout.double().transpose(0, 1)).sum(), x)
    for name, a, b in zip(("dq", "dk", "dv"), grads, exact):
        b = b.transpose(0, 1)
        once = (b.to(TD[dtype]).double() - b).norm()
        err = (a.cpu().double() - b).norm()
        assert err < math.sqrt(2) * 7 / 6 * once, (name, float(err / once))


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 40), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("lens,hk,group,left,right,sinks", [
    ([1100], 1, 3, -1, 0, 0), ([700, 333], 1, 5, 600, 600, 40), ([2050], 1, 1, 1200, -1, 3)])
def test_attention_long_walks(dtype, dim, lens, hk, group, left, right, sinks):
    """Few tiles with long walks: split over the keys in the forward, over the rows in the gradient of keys and values."""
    run_case(lens, lens, hk, group, dim, dtype, left, right, sinks)
