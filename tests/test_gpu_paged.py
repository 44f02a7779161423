"""The operators over a paged cache on the GPU against their 64-bit forms, with
elementwise bounds of the roundings on the way (tests/tokens_ref.py).

Pools hold NaN in every slot that is no key of the call, and page tables hold
numbers past the pool behind a sequence's pages: neither may reach a result.
Bounds: the parts of a row's keys and their join are some of the roundings that
tokens_ref counts one for each key."""
import math

import pytest
import torch

from tests import tokens_ref as R
from tests.helpers import say
from tests.test_gpu_tokens import DEV, TD, check, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")

LAYOUTS = ("plain", "beside", "heads", "halves")


def pool(pages, page, hk, dim, dtype, layout, device=DEV, fill=math.nan):
    """k_pages and v_pages [pages, page, hk, dim] in one of four layouts."""
    def new(*shape):
        return torch.full(shape, fill, dtype=dtype, device=device)

    if layout == "plain":
        return new(pages, page, hk, dim), new(pages, page, hk, dim)
    if layout == "beside":  # a token's keys and values in one row
        return new(pages, page, 2 * hk, dim).split([hk, hk], 2)
    if layout == "heads":  # heads before slots, the strides of k and v unlike
        return new(pages, hk, page, dim).transpose(1, 2), new(pages, hk + 1, page, dim)[:, 1:].transpose(1, 2)
    return new(pages, 2, page, hk, dim).unbind(1)  # a page's keys, then its values


def tables(g, keys, page, prefix=0, spare=3, wider=2):
    """Random pages for every sequence and the prefix; numbers past the pool behind them."""
    need = [-(-n // page) for n in keys]
    n_pre = -(-prefix // page)
    pages = sum(need) + n_pre + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(keys), max(need) + wider), 2 ** 31 - 1, dtype=torch.int32)
    at = n_pre
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table, order[:n_pre].contiguous()


def place(t, table_row, page, x):
    """Rows x to slots 0 .. of the pages of a table row, of a pool on the CPU or GPU."""
    j = torch.arange(x.shape[0])
    t[table_row[j // page].long().to(t.device), (j % page).to(t.device)] = x.to(t.device)


def offsets(lens):
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32)


# ---------------------------------------------------------------------------
# Norm, rotation and append
# ---------------------------------------------------------------------------
# new tokens, keys before them, page, hq, hk, dim, dtype, axes, interleaved, gain, norm, layout
APPEND = [
    ([1], [0], 8, 1, 1, 8, "f32", 1, False, "none", True, "plain"),
    ([1] * 32, [5, 100, 0, 63] * 8, 16, 16, 4, 128, "bf16", 1, False, "shared", True, "beside"),
    ([2] * 5, [31, 7, 8, 0, 14], 8, 3, 1, 24, "f16", 3, True, "heads", True, "heads"),
    ([137, 1, 0, 64, 12], [0, 77, 5, 1, 130], 16, 6, 2, 72, "f32", 3, False, "none", False, "halves"),
    ([300, 45], [17, 0], 64, 5, 5, 64, "bf16", 3, True, "heads", True, "heads"),
    ([0, 0, 33, 0], [3, 0, 8, 1], 32, 2, 2, 96, "f16", 2, True, "shared", True, "beside"),
    ([700], [0], 128, 9, 3, 40, "bf16", 2, False, "shared", True, "plain"),
    ([3] * 300, list(range(300)), 16, 2, 1, 16, "f32", 1, False, "none", False, "halves"),
    ([5000, 1, 800], [1, 2000, 0], 16, 7, 1, 120, "f16", 1, False, "heads", True, "plain"),
]


def append_inputs(case, seed=5, behind=3):
    new, before, page, hq, hk, dim, dtype, axes, il, gain, norm, layout = case
    g = gen(seed)
    dt = TD[dtype]
    n = sum(new) + (behind if min(new) != max(new) else 0)  # rows behind the last sequence
    qkv = randn(g, n, hq + 2 * hk, dim, dtype=dt, scale=1.7)
    coords = torch.randint(0, 64, (n, 4), generator=g, dtype=torch.int32)
    freqs = sc.rope_frequencies(dim, axes, device="cpu")
    shape = {"none": None, "shared": (dim,), "heads": (0, dim)}[gain]
    gains = [None if shape is None else 1 + 0.2 * torch.randn((h if shape[0] == 0 else dim,) + shape[1:], generator=g)
             for h in (hq, hk)]
    keys = [a + b for a, b in zip(new, before)]
    pages, table, _ = tables(g, keys, page)
    return qkv, coords, freqs, gains, keys, pages, table


def run_append(case, inputs, q_out=None, **more):
    new, before, page, hq, hk, dim, dtype, axes, il, gain, norm, layout = case
    qkv, coords, freqs, gains, keys, pages, table = inputs
    d = qkv.to(DEV)
    q, k, v = d.split([hq, hk, hk], 1)
    kp, vp = pool(pages, page, hk, dim, TD[dtype], layout)
    cu = offsets(new).to(DEV) if min(new) != max(new) or len(new) != len(keys) else None
    out = sc.qk_norm_rope_append(q, k, v, coords.to(DEV)[:, 1:1 + axes], freqs.to(DEV), kp, vp, table.to(DEV),
                                 torch.tensor(keys, dtype=torch.int32, device=DEV), cu_q=cu,
                                 q_gain=None if gains[0] is None else gains[0].to(DEV),
                                 k_gain=None if gains[1] is None else gains[1].to(DEV), interleaved=il, eps=1e-5, norm=norm,
                                 q_out=q_out, **more)
    return out, kp, vp


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[2:])))
def test_append(case):
    new, before, page, hq, hk, dim, dtype, axes, il, gain, norm, layout = case
    say("[append]", case[2:])
    dt = TD[dtype]
    inputs = append_inputs(case)
    qkv, coords, freqs, gains, keys, pages, table = inputs
    q, k, v = qkv.split([hq, hk, hk], 1)
    room = torch.full((q.shape[0], hq + 1, dim), 7.0, dtype=dt, device=DEV)
    out, kp, vp = run_append(case, inputs, q_out=room[:, 1:])
    ang = R.angles(coords[:, 1:1 + axes], freqs, [dim // 2 // axes] * axes)

    def turned(x, gn):
        if norm:
            return R.norm_rope(x, gn, ang, il, 1e-5), R.norm_rope_bound(x, gn, ang, il, 1e-5, dt)
        ref, mag = R.rotate_pairs(x.double(), ang, il), x.double().abs()
        # sine, cosine and the turn as in norm_rope_bound, the norm's roundings less
        return ref, 16 * R.E * (mag + R.swap_pairs(mag, il)) + R.U[dt] * ref.abs() + R.U[dt] * R.TINY[dt]

    total = sum(new)
    ref, tol = turned(q, gains[0])
    check(out[:total], ref[:total], tol[:total], "q")
    assert bool((room[:, 0] == 7).all()) and bool((room[total:] == 7).all())  # beside and behind
    ref, tol = turned(k, gains[1])
    kc, vc = kp.cpu(), vp.cpu()
    wk, wv = pool(pages, page, hk, dim, dt, "plain", "cpu")
    t = 0
    for b, n in enumerate(new):
        for i in range(n):
            j = before[b] + i
            p, s = int(table[b, j // page]), j % page
            wk[p, s], wv[p, s] = 1, v[t]
            if t < 40 or t % 37 == 0 or t == total - 1:
                check(kc[p, s], ref[t], tol[t], f"key of token {t}")
            t += 1
    assert torch.equal(bits(vc), bits(wv))
    assert torch.equal(torch.isnan(kc), torch.isnan(wk))  # nothing else is touched


def test_append_all_keys_of_many_tokens():
    """Every key of a long call against a gather, through the operator without pages."""
    case = ([9000, 777], [13, 4], 16, 4, 2, 64, "bf16", 3, True, "heads", True, "beside")
    inputs = append_inputs(case)
    qkv, coords, freqs, gains, keys, pages, table = inputs
    out, kp, vp = run_append(case, inputs)
    d = qkv.to(DEV)
    want_q, want_k = sc.qk_norm_rope(d[:, :4], d[:, 4:6], coords.to(DEV)[:, 1:], freqs.to(DEV), gains[0].to(DEV),
                                     gains[1].to(DEV), interleaved=True, eps=1e-5)
    assert torch.equal(out[:9777], want_q[:9777])
    t = 0
    for b, (n, total) in enumerate(zip([9000, 777], keys)):
        j = torch.arange(total - n, total)
        p, s = table[b, j // 16].long().to(DEV), (j % 16).to(DEV)
        assert torch.equal(kp[p, s], want_k[t:t + n]) and torch.equal(vp[p, s], d[t:t + n, 6:])
        t += n


def test_append_in_place_and_lengths_that_do_not_fit():
    """q_out = q. Keys that the length or the table leaves no place, pages that are none: not stored; their queries are."""
    dim, page = 64, 8
    g = gen(6)
    new = [4, 4, 4, 4, 4]
    keys = [2, 4, 18, 10, 2 ** 31 - 1]  # two tokens before the first key; all; two past the table; a bad page; far past
    qkv = randn(g, 20, 4, dim, dtype=torch.bfloat16).to(DEV)
    q, k, v = qkv.split([2, 1, 1], 1)
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, -1], [7, 9]], dtype=torch.int32, device=DEV)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    freqs = sc.rope_frequencies(dim, device=DEV)
    want = sc.qk_norm_rope(q, k, pos, freqs)
    kp, vp = pool(9, page, 1, dim, torch.bfloat16, "plain")
    v0 = v.clone()
    out = sc.qk_norm_rope_append(q, k, v, pos, freqs, kp, vp, table,
                                 torch.tensor(keys, dtype=torch.int32, device=DEV), q_out=q)
    assert out is q and torch.equal(q, want[0])
    seen = {}
    for b, (n, total) in enumerate(zip(new, keys)):
        for i in range(n):
            j = total - n + i
            if 0 <= j < 16 and 0 <= int(table[b, j // page]) < 9:
                seen[(int(table[b, j // page]), j % page)] = 4 * b + i
    assert len(seen) == 2 + 4 + 2 + 2
    for p in range(9):
        for s in range(page):
            t = seen.get((p, s))
            if t is None:
                assert bool(torch.isnan(kp[p, s]).all()) and bool(torch.isnan(vp[p, s]).all())
            else:
                assert torch.equal(kp[p, s], want[1][t]) and torch.equal(vp[p, s], v0[t])


def test_append_values_bit_by_bit():
    """NaN payloads, signed zeros and infinities of the values arrive as they are."""
    x = torch.tensor([0x7FC1, 0xFF81, 0x8000, 0x7F80, 0x0001, 0xFFFF, 0x3F80, 0x7F81] * 2, dtype=torch.int32)
    v = x.to(torch.int16).view(torch.bfloat16).reshape(1, 1, 16).to(DEV)
    q = torch.ones(1, 1, 16, dtype=torch.bfloat16, device=DEV)
    kp, vp = pool(1, 8, 1, 16, torch.bfloat16, "plain", fill=0.0)
    sc.qk_norm_rope_append(q, q, v, torch.zeros(1, dtype=torch.int32, device=DEV), sc.rope_frequencies(16, device=DEV), kp,
                           vp, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                           torch.ones(1, dtype=torch.int32, device=DEV))
    assert torch.equal(bits(vp[0, 0]), bits(v[0]))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def attend_inputs(new, keys, page, hq, hk, dim, dtype, layout, prefix=0, seed=9, behind=2):
    g = gen(seed)
    dt = TD[dtype]
    n = sum(new) + (behind if min(new) != max(new) else 0)
    q = randn(g, n, hq, dim, dtype=dt, scale=1.3)
    own = [(randn(g, m, hk, dim, dtype=dt, scale=1.3), randn(g, m, hk, dim, dtype=dt)) for m in keys]
    pre = (randn(g, prefix, hk, dim, dtype=dt, scale=1.3), randn(g, prefix, hk, dim, dtype=dt))
    pages, table, pre_pages = tables(g, keys, page, prefix)
    kp, vp = pool(pages, page, hk, dim, dt, layout)
    for b, (k, v) in enumerate(own):
        place(kp, table[b], page, k)
        place(vp, table[b], page, v)
    if prefix:
        place(kp, pre_pages, page, pre[0])
        place(vp, pre_pages, page, pre[1])
    return q, own, pre, kp, vp, table.to(DEV), pre_pages.to(DEV)


def verify(out, lse, q, own, pre, new, left, right, sinks, scale):
    """Every row of every sequence; rows behind them are 7."""
    hq, hk = q.shape[1], pre[0].shape[1]
    out, lse, t = out.cpu(), lse.cpu(), 0
    for b, n in enumerate(new):
        k, v = (torch.cat([x, y]) for x, y in zip(pre, own[b]))
        see = R.visible(n, k.shape[0], left, right, sinks)
        for h in range(hq if n else 0):
            r = R.attention(q[t:t + n, h], k[:, h * hk // hq], v[:, h * hk // hq], see, scale)
            check(out[t:t + n, h], r["out"], r["out_tol"], f"sequence {b} head {h} out")
            check(lse[h, t:t + n], r["lse"], r["lse_tol"], f"sequence {b} head {h} lse")
        t += n
    assert bool((out[t:] == 7).all())


def attend(q, kp, vp, table, keys, new, pre_pages, prefix, **how):
    cu = None if min(new) == max(new) else offsets(new).to(DEV)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lens = torch.tensor(keys, dtype=torch.int32, device=DEV)
    if prefix is None:
        return sc.paged_window_attention(q.to(DEV), kp, vp, table, lens, cu_q=cu, return_lse=True, out=out, **how)
    return sc.shared_prefix_attention(q.to(DEV), kp, vp, table, lens, pre_pages, prefix, cu_q=cu, return_lse=True, out=out,
                                      **how)


# new tokens, keys, page, hq, hk, dim, dtype, left, right, sinks, layout
PAGED = [
    ([1], [1], 8, 1, 1, 8, "f32", -1, -1, 0, "plain"),
    ([1], [0], 8, 2, 1, 16, "bf16", -1, 0, 0, "plain"),
    ([1] * 8, [450, 31, 32, 33, 1, 0, 127, 300], 16, 8, 8, 64, "bf16", -1, 0, 0, "beside"),
    ([1] * 5, [1500, 700, 64, 1499, 3], 16, 16, 4, 128, "bf16", 511, 0, 4, "heads"),
    ([1], [9000], 64, 8, 2, 128, "f16", -1, 0, 0, "halves"),
    ([1], [5000], 8, 6, 1, 72, "f32", 2047, 0, 17, "plain"),
    ([5] * 6, [400, 5, 3, 77, 256, 2047], 8, 6, 2, 80, "f32", 255, 0, 3, "heads"),
    ([3] * 4, [90, 2, 0, 800], 32, 4, 1, 40, "f16", 20, 5, 1, "beside"),
    ([130, 1, 0, 77], [400, 900, 50, 77], 16, 4, 2, 64, "bf16", -1, 0, 0, "halves"),
    ([257, 40], [257, 300], 64, 4, 1, 128, "bf16", 63, 0, 4, "beside"),
    ([200, 9], [150, 1000], 128, 6, 2, 96, "f16", -1, 0, 0, "plain"),  # rows before the first key see nothing
    ([70, 64], [333, 64], 8, 3, 3, 24, "f32", 40, 7, 2, "halves"),
    ([40], [40], 1024, 12, 1, 32, "bf16", 16, 16, 0, "heads"),
    ([2] * 70, [(37 * i) % 200 for i in range(70)], 16, 8, 2, 48, "bf16", -1, 0, 0, "plain"),
    ([1] * 3, [2600, 17, 1300], 256, 32, 1, 112, "f16", 100, 0, 128, "beside"),
    ([33, 1, 1, 1, 1, 1], [60, 900, 901, 902, 1, 30], 16, 8, 2, 128, "f32", -1, 0, 0, "plain"),
    # few rows over many keys: units dealt to waves
    ([1] * 6, [2600, 17, 0, 5000, 4097, 64], 16, 8, 4, 64, "bf16", -1, 0, 0, "beside"),
    ([2] * 3, [3000, 1, 2300], 8, 8, 2, 128, "bf16", -1, 0, 0, "heads"),
    ([1, 0, 7, 3], [2500, 40, 2900, 3], 32, 6, 3, 96, "f16", -1, 0, 0, "halves"),
    ([4] * 2, [900, 1300], 16, 4, 2, 40, "f32", -1, 0, 0, "plain"),
    ([1] * 5, [700, 5, 0, 33, 1200], 8, 8, 2, 128, "f32", 600, 0, 9, "beside"),
    ([1] * 600, [(7 * i) % 64 for i in range(600)], 16, 2, 2, 32, "bf16", -1, 0, 0, "plain"),  # many short sequences
    ([3] * 2, [2200, 2300], 64, 80, 40, 16, "f16", -1, 0, 0, "plain"),  # many heads
    ([i % 3 for i in range(200)], [(11 * i) % 90 for i in range(200)], 8, 8, 4, 24, "bf16", -1, 0, 0, "halves"),
    ([1] * 3, [500, 1, 2400], 16, 40, 1, 64, "bf16", -1, 0, 0, "plain"),  # more rows a token than a wave holds
    # many rows: units dealt to workgroups, and a workgroup an item
    ([300, 0, 5, 290], [700, 40, 5, 1500], 16, 8, 4, 128, "f16", 500, 0, 4, "heads"),
    ([160, 90], [200, 90], 8, 2, 2, 72, "f32", -1, 0, 0, "halves"),
    ([1400, 3], [1400, 77], 32, 256, 256, 8, "bf16", 30, 0, 0, "beside"),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(map(str, c[2:])) + f"-{len(c[0])}")
def test_paged_window_attention(case):
    new, keys, page, hq, hk, dim, dtype, left, right, sinks, layout = case
    say("[paged]", case[2:], len(new))
    q, own, pre, kp, vp, table, _ = attend_inputs(new, keys, page, hq, hk, dim, dtype, layout)
    how = dict(left=left, right=right, sinks=sinks)
    out, lse = attend(q, kp, vp, table, keys, new, None, None, **how)
    verify(out, lse, q, own, pre, new, left, right, sinks, dim ** -0.5)
    again, lse2 = attend(q, kp, vp, table, keys, new, None, None, **how)
    assert torch.equal(out, again) and torch.equal(lse[:, :sum(new)], lse2[:, :sum(new)])


# new tokens, own keys, prefix, page, hq, hk, dim, dtype, left, right, sinks, layout
PREFIX = [
    ([1], [1], 1, 8, 1, 1, 8, "f32", -1, -1, 0, "plain"),
    ([1] * 4, [450, 1, 77, 300], 1369, 16, 4, 4, 64, "f16", -1, 0, 0, "beside"),
    ([1] * 9, [0, 1, 2, 3, 70, 128, 129, 40, 5], 1000, 64, 16, 4, 128, "bf16", -1, 0, 0, "halves"),
    ([3] * 7, [96, 3, 50, 10, 2, 0, 64], 733, 8, 6, 2, 80, "f32", 255, 0, 4, "heads"),
    ([1] * 70, [(13 * i) % 90 for i in range(70)], 517, 16, 8, 2, 64, "bf16", -1, 0, 0, "plain"),
    ([2] * 40, [(7 * i) % 60 for i in range(40)], 300, 32, 8, 1, 96, "f16", 200, 0, 7, "beside"),  # sinks in the prefix
    ([1] * 5, [40, 30, 20, 10, 0], 5, 8, 4, 2, 32, "bf16", 16, 0, 17, "plain"),  # sinks past the prefix
    ([1, 0, 5, 33, 2], [3, 10, 60, 33, 100], 130, 16, 8, 4, 128, "bf16", -1, 0, 0, "heads"),
    ([60, 1, 7], [60, 400, 3], 200, 128, 4, 2, 72, "f32", 100, 3, 1, "plain"),  # rows inside the prefix
    ([1] * 3, [30, 31, 32], 4000, 16, 8, 1, 128, "f16", 24, 0, 0, "beside"),  # the prefix hardly in the window
    ([1] * 6, [5, 5, 5, 5, 5, 5], 64, 8, 2, 2, 16, "f32", 2, 0, 0, "halves"),  # not at all
    ([1] * 33, list(range(33)), 2100, 64, 12, 3, 40, "f32", -1, 0, 0, "plain"),
    # units dealt to waves, prefix and own keys in one list
    ([1] * 4, [500, 0, 77, 1300], 2500, 16, 8, 4, 64, "bf16", -1, 0, 0, "halves"),
    ([2, 0, 1], [30, 9, 700], 3000, 8, 4, 2, 128, "f16", -1, 0, 0, "beside"),
    ([1] * 3, [50, 60, 3], 1500, 8, 4, 1, 96, "f32", 1300, 0, 5, "heads"),
    # the prefix to workgroups, the own keys to waves
    ([1] * 20, [(31 * i) % 300 for i in range(20)], 3000, 16, 16, 4, 128, "bf16", -1, 0, 0, "beside"),
    ([2, 0, 1, 3, 1, 1, 2, 1, 1, 1] * 3, [(17 * i) % 150 + 3 for i in range(30)], 2600, 16, 4, 2, 64, "f16", -1, 0, 0, "heads"),
    ([1] * 40, [(9 * i) % 70 for i in range(40)], 4100, 64, 4, 2, 80, "bf16", 4000, 0, 3, "plain"),
    ([1] * 300, [i % 5 for i in range(300)], 700, 8, 4, 2, 32, "f32", -1, 0, 0, "plain"),
    ([2] * 9, [3] * 9, 2100, 16, 96, 48, 16, "bf16", -1, 0, 0, "plain"),  # many heads
    ([i % 2 for i in range(130)], [(5 * i) % 40 for i in range(130)], 2050, 16, 4, 1, 40, "f16", -1, 0, 0, "halves"),
    ([1] * 3, [40, 1, 9], 600, 16, 72, 1, 32, "f32", -1, 0, 0, "plain"),  # more rows a token than a wave holds
    # workgroups take both
    ([140, 3, 0, 90], [300, 3, 20, 90], 1100, 16, 4, 2, 128, "f16", -1, 0, 0, "beside"),
    ([70, 66], [70, 200], 400, 8, 2, 1, 64, "f32", 300, 0, 2, "halves"),
]


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c[2:])) + f"-{len(c[0])}")
def test_shared_prefix_attention(case):
    new, keys, prefix, page, hq, hk, dim, dtype, left, right, sinks, layout = case
    say("[prefix]", case[2:], len(new))
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, page, hq, hk, dim, dtype, layout, prefix)
    how = dict(left=left, right=right, sinks=sinks)
    out, lse = attend(q, kp, vp, table, keys, new, pre_pages, prefix, **how)
    verify(out, lse, q, own, pre, new, left, right, sinks, dim ** -0.5)
    again, lse2 = attend(q, kp, vp, table, keys, new, pre_pages, prefix, **how)
    assert torch.equal(out, again) and torch.equal(lse[:, :sum(new)], lse2[:, :sum(new)])


def test_prefix_of_nothing_is_paged_attention():
    new, keys = [2] * 3, [40, 3, 200]
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 4, 2, 64, "bf16", "plain")
    a = attend(q, kp, vp, table, keys, new, None, None, left=30, right=0, sinks=2)
    b = attend(q, kp, vp, table, keys, new, pre_pages, 0, left=30, right=0, sinks=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("scale", [0.03, 1.7])
def test_scale(scale):
    new, keys = [3, 1], [700, 90]
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 4, 2, 64, "f16", "plain", 60)
    out, lse = attend(q, kp, vp, table, keys, new, pre_pages, 60, right=0, scale=scale)
    verify(out, lse, q, own, pre, new, -1, 0, 0, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,prefix", [([1, 1], 0), ([1, 1], 96), ([1, 1], 3000), ([12, 12], 3000), ([150, 3], 0),
                                        ([150, 3], 96)])
def test_pages_that_are_none_read_as_zeros(dtype, new, prefix):
    """Page numbers past the pool or negative inside a sequence or the prefix: keys and values of zero, and no read outside."""
    keys, page, dim = [300, 180], 16, 64
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, page, 4, 2, dim, dtype, "beside", prefix)
    for b, at, bad in ((0, 3, -1), (0, 18, 2 ** 31 - 1), (1, 0, kp.shape[0])):
        table[b, at] = bad
        for x in own[b]:
            x[at * page:(at + 1) * page] = 0
    if prefix:
        pre_pages[2] = -2 ** 31
        for x in pre:
            x[2 * page:3 * page] = 0
    out, lse = attend(q, kp, vp, table, keys, new, pre_pages, prefix, right=0)
    verify(out, lse, q, own, pre, new, -1, 0, 0, dim ** -0.5)


def test_lengths_are_clamped_to_the_table():
    page, dim = 8, 32
    q, own, pre, kp, vp, table, _ = attend_inputs([1, 1, 1], [16, 16, 16], page, 2, 1, dim, "f32", "plain")
    table = table[:, :2].contiguous()
    want = attend(q, kp, vp, table, [16, 0, 16], [1, 1, 1], None, None)
    got = attend(q, kp, vp, table, [2 ** 31 - 1, -5, 17], [1, 1, 1], None, None)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert bool((got[0][1] == 0).all()) and bool(torch.isinf(got[1][:, 1]).all())
    none = attend(q, kp, vp, table[:, :0], [5, 5, 5], [1, 1, 1], None, None)  # a table without pages
    assert bool((none[0] == 0).all()) and bool((none[1] == -math.inf).all())
    none = attend(q, kp[:0], vp[:0], table, [5, 5, 5], [1, 1, 1], None, None)  # a pool without pages
    assert bool((none[0] == 0).all()) and bool((none[1] == -math.inf).all())


def test_no_tokens():
    _, own, pre, kp, vp, table, pre_pages = attend_inputs([1, 1], [16, 3], 8, 2, 1, 32, "bf16", "plain", 20)
    q = torch.empty(0, 2, 32, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([16, 3], dtype=torch.int32, device=DEV)
    for cu in (None, torch.zeros(3, dtype=torch.int32, device=DEV)):
        out, lse = sc.paged_window_attention(q, kp, vp, table, lens, cu_q=cu, return_lse=True)
        assert out.shape == (0, 2, 32) and lse.shape == (2, 0)
        assert sc.shared_prefix_attention(q, kp, vp, table, lens, pre_pages, 20, cu_q=cu).shape == (0, 2, 32)
        pos = torch.empty(0, dtype=torch.int32, device=DEV)
        before = bits(kp).clone()
        assert sc.qk_norm_rope_append(q, q[:, :1], q[:, :1], pos, sc.rope_frequencies(32, device=DEV), kp, vp, table, lens,
                                      cu_q=cu).shape == (0, 2, 32)
        assert torch.equal(before, bits(kp))


# ---------------------------------------------------------------------------
# What is not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,prefix", [([6, 6], 0), ([6, 6], 70), ([6, 6], 2500), ([20, 20], 2500), ([140, 20], 0),
                                        ([140, 20], 70)])
def test_not_finite(dtype, new, prefix):
    """NaN and infinities in keys and values that a row does not see do not reach it; rows that do see them have what
    the formula gives: NaN, or the infinity of a value."""
    keys, page, dim, left = [400, 130], 16, 64, 100
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, page, 4, 2, dim, dtype, "plain", prefix)
    for b, j, e, value, what in ((0, 5, 3, math.nan, 1), (0, 299, 0, math.nan, 0), (1, 129, 63, math.inf, 1),
                                 (1, 27, 5, math.inf, 1)):
        own[b][what][j, 1, e] = value
        (kp, vp)[what][int(table[b, j // page]), j % page, 1, e] = value
    if prefix:
        for j in (60, prefix - 2):
            pre[1][j, 0, 9] = math.nan
            vp[int(pre_pages[j // page]), j % page, 0, 9] = math.nan
    out, lse = attend(q, kp, vp, table, keys, new, pre_pages, prefix, left=left, right=0, sinks=0)
    t = 0
    for b, n in enumerate(new):
        k, v = (torch.cat([x, y]) for x, y in zip(pre, own[b]))
        see = R.visible(n, k.shape[0], left, 0, 0)
        for h in range(4):
            kh, vh = k[:, h // 2], v[:, h // 2]
            clean_k, clean_v = torch.nan_to_num(kh.float(), 0, 0, 0).to(kh.dtype), torch.nan_to_num(vh.float(), 0, 0, 0)
            r = R.attention(q[t:t + n, h], clean_k, clean_v.to(vh.dtype), see, dim ** -0.5)
            bad_key = (see & ~torch.isfinite(kh.float()).all(1)[None]).any(1)
            want = r["out"].clone()
            # a value's NaN and infinities reach their own column of the rows that see them
            for j, e in (~torch.isfinite(vh.float())).nonzero().tolist():
                want[see[:, j], e] = want[see[:, j], e] + float(vh[j, e])
            want[bad_key] = math.nan
            got = out[t:t + n, h].cpu().double()
            tol = r["out_tol"]
            same = ((got - want).abs() <= tol) | (got == want) | (torch.isnan(got) & torch.isnan(want))
            assert bool(same.all()), (b, h, (~same).nonzero()[:3].tolist())
        t += n


# ---------------------------------------------------------------------------
# Places, streams, graphs, and the calls together
# ---------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Pages whose elements lie 2^32 bytes and 2^32 elements from the pool's start."""
    page, hk, dim = 64, 8, 128
    pages = (1 << 32) // (page * hk * dim) + 40
    kp = torch.empty(pages, page, hk, dim, dtype=torch.bfloat16, device=DEV)
    vp = torch.empty_like(kp)
    g = gen(12)
    new, keys = [2, 1], [150, 90]
    table = torch.tensor([[pages - 1, pages // 2 + 3, 0], [pages - 2, 1, 0]], dtype=torch.int32)
    pre_pages = torch.tensor([pages - 3, pages // 2 + 1], dtype=torch.int32)
    q = randn(g, 3, 8, dim, dtype=torch.bfloat16)
    own = [tuple(randn(g, n, hk, dim, dtype=torch.bfloat16) for _ in range(2)) for n in keys]
    pre = tuple(randn(g, 100, hk, dim, dtype=torch.bfloat16) for _ in range(2))
    pos = torch.arange(sum(keys), dtype=torch.int32, device=DEV)
    k, v = (torch.cat([own[0][i], own[1][i]]).to(DEV) for i in range(2))
    cu = offsets(keys).to(DEV)
    lens = torch.tensor(keys, dtype=torch.int32, device=DEV)
    flat = torch.zeros(dim // 2, device=DEV)
    sc.qk_norm_rope_append(k, k, v, pos, flat, kp, vp, table.to(DEV), lens, cu_q=cu, norm=False)  # no turn: a copy
    place(kp, pre_pages, page, pre[0])
    place(vp, pre_pages, page, pre[1])
    out, lse = attend(q, kp, vp, table.to(DEV), keys, new, pre_pages.to(DEV), 100, right=0)
    verify(out, lse, q, own, pre, new, -1, 0, 0, dim ** -0.5)


@pytest.mark.parametrize("prefix", [0, 40, 2300])
def test_strided_tables_and_outputs(prefix):
    """A page table inside a wider one, the sequences' rows a slice of larger tensors, the output's too."""
    new, keys, dim = [2] * 3, [70, 9, 150], 64
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 4, 2, dim, "bf16", "heads", prefix)
    wide = torch.full((3, table.shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table
    big_q = torch.randn(9, 7, dim, dtype=torch.bfloat16, device=DEV)
    big_q[2:8, 1:5] = q.to(DEV)
    room = torch.full((8, 6, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor(keys, dtype=torch.int32, device=DEV)
    out, lse = sc.shared_prefix_attention(big_q[2:8, 1:5], kp, vp, wide[:, 2:2 + table.shape[1]], lens, pre_pages, prefix,
                                          right=0, return_lse=True, out=room[1:7, 1:5])
    assert out.data_ptr() == room[1:7, 1:5].data_ptr()
    verify(out, lse, q, own, pre, new, -1, 0, 0, dim ** -0.5)
    room[1:7, 1:5] = 7
    assert bool((room == 7).all())


def test_one_page_in_many_places():
    """A page twice in a table, in two tables and in the prefix."""
    page, dim = 16, 64
    g = gen(13)
    kp, vp = (randn(g, 3, page, 2, dim, dtype=torch.bfloat16) for _ in range(2))
    table = torch.tensor([[1, 1, 0], [1, 2, 2]], dtype=torch.int32)
    pre_pages = torch.tensor([2, 1], dtype=torch.int32)
    keys, new, prefix = [40, 33], [1, 1], 20

    def rows(t, ids, n):
        return t[ids.long()].reshape(-1, 2, dim)[:n]

    own = [(rows(kp, table[b], n), rows(vp, table[b], n)) for b, n in enumerate(keys)]
    pre = (rows(kp, pre_pages, prefix), rows(vp, pre_pages, prefix))
    q = randn(g, 2, 4, dim, dtype=torch.bfloat16)
    out, lse = attend(q, kp.to(DEV), vp.to(DEV), table.to(DEV), keys, new, pre_pages.to(DEV), prefix, right=0)
    verify(out, lse, q, own, pre, new, -1, 0, 0, dim ** -0.5)


def step_inputs(batch, hq, hk, dim, dtype, g):
    qkv = randn(g, batch, hq + 2 * hk, dim, dtype=dtype, scale=1.3).to(DEV)
    return qkv.split([hq, hk, hk], 1)


def test_steps_on_another_stream_and_in_a_graph():
    """A decoding step (length + 1, append, attend behind a prefix) captured once and replayed, against eager steps."""
    batch, hq, hk, dim, page, prefix = 5, 8, 2, 64, 16, 50
    g = gen(14)
    dt = torch.bfloat16
    start = [17, 0, 40, 31, 15]
    q0, own, pre, kp, vp, table, pre_pages = attend_inputs([1] * batch, start, page, hq, hk, dim, "bf16", "beside", prefix)
    pages = torch.arange(kp.shape[0], kp.shape[0] + 5 * 8, dtype=torch.int32, device=DEV).view(5, 8)
    need = [-(-n // page) for n in start]
    wide = torch.full((batch, 8), -1, dtype=torch.int32, device=DEV)
    for b in range(batch):
        wide[b, :need[b]] = table[b, :need[b]]
        wide[b, need[b]:] = pages[b, need[b]:]
    big = torch.cat([torch.cat([kp, vp], 2), torch.full((40, page, 2 * hk, dim), math.nan, dtype=dt, device=DEV)])
    freqs = sc.rope_frequencies(dim, device=DEV)
    steps = [step_inputs(batch, hq, hk, dim, dt, g) for _ in range(6)]
    q, k, v = (torch.empty_like(x) for x in steps[0])

    def step(pool_, lens):
        lens += 1
        kp_, vp_ = pool_.split([hk, hk], 2)
        r = sc.qk_norm_rope_append(q, k, v, lens, freqs, kp_, vp_, wide, lens)
        return sc.shared_prefix_attention(r, kp_, vp_, wide, lens, pre_pages, prefix, left=60, right=0, sinks=3)

    lens0 = torch.tensor(start, dtype=torch.int32, device=DEV)
    want, eager, lens = [], big.clone(), lens0.clone()
    for s in steps:
        for x, y in zip((q, k, v), s):
            x.copy_(y)
        want.append(step(eager, lens).clone())
    # another stream
    side = torch.cuda.Stream()
    pool2, lens = big.clone(), lens0.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s, w in zip(steps, want):
            for x, y in zip((q, k, v), s):
                x.copy_(y)
            assert torch.equal(step(pool2, lens), w)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(bits(pool2), bits(eager))
    # a graph
    pool3, lens = big.clone(), lens0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(pool3, lens)
    lens.copy_(lens0)
    for s, w in zip(steps, want):
        for x, y in zip((q, k, v), s):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        torch.randn(1000, device=DEV).sum()  # work of the program's own between replays
    assert torch.equal(bits(pool3), bits(eager))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_then_tokens_as_from_a_contiguous_cache(dtype):
    """Prompts in parts, then single tokens, through append and attention over pages: the same as norm, rotation and
    window_attention over a whole sequence, within both calls' bounds."""
    dt, page, hq, hk, dim, left, sinks = TD[dtype], 16, 4, 2, 64, 90, 2
    g = gen(15)
    lens = [230, 75, 140]
    seqs = [randn(g, n, hq + 2 * hk, dim, dtype=dt, scale=1.3) for n in lens]
    freqs = sc.rope_frequencies(dim, device=DEV)
    gains = [(1 + 0.2 * torch.randn(h, dim, generator=g)).to(DEV) for h in (hq, hk)]
    pages, table, _ = tables(g, lens, page)
    kp, vp = pool(pages, page, hk, dim, dt, "heads")
    table = table.to(DEV)
    got = [torch.empty(n, hq, dim, dtype=dt) for n in lens]
    at = [0, 0, 0]
    plan = [[100, 60, 1], [128, 0, 130], [0, 13, 0], [1, 1, 1], [1, 1, 1], [0, 0, 7]]
    for part in plan:
        rows = torch.cat([s[a:a + n] for s, a, n in zip(seqs, at, part)]).to(DEV)
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(at, part)]).to(torch.int32).to(DEV)
        at = [a + n for a, n in zip(at, part)]
        k_len = torch.tensor(at, dtype=torch.int32, device=DEV)
        cu = offsets(part).to(DEV)
        q, k, v = rows.split([hq, hk, hk], 1)
        q = sc.qk_norm_rope_append(q, k, v, pos, freqs, kp, vp, table, k_len, cu_q=cu, q_gain=gains[0], k_gain=gains[1])
        o = sc.paged_window_attention(q, kp, vp, table, k_len, cu_q=cu, left=left, right=0, sinks=sinks).cpu()
        for b, x in enumerate(o.split(part)):
            got[b][at[b] - part[b]:at[b]] = x
    assert at == lens
    for b, s in enumerate(seqs):
        q, k, v = s.to(DEV).split([hq, hk, hk], 1)
        pos = torch.arange(lens[b], dtype=torch.int32, device=DEV)
        q, k = (x.cpu() for x in sc.qk_norm_rope(q, k, pos, freqs, *gains))
        see = R.visible(lens[b], lens[b], left, 0, sinks)
        for h in range(hq):
            r = R.attention(q[:, h], k[:, h // 2], v.cpu()[:, h // 2], see, dim ** -0.5)
            check(got[b][:, h], r["out"], r["out_tol"], f"sequence {b} head {h}")


def test_workspace_of_the_callers():
    new, keys, n = [1] * 3, [900, 30, 400], 5000
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 8, 2, 64, "bf16", "plain", n)
    want = attend(q, kp, vp, table, keys, new, pre_pages, n)[0]
    ws = sc.Workspace(1 << 25, DEV)
    ws.buf.fill_(0xFF)  # NaN
    assert torch.equal(attend(q, kp, vp, table, keys, new, pre_pages, n, workspace=ws)[0], want)
    with pytest.raises(ValueError, match="needed"):
        attend(q, kp, vp, table, keys, new, pre_pages, n, workspace=sc.Workspace(64, DEV))
    with pytest.raises(ValueError, match="workspace is on cpu"):
        attend(q, kp, vp, table, keys, new, pre_pages, n, workspace=sc.Workspace(1 << 25, "cpu"))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_leading_and_far_keys(dtype):
    """A key that leads the others by 18 nats in one part of the keys, with a value of zero: what the others give keeps
    the type's precision; and scores of several hundred."""
    page, dim, prefix = 16, 64, 200
    new, keys = [1, 1], [600, 90]
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, page, 2, 1, dim, dtype, "plain", prefix)
    dt = TD[dtype]
    for lead, at in ((18.0, 3), (300.0, 150)):
        k = q[0, 0].double() / q[0, 0].double().norm() ** 2 * lead * dim ** 0.5
        pre[0][at, 0], pre[1][at, 0] = k.to(dt), 0
        place(kp, pre_pages.cpu(), page, pre[0])
        place(vp, pre_pages.cpu(), page, pre[1])
        out, lse = attend(q, kp, vp, table, keys, new, pre_pages, prefix)
        verify(out, lse, q, own, pre, new, -1, -1, 0, dim ** -0.5)
