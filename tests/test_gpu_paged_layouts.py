"""Pages whose strides are no multiples of each other's, through the append and both attentions: the same bits as from
pages without gaps, and what lies in the gaps is left as it is. Tables that give two tokens one place."""
import pytest
import torch

from tests.test_gpu_paged import DEV, TD, attend, bits, offsets, tables
from tests.test_gpu_tokens import gen, randn
from tests.helpers import say

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def gapped(pages, page, hk, dim, dtype, gap, order):
    """k_pages, v_pages of one buffer, a token's keys beside its values, with `gap` elements behind every page (order:
    "pages") or behind every slot's run over the pages ("slots"); and the buffer."""
    row = 2 * hk * dim
    if order == "pages":
        strides, room = (page * row + gap, row), pages * (page * row + gap)
    else:
        strides, room = (row, pages * row + gap), page * (pages * row + gap)
    flat = torch.full((room,), 7.0, dtype=dtype, device=DEV)
    return [flat.as_strided((pages, page, hk, dim), (*strides, dim, 1), at * hk * dim) for at in (0, 1)] + [flat]


@pytest.mark.parametrize("dtype,hk,dim", [("bf16", 2, 64), ("f16", 1, 40), ("f32", 3, 24)])
@pytest.mark.parametrize("order", ["pages", "slots"])
def test_gaps(dtype, hk, dim, order):
    say("[gaps]", dtype, hk, dim, order)
    g, dt, page, hq, new, before, prefix = gen(31), TD[dtype], 8, 2 * hk, [3, 0, 40, 1], [20, 5, 0, 90], 21
    keys = [a + b for a, b in zip(new, before)]
    qkv = randn(g, sum(new), hq + 2 * hk, dim, dtype=dt).to(DEV)
    old = [randn(g, 200, page, hk, dim, dtype=dt).to(DEV) for _ in range(2)]
    pages, table, pre = tables(g, keys, page, prefix)
    pos = torch.arange(sum(new), dtype=torch.int32, device=DEV)
    freqs = sc.rope_frequencies(dim, device=DEV)

    def step(kp, vp):
        kp.copy_(old[0][:pages])
        vp.copy_(old[1][:pages])
        q, k, v = qkv.split([hq, hk, hk], 1)
        q = sc.qk_norm_rope_append(q, k, v, pos, freqs, kp, vp, table.to(DEV),
                                   torch.tensor(keys, dtype=torch.int32, device=DEV), cu_q=offsets(new).to(DEV))
        return [q, kp, vp, *attend(q, kp, vp, table.to(DEV), keys, new, None, None, right=0),
                *attend(q, kp, vp, table.to(DEV), keys, new, pre.to(DEV), prefix, left=50, right=0)]

    want = step(*(torch.empty(pages, page, hk, dim, dtype=dt, device=DEV) for _ in range(2)))
    gap = 8
    kp, vp, flat = gapped(pages, page, hk, dim, dt, gap, order)
    got = step(kp, vp)
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    kp.fill_(7.0)
    vp.fill_(7.0)
    assert bool((flat == 7).all())


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 72)])
def test_tokens_with_one_place(dtype, dim):
    """Two sequences that share a page, a page that a sequence has twice: every other place, and every query, as if each
    token had a place of its own. What the shared places hold is unspecified."""
    g, dt, page, hq, hk, n = gen(32), TD[dtype], 8, 4, 2, 40
    say("[one place]", dtype, dim)
    qkv = randn(g, 3 * n, hq + 2 * hk, dim, dtype=dt).to(DEV)
    table = torch.tensor([[0, 1, 2, 3, 4], [5, 6, 2, 7, 8], [9, 10, 11, 9, 12]], dtype=torch.int32, device=DEV)
    pos = torch.arange(3 * n, dtype=torch.int32, device=DEV)
    freqs = sc.rope_frequencies(dim, device=DEV)
    q, k, v = qkv.split([hq, hk, hk], 1)
    lens = torch.full((3,), n, dtype=torch.int32, device=DEV)

    def run(table):
        kp, vp = (torch.full((16, page, hk, dim), 7.0, dtype=dt, device=DEV) for _ in range(2))
        return sc.qk_norm_rope_append(q, k, v, pos, freqs, kp, vp, table, lens), kp, vp

    own = torch.arange(15, dtype=torch.int32, device=DEV).view(3, 5)
    got, want = run(table), run(own)
    assert torch.equal(bits(got[0]), bits(want[0]))
    for x, y in zip(got[1:], want[1:]):
        for p, o in zip(table.flatten().tolist(), own.flatten().tolist()):
            assert p in (2, 9) or torch.equal(bits(x[p]), bits(y[o]))
        assert bool((x[13:] == 7).all())
