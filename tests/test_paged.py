"""Refusals of the operators over a paged cache: the C ABI's host checks and the
binding's. No GPU needed: every call fails before anything is enqueued."""
import ctypes

import pytest
import torch

import submanifold_sparse_conv_amd as sc
from submanifold_sparse_conv_amd import _lib
from tests.test_tokens import heads, rotation, window

P = ctypes.c_void_p
A, B, C, D, F = (i << 32 for i in range(1, 6))  # addresses far from each other, never dereferenced
BAD, UNS = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def pages(k=A, v=B, ks=(2048, 128, 64), vs=(2048, 128, 64), n=100, size=16, h=2, table=0x10000, stride=8, width=8,
          length=0x20000, batch=2):
    return _lib.Pages(k, v, *ks, *vs, n, size, h, table, stride, width, length, batch)


def view(at, h, ts=None, hs=64):
    return heads(h, at, ts or h * 64, hs)


def append(L, q=None, k=None, v=None, rot=None, qg=None, kg=None, norm=1, eps=1e-6, out=None, pg=None, cu=0x30000, tokens=10,
           dim=64, dtype=_lib.BF16, drop=()):
    args = dict(q=q or view(C, 4), k=k or view(D, 2), v=v or view(F, 2), rot=rot or rotation(), out=out or view(C, 4),
                pg=pg or pages())
    r = {n: None if n in drop else ctypes.byref(x) for n, x in args.items()}
    return L.tr_sparseconv_qk_norm_rope_append(r["q"], r["k"], r["v"], r["rot"], qg, 1, kg, 1, norm, eps, r["out"], r["pg"],
                                               cu, tokens, dim, dtype, None)


POOLS = [
    (pages(h=3), BAD), (pages(size=0), UNS), (pages(size=4), UNS), (pages(size=24), UNS), (pages(size=1 << 17), UNS),
    (pages(size=-16), UNS), (pages(n=-1), BAD), (pages(n=1 << 31), BAD), (pages(batch=0), BAD),
    (pages(batch=(1 << 20) + 1), BAD), (pages(width=-1), BAD), (pages(width=1 << 27), BAD), (pages(stride=-1), BAD),
    (pages(length=None), BAD), (pages(table=None), BAD), (pages(k=None), BAD), (pages(v=None), BAD),
    (pages(k=A + 8), BAD), (pages(vs=(2048, 128, 60)), BAD), (pages(ks=(2052, 128, 64)), BAD),
    (pages(ks=(-2048, 128, 64)), BAD), (pages(vs=(1 << 41, 128, 64)), BAD),
    (pages(ks=(1 << 30, 1 << 23, 64)), UNS),
]


@pytest.mark.parametrize("pg,code", POOLS)
def test_pool_refusals(L, pg, code):
    assert append(L, pg=pg) == code
    assert b"qk_norm_rope_append" in L.tr_sparseconv_last_error()
    assert attend(L, pg=pg) == code
    assert attend(L, pg=pg, prefix=(0x50000, 20)) == code


@pytest.mark.parametrize("how,code", [
    *[(dict(drop=(n,)), BAD) for n in ("q", "k", "v", "rot", "out", "pg")],
    (dict(dtype=9), UNS), (dict(dim=12), UNS), (dict(dim=136), UNS), (dict(tokens=-1), BAD),
    (dict(tokens=(1 << 30) + 1), BAD), (dict(cu=None, tokens=11), BAD), (dict(k=view(D, 3)), BAD), (dict(v=view(F, 1)), BAD),
    (dict(v=view(None, 2)), BAD), (dict(v=view(F + 2, 2)), BAD), (dict(out=view(C, 3)), BAD),
    (dict(out=view(C, 4, ts=320)), BAD),         # q's memory, other strides
    (dict(out=view(D, 4)), BAD), (dict(out=view(F, 4)), BAD), (dict(out=view(A + 512, 4)), BAD),
    (dict(out=view(B, 4)), BAD), (dict(k=view(A, 2)), BAD), (dict(v=view(B + 4096, 2)), BAD),
    (dict(q=view(B, 4), out=view(C, 4)), BAD), (dict(out=view(C, 4, ts=128)), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(norm=0, qg=0x40000), BAD), (dict(norm=0, kg=0x40000), BAD),
    (dict(rot=rotation(axes=0)), BAD), (dict(rot=rotation(pairs=(33, 0, 0))), BAD), (dict(rot=rotation(pos=None)), BAD),
])
def test_append_refusals(L, how, code):
    assert append(L, **how) == code
    assert b"qk_norm_rope_append" in L.tr_sparseconv_last_error()


@pytest.mark.parametrize("pg", [
    pages(v=A), pages(v=A + 64), pages(v=A + 256),                                # k's own rows
    pages(v=A + 128, ks=(4096, 256, 64), vs=(4096, 256, 64)),                     # a head of k's
    pages(v=A + 2048 * 2, ks=(2048, 128, 64), vs=(4096, 128, 64)),                # unlike strides in one range
    pages(ks=(2048, 64, 64)), pages(ks=(1024, 128, 64)), pages(vs=(2048, 128, 32)),  # rows that overlap
    pages(vs=(0, 128, 64)), pages(ks=(2048, 0, 64)),
])
def test_append_refuses_pages_that_overlap(L, pg):
    assert append(L, pg=pg) == BAD
    assert b"overlap" in L.tr_sparseconv_last_error()


def test_append_takes_pages_side_by_side(L):
    """Keys and values in one tensor, at any level. The call is refused for its q_out inside the pages, which is looked
    at after them."""
    for how in (dict(v=A + 256, ks=(4096, 256, 64), vs=(4096, 256, 64)),          # in a token's row
                dict(v=A + 2 * 2048, ks=(4096, 128, 64), vs=(4096, 128, 64)),     # a page's keys, then its values
                dict(v=A + 2 * 64, ks=(4096, 256, 128), vs=(4096, 256, 128)),     # head by head
                dict(v=A + 2 * 1024, ks=(4096, 64, 2048), vs=(4096, 64, 2048)),   # heads before slots, head by head
                dict(v=A + 100 * 4096)):                                          # one after the other
        assert append(L, pg=pages(**how), out=view(A, 4)) == BAD
        assert b"q_out overlaps the pages" in L.tr_sparseconv_last_error(), how


def attend(L, q=None, pg=None, win=None, out=None, lse=None, nq=10, dim=64, dtype=_lib.BF16, ws=P(0x100000),
           nbytes=1 << 40, prefix=None, drop=()):
    args = dict(q=q or view(C, 4), pg=pg or pages(), win=win or window(cu_q=0x30000, batch=2), out=out or view(D, 4))
    r = {n: None if n in drop else ctypes.byref(x) for n, x in args.items()}
    if prefix is None:
        return L.tr_sparseconv_paged_window_attention(r["q"], r["pg"], r["win"], r["out"], lse, nq, dim, dtype, ws, nbytes,
                                                      None)
    return L.tr_sparseconv_shared_prefix_attention(r["q"], r["pg"], *prefix, r["win"], r["out"], lse, nq, dim, dtype, ws,
                                                   nbytes, None)


@pytest.mark.parametrize("how,code", [
    *[(dict(drop=(n,)), BAD) for n in ("q", "pg", "win", "out")],
    (dict(dtype=4), UNS), (dict(dim=20), UNS), (dict(dim=256), UNS), (dict(nq=-1), BAD), (dict(nq=1 << 30), UNS),
    (dict(q=view(C, 3)), BAD), (dict(q=view(None, 4)), BAD), (dict(q=view(C + 4, 4)), BAD), (dict(out=view(D, 2)), BAD),
    (dict(out=view(D, 4, hs=0)), BAD), (dict(pg=pages(h=0)), BAD), (dict(pg=pages(h=5000)), BAD),
    (dict(win=window(cu_q=0x30000, batch=3)), BAD), (dict(win=window(batch=2, cu_q=0x30000, cu_k=0x30000)), BAD),
    (dict(win=window(batch=2, cu_q=0x30000, k_len=0x30000)), BAD), (dict(win=window(batch=2), nq=11), BAD),
    (dict(win=window(cu_q=0x30000, batch=2, left=-2)), BAD), (dict(win=window(cu_q=0x30000, batch=2, right=-2)), BAD),
    (dict(win=window(cu_q=0x30000, batch=2, sinks=-1)), BAD), (dict(win=window(cu_q=0x30000, batch=2, sinks=129)), BAD),
    (dict(win=window(cu_q=0x30000, batch=2, scale=0.0)), BAD),
    (dict(win=window(cu_q=0x30000, batch=2, scale=float("nan"))), BAD),
    (dict(out=view(C, 4)), BAD), (dict(out=view(A, 4)), BAD), (dict(out=view(B + 1024, 4)), BAD), (dict(lse=C), BAD),
    (dict(lse=D), BAD), (dict(lse=A + 64), BAD),
])
def test_attention_refusals(L, how, code):
    assert attend(L, **how) == code
    assert b"paged_window_attention" in L.tr_sparseconv_last_error()
    assert attend(L, prefix=(0x50000, 33), **how) == code
    assert b"shared_prefix_attention" in L.tr_sparseconv_last_error()


def test_prefix_refusals(L):
    assert attend(L, prefix=(None, 5)) == BAD
    assert attend(L, prefix=(0x50000, -1)) == BAD
    assert attend(L, prefix=(0x50000, 1 << 30)) == BAD
    assert attend(L, prefix=(0x50000, 5), pg=pages(n=0)) == BAD


def test_workspace(L):
    b = ctypes.byref
    W = L.tr_sparseconv_paged_attention_workspace_bytes
    win = window(cu_q=0x30000, batch=2, left=-1)
    far = pages(width=8192, stride=8192)
    need = W(b(far), b(win), 0, 2, 4, 64, _lib.BF16)
    assert need > 0
    assert W(b(far), b(win), 5000, 2, 4, 64, _lib.BF16) > 0
    assert W(b(far), b(win), 0, 2, 3, 64, _lib.BF16) == W(b(far), b(win), 0, -1, 4, 64, _lib.BF16) == 0
    assert W(b(far), b(win), 5000, 0, 4, 64, _lib.BF16) == W(b(far), b(window(batch=2)), 0, 0, 4, 64, _lib.F32) == 0
    assert W(None, b(win), 0, 2, 4, 64, _lib.BF16) == W(b(far), None, 0, 2, 4, 64, _lib.BF16) == 0
    assert attend(L, pg=far, win=win, nq=2, nbytes=need - 1) == _lib.ERR_WORKSPACE
    assert attend(L, pg=far, win=win, nq=2, ws=None) == BAD
    assert attend(L, pg=far, win=win, nq=2, ws=P(0x100010)) == BAD


def test_binding_refuses_cpu_tensors_and_shapes():
    q = torch.zeros(4, 2, 16)
    pool = torch.zeros(3, 8, 2, 16)
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    pos, f = torch.zeros(4, dtype=torch.int32), sc.rope_frequencies(16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        sc.qk_norm_rope_append(q, q, q, pos, f, pool, pool, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        sc.paged_window_attention(q, pool, pool, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        sc.shared_prefix_attention(q, pool, pool, table, lens, lens, 3)
    with pytest.raises(ValueError, match="type"):
        sc.paged_window_attention(q.double(), pool, pool, table, lens)
    with pytest.raises(ValueError, match="prefix"):
        sc.shared_prefix_attention(q, pool, pool, table, lens, lens, 33)
    with pytest.raises(ValueError, match="prefix_len"):
        sc.shared_prefix_attention(q, pool, pool, table, lens, lens, -1)
    with pytest.raises(ValueError, match="prefix_len"):
        sc.shared_prefix_attention(q, pool, pool, table, lens, lens, 1 << 40)
