"""Outputs of the token operators that overlap their inputs or each other are refused. No GPU needed: the calls of
the norm's gradient that are accepted fail too, at the last check. (tests/test_gpu_tokens_overlap.py has accepted calls
of the attention.)"""
import ctypes
import random

import numpy as np
import pytest

from submanifold_sparse_conv_amd import _lib

P = ctypes.c_void_p
BASE = 0x1000000  # never dereferenced
FAR = 0x4000000000
NO, YES = "the gradient of a gain that is not there", "overlap"


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def view(at, ts, hs, h=1):
    """at, strides in bf16 elements."""
    return _lib.Heads(BASE + 2 * at, ts, hs, h)


def far(i, h=1):
    return _lib.Heads(FAR * (i + 1), 1 << 16, 64, h)


def norm_backward(L, tokens, dim, dq, dk, q=None, k=None, dq_out=None, dk_out=None):
    b = ctypes.byref
    rot = _lib.Rotation(FAR, 1, FAR, 1, (ctypes.c_int * 3)(dim // 2, 0, 0), 0)
    q, k = q or far(0, dq.heads), k or far(1, dk.heads)
    dq_out, dk_out = dq_out or far(2, dq.heads), dk_out or far(3, dk.heads)
    code = L.tr_sparseconv_qk_norm_rope_backward(b(dq_out), b(dk_out), b(q), b(k), b(rot), None, 1, None, 1, 1e-6, b(dq),
                                                 b(dk), 5 * FAR, None, tokens, dim, _lib.BF16, P(6 * FAR), 1 << 30, None)
    assert code == _lib.ERR_INVALID_ARG
    text = L.tr_sparseconv_last_error().decode()
    return next(t for t in (NO, YES) if t in text)


def cells(at, ts, hs, h, tokens, dim):
    t, i, d = np.ogrid[:tokens, :h, :dim]
    return (at + t * ts + i * hs + d).ravel()


def test_norm_gradient_in_place(L):
    w = 8 * 64  # rows of a projection: four query heads, two key heads, two others
    q, k = view(0, w, 64, 4), view(4 * 64, w, 64, 2)
    assert norm_backward(L, 100, 64, q, k) == NO                              # slices of the same rows
    assert norm_backward(L, 100, 64, q, k, q=q, k=k) == NO                    # the inputs themselves
    assert norm_backward(L, 100, 64, q, k, dq_out=q, dk_out=k) == NO
    p = view(4 * 64, w, 64, 4)
    assert norm_backward(L, 100, 64, q, p, dq_out=p, dk_out=q) == YES         # each other's
    assert norm_backward(L, 100, 64, q, view(3 * 64, w, 64, 2)) == YES        # one head in common
    assert norm_backward(L, 100, 64, q, k, q=view(64, w, 64, 4)) == YES       # a head further
    assert norm_backward(L, 100, 64, q, k, q=view(w, w, 64, 4)) == YES        # a token further
    assert norm_backward(L, 100, 64, q, k, q=view(100 * w, w, 64, 4)) == NO   # all tokens further
    assert norm_backward(L, 100, 64, q, k, q=view(0, 2 * w, 64, 4)) == YES    # other strides, the same start
    assert norm_backward(L, 100, 64, view(0, w, 128, 2), view(64, w, 128, 2)) == NO   # heads that alternate
    assert norm_backward(L, 100, 64, view(0, 64, 6400, 2), view(12800, 64, 6400, 2)) == NO  # heads before tokens
    assert norm_backward(L, 100, 64, view(0, 64, 3200, 2), far(5)) == YES     # ... whose rows overlap
    assert norm_backward(L, 1, 64, view(0, 0, 64, 2), view(128, 0, 64, 2)) == NO
    assert norm_backward(L, 1, 64, view(0, 0, 64, 2), view(64, 0, 64, 2)) == YES


def test_against_enumeration(L):
    """Random views in a small range: refused where elements coincide, accepted where none do and the token strides
    are alike."""
    rng = random.Random(5)
    seen = {(o, c): 0 for o in (False, True) for c in (NO, YES)}
    for _ in range(4000):
        dim, tokens = rng.choice([8, 16]), rng.choice([1, 2, 3, 5])
        alike = rng.random() < 0.8
        ts = rng.choice([8, 16, 24, 40, 64, 96, 128])
        views = []
        for _ in range(2):
            h, hs = rng.choice([1, 2, 3]), rng.choice([8, 16, 32, 48, 80, 200])
            views.append((8 * rng.randrange(40), ts if alike else 8 * rng.randrange(2, 20), hs, h))
        if any((tokens > 1 and v[1] < dim) or (v[3] > 1 and v[2] < dim) for v in views):
            continue  # refused as it was
        sets = [cells(*v, tokens, dim) for v in views]
        meet = any(len(np.unique(s)) < len(s) for s in sets) or bool(np.intersect1d(*sets).size)
        got = norm_backward(L, tokens, dim, *(view(*v) for v in views))
        assert got in (NO, YES)
        if meet:
            assert got == YES, (dim, tokens, views)
        elif tokens == 1 or views[0][1] == views[1][1]:
            assert got == NO, (dim, tokens, views)
        seen[meet, got] += 1
    assert seen[True, YES] > 300 and seen[False, NO] > 300, seen


def attend(L, out, q, k, v, nq=100, nk=100, lse=None):
    b = ctypes.byref
    win = _lib.Window(None, None, None, 1, -1, 0, 0, 0.1)
    code = L.tr_sparseconv_window_attention(b(q), b(k), b(v), b(win), b(out), lse, nq, nk, 64, _lib.BF16, P(6 * FAR),
                                            1 << 30, None)
    return code == _lib.ERR_INVALID_ARG and b"overlaps" in L.tr_sparseconv_last_error()


def test_attention(L):
    w = 8 * 64
    q, k, v = far(0, 4), view(0, w, 64, 2), view(2 * 64, w, 64, 2)
    out = far(1, 4)
    assert attend(L, q, q, k, v)
    assert attend(L, _lib.Heads(k.data, w, 64, 4), q, k, v)
    assert attend(L, view(50 * w, w, 64, 4), q, k, v)                        # over keys and values from token 50
    assert attend(L, view(3 * 64, w, 64, 4), q, k, v)                        # over one head of the values
    assert attend(L, view(4 * 64, 256, 64, 4), q, k, v)                      # beside them in the first row only
    assert attend(L, out, q, k, v, lse=FAR + 128)                            # inside q
    assert attend(L, out, q, k, v, lse=2 * FAR + 128)                        # inside out


def test_attention_gradient(L):
    b = ctypes.byref
    nq, nk, hq, hk, dim = 10, 20, 4, 2, 64
    win = _lib.Window(None, None, None, 1, 4, 0, 0, 0.1)

    def refused(dq=9 * FAR, dk=10 * FAR, dv=11 * FAR, lse=12 * FAR):
        q, k, v, out, dout = far(0, hq), far(1, hk), far(2, hk), far(3, hq), far(4, hq)
        code = L.tr_sparseconv_window_attention_backward(b(dout), b(q), b(k), b(v), b(out), lse, b(win), dq, dk, dv, nq, nk,
                                                         dim, _lib.BF16, P(6 * FAR), 1 << 30, None)
        return code == _lib.ERR_INVALID_ARG and b"overlaps" in L.tr_sparseconv_last_error()

    for i in range(5):
        assert refused(dq=FAR * (i + 1)) and refused(dk=FAR * (i + 1)) and refused(dv=FAR * (i + 1))
    assert refused(dk=9 * FAR + 2 * nq * hq * dim - 16)                      # the last elements of dq
    assert refused(dv=10 * FAR)
    assert refused(lse=9 * FAR + 64)
