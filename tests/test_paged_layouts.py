"""Where the pages of keys and values may lie with respect to each other: the append's host check against every address
that the two hold. No GPU needed: the calls are refused for a q_out inside the pages, which is looked at afterwards."""
import itertools
import random

import pytest

from submanifold_sparse_conv_amd import _lib
from tests.test_paged import A, append, pages, view
from tests.test_tokens import rotation


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def refused_for(L, **how):
    h = how.get("h", 2)
    assert append(L, pg=pages(**how), q=view(1 << 40, 2 * h), out=view(A, 2 * h), k=view(1 << 41, h), v=view(1 << 42, h),
                  rot=rotation(pairs=(4, 0, 0)), dim=8) == _lib.ERR_INVALID_ARG
    return L.tr_sparseconv_last_error()


@pytest.mark.parametrize("how", [
    dict(v=A + 32, ks=(520, 32, 8), vs=(520, 32, 8)),     # a token's keys beside its values, eight elements behind a page
    dict(v=A + 512, ks=(712, 16, 8), vs=(712, 16, 8)),    # a page's keys, then its values, then 200 elements of neither
    dict(v=A + 16, ks=(520, 32, 16), vs=(520, 32, 16)),   # head by head
    dict(v=A + 32, ks=(32, 3208, 8), vs=(32, 3208, 8)),   # slots before pages
    dict(v=A + 16, ks=(32, 3208, 16), vs=(32, 3208, 16)),
    dict(v=A + 32 + 1040, ks=(520, 32, 8), vs=(520, 32, 8), n=2),
])
def test_gaps_that_are_no_multiple_of_a_slot(L, how):
    assert b"q_out overlaps the pages" in refused_for(L, **how), how


def rows(at, n, size, h, strides):
    return {at + 2 * (p * strides[0] + s * strides[1] + i * strides[2])
            for p, s, i in itertools.product(range(n), range(size), range(h))}


def test_against_every_address(L):
    """Pools of equal strides at all orders of their levels, gaps and offsets: refused for the overlap exactly where an
    element is in both."""
    rng, met, apart = random.Random(3), 0, 0
    for _ in range(3000):
        n, size, h = rng.choice([1, 2, 3]), 8, rng.choice([1, 2, 3])
        order, count, strides, extent = rng.sample(range(3), 3), (n, size, h), [0, 0, 0], 8
        for level in order:  # inner to outer, each with a gap now and then
            strides[level] = extent + 8 * rng.choice([0, 0, 1, 2, 5])
            extent = strides[level] * count[level]
        d = 8 * rng.randint(0, extent // 8 + 2) * rng.choice([-1, 1])
        # rows are 16 bytes at multiples of 16: they overlap where they are the same
        want = bool(rows(A, n, size, h, strides) & rows(A + 2 * d, n, size, h, strides))
        said = refused_for(L, v=A + 2 * d, ks=tuple(strides), vs=tuple(strides), n=n, size=size, h=h)
        assert (b"k pages overlap v pages" in said) == want, (n, h, strides, d, said)
        met, apart = met + want, apart + (not want)
    assert met > 500 and apart > 500
