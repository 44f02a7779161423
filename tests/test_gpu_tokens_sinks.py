"""Gradients where rows past the band see the sinks: the key blocks, the chunks of rows (which start inside a token
where the group does not divide 32) and the joins of that part of the gradient."""
import pytest

from tests.test_gpu_tokens import run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("f32", 96), ("f32", 128), ("f16", 24)])
@pytest.mark.parametrize("group", [1, 3, 5, 8])
@pytest.mark.parametrize("sinks", [40, 128])
def test_many_sinks(dtype, dim, group, sinks):
    run_case([600], [600], 1, group, dim, dtype, 20, 0, sinks)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f32", 32)])
@pytest.mark.parametrize("sinks", [1, 33, 97])
def test_more_heads_than_a_row_tile(dtype, dim, sinks):
    run_case([260], [260], 1, 40, dim, dtype, 20, 0, sinks)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 96), ("f32", 128)])
@pytest.mark.parametrize("lens_q,lens_k", [([900, 37, 0, 411], [900, 37, 5, 411]), ([400, 300], [700, 333]),
                                           ([700, 2], [300, 900])])
@pytest.mark.parametrize("hk,group", [(2, 4), (1, 6)])
def test_ragged_and_unequal(dtype, dim, lens_q, lens_k, hk, group):
    """Several sequences, keys before the first query, and rows before the first key."""
    run_case(lens_q, lens_k, hk, group, dim, dtype, 20, 0, 70, room=[n + 11 for n in lens_k])


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 128)])
def test_many_chunks(dtype, dim):
    """Chunks by the dozen, a window on both sides."""
    run_case([3000], [3000], 1, 4 if dtype == "bf16" else 1, dim, dtype, 100, 30, 128)
