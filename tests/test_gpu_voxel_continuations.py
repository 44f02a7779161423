"""The example's continuations of one prompt from a paged cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu

example = pytest.importorskip("examples.voxel_transformer")
DEV = "cuda:0"


@pytest.mark.parametrize("prompt,count,m", [(200, 3, 20), (1, 1, 1), (2100, 5, 17)])
def test_continuations(prompt, count, m):
    """Every sequence as `decode` has it from a cache of its own. Two computations of the same rows: each rounds queries,
    keys, weights and outputs (2^-8 relative, the weights' averaged), the projection of the outputs and its sum with
    the tokens: less than four roundings of the result's size between them."""
    torch.manual_seed(3)
    block = example.Block(width=64, heads=4, kv_heads=2, dim=32, window=50, sinks=3)
    t = torch.randn(prompt, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.randint(0, 64, (prompt, 3), dtype=torch.int32, device=DEV)
    tails = torch.randn(count, m, 64, dtype=torch.bfloat16, device=DEV)
    tail_pos = torch.randint(0, 64, (count, m, 3), dtype=torch.int32, device=DEV)
    got = block.continuations(t, pos, tails, tail_pos)
    assert got.shape == (count, m, 64)
    for b in range(count):
        want = block.decode(torch.cat([t, tails[b]]), torch.cat([pos, tail_pos[b]]), prompt)[prompt:]
        off = (got[b].float() - want.float()).square().mean().sqrt()
        assert float(off) <= 4 * 2 ** -8 * float(want.float().square().mean().sqrt())
