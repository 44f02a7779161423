"""The example of a transformer block over voxels: it trains, its gradients are
the plain block's, and decoding from the cache gives the causal block's rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")
from examples import voxel_transformer as vt  # noqa: E402


def test_training_lowers_the_loss():
    _, losses, *_ = vt.train(steps=12)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.8 * losses[0], losses


def plain_attention(block, t, pos, cu, causal):
    """The attention part in float64 with torch's own gradients."""
    n = t.shape[0]
    qkv = (t @ block.qkv.double()).view(n, -1, block.dim)
    q, k, v = qkv.split([block.heads, block.kv_heads, block.kv_heads], 1)
    pairs = block.dim // 2
    axis = torch.tensor([i // (pairs // 3) if i < pairs // 3 * 3 else 0 for i in range(pairs)], device=t.device)
    angle = pos.double()[:, axis] * block.freqs.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]

    def norm_rope(x, gain):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
        a, b = y.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    q, k = norm_rope(q, block.q_gain), norm_rope(k, block.k_gain)
    i = torch.arange(n, device=t.device)
    obj = torch.bucketize(i, cu[1:].long(), right=True)
    first = cu.long()[obj]
    sees = (i[None] - first[:, None] < block.sinks) | (i[None] >= i[:, None] - block.left)
    sees &= (obj[:, None] == obj) & (i[None] <= i[:, None] + (0 if causal else block.left))
    out = []
    for h in range(block.heads):
        g = h * block.kv_heads // block.heads
        z = (q[:, h] @ k[:, g].T * block.dim ** -0.5).masked_fill(~sees, float("-inf"))
        out.append(torch.softmax(z, -1) @ v[:, g])
    return t + torch.cat(out, -1) @ block.proj.double()


def test_gradients_are_the_plain_blocks():
    torch.manual_seed(3)
    coords, kmap, cu = vt.voxels(objects=2)
    # the first 300 tokens of either object
    rows = torch.cat([torch.arange(int(b), int(b) + 300) for b in cu[:2]]).cuda()
    cu2 = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
    pos = coords[rows, 1:]
    block = vt.Block()
    t = torch.randn(600, 128, dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(600, 128, dtype=torch.bfloat16, device="cuda")
    params = [block.qkv, block.proj, block.q_gain, block.k_gain]

    def run(plain):
        x = t.clone().requires_grad_()
        if plain:
            xd = x.double()
            y = plain_attention(block, xd, pos, cu2, False)
        else:
            q, k, v = block.rotated(x, pos)
            o = vt.WindowAttention.apply(q, k, v, dict(cu_q=cu2, cu_k=cu2, left=block.left, right=block.left,
                                                       sinks=block.sinks))
            y = x + o.flatten(1) @ block.proj
        return [y, *torch.autograd.grad((y.double() * dy.double()).sum(), [x, *params])]

    for name, a, b in zip(("y", "x", "qkv", "proj", "q_gain", "k_gain"), run(False), run(True)):
        # bf16 products and results on the way: a few roundings of 2^-9 (rms) each, at most ten in a row
        err = (a.double() - b.double()).norm() / b.double().norm()
        assert err < 10 * 2.0 ** -9, (name, float(err))


def test_decoding_from_the_cache_is_the_causal_block():
    torch.manual_seed(4)
    coords, kmap, cu = vt.voxels(objects=1)
    block = vt.Block()
    x = torch.randn(coords.shape[0], 64, dtype=torch.bfloat16, device="cuda")
    n = 200
    with torch.no_grad():
        t = sc.forward(kmap, x, block.conv)[:n].contiguous()
        pos = coords[:n, 1:]
        got = block.decode(t, pos, prompt=130)
        ref = plain_attention(block, t.double(), pos, torch.tensor([0, n], dtype=torch.int32, device="cuda"), True)
    err = (got.double() - ref).norm() / ref.norm()
    assert err < 5 * 2.0 ** -9, float(err)
