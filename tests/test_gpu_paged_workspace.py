"""A workspace whose buffer nothing but the call holds."""
import pytest
import torch

from tests.test_gpu_paged import DEV, attend, attend_inputs

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


class Passing:
    """Gives its bytes to the first who asks and keeps nothing of them."""

    def __init__(self, nbytes, device):
        self.nbytes, self.device, self.asked = nbytes, device, 0

    @property
    def buf(self):
        self.asked += 1
        return torch.empty(self.nbytes + 256, dtype=torch.uint8, device=self.device)


def test_buffer_is_held_by_the_call():
    new, keys, n = [1] * 3, [900, 30, 400], 5000
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 8, 2, 64, "bf16", "plain", n)
    want = attend(q, kp, vp, table, keys, new, pre_pages, n)[0]
    ws = Passing(1 << 25, DEV)
    assert torch.equal(attend(q, kp, vp, table, keys, new, pre_pages, n, workspace=ws)[0], want) and ws.asked == 1
    with pytest.raises(ValueError, match="workspace is on cpu"):
        attend(q, kp, vp, table, keys, new, pre_pages, n, workspace=Passing(1 << 25, "cpu"))


def test_what_is_no_workspace():
    """Its own error comes through, not one raised on top of it."""
    new, keys = [1] * 3, [900, 30, 400]
    q, own, pre, kp, vp, table, _ = attend_inputs(new, keys, 16, 8, 2, 64, "bf16", "plain")

    class Broken:
        buf = None

        @property
        def nbytes(self):
            raise KeyError("no bytes")

    class Words:
        buf, nbytes = None, "many"

    with pytest.raises(KeyError, match="no bytes"):
        attend(q, kp, vp, table, keys, new, None, None, workspace=Broken())
    with pytest.raises(TypeError):
        attend(q, kp, vp, table, keys, new, None, None, workspace=Words())
    Words.nbytes = 1 << 30
    with pytest.raises(ValueError, match="must be a Workspace"):
        attend(q, kp, vp, table, keys, new, None, None, workspace=Words())
