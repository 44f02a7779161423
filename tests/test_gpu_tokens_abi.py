"""Calls of the token operators' C interface that the binding does not make."""
import ctypes

import pytest
import torch

from submanifold_sparse_conv_amd import _lib
from tests.test_gpu_tokens import DEV, gen, randn

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


@pytest.mark.parametrize("rows", [0, -7, 5, 1 << 24, (1 << 31) - 1])
def test_rows_of_a_gain_that_is_not_there(rows):
    """The row count beside a NULL gain is not read, with the other side's gradient wanted or not."""
    n, hq, hk, dim = 40, 3, 2, 128
    g = gen(71)
    q, k, dq, dk = (randn(g, n, h, dim, dtype=torch.float32).to(DEV) for h in (hq, hk, hq, hk))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freqs = sc.rope_frequencies(dim, device=DEV)
    gain = (1 + 0.2 * torch.randn(hk, dim, generator=g)).to(DEV)
    want_y = sc.qk_norm_rope(q, k, pos, freqs, None, gain)
    want = sc.qk_norm_rope_backward(dq, dk, q, k, pos, freqs, None, gain)
    L, b = _lib.lib(), ctypes.byref

    def view(t):
        return _lib.Heads(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1])

    rot = _lib.Rotation(pos.data_ptr(), 1, freqs.data_ptr(), 1, (ctypes.c_int * 3)(dim // 2, 0, 0), 0)
    yq, yk, xq, xk, dg = (torch.empty_like(t) for t in (q, k, q, k, gain))
    ws = sc.Workspace(L.tr_sparseconv_qk_norm_rope_backward_workspace_bytes(n, hq, hk, dim), DEV)
    st = torch.cuda.current_stream().cuda_stream
    q_, k_, dq_, dk_, yq_, yk_, xq_, xk_ = (view(t) for t in (q, k, dq, dk, yq, yk, xq, xk))
    assert L.tr_sparseconv_qk_norm_rope(b(q_), b(k_), b(rot), None, rows, gain.data_ptr(), hk, 1e-6, b(yq_), b(yk_), n,
                                        dim, _lib.F32, st) == 0
    assert L.tr_sparseconv_qk_norm_rope_backward(b(dq_), b(dk_), b(q_), b(k_), b(rot), None, rows, gain.data_ptr(), hk,
                                                 1e-6, b(xq_), b(xk_), None, dg.data_ptr(), n, dim, _lib.F32, ws.ptr,
                                                 ws.nbytes, st) == 0, L.tr_sparseconv_last_error()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((yq, yk, xq, xk, dg), (*want_y, want[0], want[1], want[3])))
