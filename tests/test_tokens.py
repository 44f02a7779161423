"""Refusals of the token operators: the C ABI's host checks and the binding's.
No GPU needed: every call fails before anything is enqueued."""
import ctypes

import pytest
import torch

from submanifold_sparse_conv_amd import _lib
import submanifold_sparse_conv_amd as sc

P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def heads(h=2, data=FAKE, ts=256, hs=64):
    return _lib.Heads(data, ts, hs, h)


def rotation(pos=FAKE, stride=1, freqs=FAKE, axes=1, pairs=(32, 0, 0), il=0):
    return _lib.Rotation(pos, stride, freqs, axes, (ctypes.c_int * 3)(*pairs), il)


def window(cu_q=None, cu_k=None, k_len=None, batch=1, left=4, right=0, sinks=0, scale=0.1):
    return _lib.Window(cu_q, cu_k, k_len, batch, left, right, sinks, scale)


def norm(L, q=None, k=None, rot=None, qg=None, qr=1, kg=None, kr=1, eps=1e-6, qo=None, ko=None, tokens=10, dim=64,
         dtype=_lib.BF16, drop=()):
    args = dict(q=q or heads(), k=k or heads(), rot=rot or rotation(), qo=qo or heads(), ko=ko or heads())
    r = {n: None if n in drop else ctypes.byref(v) for n, v in args.items()}
    return L.tr_sparseconv_qk_norm_rope(r["q"], r["k"], r["rot"], qg, qr, kg, kr, eps, r["qo"], r["ko"], tokens, dim,
                                        dtype, None)


@pytest.mark.parametrize("how,code", [
    (dict(drop=("q",)), _lib.ERR_INVALID_ARG), (dict(drop=("k",)), _lib.ERR_INVALID_ARG),
    (dict(drop=("rot",)), _lib.ERR_INVALID_ARG), (dict(drop=("qo",)), _lib.ERR_INVALID_ARG),
    (dict(drop=("ko",)), _lib.ERR_INVALID_ARG), (dict(dtype=7), _lib.ERR_UNSUPPORTED),
    (dict(dim=0), _lib.ERR_INVALID_ARG), (dict(dim=12), _lib.ERR_UNSUPPORTED), (dict(dim=136), _lib.ERR_UNSUPPORTED),
    (dict(tokens=-1), _lib.ERR_INVALID_ARG), (dict(tokens=(1 << 30) + 1), _lib.ERR_INVALID_ARG),
    (dict(q=heads(0)), _lib.ERR_INVALID_ARG), (dict(k=heads(5000)), _lib.ERR_INVALID_ARG),
    (dict(q=heads(data=None)), _lib.ERR_INVALID_ARG), (dict(q=heads(data=FAKE + 8)), _lib.ERR_INVALID_ARG),
    (dict(q=heads(ts=257)), _lib.ERR_INVALID_ARG), (dict(k=heads(hs=-64)), _lib.ERR_INVALID_ARG),
    (dict(qo=heads(3)), _lib.ERR_INVALID_ARG), (dict(qo=heads(ts=0)), _lib.ERR_INVALID_ARG),
    (dict(ko=heads(hs=32)), _lib.ERR_INVALID_ARG), (dict(eps=-1.0), _lib.ERR_INVALID_ARG),
    (dict(eps=float("nan")), _lib.ERR_INVALID_ARG), (dict(rot=rotation(axes=0)), _lib.ERR_INVALID_ARG),
    (dict(rot=rotation(axes=4)), _lib.ERR_INVALID_ARG), (dict(rot=rotation(pairs=(33, 0, 0))), _lib.ERR_INVALID_ARG),
    (dict(rot=rotation(axes=2, pairs=(2, -1, 0))), _lib.ERR_INVALID_ARG),
    (dict(rot=rotation(axes=3, pairs=(2147483647, 2147483647, 2))), _lib.ERR_INVALID_ARG),
    (dict(rot=rotation(pos=None)), _lib.ERR_INVALID_ARG), (dict(rot=rotation(freqs=None)), _lib.ERR_INVALID_ARG),
    (dict(rot=rotation(stride=-1)), _lib.ERR_INVALID_ARG), (dict(qg=FAKE, qr=3), _lib.ERR_INVALID_ARG),
])
def test_norm_rope_refusals(L, how, code):
    assert norm(L, **how) == code
    assert b"qk_norm_rope" in L.tr_sparseconv_last_error()


def test_norm_rope_backward_refusals(L):
    h, rot = heads(), rotation()
    b = ctypes.byref

    def call(qg=None, dqg=None, ws=P(0x10000), nbytes=1 << 30, dq=h):
        return L.tr_sparseconv_qk_norm_rope_backward(b(h), b(h), b(h), b(h), b(rot), qg, 1, None, 1, 1e-6, b(dq), b(h),
                                                     dqg, None, 10, 64, _lib.BF16, ws, nbytes, None)

    assert call(dqg=FAKE) == _lib.ERR_INVALID_ARG          # a gradient without its gain
    assert call(nbytes=64) == _lib.ERR_WORKSPACE
    assert call(ws=P(0x10010)) == _lib.ERR_INVALID_ARG      # misaligned
    assert call(ws=None) == _lib.ERR_INVALID_ARG
    assert call(dq=heads(ts=32)) == _lib.ERR_INVALID_ARG    # rows overlap
    W = L.tr_sparseconv_qk_norm_rope_backward_workspace_bytes
    assert W(-1, 1, 1, 64) == W(10, 0, 1, 64) == W(10, 1, 1, 12) == W(10, 1, 1, 136) == 0
    assert W(0, 1, 1, 64) == 0 < W(1, 1, 1, 64) <= W(10 ** 6, 1, 1, 64) <= 1024 * 4 * 2 * 64 * 4


def attend(L, q=None, k=None, v=None, win=None, out=None, nq=10, nk=20, dim=64, dtype=_lib.BF16, ws=None, nbytes=0,
           drop=()):
    args = dict(q=q or heads(4), k=k or heads(2), v=v or heads(2), win=win or window(), out=out or heads(4))
    r = {n: None if n in drop else ctypes.byref(x) for n, x in args.items()}
    return L.tr_sparseconv_window_attention(r["q"], r["k"], r["v"], r["win"], r["out"], None, nq, nk, dim, dtype, ws,
                                            nbytes, None)


@pytest.mark.parametrize("how,code", [
    *[(dict(drop=(n,)), _lib.ERR_INVALID_ARG) for n in ("q", "k", "v", "win", "out")],
    (dict(dtype=3), _lib.ERR_UNSUPPORTED), (dict(dim=20), _lib.ERR_UNSUPPORTED), (dict(dim=256), _lib.ERR_UNSUPPORTED),
    (dict(dim=-8), _lib.ERR_INVALID_ARG), (dict(nq=-1), _lib.ERR_INVALID_ARG), (dict(nk=-1), _lib.ERR_INVALID_ARG),
    (dict(nk=(1 << 30) + 1), _lib.ERR_INVALID_ARG), (dict(q=heads(3)), _lib.ERR_INVALID_ARG),
    (dict(v=heads(1)), _lib.ERR_INVALID_ARG), (dict(out=heads(2)), _lib.ERR_INVALID_ARG),
    (dict(out=heads(4, hs=0)), _lib.ERR_INVALID_ARG), (dict(k=heads(2, data=None)), _lib.ERR_INVALID_ARG),
    (dict(k=heads(2, data=FAKE + 2)), _lib.ERR_INVALID_ARG), (dict(v=heads(2, ts=4)), _lib.ERR_INVALID_ARG),
    (dict(win=window(batch=0)), _lib.ERR_INVALID_ARG), (dict(win=window(batch=2)), _lib.ERR_INVALID_ARG),
    (dict(win=window(left=-2)), _lib.ERR_INVALID_ARG), (dict(win=window(right=-2)), _lib.ERR_INVALID_ARG),
    (dict(win=window(sinks=-1)), _lib.ERR_INVALID_ARG), (dict(win=window(sinks=129)), _lib.ERR_INVALID_ARG),
    (dict(win=window(scale=0.0)), _lib.ERR_INVALID_ARG), (dict(win=window(scale=-1.0)), _lib.ERR_INVALID_ARG),
    (dict(win=window(scale=float("inf"))), _lib.ERR_INVALID_ARG),
    (dict(win=window(scale=float("nan"))), _lib.ERR_INVALID_ARG),
    (dict(nq=1 << 30), _lib.ERR_UNSUPPORTED),
])
def test_attention_refusals(L, how, code):
    assert attend(L, **how) == code
    assert b"window_attention" in L.tr_sparseconv_last_error()


def test_attention_workspace(L):
    """Few rows over many keys are split, and the parts need room."""
    b = ctypes.byref
    W = L.tr_sparseconv_window_attention_workspace_bytes
    far = window(left=-1)
    need = W(b(far), 1, 100000, 4, 2, 64, _lib.BF16)
    assert need > 0
    assert W(b(far), 100000, 100000, 4, 2, 64, _lib.BF16) == 0
    assert W(b(window(sinks=500)), 1, 100000, 4, 2, 64, _lib.BF16) == 0
    assert attend(L, win=far, nq=1, nk=100000, ws=P(0x10000), nbytes=need - 1) == _lib.ERR_WORKSPACE
    assert attend(L, win=far, nq=1, nk=100000, ws=P(0x10010), nbytes=need) == _lib.ERR_INVALID_ARG
    B = L.tr_sparseconv_window_attention_backward_workspace_bytes
    assert B(b(window(sinks=8)), 1000, 1000, 4, 2, 64, _lib.F32) > B(b(window()), 1000, 1000, 4, 2, 64, _lib.F32) >= 16000


def test_attention_backward_refusals(L):
    b = ctypes.byref
    q, k, win = heads(4), heads(2), window(sinks=2)

    def call(lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=P(0x10000), nbytes=1 << 30, dout=q):
        return L.tr_sparseconv_window_attention_backward(b(dout), b(q), b(k), b(k), b(q), lse, b(win), dq, dk, dv, 10,
                                                         20, 64, _lib.BF16, ws, nbytes, None)

    for how in (dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=FAKE + 4), dict(ws=None), dict(ws=P(0x10010)),
                dict(dout=heads(2))):
        assert call(**how) == _lib.ERR_INVALID_ARG, how
    assert call(nbytes=0, ws=None) == _lib.ERR_WORKSPACE


def test_binding_refuses_cpu_tensors_and_shapes():
    q = torch.zeros(4, 2, 16)
    pos = torch.zeros(4, 1, dtype=torch.int32)
    f = sc.rope_frequencies(16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        sc.qk_norm_rope(q, q, pos, f)
    with pytest.raises(ValueError, match="GPU"):
        sc.window_attention(q, q, q)
    with pytest.raises(ValueError, match="type"):
        sc.window_attention(q.double(), q, q)
    with pytest.raises(ValueError):
        sc.rope_frequencies(15)
    with pytest.raises(ValueError):
        sc.rope_frequencies(16, axes=4)


def test_rope_frequencies():
    f = sc.rope_frequencies(128, axes=3, theta=100.0, device="cpu")
    assert f.shape == (64,) and f.dtype == torch.float32
    assert torch.equal(f[:21], f[21:42]) and torch.equal(f[:21], f[42:63]) and float(f[63]) == 0.0
    assert float(f[0]) == 1.0 and abs(float(f[20]) - 100.0 ** (-20 / 21)) < 1e-7
