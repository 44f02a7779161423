"""Operators over voxel tokens: per-head norm with position rotation, and
attention in a window with sinks (the calls of the same names, with the
tr_sparseconv_ prefix, in include/tr_sparseconv.h).

    q, k = qk_norm_rope(q, k, coords[:, 1:], rope_frequencies(dim, axes=3))
    y = window_attention(q, k, v, cu_q=cu, cu_k=cu, left=512, right=512, sinks=4)

Tensors of heads are [tokens, heads, dim]; their rows' elements are adjacent,
tokens and heads may be strided (slices of one projection's rows) by multiples
of 16 bytes. The calls record no gradients: the *_backward calls compute them
(examples/voxel_transformer.py has autograd functions around both).
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import Heads, Rotation, Window, check

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
_byref = ctypes.byref
_Pairs = ctypes.c_int * 3
_FIELD_MOST = 1 << 31  # a number past its C field would be taken modulo its range


def _heads(t, name: str, tokens=None, heads=None, dim=None, like: torch.Tensor | None = None) -> Heads:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(shape)}")
    n, h, d = shape
    if h >= _FIELD_MOST or d >= _FIELD_MOST:
        raise ValueError(f"{name} has {h} heads of {d} elements, past 2^31")
    if like is not None:
        if d != dim or (tokens is not None and n != tokens) or (heads is not None and h != heads):
            want = ["*" if w is None else w for w in (tokens, heads, dim)]
            raise ValueError(f"{name} must be [{want[0]}, {want[1]}, {want[2]}], got {tuple(shape)}")
        if t.dtype is not like.dtype or t.device != like.device:
            raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    # a stride that is never taken may be anything
    return Heads(t.data_ptr() if n else None, st if n > 1 else 0, sh if h > 1 else 0, h)


def _dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise ValueError(f"{name} has unsupported type {getattr(t, 'dtype', type(t))}")
    return _DTYPES[t.dtype]


def _ints(t, name: str, n: int, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 or t.dim() != 1 \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector on {device}")
    if n >= 0 and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")
    return t.data_ptr()


def _scratch(nbytes: int, device, given):
    """(pointer, bytes, owner) of a workspace; torch's own blocks are aligned to 256 bytes and more."""
    if given is not None:
        if given.nbytes < nbytes:
            raise ValueError(f"workspace of {given.nbytes} bytes, {nbytes} needed")
        if given.buf.device != device:
            raise ValueError(f"the workspace is on {given.buf.device}, the tensors on {device}")
        return given.ptr, given.nbytes, given
    if nbytes == 0:
        return None, 0, None
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf.data_ptr(), nbytes, buf


def _out(out, name: str, tokens: int, heads: int, dim: int, like: torch.Tensor):
    """An output of the caller's, or a new contiguous one, with its view."""
    if out is not None:
        return out, _heads(out, name, tokens, heads, dim, like)
    out = like.new_empty((tokens, heads, dim))
    return out, Heads(out.data_ptr() if tokens else None, heads * dim if tokens > 1 else 0, dim if heads > 1 else 0,
                      heads)


# The stream's address without a Stream object around it, where torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, device, *args) -> None:
    """fn(*args, stream) on the device's current stream. (A call of a few
    microseconds: the context manager is entered only for another device.)"""
    stream = _raw_stream(device.index)
    if torch.cuda.current_device() == device.index:
        check(fn(*args, stream))
    else:
        with torch.cuda.device(device):
            check(fn(*args, stream))


def rope_frequencies(dim: int, axes: int = 1, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Frequencies (radians a step) for qk_norm_rope, fp32 [dim / 2]: each axis
    has dim / 2 // axes pairs, pair i of them theta^(-i / pairs); pairs left over
    (which do not turn) have 0."""
    if dim <= 0 or dim % 2 or not 1 <= axes <= 3:
        raise ValueError(f"dim = {dim} must be even and axes = {axes} in 1 .. 3")
    n = dim // 2 // axes
    f = [theta ** (-i / n) for _ in range(axes) for i in range(n)]
    return torch.tensor(f + [0.0] * (dim // 2 - len(f)), dtype=torch.float32, device=device)


def _rotation(pos, freqs, sections, interleaved, tokens, dim, device) -> Rotation:
    if not isinstance(pos, torch.Tensor) or pos.device != device or pos.dtype != torch.int32:
        raise ValueError(f"pos must be an int32 tensor on {device}")
    if pos.dim() == 1:
        pos = pos[:, None]
    shape = pos.shape
    if len(shape) != 2 or shape[0] != tokens or not 1 <= shape[1] <= 3:
        raise ValueError(f"pos must be [{tokens}, 1 .. 3 axes], got {tuple(shape)}")
    axes = shape[1]
    if axes > 1 and pos.stride(1) != 1:
        raise ValueError("the axes of a position must be adjacent")
    if not isinstance(freqs, torch.Tensor) or freqs.device != device or freqs.dtype != torch.float32 \
            or freqs.shape != (dim // 2,) or not freqs.is_contiguous():
        raise ValueError(f"freqs must be fp32 [{dim // 2}] on {device}")
    if sections is None:
        sections = [dim // 2 // axes] * axes
    if len(sections) != axes or not all(0 <= s <= dim for s in sections):
        raise ValueError(f"{axes} axes need {axes} sections of pairs, got {list(sections)}")
    return Rotation(pos.data_ptr() if tokens else None, pos.stride(0) if tokens > 1 else 0, freqs.data_ptr(), axes,
                    _Pairs(*sections), bool(interleaved))


def _gain(g, name: str, heads: int, dim: int, device):
    """(pointer, rows) of a gain [dim] or [heads, dim]."""
    if g is None:
        return None, 1
    if not isinstance(g, torch.Tensor) or g.device != device or g.dtype != torch.float32 or not g.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor on {device}")
    if g.shape == (dim,):
        return g.data_ptr(), 1
    if g.shape == (heads, dim):
        return g.data_ptr(), heads
    raise ValueError(f"{name} must be [{dim}] or [{heads}, {dim}], got {tuple(g.shape)}")


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, freqs: torch.Tensor,
                 q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None, sections=None,
                 interleaved: bool = False, eps: float = 1e-6, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None):
    """RMS norm of every query and key row, its gain, and the position rotation,
    in one pass (tr_sparseconv_qk_norm_rope). Returns (q_out, k_out).

    pos: int32 [tokens, axes] (1 to 3; coords[:, 1:] serves) or [tokens]; freqs:
    fp32 [dim / 2], radians a step (rope_frequencies); sections: pairs of each
    axis, default dim / 2 // axes. Gains: fp32 [dim] (shared) or [heads, dim].
    q_out / k_out may be q / k themselves; other overlaps are refused."""
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    hk = _heads(k, "k", n, None, dim, q)
    dev = q.device
    rot = _rotation(pos, freqs, sections, interleaved, n, dim, dev)
    qg, qr = _gain(q_gain, "q_gain", hq.heads, dim, dev)
    kg, kr = _gain(k_gain, "k_gain", hk.heads, dim, dev)
    q_out, ho = _out(q_out, "q_out", n, hq.heads, dim, q)
    k_out, hp = _out(k_out, "k_out", n, hk.heads, dim, q)
    _call(_lib.lib().tr_sparseconv_qk_norm_rope, dev, _byref(hq), _byref(hk), _byref(rot), qg, qr, kg, kr, eps,
          _byref(ho), _byref(hp), n, dim, dt)
    return q_out, k_out


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          pos: torch.Tensor, freqs: torch.Tensor, q_gain: torch.Tensor | None = None,
                          k_gain: torch.Tensor | None = None, sections=None, interleaved: bool = False,
                          eps: float = 1e-6, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                          workspace=None):
    """Gradients of L = sum <q_out, dq_out> + sum <k_out, dk_out> of qk_norm_rope
    with the same further arguments (tr_sparseconv_qk_norm_rope_backward):
    (dq, dk, dq_gain, dk_gain), the last two fp32, None without that gain."""
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    hk = _heads(k, "k", n, None, dim, q)
    dev = q.device
    gq, gk = _heads(dq_out, "dq_out", n, hq.heads, dim, q), _heads(dk_out, "dk_out", n, hk.heads, dim, q)
    rot = _rotation(pos, freqs, sections, interleaved, n, dim, dev)
    qg, qr = _gain(q_gain, "q_gain", hq.heads, dim, dev)
    kg, kr = _gain(k_gain, "k_gain", hk.heads, dim, dev)
    dq, oq = _out(dq, "dq", n, hq.heads, dim, q)
    dk, ok = _out(dk, "dk", n, hk.heads, dim, q)
    dqg = None if q_gain is None else torch.empty_like(q_gain)
    dkg = None if k_gain is None else torch.empty_like(k_gain)
    L = _lib.lib()
    ptr, nbytes, _keep = _scratch(
        L.tr_sparseconv_qk_norm_rope_backward_workspace_bytes(n, hq.heads, hk.heads, dim), dev, workspace)
    _call(L.tr_sparseconv_qk_norm_rope_backward, dev, _byref(gq), _byref(gk), _byref(hq), _byref(hk), _byref(rot), qg,
          qr, kg, kr, eps, _byref(oq), _byref(ok), None if dqg is None else dqg.data_ptr(),
          None if dkg is None else dkg.data_ptr(), n, dim, dt, ptr, nbytes)
    return dq, dk, dqg, dkg


def _window(cu_q, cu_k, k_len, left, right, sinks, scale, dim, device) -> Window:
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    if cu_q is not None and isinstance(cu_q, torch.Tensor) and cu_q.dim() == 1 and cu_q.shape[0] < 2:
        raise ValueError("cu_q needs two elements at least (one sequence)")
    if not (-1 <= left < 1 << 63 and -1 <= right < 1 << 63 and 0 <= sinks < _FIELD_MOST):
        raise ValueError(f"window ({left}, {right}) with {sinks} sinks: sides are -1 or more, sinks 0 or more")
    batch = 1 if cu_q is None else len(cu_q) - 1
    if batch >= _FIELD_MOST:
        raise ValueError(f"{batch} sequences, past 2^31")
    return Window(_ints(cu_q, "cu_q", -1, device), _ints(cu_k, "cu_k", batch + 1, device),
                  _ints(k_len, "k_len", batch, device), batch, left, right, sinks,
                  dim ** -0.5 if scale is None else scale)


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor | None = None,
                     cu_k: torch.Tensor | None = None, k_len: torch.Tensor | None = None, left: int = -1,
                     right: int = -1, sinks: int = 0, scale: float | None = None, return_lse: bool = False,
                     out: torch.Tensor | None = None, workspace=None):
    """Attention in a window that moves with the query, plus the first `sinks`
    keys of the sequence (tr_sparseconv_window_attention). Returns out, or
    (out, lse [q heads, tokens] fp32) with return_lse.

    Query i of a sequence with Lq queries and Lk keys stands at p = i + Lk - Lq and
    sees key j when j <= p + right and (j >= p - left or j < sinks); -1 lifts the
    limit of a side, right = 0 is causal. Sequences lie one after the other: b has
    the rows cu_q[b] .. cu_q[b + 1] of q and cu_k[b] .. cu_k[b + 1] of k and v, of
    which only the first k_len[b] count when given (a cache with room to grow).
    Without cu_q and cu_k all rows are one sequence. Query heads are a multiple of
    the key-value heads."""
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    hk = _heads(k, "k", None, None, dim, q)
    m = k.shape[0]
    hv = _heads(v, "v", m, hk.heads, dim, q)
    dev = q.device
    win = _window(cu_q, cu_k, k_len, left, right, sinks, scale, dim, dev)
    out, ho = _out(out, "out", n, hq.heads, dim, q)
    lse = torch.empty((hq.heads, n), dtype=torch.float32, device=dev) if return_lse else None
    L = _lib.lib()
    ptr, nbytes, _keep = _scratch(
        L.tr_sparseconv_window_attention_workspace_bytes(_byref(win), n, m, hq.heads, hk.heads, dim, dt), dev,
        workspace)
    _call(L.tr_sparseconv_window_attention, dev, _byref(hq), _byref(hk), _byref(hv), _byref(win), _byref(ho),
          None if lse is None else lse.data_ptr(), n, m, dim, dt, ptr, nbytes)
    return (out, lse) if return_lse else out


def window_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              out: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor | None = None,
                              cu_k: torch.Tensor | None = None, k_len: torch.Tensor | None = None, left: int = -1,
                              right: int = -1, sinks: int = 0, scale: float | None = None, workspace=None):
    """(dq, dk, dv) of L = sum <out, dout> of window_attention with the same
    further arguments (tr_sparseconv_window_attention_backward); out and lse are
    the forward's on these tensors."""
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    hk = _heads(k, "k", None, None, dim, q)
    m = k.shape[0]
    hv = _heads(v, "v", m, hk.heads, dim, q)
    dev = q.device
    hd, ho = _heads(dout, "dout", n, hq.heads, dim, q), _heads(out, "out", n, hq.heads, dim, q)
    if not isinstance(lse, torch.Tensor) or lse.device != dev or lse.dtype != torch.float32 \
            or tuple(lse.shape) != (hq.heads, n) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 tensor [{hq.heads}, {n}] on {dev}")
    win = _window(cu_q, cu_k, k_len, left, right, sinks, scale, dim, dev)
    dq = torch.empty((n, hq.heads, dim), dtype=q.dtype, device=dev)
    dk, dv = (torch.empty((m, hk.heads, dim), dtype=q.dtype, device=dev) for _ in range(2))
    L = _lib.lib()
    ptr, nbytes, _keep = _scratch(
        L.tr_sparseconv_window_attention_backward_workspace_bytes(_byref(win), n, m, hq.heads, hk.heads, dim, dt),
        dev, workspace)
    _call(L.tr_sparseconv_window_attention_backward, dev, _byref(hd), _byref(hq), _byref(hk), _byref(hv), _byref(ho),
          lse.data_ptr(), _byref(win), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), n, m, dim, dt, ptr, nbytes)
    return dq, dk, dv
