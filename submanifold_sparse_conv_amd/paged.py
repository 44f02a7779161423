"""Operators over a paged key-value cache of voxel tokens (the calls of the same
names, with the tr_sparseconv_ prefix, in include/tr_sparseconv.h).

    q = qk_norm_rope_append(q, k, v, pos, freqs, k_pages, v_pages, page_table, k_len)
    y = paged_window_attention(q, k_pages, v_pages, page_table, k_len, right=0)

The pool is two tensors [pages, page_size, heads, dim], of any layout whose rows'
elements are adjacent (heads before slots, keys and values side by side in one
tensor); page_size is a power of two from 8. Key j of sequence b is
k_pages[page_table[b, j // page_size], j % page_size], and the sequence has
k_len[b] keys, those of the step's new tokens among them: k_len is advanced
first, then a step appends and attends with the same k_len. cu_q has the offsets
of the sequences' tokens; without it each has the same number, tokens / batch. The
calls read no length on the host and record no gradients.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import Pages, Window
from .tokens import _byref, _call, _dtype, _gain, _heads, _ints, _out, _rotation, _scratch


def _pages(k_pages, v_pages, page_table, k_len, dim: int, like: torch.Tensor) -> Pages:
    device, shape = like.device, None
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype is not like.dtype or t.device != device:
            raise ValueError(f"{name} must be a {like.dtype} tensor [pages, page_size, heads, dim] on {device}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"k_pages {tuple(shape)} and v_pages {tuple(t.shape)} must have one shape")
        shape = t.shape
        if t.stride(3) != 1 and dim > 1:
            raise ValueError(f"the elements of a row of {name} must be adjacent")
    pages, size, heads, d = shape
    if d != dim:
        raise ValueError(f"the pages' heads have {d} elements, q's {dim}")
    if not isinstance(page_table, torch.Tensor) or page_table.device != device or page_table.dtype != torch.int32 \
            or page_table.dim() != 2:
        raise ValueError(f"page_table must be an int32 tensor [batch, pages] on {device}")
    batch, width = page_table.shape
    if width > 1 and page_table.stride(1) != 1:
        raise ValueError("the entries of a row of page_table must be adjacent")
    length = _ints(k_len, "k_len", batch, device)
    if length is None:
        raise ValueError("k_len must be given")
    if batch < 1:
        raise ValueError("page_table needs a sequence at least")
    ks, vs = k_pages.stride(), v_pages.stride()
    keep = (pages > 1, size > 1, heads > 1)  # a stride that is never taken may be anything
    return Pages(k_pages.data_ptr() if pages else None, v_pages.data_ptr() if pages else None,
                 *(s if on else 0 for s, on in zip(ks, keep)), *(s if on else 0 for s, on in zip(vs, keep)), pages, size,
                 heads, page_table.data_ptr() if width else None, page_table.stride(0) if batch > 1 else 0, width, length,
                 batch)


def qk_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, freqs: torch.Tensor,
                        k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, k_len: torch.Tensor,
                        cu_q: torch.Tensor | None = None, q_gain: torch.Tensor | None = None,
                        k_gain: torch.Tensor | None = None, sections=None, interleaved: bool = False, eps: float = 1e-6,
                        norm: bool = True, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope of new tokens, their keys and values to the pages in the same
    pass (tr_sparseconv_qk_norm_rope_append). Returns q_out.

    q [tokens, q heads, dim], k and v [tokens, kv heads, dim]; pos, freqs, gains,
    sections, interleaved and eps as in qk_norm_rope; norm=False: rotation alone,
    without gains. Token i of a sequence's Lq is its key k_len[b] - Lq + i. Tokens
    of no sequence (behind cu_q's last) are neither stored nor written to q_out;
    one whose key is none of the table is not stored. q_out may be q itself."""
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    hk = _heads(k, "k", n, None, dim, q)
    hv = _heads(v, "v", n, hk.heads, dim, q)
    dev = q.device
    rot = _rotation(pos, freqs, sections, interleaved, n, dim, dev)
    qg, qr = _gain(q_gain, "q_gain", hq.heads, dim, dev)
    kg, kr = _gain(k_gain, "k_gain", hk.heads, dim, dev)
    pages = _pages(k_pages, v_pages, page_table, k_len, dim, q)
    cu = _ints(cu_q, "cu_q", pages.batch + 1, dev)
    q_out, ho = _out(q_out, "q_out", n, hq.heads, dim, q)
    _call(_lib.lib().tr_sparseconv_qk_norm_rope_append, dev, _byref(hq), _byref(hk), _byref(hv), _byref(rot), qg, qr, kg,
          kr, bool(norm), eps, _byref(ho), _byref(pages), cu, n, dim, dt)
    return q_out


def _attend(q, k_pages, v_pages, page_table, k_len, prefix, cu_q, left, right, sinks, scale, return_lse, out, workspace):
    dt = _dtype(q, "q")
    hq = _heads(q, "q")
    n, _, dim = q.shape
    dev = q.device
    pages = _pages(k_pages, v_pages, page_table, k_len, dim, q)
    # a number past its C field would be taken modulo its range
    if not (-1 <= left < 1 << 63 and -1 <= right < 1 << 63 and 0 <= sinks < 1 << 31):
        raise ValueError(f"window ({left}, {right}) with {sinks} sinks: sides are -1 or more, sinks 0 or more")
    win = Window(_ints(cu_q, "cu_q", pages.batch + 1, dev), None, None, pages.batch, left, right, sinks,
                 dim ** -0.5 if scale is None else scale)
    out, ho = _out(out, "out", n, hq.heads, dim, q)
    lse = torch.empty((hq.heads, n), dtype=torch.float32, device=dev) if return_lse else None
    L = _lib.lib()
    ptr, nbytes, _keep = _scratch(
        L.tr_sparseconv_paged_attention_workspace_bytes(_byref(pages), _byref(win), 0 if prefix is None else prefix[1], n,
                                                        hq.heads, dim, dt), dev, workspace)
    lse_ptr = None if lse is None else lse.data_ptr()
    if prefix is None:
        _call(L.tr_sparseconv_paged_window_attention, dev, _byref(hq), _byref(pages), _byref(win), _byref(ho), lse_ptr, n,
              dim, dt, ptr, nbytes)
    else:
        _call(L.tr_sparseconv_shared_prefix_attention, dev, _byref(hq), _byref(pages), prefix[0], prefix[1], _byref(win),
              _byref(ho), lse_ptr, n, dim, dt, ptr, nbytes)
    return (out, lse) if return_lse else out


def paged_window_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                           k_len: torch.Tensor, cu_q: torch.Tensor | None = None, left: int = -1, right: int = -1,
                           sinks: int = 0, scale: float | None = None, return_lse: bool = False,
                           out: torch.Tensor | None = None, workspace=None):
    """window_attention of packed queries over each sequence's pages
    (tr_sparseconv_paged_window_attention): single tokens, drafted ones, parts of
    prompts. Returns out, or (out, lse [q heads, tokens] fp32) with return_lse.

    Query i of a sequence's Lq stands at p = i + k_len - Lq and sees key j when
    j <= p + right and (j >= p - left or j < sinks); -1 lifts the limit of a side.
    Rows of out and lse that belong to no sequence are left as they are."""
    return _attend(q, k_pages, v_pages, page_table, k_len, None, cu_q, left, right, sinks, scale, return_lse, out,
                   workspace)


def shared_prefix_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                            k_len: torch.Tensor, prefix_pages: torch.Tensor, prefix_len: int,
                            cu_q: torch.Tensor | None = None, left: int = -1, right: int = -1, sinks: int = 0,
                            scale: float | None = None, return_lse: bool = False, out: torch.Tensor | None = None,
                            workspace=None):
    """paged_window_attention of sequences whose keys begin with a common prefix
    (tr_sparseconv_shared_prefix_attention): prefix_len keys in the pool's pages
    prefix_pages (int32 vector), which are read once for the batch. A sequence's
    keys are the prefix's, then its own k_len[b]; positions, window and sinks count
    over both, query i standing at p = i + prefix_len + k_len - Lq."""
    if not 0 <= prefix_len <= 1 << 30:
        raise ValueError(f"prefix_len = {prefix_len} out of [0, 2^30]")
    at = _ints(prefix_pages, "prefix_pages", -1, q.device if isinstance(q, torch.Tensor) else None)
    if at is None:
        raise ValueError("prefix_pages must be given")
    if isinstance(k_pages, torch.Tensor) and k_pages.dim() == 4 and prefix_pages.shape[0] * k_pages.shape[1] < prefix_len:
        raise ValueError(f"{prefix_pages.shape[0]} pages of {k_pages.shape[1]} do not hold a prefix of {prefix_len}")
    return _attend(q, k_pages, v_pages, page_table, k_len, (at if prefix_len else None, int(prefix_len)), cu_q, left, right,
                   sinks, scale, return_lse, out, workspace)
