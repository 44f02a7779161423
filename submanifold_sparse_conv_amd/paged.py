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
    one whose key is none of the table is not stored. q_out may be q itself. The
    table must not give two of the call's tokens the same place: it is unspecified
    what that place holds then."""
    return (_lib._binding or _lib.binding()).append(q, k, v, pos, freqs, k_pages, v_pages, page_table, k_len, cu_q, q_gain,
                                                    k_gain, sections, interleaved, eps, norm, q_out)


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
    return (_lib._binding or _lib.binding()).attend(q, k_pages, v_pages, page_table, k_len, None, 0, cu_q, left, right,
                                                    sinks, scale, return_lse, out, workspace)


def shared_prefix_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                            k_len: torch.Tensor, prefix_pages: torch.Tensor, prefix_len: int,
                            cu_q: torch.Tensor | None = None, left: int = -1, right: int = -1, sinks: int = 0,
                            scale: float | None = None, return_lse: bool = False, out: torch.Tensor | None = None,
                            workspace=None):
    """paged_window_attention of sequences whose keys begin with a common prefix
    (tr_sparseconv_shared_prefix_attention): prefix_len keys in the pool's pages
    prefix_pages (int32 vector), which are read for rows of all sequences together
    (in small calls for each sequence). A sequence's keys are the prefix's, then
    its own k_len[b]; positions, window and sinks count
    over both, query i standing at p = i + prefix_len + k_len - Lq."""
    if not 0 <= prefix_len <= 1 << 30:
        raise ValueError(f"prefix_len = {prefix_len} out of [0, 2^30]")
    if prefix_pages is None:
        raise ValueError("prefix_pages must be given")
    return (_lib._binding or _lib.binding()).attend(q, k_pages, v_pages, page_table, k_len, prefix_pages, prefix_len, cu_q,
                                                    left, right, sinks, scale, return_lse, out, workspace)
