"""Plain 64-bit forms of the token operators and elementwise error bounds of the
kernels' arithmetic (no test functions here).

Bounds. u is the unit roundoff of a tensor's type (2^-8 bf16, 2^-11 f16, 2^-24
fp32), e = 2^-24. A sum of n fp32 products is off by at most n e times the sum
of the products' magnitudes, whatever its order. Every bound below is the sum of
the roundings on the way to the element, each with its largest effect, so the
tolerances need no measurement.
"""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, torch.float64: 2.0 ** -53}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14, torch.float32: 2.0 ** -126,
        torch.float64: 2.0 ** -1022}  # smallest normal
E = 2.0 ** -24


def rotate_pairs(y, angle, interleaved):
    """y [T, H, D] with every pair turned by angle [T, D / 2]."""
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    out = torch.empty_like(y)
    d = y.shape[-1]
    a, b = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def swap_pairs(y, interleaved):
    out = torch.empty_like(y)
    d = y.shape[-1]
    a, b = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    out[..., a], out[..., b] = y[..., b], y[..., a]
    return out


def angles(pos, freqs, sections):
    """[T, D / 2] in float64: pair i turns with the axis its section names, the rest not."""
    pos, freqs = pos.double(), freqs.double()
    if pos.dim() == 1:
        pos = pos[:, None]
    out = torch.zeros(pos.shape[0], freqs.shape[0], dtype=torch.float64)
    at = 0
    for axis, n in enumerate(sections):
        out[:, at:at + n] = pos[:, axis:axis + 1] * freqs[at:at + n]
        at += n
    return out


def norm_rope(x, gain, angle, interleaved, eps):
    x = x.double()
    r = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    y = x * r * (1.0 if gain is None else gain.double())
    return rotate_pairs(y, angle, interleaved)


def norm_rope_bound(x, gain, angle, interleaved, eps, dtype):
    """Mean of squares: D + 2 roundings, halved by the root, plus 2 for it; the
    products and the turn 6 more; sine and cosine 4 ulp: 16 + D / 2 in all, of
    the two partners' magnitudes. Then one rounding to the type."""
    x = x.double()
    d = x.shape[-1]
    r = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    y = (x * r * (1.0 if gain is None else gain.double())).abs()
    both = y + swap_pairs(y, interleaved)
    ref = norm_rope(x, gain, angle, interleaved, eps)
    return (16 + d / 2) * E * both + U[dtype] * ref.abs() + U[dtype] * TINY[dtype]


def norm_rope_grad(x, gain, angle, interleaved, eps, dy):
    x, dy = x.double(), dy.double()
    g = torch.ones(x.shape[-1], dtype=torch.float64) if gain is None else gain.double()
    r = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    z = rotate_pairs(dy, -angle, interleaved)
    xn, w = x * r, z * g
    dx = r * (w - xn * (w * xn).mean(-1, keepdim=True))
    dg = z * xn
    return dx, (dg.sum((0, 1)) if g.dim() == 1 else dg.sum(0))


def norm_rope_grad_bounds(x, gain, angle, interleaved, eps, dy, dtype):
    """As above: 32 + 2 D roundings of the largest magnitudes that meet in an
    element; the gain's sums one more a term."""
    x, dy = x.double(), dy.double()
    d = x.shape[-1]
    g = torch.ones(d, dtype=torch.float64) if gain is None else gain.double()
    r = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    z = dy.abs() + swap_pairs(dy.abs(), interleaved)
    xn, w = (x * r).abs(), z * g.abs()
    dx, _ = norm_rope_grad(x, gain, angle, interleaved, eps, dy)
    bound = (32 + 2 * d) * E * r * (w + xn * (w * xn).mean(-1, keepdim=True))
    terms = z * xn
    n = x.shape[0] * (x.shape[1] if g.dim() == 1 else 1)
    dg = (32 + d + n) * E * (terms.sum((0, 1)) if g.dim() == 1 else terms.sum(0))
    return bound + U[dtype] * dx.abs() + U[dtype] * TINY[dtype], dg + 1e-30


def visible(lq, lk, left, right, sinks):
    """[lq, lk] bool."""
    p = torch.arange(lq)[:, None] + lk - lq
    j = torch.arange(lk)[None]
    see = torch.ones(lq, lk, dtype=torch.bool)
    if right >= 0:
        see &= j <= p + right
    if left >= 0:
        see &= (j >= p - left) | (j < sinks)
    return see


def attention(q, k, v, see, scale, dout=None):
    """One sequence and one head in float64, touching only what is seen: dict of
    out, lse and, with dout, dq, dk, dv; and the same names with "_tol" for inputs
    of dtype q.dtype."""
    dtype = q.dtype
    u, d = U[dtype], q.shape[-1]
    up = u if u > 2 * E else 0.0  # weights and score gradients are rounded to the type
    q, k, v = q.double(), k.double(), v.double()
    lq, lk = see.shape
    rows, cols = see.any(1), see.any(0)
    # what nobody sees is not touched; a row's or key's unseen partners drop out through zero weights
    kz, vz = torch.where(cols[:, None], k, 0.0), torch.where(cols[:, None], v, 0.0)
    qz = torch.where(rows[:, None], q, 0.0)
    s = (qz @ kz.T * scale).masked_fill(~see, -math.inf)
    mag = qz.abs() @ kz.abs().T * scale
    m = s.amax(1, keepdim=True) if lk else torch.zeros(lq, 1, dtype=torch.float64)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    ex = torch.exp(s - m)
    l = ex.sum(1, keepdim=True)
    p = torch.where(l > 0, ex / l.clamp_min(1e-300), torch.zeros_like(ex))
    out = p @ vz
    lse = torch.where(l > 0, m + torch.log(l.clamp_min(1e-300)), torch.full_like(l, -math.inf))[:, 0]
    # relative error of a weight: the score's (D products, the scaling), the
    # exponential's argument and value, of itself and of the sum; n terms summed
    smax = torch.where(see, s.abs(), torch.zeros_like(s)).amax() if lk and see.any() else torch.zeros(())
    amax = torch.where(see, mag, torch.zeros_like(mag)).amax() if lk and see.any() else torch.zeros(())
    ep = 2 * ((d + 2) * E * float(amax) + 6 * E * float(smax) + 8 * E) + (lk + 64) * E
    r = dict(out=out, lse=lse)
    wide = p @ vz.abs()
    r["out_tol"] = u * out.abs() + (up + ep) * 1.01 * wide + u * TINY[dtype]
    r["lse_tol"] = torch.full_like(lse, ep + 8 * E) + 4 * E * torch.where(torch.isinf(lse), 0.0, lse.abs())
    if dout is None:
        return r
    g = torch.where(rows[:, None], dout.double(), 0.0)
    dp = g @ vz.T
    delta = (p * dp).sum(1, keepdim=True)
    ds = p * (dp - delta)
    r["dq"], r["dk"], r["dv"] = scale * ds @ kz, scale * ds.T @ qz, p.T @ g
    # the kernel's delta is the sum of dout times the rounded output
    gv, gw = g.abs() @ vz.abs().T, (g.abs() * wide).sum(1, keepdim=True)
    eds = (up + ep + 2 * E) * ds.abs() + p * (1 + ep) * (
        (d + 2) * E * gv + ((d + 2) * E + u + up + ep) * gw + ep * (dp.abs() + delta.abs()))
    n = max(lq, lk) + 64
    r["dq_tol"] = u * r["dq"].abs() + 1.01 * scale * (eds + n * E * ds.abs()) @ kz.abs() + u * TINY[dtype]
    r["dk_tol"] = u * r["dk"].abs() + 1.01 * scale * (eds + n * E * ds.abs()).T @ qz.abs() + u * TINY[dtype]
    r["dv_tol"] = u * r["dv"].abs() + 1.01 * ((up + ep + n * E) * p).T @ g.abs() + u * TINY[dtype]
    return r
