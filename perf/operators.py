"""Cases of the sparse transformer operators: per-head query/key norm with
position rotation (qk_norm_rope, qk_norm_rope_backward) and windowed attention
with sinks (window_attention, window_attention_backward).

The tokens are the voxels of one or more objects, object after object, or the
tokens of a sequence with its key-value cache. `run` computes each operator with
elementary torch operations (own = False) or with the package's kernels
(own = True); `exact` computes it from the definition in float64.

    qk_norm_rope: for every token t and head h, xn = x / sqrt(mean(x^2) + eps) * gain[h],
    then each pair of elements is rotated by the angle pos[t, axis of the pair] * freq[pair].

    window_attention: row i of a sequence with Lq queries and Lk keys stands at
    p = i + Lk - Lq and sees key j when j <= p + right and (j >= p - left or
    j < sinks); out = softmax(scale q k^T) v over the keys it sees, 0 if it sees none.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _ints(text):
    return [int(t) for t in str(text).split(",")]


def listed():
    return [
        # One new token of 32 sequences: the smallest call, latency only.
        dict(name="rotate, a token of 32", kind="rotate", tokens=32, q_heads=16, kv_heads=4, dim=128, axes=1,
             span=131072, interleaved=False, shared=True, dtype="bf16"),
        # Four 64^3 objects at the width of the 1024-channel workload: the streaming case.
        dict(name="rotate, four objects", kind="rotate", tokens=73881, q_heads=16, kv_heads=16, dim=64, axes=3,
             span=64, interleaved=True, shared=False, dtype="bf16"),
        # fp32 features of one 64^3 object, an odd head size.
        dict(name="rotate, fp32 dim 72", kind="rotate", tokens=16219, q_heads=12, kv_heads=4, dim=72, axes=3,
             span=256, interleaved=False, shared=False, dtype="f32"),
        # Training step of the norm and rotation at the latent flow's longest set, 12 heads of 128.
        dict(name="rotate gradient", kind="rotate_grad", tokens=15800, q_heads=12, kv_heads=12, dim=128, axes=3,
             span=64, interleaved=True, shared=False, dtype="bf16"),
        # The 16^3 sphere shell: a small call, latency counts.
        dict(name="attend, small shell", kind="attend", lens="450", q_heads=8, kv_heads=8, dim=64, left=64, right=64,
             sinks=4, dtype="bf16"),
        # Four objects in one packed call, 16 heads of 64, a window along the voxel order on both sides.
        dict(name="attend, four objects", kind="attend", lens="16219,22483,19872,15307", q_heads=16, kv_heads=16,
             dim=64, left=512, right=512, sinks=8, dtype="bf16"),
        # Prompt of an autoregressive model over voxel tokens: causal, shared key-value heads.
        dict(name="attend, long prompt", kind="attend", lens="32768", q_heads=16, kv_heads=4, dim=128, left=4095,
             right=0, sinks=4, dtype="bf16"),
        # fp32, odd lengths down to one token, odd head size.
        dict(name="attend, fp32 odd", kind="attend", lens="2047,1,733,96", q_heads=6, kv_heads=2, dim=80, left=255,
             right=255, sinks=3, dtype="f32"),
        # Training step, forward and gradients: the latent flow's longest set, 12 heads of 128.
        dict(name="attend gradient", kind="attend_grad", lens="15800", q_heads=12, kv_heads=12, dim=128, left=512,
             right=512, sinks=8, dtype="bf16"),
        # Training step, causal, shared key-value heads, ragged.
        dict(name="attend gradient, shared heads", kind="attend_grad", lens="4099,517", q_heads=16, kv_heads=4, dim=64,
             left=1023, right=0, sinks=4, dtype="f16"),
        # One new token of 32 sequences against their caches.
        dict(name="token, 32 caches", kind="token", slots=8192, batch=32, q_heads=16, kv_heads=4, dim=128, left=4095,
             sinks=4, dtype="bf16"),
        # One new token of one sequence against a long cache: few rows, one long axis.
        dict(name="token, one long cache", kind="token", slots=131072, batch=1, q_heads=16, kv_heads=4, dim=128,
             left=65535, sinks=4, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 4e12, w["flops"] / 5e14)


def draw(rng):
    kind = rng.choice(["rotate", "rotate_grad", "attend", "attend_grad", "token"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    dim = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4]) if kv < 8 else 1
    case = dict(kind=kind, q_heads=kv * group, kv_heads=kv, dim=dim, dtype=dtype)
    if kind in ("rotate", "rotate_grad"):
        axes = 3 if dtype == "f32" else rng.choice([1, 3])
        case.update(tokens=_log(rng, 1, 60000 if kind == "rotate" else 16000), axes=axes,
                    span=rng.choice([16, 64, 256]) if axes == 3 else _log(rng, 64, 131072),
                    interleaved=rng.random() < 0.5, shared=rng.random() < 0.5)
    elif kind == "token":
        case.update(batch=_log(rng, 1, 64), slots=_log(rng, 16, 16384), left=_log(rng, 16, 8192),
                    sinks=rng.choice([0, 1, 4, 17]))
    else:
        top = (16000 if dtype != "f32" else 3000) // (1 if kind == "attend" else 2)
        # one sequence at least has more than a few keys: with one key the gradient of q is zero
        lens = [_log(rng, 32, top)] + [_log(rng, 1, top) for _ in range(rng.choice([0, 0, 1, 2, 4]))]
        left = _log(rng, 16, 2048)
        case.update(lens=",".join(map(str, lens)), left=left, right=rng.choice([0, left]),
                    sinks=rng.choice([0, 1, 4, 17]))
    most = max(_cost(c) for c in listed() if c["kind"] == kind)
    while _cost(case) > most:
        if "tokens" in case:
            case["tokens"] = max(1, case["tokens"] * 2 // 3)
        elif kind == "token":
            case["batch"] = max(1, case["batch"] * 2 // 3)
        else:
            n, *more = _ints(case["lens"])
            case["lens"] = ",".join(map(str, [max(32, n * 2 // 3)] + [max(1, m * 2 // 3) for m in more]))
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _token_lens(case):
    """Tokens in each cache: between half a window and the whole cache, seeded by the sizes alone."""
    r = np.random.default_rng(case["batch"] * 1000003 + case["slots"])
    hi = case["slots"]
    lo = max(1, hi - hi // 4) if case["batch"] == 1 else max(1, min(hi, case["left"] // 2))
    return r.integers(lo, hi + 1, size=case["batch"]).tolist()


def _sections(case):
    """Pairs rotated by each axis; with three axes the pairs left over stay as they are."""
    return [case["dim"] // 2 // case["axes"]] * case["axes"]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    dt = _TYPES[case["dtype"]]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    s = dict(case=case, kind=case["kind"], hq=hq, hk=hk, d=d, dtype=dt)
    if case["kind"].startswith("rotate"):
        t = case["tokens"]
        qkv = normal(t, hq + 2 * hk, d, scale=1.7)  # one projection's rows: queries, keys, values
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        if case["axes"] == 1:
            s["pos"] = torch.randint(0, case["span"], (t, 1), generator=g, device=dev, dtype=torch.int32)
        else:
            coords = torch.randint(0, case["span"], (t, 4), generator=g, device=dev, dtype=torch.int32)
            s["pos"] = coords[:, 1:]  # the voxels' own rows (b, x, y, z)
        sec = _sections(case)
        f = [10000.0 ** (-i / n) for n in sec for i in range(n)]
        s["freqs"] = torch.tensor(f + [0.0] * (d // 2 - len(f)), dtype=torch.float32, device=dev)
        s["sections"] = sec
        axis = [a for a, n in enumerate(sec) for _ in range(n)] + [0] * (d // 2 - sum(sec))
        s["axis"] = torch.tensor(axis, device=dev)
        shape = (d,) if case["shared"] else None
        s["q_gain"] = 1 + 0.2 * torch.randn(shape or (hq, d), generator=g, device=dev)
        s["k_gain"] = 1 + 0.2 * torch.randn(shape or (hk, d), generator=g, device=dev)
        if case["kind"] == "rotate_grad":
            s["dq"], s["dk"] = normal(t, hq, d), normal(t, hk, d)
        return s
    if case["kind"] == "token":
        lens_q, lens_k = [1] * case["batch"], _token_lens(case)
        rows_k, starts = case["batch"] * case["slots"], [b * case["slots"] for b in range(case["batch"] + 1)]
        s["right"] = 0
        s["q"] = normal(case["batch"], hq, d, scale=1.3)
        s["k"], s["v"] = normal(rows_k, hk, d, scale=1.3), normal(rows_k, hk, d)
        s["k_len"] = torch.tensor(lens_k, dtype=torch.int32, device=dev)
    else:
        lens_q = lens_k = _ints(case["lens"])
        starts = np.concatenate([[0], np.cumsum(lens_k)]).tolist()
        s["right"] = case["right"]
        t = starts[-1]
        qk = normal(t, hq + hk, d, scale=1.3)  # rotated queries and keys side by side
        s["q"], s["k"] = qk[:, :hq], qk[:, hq:]
        s["v"] = normal(t, hq + 2 * hk, d)[:, hq + hk:]  # values inside a projection's rows
        s["k_len"] = None
    s["left"], s["sinks"] = case["left"], case["sinks"]
    s["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(lens_q)]).tolist(), dtype=torch.int32, device=dev)
    s["cu_k"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["lens_q"], s["lens_k"] = lens_q, lens_k
    if case["kind"] == "attend_grad":
        s["dout"] = normal(t, hq, d)
    return s


# ---------------------------------------------------------------------------
# The operators in their plain form (32 bits, rounded once at the end)
# ---------------------------------------------------------------------------
def _angles(s):
    a = s["pos"].float()[:, s["axis"]] * s["freqs"]  # [T, d / 2]
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def _split(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)


def _join(a, b, interleaved):
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _rotate_plain(s):
    c, n = _angles(s)
    il = s["case"]["interleaved"]
    out = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
        a, b = _split(y, il)
        out.append(_join(a * c - b * n, a * n + b * c, il).to(s["dtype"]))
    return out


def _rotate_grad_plain(s):
    c, n = _angles(s)
    il = s["case"]["interleaved"]
    dx, dg = [], []
    for x, gain, dy in ((s["q"], s["q_gain"], s["dq"]), (s["k"], s["k_gain"], s["dk"])):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        a, b = _split(dy.float(), il)
        dz = _join(a * c + b * n, b * c - a * n, il)
        xn = x * r
        w = dz * gain
        dx.append((r * (w - xn * (w * xn).mean(-1, keepdim=True))).to(s["dtype"]))
        dg.append((dz * xn).sum((0, 1) if gain.dim() == 1 else 0))
    return dx + dg


def _window(s):
    """Blocks of rows, each with the columns (sinks, then the band) that its rows can see."""
    dev = s["q"].device
    lq, lk = s["lens_q"], s["lens_k"]
    bs = min(256, max(lq))
    n_q = s["cu_q"][1:] - s["cu_q"][:-1]
    n_k = s["k_len"] if s["k_len"] is not None else s["cu_k"][1:] - s["cu_k"][:-1]
    total = sum(-(-n // bs) for n in lq)
    blocks = (n_q + bs - 1) // bs
    seq = torch.repeat_interleave(torch.arange(len(lq), device=dev), blocks, output_size=total)
    first = (torch.arange(total, device=dev) - (torch.cumsum(blocks, 0) - blocks)[seq]) * bs
    i = first[:, None] + torch.arange(bs, device=dev)  # [blocks, bs] row in its sequence
    p = i + (n_k - n_q)[seq][:, None]
    band = min(max(lk), bs + s["left"] + s["right"])
    start = (p[:, 0] - s["left"]).clamp_min(0)
    sinks = torch.arange(min(s["sinks"], max(lk)), device=dev).expand(total, -1)
    j = torch.cat([sinks, start[:, None] + torch.arange(band, device=dev)], 1)
    twice = torch.cat([sinks >= start[:, None], torch.zeros(total, band, dtype=torch.bool, device=dev)], 1)
    j3, p3 = j[:, None], p[:, :, None]
    sees = (j3 <= p3 + s["right"]) & ((j3 >= p3 - s["left"]) | (j3 < s["sinks"]))
    sees &= ((j < n_k[seq][:, None]) & ~twice)[:, None] & (i < n_q[seq][:, None])[:, :, None]
    rows = torch.where(i < n_q[seq][:, None], s["cu_q"][:-1][seq][:, None] + i, s["q"].shape[0])
    cols = (s["cu_k"][:-1][seq][:, None] + j).clamp(0, s["k"].shape[0] - 1)
    return rows, cols, sees


def _take_rows(s, x, rows):
    """[blocks * kv heads, group * bs, d] in 32 bits."""
    nb, bs = rows.shape
    x = x[rows.clamp_max(x.shape[0] - 1)].float()
    return x.view(nb, bs, s["hk"], s["hq"] // s["hk"], s["d"]).permute(0, 2, 3, 1, 4).reshape(nb * s["hk"], -1, s["d"])


def _put_rows(s, x, rows):
    nb, bs = rows.shape
    out = torch.zeros(s["q"].shape[0] + 1, s["hq"], s["d"], device=x.device)
    out[rows] = x.view(nb, s["hk"], s["hq"] // s["hk"], bs, s["d"]).permute(0, 3, 1, 2, 4).reshape(nb, bs, s["hq"], -1)
    return out[:-1].to(s["dtype"])


def _take_cols(s, x, cols):
    return x[cols].float().permute(0, 2, 1, 3).reshape(-1, cols.shape[1], s["d"])


def _attend_plain(s):
    rows, cols, sees = _window(s)
    nb, bs = rows.shape
    scale = s["d"] ** -0.5
    q, k, v = _take_rows(s, s["q"], rows), _take_cols(s, s["k"], cols), _take_cols(s, s["v"], cols)
    z = torch.bmm(q, k.transpose(1, 2)).view(nb, s["hk"], -1, bs, cols.shape[1]) * scale
    z = z.masked_fill(~sees[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    e = (e / e.sum(-1, keepdim=True).clamp_min(1e-30)).view(q.shape[0], q.shape[1], -1)
    o = torch.bmm(e, v)
    out = _put_rows(s, o, rows)
    if s["kind"] != "attend_grad":
        return out
    do = _take_rows(s, s["dout"], rows)
    ds = e * (torch.bmm(do, v.transpose(1, 2)) - (do * o).sum(-1, keepdim=True)) * scale
    dq = _put_rows(s, torch.bmm(ds, k), rows)
    back = []
    for a, b in ((ds, q), (e, do)):
        x = torch.bmm(a.transpose(1, 2), b).view(nb, s["hk"], -1, s["d"]).permute(0, 2, 1, 3)
        to = torch.zeros(s["k"].shape[0], s["hk"], s["d"], device=x.device)
        back.append(to.index_add_(0, cols.reshape(-1), x.reshape(-1, s["hk"], s["d"])).to(s["dtype"]))
    return [out, dq] + back


# ---------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        plain = dict(rotate=_rotate_plain, rotate_grad=_rotate_grad_plain, attend=_attend_plain,
                     attend_grad=_attend_plain, token=_attend_plain)
        return plain[s["kind"]](s)
    import submanifold_sparse_conv_amd as sc

    if s["kind"].startswith("rotate"):
        how = dict(q_gain=s["q_gain"], k_gain=s["k_gain"], sections=s["sections"],
                   interleaved=s["case"]["interleaved"], eps=EPS)
        if s["kind"] == "rotate":
            return list(sc.qk_norm_rope(s["q"], s["k"], s["pos"], s["freqs"], **how))
        return list(sc.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freqs"], **how))
    how = dict(cu_q=s["cu_q"], cu_k=s["cu_k"], k_len=s["k_len"], left=s["left"], right=s["right"], sinks=s["sinks"])
    if s["kind"] != "attend_grad":
        return sc.window_attention(s["q"], s["k"], s["v"], **how)
    out, lse = sc.window_attention(s["q"], s["k"], s["v"], return_lse=True, **how)
    return [out, *sc.window_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)]


def _pairs(case):
    """(row, key) pairs that the rows of one head see."""
    if case["kind"] == "token":
        lens, right, first = _token_lens(case), 0, [n - 1 for n in _token_lens(case)]
    else:
        lens, right = _ints(case["lens"]), case["right"]
        first = [0] * len(lens)
    n = 0
    for lk, p0 in zip(lens, first):
        p = np.arange(p0, lk, dtype=np.int64)
        lo, hi = np.maximum(0, p - case["left"]), np.minimum(lk, p + right + 1)
        n += int((np.maximum(0, hi - lo) + np.minimum(np.minimum(case["sinks"], hi), lo)).sum())
    return n


def work(case):
    e = torch.empty(0, dtype=_TYPES[case["dtype"]]).element_size()
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["kind"].startswith("rotate"):
        t, grad = case["tokens"], case["kind"] == "rotate_grad"
        values = t * (hq + hk) * d
        gains = (2 * d if case["shared"] else (hq + hk) * d) * 4
        return {"bytes": values * e * (3 if grad else 2) + t * case["axes"] * 4 + gains * (2 if grad else 1),
                "flops": values * (16 if grad else 8)}
    pairs = _pairs(case)
    if case["kind"] == "token":
        lens = _token_lens(case)
        keys = sum(min(n, case["left"] + 1 + case["sinks"]) for n in lens)
        return {"bytes": (2 * keys * hk * d + 2 * len(lens) * hq * d) * e, "flops": 4 * pairs * hq * d}
    t = sum(_ints(case["lens"]))
    if case["kind"] == "attend":
        return {"bytes": (2 * hq + 2 * hk) * t * d * e, "flops": 4 * pairs * hq * d}
    return {"bytes": (4 * hq + 4 * hk) * t * d * e, "flops": 14 * pairs * hq * d}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotate(s):
    """Each pair as a complex number times exp(i angle)."""
    d, il = s["d"], s["case"]["interleaved"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["pos"].double()[:, s["axis"]] * s["freqs"].double())[:, None]
    pair = torch.arange(d, device=s["q"].device)
    even, odd = (pair[0::2], pair[1::2]) if il else (pair[:d // 2], pair[d // 2:])
    outs, grads, gains = [], [], []
    for x, gain, dy in ((s["q"], s["q_gain"], s.get("dq")), (s["k"], s["k_gain"], s.get("dk"))):
        x, gain = x.double(), gain.double()
        norm = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        if dy is None:
            y = x / norm * gain
            z = torch.complex(y[..., even], y[..., odd]) * turn
            out = torch.empty_like(y)
            out[..., even], out[..., odd] = z.real, z.imag
            outs.append(out)
            continue
        dy = dy.double()
        z = torch.complex(dy[..., even], dy[..., odd]) * turn.conj()
        back = torch.empty_like(x)
        back[..., even], back[..., odd] = z.real, z.imag
        grads.append(gain * back / norm - x * (gain * back * x).sum(-1, keepdim=True) / (d * norm.pow(3)))
        w = back * x / norm
        gains.append(w.sum(0).sum(0) if gain.dim() == 1 else w.sum(0))
    return outs or grads + gains


def _exact_attend(s):
    q, k, v = s["q"], s["k"], s["v"]
    dev, d, group = q.device, s["d"], s["hq"] // s["hk"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    grad = s["kind"] == "attend_grad"
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=dev) for x in ((q, k, v) if grad else (q[:0],) * 3))
    q0 = 0
    for lq, lk, k0 in zip(s["lens_q"], s["lens_k"], s["cu_k"].tolist()):
        for r in range(0, lq, 2048):
            n = min(2048, lq - r)
            p = torch.arange(r, r + n, device=dev) + (lk - lq)
            lo, hi = max(0, r + lk - lq - s["left"]), min(lk, r + n + lk - lq + s["right"])
            j = torch.cat([torch.arange(0, min(s["sinks"], lo, max(hi, 0)), device=dev),
                           torch.arange(lo, max(lo, hi), device=dev)])
            hidden = (j > p[:, None] + s["right"]) | ((j < p[:, None] - s["left"]) & (j >= s["sinks"]))
            for h in range(s["hq"]):
                a, c = q[q0 + r:q0 + r + n, h].double(), k[k0 + j, h // group].double()
                u = v[k0 + j, h // group].double()
                w = torch.softmax((a @ c.T / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
                w = torch.where(hidden, torch.zeros_like(w), w)
                out[q0 + r:q0 + r + n, h] = w @ u
                if grad:
                    t = s["dout"][q0 + r:q0 + r + n, h].double()
                    x = t @ u.T
                    x = w * (x - (w * x).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[q0 + r:q0 + r + n, h] = x @ c
                    dk[k0 + j, h // group] += x.T @ a
                    dv[k0 + j, h // group] += w.T @ t
        q0 += lq
    return [out, dq, dk, dv] if grad else out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rotate(s) if case["kind"].startswith("rotate") else _exact_attend(s)
