"""Cases of the operators that serve voxel token models from a paged key-value
cache: norm and rotation with the append of keys and values to the pages
(qk_norm_rope_append), attention over the pages (paged_window_attention), and
attention of a batch whose sequences share a prefix (shared_prefix_attention).

`run` computes each operator with elementary torch operations (own = False) or
with the package's kernels (own = True); `exact` computes it from the definition
in float64.

    Pages: key j of sequence b is k_pages[table[b, j // page], j % page], of
    [kv heads, dim]; the sequence has k_len[b] keys, the new tokens' included.

    qk_norm_rope_append: token i of the Lq new ones of sequence b is its key
    j = k_len[b] - Lq + i. Queries and keys are normed (xn = x / sqrt(mean(x^2) + eps)
    * gain, or left as they are), each pair of elements turned by pos * freq; the
    queries are returned, the keys and the unchanged values go to their place.

    paged_window_attention: query i of Lq stands at p = i + Lk - Lq and sees key j
    when j <= p + right and (j >= p - left or j < sinks), right = 0 here; out =
    softmax(scale q k^T) v over the keys it sees, 0 if it sees none.

    shared_prefix_attention: the same with Lk = prefix_len + k_len[b], the first
    prefix_len keys the batch's common ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # One new token of each of 32 sequences: latency only.
        dict(name="append, a token of 32", kind="append", batch=32, tokens="1", slots=8192, page=16, q_heads=16,
             kv_heads=4, dim=128, axes=1, span=131072, interleaved=False, shared=True, norm=True, dtype="bf16"),
        # The prompts of four 64^3 objects into empty caches, positions from the voxels: the streaming case.
        dict(name="append, four objects", kind="append", batch=4, tokens="16219,22483,19872,15307", slots=0, page=64,
             q_heads=16, kv_heads=16, dim=64, axes=3, span=64, interleaved=True, shared=False, norm=True,
             dtype="bf16"),
        # Odd lengths behind what is there, rotation alone, an odd head size, fp32.
        dict(name="append, fp32 dim 72", kind="append", batch=4, tokens="2047,1,733,96", slots=512, page=8, q_heads=12,
             kv_heads=4, dim=72, axes=3, span=256, interleaved=False, shared=False, norm=False, dtype="f32"),
        # A step of a few short sequences: a small call, latency counts.
        dict(name="paged, 8 short caches", kind="paged", batch=8, tokens="1", slots=450, page=16, q_heads=8,
             kv_heads=8, dim=64, left=-1, sinks=0, dtype="bf16"),
        # One new token of 32 sequences of unlike lengths, a window over each.
        dict(name="paged, 32 caches", kind="paged", batch=32, tokens="1", slots=8192, page=16, q_heads=16, kv_heads=4,
             dim=128, left=4095, sinks=4, dtype="bf16"),
        # One new token of one sequence against all of a long cache: few rows, one long axis.
        dict(name="paged, one long cache", kind="paged", batch=1, tokens="1", slots=131072, page=64, q_heads=16,
             kv_heads=4, dim=128, left=-1, sinks=0, dtype="f16"),
        # Parts of four prompts against what the caches hold already: the matrix units' case.
        dict(name="paged, prompt parts", kind="paged", batch=4, tokens="512,300,512,77", slots=8192, page=64,
             q_heads=16, kv_heads=4, dim=128, left=-1, sinks=0, dtype="bf16"),
        # Five drafted tokens of six sequences, fp32, an odd head size, a short window and the smallest pages.
        dict(name="paged, fp32 drafts", kind="paged", batch=6, tokens="5", slots=2047, page=8, q_heads=6, kv_heads=2,
             dim=80, left=255, sinks=3, dtype="f32"),
        # Four samples of one image: its 1369 tokens are the prefix; a small call.
        dict(name="prefix, four samples", kind="prefix", batch=4, tokens="1", slots=450, page=16, prefix=1369,
             q_heads=16, kv_heads=16, dim=64, left=-1, sinks=0, dtype="f16"),
        # 32 continuations of one object.
        dict(name="prefix, 32 continuations", kind="prefix", batch=32, tokens="1", slots=1024, page=64, prefix=16219,
             q_heads=16, kv_heads=4, dim=128, left=-1, sinks=0, dtype="bf16"),
        # A large batch behind one long prompt.
        dict(name="prefix, 256 sequences", kind="prefix", batch=256, tokens="1", slots=512, page=16, prefix=8192,
             q_heads=16, kv_heads=4, dim=128, left=-1, sinks=0, dtype="bf16"),
        # Drafted tokens, fp32, odd sizes, a window that ends inside the prefix and its first tokens as sinks.
        dict(name="prefix, fp32 window", kind="prefix", batch=7, tokens="3", slots=96, page=8, prefix=733, q_heads=6,
             kv_heads=2, dim=80, left=255, sinks=4, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 4e12, w["flops"] / (5e14 if case["dtype"] != "f32" else 5e13))


def draw(rng):
    kind = rng.choice(["append", "paged", "paged", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    kv = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 2, 3, 4, 8]) if kv < 8 else 1
    case = dict(kind=kind, q_heads=kv * group, kv_heads=kv, dim=rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128]),
                page=rng.choice([8, 16, 16, 32, 64, 128]), dtype=dtype)
    if kind == "append":
        case["batch"] = _log(rng, 1, 256)
        if rng.random() < 0.5:
            case["tokens"] = str(rng.choice([1, 1, 2, 5]))
        else:
            case["batch"] = min(case["batch"], 8)
            case["tokens"] = ",".join(str(_log(rng, 1, 16000)) for _ in range(case["batch"]))
        case["axes"] = rng.choice([1, 3])
        case.update(slots=rng.choice([0, _log(rng, 16, 8192)]),
                    span=rng.choice([16, 64, 256]) if case["axes"] == 3 else _log(rng, 64, 131072),
                    interleaved=rng.random() < 0.5, shared=rng.random() < 0.5, norm=rng.random() < 0.75)
    else:
        left = rng.choice([-1, -1, _log(rng, 16, 8192)])
        case.update(batch=_log(rng, 1, 256), left=left, sinks=0 if left < 0 else rng.choice([0, 1, 4, 17]),
                    slots=_log(rng, 16, 16384 if kind == "paged" else 2048))
        case["tokens"] = str(rng.choice([1, 1, 1, 2, 3, 5]))
        if kind == "prefix":
            case["prefix"] = _log(rng, 16, 16384)
        elif rng.random() < 0.4:
            case["batch"] = min(case["batch"], 6)
            case["slots"] = max(64, case["slots"])
            case["tokens"] = ",".join(str(_log(rng, 1, min(600, case["slots"] // 2))) for _ in range(case["batch"]))
    # no dearer than the dearest listed one, its memory in the plain form included
    most = max(_cost(c) for c in listed() if c["kind"] == kind)
    while _cost(case) > most or _cells(case) > 1 << 28:
        if kind != "append" and case["slots"] > 4096:
            case["slots"] = case["slots"] * 2 // 3
        elif case["batch"] > 1:
            case["batch"] = max(1, case["batch"] * 2 // 3)
            if "," in case["tokens"]:
                case["tokens"] = ",".join(case["tokens"].split(",")[:case["batch"]])
        elif kind == "prefix" and case["prefix"] > 64:
            case["prefix"] = case["prefix"] * 2 // 3
        else:
            case["tokens"] = str(max(1, _lens(case)[0][0] * 2 // 3))
    return case


def _lens(case):
    """New tokens and keys (the new ones included, a prefix not) of each sequence, from the sizes alone."""
    r = np.random.default_rng(case["batch"] * 1000003 + case["slots"])
    new = [int(t) for t in case["tokens"].split(",")]
    new = new * case["batch"] if len(new) == 1 else new
    if case["kind"] == "append":  # behind up to `slots` keys
        return new, [n + int(r.integers(0, case["slots"] + 1)) for n in new]
    lo = case["slots"] - case["slots"] // 4 if case["batch"] == 1 else max(1, case["slots"] // 4)
    return new, [max(n, int(r.integers(lo, case["slots"] + 1))) for n in new]


def _cells(case):
    """Scores that the plain form holds at once."""
    if case["kind"] == "append":
        return 0
    new, keys = _lens(case)
    return case["batch"] * case["q_heads"] * max(new) * (max(keys) + case.get("prefix", 0))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    dt = _TYPES[case["dtype"]]
    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    new, keys = _lens(case)
    t, pre = sum(new), case.get("prefix", 0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    # a pool with room, pages in no order; a table as wide as the longest sequence, -1 past a sequence's pages
    need = [-(-n // page) for n in keys]
    n_pre = -(-pre // page)
    pages = sum(need) + n_pre + 8
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((case["batch"], max(need) + 1), -1, dtype=torch.int32, device=dev)
    at = n_pre
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case=case, kind=case["kind"], hq=hq, hk=hk, d=d, page=page, dtype=dt, new=new, keys=keys, table=table,
             k_len=ints(keys), cu_q=ints(np.concatenate([[0], np.cumsum(new)]).tolist()), cu_arg=None)
    if min(new) != max(new):
        s["cu_arg"] = s["cu_q"]  # sequences of like counts need no offsets
    if case["kind"] == "append":
        qkv = normal(t, hq + 2 * hk, d, scale=1.7)  # one projection's rows: queries, keys, values
        s["q"], s["k"], s["v"] = qkv.split([hq, hk, hk], 1)
        s["k_pages"], s["v_pages"] = normal(pages, page, hk, d), normal(pages, page, hk, d)
        if case["axes"] == 1:
            s["pos"] = torch.randint(0, case["span"], (t, 1), generator=g, device=dev, dtype=torch.int32)
        else:
            coords = torch.randint(0, case["span"], (t, 4), generator=g, device=dev, dtype=torch.int32)
            s["pos"] = coords[:, 1:]  # the voxels' own rows (b, x, y, z)
        sec = [d // 2 // case["axes"]] * case["axes"]
        f = [10000.0 ** (-i / n) for n in sec for i in range(n)]
        s["freqs"] = torch.tensor(f + [0.0] * (d // 2 - len(f)), dtype=torch.float32, device=dev)
        s["axis"] = torch.tensor([a for a, n in enumerate(sec) for _ in range(n)] + [0] * (d // 2 - sum(sec)), device=dev)
        s["q_gain"] = s["k_gain"] = None
        if case["norm"]:
            s["q_gain"] = 1 + 0.2 * torch.randn((d,) if case["shared"] else (hq, d), generator=g, device=dev)
            s["k_gain"] = 1 + 0.2 * torch.randn((d,) if case["shared"] else (hk, d), generator=g, device=dev)
        return s
    s["q"] = normal(t, hq, d, scale=1.3)
    pool = normal(pages, page, 2 * hk, d)  # keys and values of a token side by side
    s["k_pages"], s["v_pages"] = pool.split([hk, hk], 2)
    s["left"], s["sinks"], s["prefix"] = case["left"], case["sinks"], pre
    s["prefix_pages"] = order[:n_pre].contiguous()
    return s


# ---------------------------------------------------------------------------
# The operators in their plain form (32 bits, rounded once at the end)
# ---------------------------------------------------------------------------
def _split(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)


def _append_plain(s):
    dev, il = s["q"].device, s["case"]["interleaved"]
    angle = s["pos"].double()[:, s["axis"]] * s["freqs"].double()
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        y = x.float()
        if s["case"]["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain
        a, b = _split(y, il)
        y = [a * c - b * n, a * n + b * c]
        out.append((torch.stack(y, -1).flatten(-2) if il else torch.cat(y, -1)).to(s["dtype"]))
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    t = s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), new, output_size=t)
    j = torch.arange(t, device=dev) - s["cu_q"][seq] + (s["k_len"] - new)[seq]
    at = s["table"][seq, j // s["page"]].long(), j % s["page"]
    s["k_pages"][at] = out[1]
    s["v_pages"][at] = s["v"]
    return [out[0], s["k_pages"], s["v_pages"]]


def _part(q, k, v, sees, scale):
    """Largest score, sum of exponentials and weighted sum of values: q [n, rows, d], k, v [n, cols, d]."""
    z = (torch.bmm(q, k.transpose(1, 2)) * scale).masked_fill(~sees, -math.inf)
    m = z.amax(-1, keepdim=True) if z.shape[-1] else z.new_full((*z.shape[:2], 1), -math.inf)
    e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, e.sum(-1, keepdim=True), torch.bmm(e, v)


def _attend_plain(s):
    dev, d, hk, group = s["q"].device, s["d"], s["hk"], s["hq"] // s["hk"]
    batch, lq, pre = len(s["new"]), max(s["new"]), s["prefix"]
    left = s["left"] if s["left"] >= 0 else 1 << 40
    n_q, n_k = s["cu_q"][1:] - s["cu_q"][:-1], s["k_len"]
    i = torch.arange(lq, device=dev)
    rows = torch.where(i < n_q[:, None], s["cu_q"][:-1, None] + i, s["q"].shape[0])  # [batch, lq]
    p = i + (n_k - n_q)[:, None]  # position among the sequence's own keys
    x = s["q"][rows.clamp_max(s["q"].shape[0] - 1)].float().view(batch, lq, hk, group, d)
    scale = d ** -0.5
    # own keys: the window's, and the sinks before them
    own_sinks = max(0, min(s["sinks"], max(s["keys"]) + pre) - pre)
    band = min(max(s["keys"]), lq + left)
    start = (p[:, 0] - left).clamp_min(0)
    sink = torch.arange(own_sinks, device=dev).expand(batch, -1)
    j = torch.cat([sink, start[:, None] + torch.arange(band, device=dev)], 1)  # [batch, cols]
    once = torch.cat([sink < start[:, None], torch.ones(batch, band, dtype=torch.bool, device=dev)], 1)
    j3, p3 = j[:, None], p[:, :, None]
    sees = (j3 <= p3) & ((j3 >= p3 - left) | (j3 < own_sinks)) & (once & (j < n_k[:, None]))[:, None]
    jc = torch.minimum(j, n_k[:, None] - 1).clamp_min(0)
    page = torch.gather(s["table"].long(), 1, jc // s["page"]).clamp_min(0)
    k, v = (t[page, jc % s["page"]].float().permute(0, 2, 1, 3).reshape(batch * hk, -1, d)
            for t in (s["k_pages"], s["v_pages"]))
    q = x.permute(0, 2, 3, 1, 4).reshape(batch * hk, group * lq, d)
    m, l, o = _part(q, k, v, sees.repeat_interleave(hk, 0).repeat(1, group, 1), scale)
    if pre:
        # the prefix: one product for the batch
        j = torch.arange(pre, device=dev)
        page = s["prefix_pages"].long()[j // s["page"]]
        k, v = (t[page, j % s["page"]].float().permute(1, 0, 2).contiguous() for t in (s["k_pages"], s["v_pages"]))
        sees = (j <= p3 + pre) & ((j >= p3 + pre - left) | (j < s["sinks"]))
        sees = sees[:, None].expand(-1, group, -1, -1).reshape(1, -1, pre)
        q = x.permute(2, 0, 3, 1, 4).reshape(hk, -1, d)
        m2, l2, o2 = (y.view(hk, batch, group * lq, -1).transpose(0, 1).reshape(batch * hk, group * lq, -1)
                      for y in _part(q, k, v, sees, scale))
        top = torch.maximum(m, m2)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        a, b = torch.exp(m - top), torch.exp(m2 - top)
        l, o = l * a + l2 * b, o * a + o2 * b
    o = (o / l.clamp_min(1e-30)).view(batch, hk, group, lq, d).permute(0, 3, 1, 2, 4).reshape(batch, lq, s["hq"], d)
    out = torch.zeros(s["q"].shape[0] + 1, s["hq"], d, device=dev)
    out[rows] = o
    return out[:-1].to(s["dtype"])


# ---------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return _append_plain(s) if s["kind"] == "append" else _attend_plain(s)
    import submanifold_sparse_conv_amd as sc

    if s["kind"] == "append":
        q = sc.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freqs"], s["k_pages"], s["v_pages"],
                                   s["table"], s["k_len"], cu_q=s["cu_arg"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                                   interleaved=s["case"]["interleaved"], eps=EPS, norm=s["case"]["norm"])
        return [q, s["k_pages"], s["v_pages"]]
    how = dict(cu_q=s["cu_arg"], left=s["left"], right=0, sinks=s["sinks"])
    if s["kind"] == "paged":
        return sc.paged_window_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["k_len"], **how)
    return sc.shared_prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["k_len"], s["prefix_pages"],
                                      s["prefix"], **how)


def work(case):
    e = torch.empty(0, dtype=_TYPES[case["dtype"]]).element_size()
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    new, keys = _lens(case)
    t = sum(new)
    if case["kind"] == "append":
        gains = (2 * d if case["shared"] else (hq + hk) * d) * 4 if case["norm"] else 0
        return {"bytes": 2 * t * (hq + 2 * hk) * d * e + t * case["axes"] * 4 + gains,
                "flops": t * (hq + hk) * d * (8 if case["norm"] else 3)}
    pre = case.get("prefix", 0)
    left = case["left"] if case["left"] >= 0 else 1 << 40
    pairs, seen, first = 0, 0, pre
    for n, own_keys in zip(new, keys):
        p = np.arange(n, dtype=np.int64) + pre + own_keys - n
        lo = np.maximum(0, p - left)
        pairs += int((p + 1 - lo + np.minimum(case["sinks"], lo)).sum())
        least = max(int(lo[0]), min(case["sinks"], pre))
        first = min(first, least)
        own_sinks = max(0, case["sinks"] - pre)
        seen += min(own_keys, own_keys - max(0, least - pre) + own_sinks)
    shared = pre - first + min(case["sinks"], first)
    return {"bytes": (2 * (seen + shared) * hk * d + 2 * t * hq * d) * e, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_append(s):
    """Each pair as a complex number times exp(i angle), token by token to its place."""
    d, il = s["d"], s["case"]["interleaved"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["pos"].double()[:, s["axis"]] * s["freqs"].double())[:, None]
    pair = torch.arange(d, device=s["q"].device)
    even, odd = (pair[0::2], pair[1::2]) if il else (pair[:d // 2], pair[d // 2:])
    turned = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        y = x.double()
        if s["case"]["norm"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * gain.double()
        z = torch.complex(y[..., even], y[..., odd]) * turn
        out = torch.empty_like(y)
        out[..., even], out[..., odd] = z.real, z.imag
        turned.append(out)
    pools = [s["k_pages"].double(), s["v_pages"].double()]
    t = 0
    for b, (n, keys) in enumerate(zip(s["new"], s["keys"])):
        j = torch.arange(keys - n, keys, device=s["q"].device)
        at = s["table"][b].long()[j // s["page"]] * s["page"] + j % s["page"]
        for pool, x in zip(pools, (turned[1], s["v"].double())):
            pool.view(-1, s["hk"], d)[at] = x[t:t + n]
        t += n
    return [turned[0], *pools]


def _exact_attend(s):
    q, dev, d, group, pre = s["q"], s["q"].device, s["d"], s["hq"] // s["hk"], s["prefix"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    t = 0
    for b, (n, own_keys) in enumerate(zip(s["new"], s["keys"])):
        lk = pre + own_keys
        p = torch.arange(n, device=dev) + lk - n
        every = torch.cat([s["prefix_pages"].long().repeat_interleave(s["page"])[:pre],
                           s["table"][b].long().repeat_interleave(s["page"])[:own_keys]])
        place = torch.cat([torch.arange(pre, device=dev), torch.arange(own_keys, device=dev)]) % s["page"]
        j = torch.arange(lk, device=dev)
        hidden = j > p[:, None]
        if s["left"] >= 0:
            hidden |= (j < p[:, None] - s["left"]) & (j >= s["sinks"])
        seen = (~hidden).any(0).nonzero()[:, 0]
        k, v = (x[every[seen], place[seen]].double().permute(1, 2, 0).contiguous() for x in (s["k_pages"], s["v_pages"]))
        x = q[t:t + n].double().view(n, s["hk"], group, d).permute(1, 2, 0, 3).reshape(s["hk"], group * n, d)
        z = (x @ k / math.sqrt(d)).masked_fill(hidden[:, seen].repeat(group, 1), -math.inf)
        y = torch.softmax(z, -1) @ v.transpose(1, 2).contiguous()
        out[t:t + n] = y.view(s["hk"], group, n, d).permute(2, 0, 1, 3).reshape(n, s["hq"], d)
        t += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["kind"] == "append" else _exact_attend(s)
