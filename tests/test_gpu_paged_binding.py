"""Arguments that the binding of the calls over a paged cache refuses itself; none of them reaches a kernel. And two
calls at once."""
import pytest
import torch

from tests.test_gpu_paged import DEV, attend, attend_inputs

pytestmark = pytest.mark.gpu

sc = pytest.importorskip("submanifold_sparse_conv_amd")


def arguments():
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    q, k = torch.zeros(6, 4, 64, **bf16), torch.zeros(6, 2, 64, **bf16)
    kp, vp = torch.zeros(5, 8, 2, 64, **bf16), torch.zeros(5, 8, 2, 64, **bf16)
    return dict(q=q, k=k, v=k.clone(), pos=torch.zeros(6, dtype=torch.int32, device=DEV),
                freqs=sc.rope_frequencies(64, device=DEV), k_pages=kp, v_pages=vp,
                page_table=torch.zeros(2, 2, dtype=torch.int32, device=DEV),
                k_len=torch.full((2,), 9, dtype=torch.int32, device=DEV))


POOL = [
    (dict(q=torch.zeros(6, 4, 64, dtype=torch.float64, device="cpu")), "type"), (dict(q=3), "type"),
    (dict(q=torch.zeros(6, 256, dtype=torch.bfloat16)), "GPU"), (dict(k_pages=None), "k_pages"), (dict(v_pages=7), "v_pages"),
    (dict(page_table=None), "page_table"), (dict(k_len=None), "k_len"),
]


@pytest.mark.parametrize("how,word", POOL, ids=range(len(POOL)))
def test_kinds(how, word):
    a = {**arguments(), **how}
    with pytest.raises(ValueError, match=word):
        sc.qk_norm_rope_append(**a)
    a = {n: a[n] for n in ("q", "k_pages", "v_pages", "page_table", "k_len")}
    with pytest.raises(ValueError, match=word):
        sc.paged_window_attention(**a)


def changed(name):
    a = arguments()
    t = a[name]
    return {
        "cpu": lambda: t.cpu(), "type": lambda: t.to(torch.int64 if t.dtype == torch.int32 else torch.float16),
        "long": lambda: torch.cat([t, t]), "deep": lambda: t[None], "wide": lambda: t.repeat_interleave(2, -1)[..., ::2],
    }


@pytest.mark.parametrize("name", ["k", "v", "pos", "freqs", "k_pages", "v_pages", "page_table", "k_len"])
@pytest.mark.parametrize("how", ["cpu", "type", "long", "deep", "wide"])
def test_shapes_types_devices(name, how):
    a = arguments()
    a[name] = changed(name)[how]()
    fine = name == "pos" and how == "wide"  # positions at a stride of two are positions
    fine = fine or (how == "wide" and a[name].shape[-1] == 1)
    if fine:
        sc.qk_norm_rope_append(**a)
        return
    with pytest.raises((ValueError, sc.TrSparseConvError)):
        sc.qk_norm_rope_append(**a)
    if name in ("k_pages", "v_pages", "page_table", "k_len"):
        with pytest.raises((ValueError, sc.TrSparseConvError)):
            sc.paged_window_attention(**{n: a[n] for n in ("q", "k_pages", "v_pages", "page_table", "k_len")})


@pytest.mark.parametrize("how", [
    dict(cu_q=torch.zeros(2, dtype=torch.int32)), dict(q_gain=torch.ones(64)), dict(eps=-1.0), dict(sections=[33]),
    dict(sections=[16, 16]), dict(sections=[1 << 40]), dict(sections=[-1]), dict(norm=False, gain=True), dict(q_out="short"),
    dict(q_out="k"), dict(cu="short"),
])
def test_append_refusals(how):
    a, how = arguments(), dict(how)
    if how.pop("gain", False):
        how["q_gain"] = torch.ones(64, device=DEV)
    if how.get("q_out") == "short":
        how["q_out"] = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device=DEV)
    if how.get("q_out") == "k":
        how["q_out"] = torch.zeros(6, 4, 64, dtype=torch.float16, device=DEV)
    if how.pop("cu", None):
        how["cu_q"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises((ValueError, sc.TrSparseConvError)):
        sc.qk_norm_rope_append(**a, **how)


@pytest.mark.parametrize("how", [
    dict(left=-2), dict(right=1 << 64), dict(left=-(1 << 64)), dict(sinks=1 << 32), dict(sinks=-1), dict(sinks=129),
    dict(scale=0.0), dict(scale=float("nan")), dict(workspace=5), dict(cu_q=torch.zeros(3)), dict(out=torch.zeros(6, 4, 64)),
])
def test_attention_refusals(how):
    a = arguments()
    a = [a[n] for n in ("q", "k_pages", "v_pages", "page_table", "k_len")]
    with pytest.raises((ValueError, AttributeError, sc.TrSparseConvError)):
        sc.paged_window_attention(*a, **how)
    pre = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises((ValueError, AttributeError, sc.TrSparseConvError)):
        sc.shared_prefix_attention(*a, pre, 16, **how)
    for prefix, n in ((pre, 17), (pre.cpu(), 3), (None, 3), (pre, -1), (pre.long(), 3)):
        with pytest.raises(ValueError):
            sc.shared_prefix_attention(*a, prefix, n)


def test_references_are_given_back():
    """Calls, refused ones too, keep no reference to their arguments."""
    import sys

    a = arguments()
    before = {n: sys.getrefcount(t) for n, t in a.items()}
    for _ in range(50):
        sc.qk_norm_rope_append(**a, q_out=a["q"])
        sc.paged_window_attention(a["q"], a["k_pages"], a["v_pages"], a["page_table"], a["k_len"], return_lse=True)
        with pytest.raises(ValueError):
            sc.paged_window_attention(a["q"], a["k_pages"], a["v_pages"], a["page_table"], a["k_len"], left=-2)
    assert before == {n: sys.getrefcount(t) for n, t in a.items()}


def test_two_streams_at_once():
    """Calls that share pools and tables run side by side, each with its workspace."""
    new, keys, n = [1] * 6, [3000, 40, 1200, 7, 0, 2600], 2500
    q, own, pre, kp, vp, table, pre_pages = attend_inputs(new, keys, 16, 8, 4, 128, "bf16", "beside", n)
    want = [attend(q * (i + 1) / 4, kp, vp, table, keys, new, pre_pages, n, right=0)[0] for i in range(4)]
    qs = [(q * (i + 1) / 4).to(DEV) for i in range(4)]
    lens = torch.tensor(keys, dtype=torch.int32, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sc.shared_prefix_attention(qs[i], kp, vp, table, lens, pre_pages, n, right=0))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert all(torch.equal(g, w) for g in got[i])
