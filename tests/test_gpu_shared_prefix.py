"""vt_shared_prefix_decode against attention of each request over all its pages in 64 bits."""
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import make_cache, make_q, scale_of
from cache_ref import attend_ref, check_attend

pytestmark = pytest.mark.gpu

HEADS = [(1, 1, 64), (2, 1, 128), (6, 2, 64), (4, 1, 128), (10, 2, 128), (12, 2, 64), (7, 1, 128),
         (16, 2, 128), (8, 8, 64)]
GROUPS = {  # group sizes, prefix pages of each, own tokens of each request
    "alone": ([1], [0], [1]),
    "alone_prefix": ([1], [9], [0]),
    "pair": ([2], [1], [1, 37]),
    "none_shared": ([3], [0], [20, 400, 16]),
    "ends_with_prefix": ([4], [5], [0, 0, 16, 5]),
    "groups": ([3, 0, 1, 5], [40, 7, 12, 17], [3, 16, 300, 150, 1, 0, 33, 17, 129]),
    "long": ([6], [150], [700, 1, 128, 127, 129, 2100]),
    "wide": ([150, 30], [20, 3], [(13 * i) % 60 for i in range(180)]),
}


def build(sizes, prefix, own, hq, hkv, d, seed=0, **kw):
    start = [0]
    for n in sizes:
        start.append(start[-1] + n)
    lead = [p for n, p in zip(sizes, prefix) for _ in range(n)]
    seq = [16 * p + t for p, t in zip(lead, own)]
    k, v, table, seq_t = make_cache(seq, hkv, d, seed, shared=(start, prefix), **kw)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=make_q(len(own), hq, d, seed), k_pool=k, v_pool=v, page_table=table,
                seq_lens=seq_t, group_start=torch.tensor(start, **i32),
                prefix_pages=torch.tensor(prefix, **i32), sm_scale=scale_of(d))


def run(c, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = vt.vt_shared_prefix_decode(**c, status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def ref_of(c, **kw):
    return attend_ref(c["q"], c["k_pool"], c["v_pool"], c["page_table"], c["seq_lens"],
                      [1] * c["q"].shape[0], c["sm_scale"], **kw)


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_groups_and_heads(name, hq, hkv, d):
    c = build(*GROUPS[name], hq, hkv, d, seed=hq + d)
    out, lse, st = run(c)
    assert st == 0
    check_attend(out, lse, ref_of(c))


@pytest.mark.parametrize("layout", ["hpd", "shard", "pad"])
def test_pool_layouts(layout):
    c = build(*GROUPS["groups"], 10, 2, 128, layout=layout)
    out, lse, st = run(c)
    assert st == 0
    check_attend(out, lse, ref_of(c))


def test_sharing_is_only_a_matter_of_speed():
    """The same requests with their prefix declared, half declared, or not at all."""
    c = build([7], [30], [5, 90, 16, 0, 1, 200, 31], 8, 2, 128)
    ref = ref_of(c)
    for pages in (30, 15, 1, 0):
        c["prefix_pages"].fill_(pages)
        out, lse, st = run(c)
        assert st == 0
        check_attend(out, lse, ref, label=pages)


@pytest.mark.parametrize("gain", [0.0, 12.0])
def test_flat_and_sharp_scores(gain):
    c = build(*GROUPS["groups"], 4, 2, 64)
    c["q"] = (c["q"] * gain).contiguous()
    out, lse, _ = run(c)
    check_attend(out, lse, ref_of(c))


def test_requests_behind_the_last_group_are_left_alone():
    c = build([4, 2], [3, 0], [9, 30, 1, 17, 50, 60], 4, 2, 64)
    ref = ref_of(c)
    c["group_start"] = c["group_start"][:2].clone()
    c["prefix_pages"] = c["prefix_pages"][:1].clone()
    c["seq_lens"][4:] = -1
    c["page_table"][4:] = 1 << 30
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    _, _, st = run(c, out=out, lse=lse)
    assert st == 0
    check_attend(out[:4], lse[:4], tuple(x[:4] for x in ref))
    assert bool((out[4:] == 7.0).all()) and bool((lse[4:] == 7.0).all())


def test_bad_lengths_give_empty_rows():
    c = build([3, 2, 2], [4, 6, 2], [9, 30, 17, 50, 60, 8, 8], 6, 2, 64)
    ref = ref_of(c)
    c["seq_lens"][1] = 16 * 4 - 1                       # shorter than its prefix
    c["seq_lens"][4] = 16 * c["page_table"].shape[1] + 1
    c["prefix_pages"][2] = c["page_table"].shape[1] + 1  # a whole group
    out, lse, st = run(c)
    assert st == vt.VT_DEV_BAD_LEN
    for b in (1, 4, 5, 6):
        assert bool((out[b] == 0).all()) and bool((lse[b] == -float("inf")).all())
    for b in (0, 2, 3):
        check_attend(out[b:b + 1], lse[b:b + 1], tuple(x[b:b + 1] for x in ref))
    for bad in (0, -7, -2**31):
        c["seq_lens"][0] = bad
        out, lse, st = run(c)
        assert st == vt.VT_DEV_BAD_LEN
        assert bool((out[0] == 0).all()) and bool((lse[0] == -float("inf")).all())
    c["prefix_pages"][1] = -1
    out, lse, st = run(c)
    assert bool((out[3:] == 0).all()) and bool((lse[3:] == -float("inf")).all())


@pytest.mark.parametrize("bad_id", [-1, 1 << 20, 2**31 - 1])
def test_bad_pages_take_no_part(bad_id):
    c = build([3, 1], [12, 1], [30, 0, 200, 16], 6, 2, 64)
    c["page_table"][:3, 5] = bad_id       # in the shared part
    c["page_table"][2, 14] = bad_id       # in a request's own part
    c["page_table"][3, :2] = bad_id       # nothing left
    out, lse, st = run(c)
    assert st == vt.VT_DEV_BAD_PAGE
    check_attend(out, lse, ref_of(c, bad_pages=[[5], [5], [5, 14], [0, 1]]))
    assert bool((lse[3] == -float("inf")).all())


@pytest.mark.parametrize("start", [[1, 2, 4], [0, 3, 2], [0, 2, 5], [0, -1, 4]])
def test_bad_starts_compute_nothing(start):
    c = build([2, 2], [1, 1], [4, 4, 4, 4], 2, 1, 64)
    c["group_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.full_like(c["q"], 3.0)
    _, _, st = run(c, out=out)
    assert st == vt.VT_DEV_BAD_START and bool((out == 3.0).all())


def test_many_requests_and_groups():
    """More units than one step of the planner takes."""
    sizes = [1 + i % 3 for i in range(1500)]
    prefix = [i % 4 for i in range(1500)]
    own = [1 + (7 * i) % 40 for i in range(sum(sizes))]
    c = build(sizes, prefix, own, 2, 1, 64, poison=False)
    out, lse, st = run(c)
    assert st == 0
    for b in list(range(0, len(own), 131)) + [len(own) - 1]:
        one = attend_ref(c["q"][b:b + 1], c["k_pool"], c["v_pool"], c["page_table"][b:b + 1],
                         c["seq_lens"][b:b + 1], [1], c["sm_scale"])
        check_attend(out[b:b + 1], lse[b:b + 1], one, label=b)


def test_repeats_graphs_and_a_shared_workspace():
    a = build(*GROUPS["long"], 8, 2, 128, seed=1)
    b = build(*GROUPS["groups"], 8, 2, 128, seed=2)
    refs = [ref_of(a), ref_of(b)]
    args = ("q", "k_pool", "v_pool", "page_table", "seq_lens", "group_start", "prefix_pages")
    ws = max((vt.shared_prefix_workspace(*(c[n] for n in args)) for c in (a, b)),
             key=lambda t: t.numel()).fill_(255)
    want = [run(c)[:2] for c in (a, b)]
    graphs, got = [], []
    for c in (a, b):
        run(c, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(vt.vt_shared_prefix_decode(**c, workspace=ws))
        graphs.append(g)
    for g in graphs * 3:
        g.replay()
    torch.cuda.synchronize()
    for (out, lse), (w, wl), ref in zip(got, want, refs):
        assert torch.equal(out, w) and torch.equal(lse, wl)
        check_attend(out, lse, ref)
    # a shorter batch in place: the lengths are read on the device
    a["seq_lens"].sub_(1).clamp_(min=16 * 150)
    graphs[0].replay()
    torch.cuda.synchronize()
    check_attend(*got[0], ref_of(a))


def test_prepared():
    c = build(*GROUPS["groups"], 8, 2, 128)
    args = ("q", "k_pool", "v_pool", "page_table", "seq_lens", "group_start", "prefix_pages")
    ws = vt.shared_prefix_workspace(*(c[n] for n in args))
    out, lse = torch.empty_like(c["q"]), torch.empty(c["q"].shape[:2], device="cuda")
    call = vt.prepare_shared_prefix_decode(**c, out=out, lse=lse, workspace=ws)
    for _ in range(2):
        assert call.run() == (out, lse)
        want, want_lse = vt.vt_shared_prefix_decode(**c)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        c["q"].mul_(0.5)
    with pytest.raises(vt.VtError):
        vt.prepare_shared_prefix_decode(**c, out=out)


def test_binding_refusals():
    c = build([2], [1], [3, 4], 2, 1, 64)
    for over in (dict(q=c["q"].float()), dict(q=c["q"][:1]), dict(group_start=c["group_start"][:1]),
                 dict(prefix_pages=c["prefix_pages"].long()), dict(sm_scale=0.0),
                 dict(out=c["q"][:1].clone()),
                 dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(vt.VtError):
            vt.vt_shared_prefix_decode(**{**c, **over})


def test_drawn_batches():
    g = torch.Generator().manual_seed(7)

    def ri(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    for i in range(24):
        hkv, group, d = ri(1, 3), ri(1, 8), (64, 128)[ri(0, 1)]
        sizes = [ri(0, (2, 60)[ri(0, 1)]) for _ in range(ri(1, 4))]
        sizes[0] += 1
        prefix = [ri(0, (3, 90)[ri(0, 1)]) for _ in sizes]
        own = [ri(1, (20, 500)[ri(0, 1)]) for _ in range(sum(sizes))]
        c = build(sizes, prefix, own, hkv * group, hkv, d, seed=i)
        out, lse, st = run(c)
        assert st == 0
        check_attend(out, lse, ref_of(c), label=(i, sizes, prefix))
