"""vt_prefill against the definition in 64 bits: head shapes, lengths around the tiles' edges,
contexts, layouts and strides, rows that are left alone, and what it reports."""
import os
import subprocess
import sys

import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import make_cache, make_pools, make_q, scale_of, starts
from cache_ref import attend_ref, check_attend, pages_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEADS = [(1, 1, 64), (2, 1, 128), (6, 2, 64), (4, 1, 128), (10, 2, 128), (12, 2, 64), (7, 1, 128),
         (16, 2, 128), (8, 8, 64)]  # Hq, Hkv, D: every group size from 1 to 8
LENGTHS = {  # query tokens and context of each request
    "one": ([1], [0]),
    "one_far": ([1], [1290]),
    "short": ([3, 0, 17, 1, 15, 16, 0], [0, 40, 0, 0, 1, 0, 16]),
    "edges": ([127, 128, 129, 255, 257], [0, 0, 1, 127, 128]),
    "long": ([700, 33], [0, 1500]),
    "drafts": ([4] * 9, [300 + 16 * i + i for i in range(9)]),
}


def run(q, k, v, table, seq, q_lens, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = vt.vt_prefill(q, k, v, table, seq, starts(q_lens), scale_of(q.shape[2]),
                             status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def case(q_lens, ctx, hq, hkv, d, seed=0, **kw):
    seq = [a + b for a, b in zip(q_lens, ctx)]
    k, v, table, seq_t = make_cache(seq, hkv, d, seed, **kw)
    return make_q(sum(q_lens), hq, d, seed), k, v, table, seq_t


@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_lengths_and_heads(name, hq, hkv, d):
    q_lens, ctx = LENGTHS[name]
    q, k, v, table, seq = case(q_lens, ctx, hq, hkv, d, seed=hq + d)
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == 0
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(d)))


@pytest.mark.parametrize("layout", ["hpd", "shard", "pad"])
@pytest.mark.parametrize("hq,hkv,d", [(6, 2, 64), (10, 2, 128)])
def test_pool_layouts(layout, hq, hkv, d):
    q_lens, ctx = [200, 5, 64], [33, 700, 0]
    q, k, v, table, seq = case(q_lens, ctx, hq, hkv, d, layout=layout)
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == 0
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(d)))


def test_query_as_a_view_and_a_wider_table():
    q_lens, ctx = [90, 7], [0, 250]
    q, k, v, table, seq = case(q_lens, ctx, 4, 2, 128, width=40)
    packed = torch.randn((97, 4 + 2 + 2, 128), device="cuda", dtype=torch.bfloat16)
    packed[:, :4] = q
    wide = torch.full((2, 50), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :40] = table
    out, lse, st = run(packed[:, :4], k, v, wide[:, :40], seq, q_lens)
    assert st == 0
    ref, ref_lse, _ = run(q, k, v, table, seq, q_lens)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(128)))


@pytest.mark.parametrize("gain", [0.0, 12.0])
def test_flat_and_sharp_scores(gain):
    """All scores equal, and scores of some hundreds (one key has nearly all the weight)."""
    q_lens, ctx = [300], [100]
    q, k, v, table, seq = case(q_lens, ctx, 4, 1, 64)
    q = (q * gain).contiguous()
    out, lse, _ = run(q, k, v, table, seq, q_lens)
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(64)))


@pytest.mark.parametrize("at", [(70, 198, 300), (10, 140, 210, 390), (127, 128, 255, 256, 511),
                                (64, 65, 66, 447)])
@pytest.mark.parametrize("hq,d", [(2, 64), (5, 128)])
def test_scores_that_rise_by_more_than_100_bits_at_once(at, hq, d):
    """Keys whose scores are 150 bits above all before them, in either half of a step of 128 keys;
    every row's result is the value of the last of them that it sees, to rounding."""
    q_lens, ctx = [300], [260]
    q, k, v, table, seq = case(q_lens, ctx, hq, 1, d, poison=False)
    k *= 0.3
    page = table[0].long()
    for i, pos in enumerate(at):
        k[page[pos // 16], pos % 16] = 13.0 * (i + 1)      # 64 * 13 / 8 = 104, 150 in base 2
    q = torch.ones_like(q)
    out, lse, _ = run(q, k, v, table, seq, q_lens)
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(d)))


def test_rising_scores_move_the_maximum_in_every_tile():
    q_lens, ctx = [130], [1200]
    q, k, v, table, seq = case(q_lens, ctx, 2, 1, 64, poison=False)
    order = torch.arange(pages_of(1330), device="cuda", dtype=torch.float32)
    k[table[0].long()] = (0.2 * order[:, None, None, None] *
                          torch.ones_like(k[table[0].long()])).to(torch.bfloat16)
    q = q.abs()
    out, lse, _ = run(q, k, v, table, seq, q_lens)
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(64)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_row_spoils_only_itself(bad):
    q_lens, ctx = [70, 200], [300, 900]
    q, k, v, table, seq = case(q_lens, ctx, 6, 2, 64)
    ref = attend_ref(q, k, v, table, seq, q_lens, scale_of(64))
    q[5, 1, 7] = q[150, 4, 0] = bad
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == 0
    keep = torch.ones(270, 6, dtype=torch.bool, device="cuda")
    keep[5, 1] = keep[150, 4] = False
    assert bool(torch.isnan(out[~keep]).any(1).all())
    check_attend(out[keep], lse[keep], tuple(x[keep] for x in ref))


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3.0])
def test_scales(scale):
    q_lens, ctx = [40, 150], [500, 0]
    q, k, v, table, seq = case(q_lens, ctx, 4, 1, 128)
    out, lse = vt.vt_prefill(q, k, v, table, seq, starts(q_lens), scale)
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale))


def test_captured_by_a_process_that_never_called_it():
    """The first call of a process inside a stream capture."""
    code = """if True:
        import torch, paged_block_sparse_vt_b200 as vt
        i32 = dict(dtype=torch.int32, device="cuda")
        k = torch.randn(8, 16, 1, 64, device="cuda", dtype=torch.bfloat16)
        q = torch.randn(20, 2, 64, device="cuda", dtype=torch.bfloat16)
        table, seq = torch.arange(8, **i32).view(1, 8), torch.tensor([100], **i32)
        start, out = torch.tensor([0, 20], **i32), torch.zeros_like(q)
        vt.load_library()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vt.vt_prefill(q, k, k, table, seq, start, 0.1, out=out)
        g.replay()
        want, _ = vt.vt_prefill(q, k, k, table, seq, start, 0.1)
        assert torch.equal(out, want) and float(out.abs().sum()) > 0
    """
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


def test_rows_behind_the_last_prompt_are_left_alone():
    q_lens, ctx = [20, 9], [0, 77]
    q, k, v, table, seq = case(q_lens, ctx, 4, 2, 64)
    padded = torch.cat([q, torch.full_like(q[:14], float("nan"))])
    out = torch.full_like(padded, 7.0)
    lse = torch.full(padded.shape[:2], 7.0, device="cuda")
    run(padded, k, v, table, seq, q_lens, out=out, lse=lse)
    check_attend(out[:29], lse[:29], attend_ref(q, k, v, table, seq, q_lens, scale_of(64)))
    assert bool((out[29:] == 7.0).all()) and bool((lse[29:] == 7.0).all())


def test_padded_batch_and_no_lse():
    """Rows of the table behind the live requests: no query tokens, lengths and pages of any kind."""
    q_lens, ctx = [50, 0, 0], [10, 0, 0]
    q, k, v, table, seq = case(q_lens, ctx, 2, 2, 128)
    seq[1], seq[2] = -5, 1 << 20
    table[1:] = -1
    out, lse, st = run(q, k, v, table, seq, q_lens, want_lse=False)
    assert lse is None and st == 0
    check_attend(out, None, attend_ref(q[:50], k, v, table[:1], seq[:1], [50], scale_of(128)))


def test_bad_lengths_give_empty_rows():
    q_lens, ctx = [40, 30, 20, 10], [5, 6, 7, 8]
    q, k, v, table, seq = case(q_lens, ctx, 4, 2, 64)
    ref = attend_ref(q, k, v, table, seq, q_lens, scale_of(64))
    seq[1] = 29                                   # fewer tokens than query rows
    seq[3] = 16 * table.shape[1] + 1              # more pages than the table has
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == vt.VT_DEV_BAD_LEN
    for lo, hi in ((40, 70), (90, 100)):
        assert bool((out[lo:hi] == 0).all()) and bool((lse[lo:hi] == -float("inf")).all())
    for lo, hi in ((0, 40), (70, 90)):
        check_attend(out[lo:hi], lse[lo:hi], tuple(x[lo:hi] for x in ref))


@pytest.mark.parametrize("bad_id", [-1, 1 << 20, 2**31 - 1, -2**31])
@pytest.mark.parametrize("where", [[0], [3, 4], [20], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]])
def test_bad_pages_take_no_part(bad_id, where):
    q_lens, ctx = [170, 40], [160, 0]
    q, k, v, table, seq = case(q_lens, ctx, 6, 2, 64)
    table[0, where] = bad_id
    table[1, 0] = bad_id                          # rows 0 .. 15 of request 1 see nothing else
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == vt.VT_DEV_BAD_PAGE
    check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(64),
                                      bad_pages=[where, [0]]))
    assert bool((lse[170:186] == -float("inf")).all())


@pytest.mark.parametrize("start", [[1, 5, 9], [0, 6, 5], [0, 5, 11], [0, -1, 4], [-3, 2, 4]])
def test_bad_starts_compute_nothing(start):
    q, k, v, table, seq = case([5, 5], [0, 0], 2, 1, 64)
    out = torch.full_like(q, 3.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vt.vt_prefill(q, k, v, table, seq, torch.tensor(start, dtype=torch.int32, device="cuda"), 0.1,
                  out=out, status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_START and bool((out == 3.0).all())


def test_offsets_past_32_bits():
    """Pages near the end of pools of more than 2^31 elements each."""
    P, hkv, d = 140_000, 8, 128
    k = torch.empty((P, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = torch.tensor([P - 1, 3, P - 2, P - 70_000], device="cuda")
    for pool, small in zip((k, v), make_pools(4, hkv, d)):
        pool[ids] = small
    table = ids.to(torch.int32).view(1, 4)
    seq = torch.tensor([64], dtype=torch.int32, device="cuda")
    q = make_q(60, 8, d)
    out, lse, st = run(q, k, v, table, seq, [60])
    assert st == 0
    check_attend(out, lse, attend_ref(q, k, v, table, seq, [60], scale_of(d)))


def test_many_short_prompts():
    """More requests than one step of the planner takes, some without query tokens."""
    q_lens = [(7 * i) % 5 for i in range(3000)]
    ctx = [(11 * i) % 50 for i in range(3000)]
    q, k, v, table, seq = case(q_lens, ctx, 2, 1, 64, poison=False)
    out, lse, st = run(q, k, v, table, seq, q_lens)
    assert st == 0
    # the definition for a sample of them
    at = [0]
    for n in q_lens:
        at.append(at[-1] + n)
    for b in list(range(0, 3000, 97)) + [2999]:
        rows = slice(at[b], at[b + 1])
        check_attend(out[rows], lse[rows],
                     attend_ref(q[rows], k, v, table[b:b + 1], seq[b:b + 1], [q_lens[b]],
                                scale_of(64)), label=b)


def test_calls_repeat_bit_for_bit_and_share_a_workspace():
    q_lens, ctx = [300, 2, 45], [0, 3000, 600]
    q, k, v, table, seq = case(q_lens, ctx, 8, 2, 128)
    first, first_lse, _ = run(q, k, v, table, seq, q_lens)
    ws = vt.prefill_workspace(q, k, v, table, seq, starts(q_lens))
    ws.fill_(255)
    other = case([50], [60], 8, 2, 128, seed=5)
    for _ in range(3):
        out, lse, _ = run(q, k, v, table, seq, q_lens, workspace=ws)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)
        # another shape on the same workspace in between (a smaller call)
        run(*other, [50], workspace=ws)


def test_graphs_that_share_a_workspace_and_new_lengths():
    """Two captured calls on one workspace, replayed in turn, lengths and pages changed in place."""
    q_lens, ctx = [64, 30], [500, 1]
    a = case(q_lens, ctx, 4, 2, 128, seed=1)
    b = case(q_lens, ctx, 4, 2, 128, seed=2)
    ws = vt.prefill_workspace(*a, starts(q_lens))
    start, scale = starts(q_lens), scale_of(128)
    outs = [torch.empty_like(a[0]), torch.empty_like(b[0])]
    vt.vt_prefill(*a, start, scale, out=outs[0], want_lse=False, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for c, out in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vt.vt_prefill(*c, start, scale, out=out, want_lse=False, workspace=ws)
        graphs.append(g)
    for lens in (q_lens, [90, 4]):
        start.copy_(starts(lens))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, out in zip((a, b), outs):
            check_attend(out, None, attend_ref(*c, lens, scale))


@pytest.mark.parametrize("q_lens,ctx", [([300, 41], [90, 2000]), ([9], [0])])
def test_prepared(q_lens, ctx):
    """The prepared call gives what the plain one gives, also after its inputs changed in place."""
    q, k, v, table, seq = case(q_lens, ctx, 4, 2, 128)
    start, scale = starts(q_lens), scale_of(128)
    ws = vt.prefill_workspace(q, k, v, table, seq, start)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    call = vt.prepare_prefill(q, k, v, table, seq, start, scale, out, lse, workspace=ws)
    for _ in range(2):
        assert call.run() == (out, lse)
        want, want_lse = vt.vt_prefill(q, k, v, table, seq, start, scale)
        n = int(start[-1])                       # (rows behind it are nobody's)
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])
        q.mul_(0.5)
        seq.sub_(1)
        start.clamp_(max=int(start[-1]) - 1)
        seq[-1:].clamp_(min=int(start[-1] - start[-2]))
    if ws is not None:
        with pytest.raises(vt.VtError):
            vt.prepare_prefill(q, k, v, table, seq, start, scale, out)
    with pytest.raises(vt.VtError):
        vt.prepare_prefill(q, k, v, table, seq, start, scale, out[:1], workspace=ws)


def test_two_streams_at_once():
    q_lens, ctx = [400, 100], [900, 0]
    cases = [case(q_lens, ctx, 4, 2, 64, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    start = starts(q_lens)
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(vt.vt_prefill(*c, start, scale_of(64)))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        c = cases[i % 2]
        assert torch.equal(out, outs[i % 2][0])
        if i < 2:
            check_attend(out, lse, attend_ref(*c, q_lens, scale_of(64)))


def test_binding_refusals():
    q, k, v, table, seq = case([300], [300], 2, 1, 64)   # (of a size that needs a workspace)
    start = starts([300])
    bad = [dict(q=q.float()), dict(q=q[..., ::2]), dict(q=q.transpose(0, 1)), dict(seq_lens=seq.long()),
           dict(q_start=start[:1]), dict(k_pool=k.half()), dict(out=q.float()),
           dict(out=q[:4].clone()), dict(lse=torch.empty(5, 1, device="cuda")),
           dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
           dict(sm_scale=-1.0), dict(page_table=table.long())]
    for over in bad:
        kw = dict(q=q, k_pool=k, v_pool=v, page_table=table, seq_lens=seq, q_start=start,
                  sm_scale=0.1)
        kw.update(over)
        with pytest.raises(vt.VtError):
            vt.vt_prefill(**kw)


def test_drawn_batches():
    g = torch.Generator().manual_seed(99)

    def ri(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    for i in range(24):
        hkv, group, d = ri(1, 3), ri(1, 8), (64, 128)[ri(0, 1)]
        q_lens = [ri(0, (3, 40, 400)[ri(0, 2)]) for _ in range(ri(1, 6))]
        ctx = [ri(0, (20, 2000)[ri(0, 1)]) for _ in q_lens]
        q_lens[0] += 1
        q, k, v, table, seq = case(q_lens, ctx, hkv * group, hkv, d, seed=i)
        out, lse, st = run(q, k, v, table, seq, q_lens)
        assert st == 0
        check_attend(out, lse, attend_ref(q, k, v, table, seq, q_lens, scale_of(d)),
                     label=(i, hkv, group, d, q_lens, ctx))
