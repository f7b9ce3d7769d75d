"""The serving-cache calls where offsets pass 32 bits, on two streams at once, and with scores that
fall, rise and jump from tile to tile."""
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import make_cache, make_pools, make_q, scale_of, starts
from cache_ref import attend_ref, check_attend, pages_of

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def test_shared_prefix_offsets_past_32_bits():
    P, hkv, d = 140_000, 8, 128
    k = torch.empty((P, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = torch.tensor([P - 1, 3, P - 2, P - 70_000, P - 5, 17], device="cuda")
    for pool, small in zip((k, v), make_pools(6, hkv, d)):
        pool[ids] = small
    x = ids.to(torch.int32)
    table = torch.stack([x[[0, 1, 2, 4]], x[[0, 1, 3, 5]]])
    seq = i32([64, 50])
    q = make_q(2, 16, d)
    out, lse = vt.vt_shared_prefix_decode(q, k, v, table, seq, i32([0, 2]), i32([2]), scale_of(d))
    check_attend(out, lse, attend_ref(q, k, v, table, seq, [1, 1], scale_of(d)))


def test_page_operations_past_32_bits():
    """Copies, a fork's last page and a compaction in pools of more than 2^32 bytes each."""
    P, hkv, d = 140_000, 8, 128
    k = torch.zeros((P, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    used = torch.tensor([P - 1, P - 2, 2, P - 70_000], device="cuda")
    for i, pool in enumerate((k, v)):
        pool[used] = (torch.arange(4, device="cuda") + 10 * i + 1).view(4, 1, 1, 1).to(pool.dtype)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    table[0] = used.to(torch.int32)
    lens, refs, status = i32([60, 0]), torch.zeros(P, dtype=torch.int32, device="cuda"), i32([0])
    refs[used] = 1
    refs[:2] = 1                                   # (somebody's: the fork's page is 3)
    vt.vt_fork_requests(k, v, table, lens, refs, i32([0]), i32([1]), status=status)
    assert table[1].tolist() == [P - 1, P - 2, 2, 3]
    vt.vt_copy_pages(k, v, i32([P - 2]), i32([P - 3]), status=status)
    assert torch.equal(k[P - 3], k[P - 2]) and torch.equal(v[P - 3], v[P - 2])
    n = vt.vt_compact_pages(k, v, table, lens, refs, status=status)
    assert int(n.item()) == 7 and int(status.item()) == 0
    assert table.tolist() == [[6, 5, 2, 4], [6, 5, 2, 3]]
    for i, pool in enumerate((k, v)):
        assert [float(pool[p].float().mean()) for p in (6, 5, 2, 4, 3)] == \
            [10 * i + x for x in (1, 2, 3, 4, 4)]


def test_shared_prefixes_on_two_streams():
    cases = []
    for seed in (1, 2):
        groups, own = ([0, 9, 20], [12, 40]), [(37 * i) % 300 + 1 for i in range(20)]
        seq = [16 * groups[1][int(b >= 9)] + own[b] for b in range(20)]
        k, v, table, lens = make_cache(seq, 2, 128, seed, shared=groups)
        cases.append((make_q(20, 8, 128, seed), k, v, table, lens, i32(groups[0]), i32(groups[1])))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(vt.vt_shared_prefix_decode(*c, scale_of(128)))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        q, k, v, table, lens = cases[i % 2][:5]
        assert torch.equal(out, outs[i % 2][0]) and torch.equal(lse, outs[i % 2][1])
        if i < 2:
            check_attend(out, lse, attend_ref(q, k, v, table, lens, [1] * 20, scale_of(128)))


SHAPES = {  # a factor for the keys of each tile of 128, cycled
    "falls": [8.0, 1.0, 0.1, 0.01],
    "sink": [20.0] + [0.3] * 40,
    "jumps": [0.1, 9.0, 0.1, 30.0, -30.0, 5.0],
    "slow_rise": [0.5 + 0.25 * i for i in range(40)],
    "below_then_zero": [-25.0, -25.0, 0.0],
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 64), (8, 1, 128)])
def test_scores_that_change_from_tile_to_tile(name, hq, hkv, d):
    """All keys near one direction, and the queries with it: a tile's scores are its factor's."""
    q_lens, ctx = [290, 1, 33], [1500, 2100, 77]
    seq = [a + b for a, b in zip(q_lens, ctx)]
    k, v, table, seq_t = make_cache(seq, hkv, d, poison=False)
    f = SHAPES[name]
    for b, n in enumerate(seq):
        page = table[b, :pages_of(n)].long()
        for i in range(page.numel()):
            k[page[i]] = (f[i // 8 % len(f)] * (1 + 0.05 * k[page[i]].float())).to(k.dtype)
    q = (make_q(sum(q_lens), hq, d).float().abs() * 0.5 + 0.5).to(torch.bfloat16)
    scale = scale_of(d)
    out, lse = vt.vt_prefill(q, k, v, table, seq_t, starts(q_lens), scale)
    check_attend(out, lse, attend_ref(q, k, v, table, seq_t, q_lens, scale))
    last = q[[289, 290, 323]].contiguous()
    for groups, prefix in (([0, 1, 2, 3], [50, 40, 0]), ([0, 3], [0])):
        out, lse = vt.vt_shared_prefix_decode(last, k, v, table, seq_t, i32(groups), i32(prefix),
                                              scale)
        check_attend(out, lse, attend_ref(last, k, v, table, seq_t, [1] * 3, scale))
