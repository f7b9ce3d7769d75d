"""Page tables that are some columns of a wider one, or of one allocation's end: requests have the
view's entries, and what is between the rows is neither read nor written."""
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import make_cache, make_pools, make_q, scale_of, starts
from cache_ref import attend_ref, check_attend

pytestmark = pytest.mark.gpu
GUARD = 1 << 29   # no page's id: read as one, it is reported

VIEWS = {"left": slice(0, 6), "right": slice(4, 10), "middle": slice(2, 8)}


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.fixture(params=list(VIEWS))
def view(request):
    """A table of 4 rows, 6 of 10 columns wide, and what it is a view of (guards behind it)."""
    store = torch.full((4 * 10 + 64,), GUARD, dtype=torch.int32, device="cuda")
    cols = VIEWS[request.param]
    table = store[:40].view(4, 10)[:, cols]
    table.fill_(-1)
    outside = torch.ones(104, dtype=torch.bool, device="cuda")
    outside[:40].view(4, 10)[:, cols] = False
    return table, store, outside


def untouched(store, outside):
    return bool((store[outside] == GUARD).all())


def test_growth_ends_at_the_view(view):
    table, store, outside = view
    lens, refs = i32([0] * 4), i32([0] * 40)
    status = i32([0])
    vt.vt_extend_requests(table, lens, refs, i32([0, 1, 2, 3]), i32([96, 97, 95, 160]),
                          status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_LEN
    assert lens.tolist() == [96, 0, 95, 0] and int(refs.sum()) == 12
    assert table[0].tolist() == list(range(6)) and table[2].tolist() == list(range(6, 12))
    vt.vt_extend_requests(table, lens, refs, i32([0, 2, 3]), i32([1, 1, 96]), status=status)
    assert lens.tolist() == [96, 0, 96, 96]
    assert table[3].tolist() == list(range(12, 18))
    assert untouched(store, outside)


def test_fork_free_and_compaction_end_at_the_view(view):
    table, store, outside = view
    k, v = make_pools(40, 1, 64)
    lens, refs, status = i32([0] * 4), i32([0] * 40), i32([0])
    vt.vt_extend_requests(table, lens, refs, i32([1]), i32([90]))
    vt.vt_fork_requests(k, v, table, lens, refs, i32([1]), i32([3]), status=status)
    assert int(status.item()) == 0 and lens.tolist() == [0, 90, 0, 90]
    assert table[3].tolist() == [0, 1, 2, 3, 4, 6]
    lens[1] = 97                                   # a length that the row has no entries for
    vt.vt_fork_requests(k, v, table, lens, refs, i32([1]), i32([0]), status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_LEN and lens.tolist() == [0, 97, 0, 90]
    status.zero_()
    n = vt.vt_compact_pages(k, v, table, lens, refs, status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_LEN and int(n.item()) == 7
    status.zero_()
    vt.vt_free_requests(table, lens, refs, i32([1]), status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_LEN and lens.tolist() == [0, 0, 0, 90]
    assert int(refs.sum()) == 6                    # the fork's own
    assert untouched(store, outside)


@pytest.mark.parametrize("name", list(VIEWS))
def test_prompts_longer_than_the_view_are_bad_lengths(name):
    q_lens, seq = [40, 5, 7, 96], [96, 70, 7, 96]
    k, v, table, seq_t = make_cache(seq, 2, 64, width=6)
    wide = torch.full((4, 10), GUARD, dtype=torch.int32, device="cuda")
    wide[:, VIEWS[name]] = table
    q = make_q(sum(q_lens), 4, 64)
    ref = attend_ref(q, k, v, table, seq_t, q_lens, scale_of(64))
    seq_t = seq_t.clone()
    seq_t[1] = 97                                  # past the view, inside the wider row
    status = i32([0])
    out, lse = vt.vt_prefill(q, k, v, wide[:, VIEWS[name]], seq_t, starts(q_lens), scale_of(64),
                             status=status)
    assert int(status.item()) == vt.VT_DEV_BAD_LEN  # (and no bad page: none was read)
    assert bool((out[40:45] == 0).all()) and bool((lse[40:45] == -torch.inf).all())
    keep = [i for i in range(148) if not 40 <= i < 45]
    check_attend(out[keep], lse[keep], tuple(x[keep] for x in ref))


@pytest.mark.parametrize("name", list(VIEWS))
def test_shared_prefixes_longer_than_the_view_are_bad_lengths(name):
    seq, groups = [64, 90, 33, 96], ([0, 2, 4], [3, 0])
    k, v, table, seq_t = make_cache(seq, 2, 128, width=6, shared=groups)
    wide = torch.full((4, 10), GUARD, dtype=torch.int32, device="cuda")
    wide[:, VIEWS[name]] = table
    q = make_q(4, 8, 128)
    ref = attend_ref(q, k, v, table, seq_t, [1] * 4, scale_of(128))

    def run(lens, prefix):
        status = i32([0])
        out, lse = vt.vt_shared_prefix_decode(q, k, v, wide[:, VIEWS[name]], lens, i32(groups[0]),
                                              i32(prefix), scale_of(128), status=status)
        return out, lse, int(status.item())

    out, lse, st = run(seq_t, groups[1])
    assert st == 0
    check_attend(out, lse, ref)
    long = seq_t.clone()
    long[3] = 97
    for lens, prefix, gone in ((long, [3, 0], [3]), (seq_t, [7, 0], [0, 1])):
        out, lse, st = run(lens, prefix)
        keep = [b for b in range(4) if b not in gone]
        assert st == vt.VT_DEV_BAD_LEN
        assert bool((out[gone] == 0).all()) and bool((lse[gone] == -torch.inf).all())
        check_attend(out[keep], lse[keep], tuple(x[keep] for x in ref))
