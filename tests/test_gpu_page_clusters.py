"""The page lists by one CTA (small pools) and by a cluster of eight, against the model of the books:
pools around the size where the cluster takes over, lists that stay in shared memory and lists that
do not, free pages across the CTAs' shares, and too few of them."""
import numpy as np
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_ref import pages_of
from test_gpu_pages import Cache

pytestmark = pytest.mark.gpu

LARGE = 16384


@pytest.mark.parametrize("pages", [4096, 4097, 12000, LARGE, LARGE + 1, 3 * LARGE + 7])
def test_a_life_at_the_boundary(pages):
    c = Cache([33, 16, 100, 1, 0, 0, 0, 0], 10, pages, hkv=1, seed=pages)
    c.fork([0, 1, 2, 0, 0], [4, 5, 6, 7, 5])
    assert c.bits() == vt.VT_DEV_BAD_REQ
    c.extend([4, 5, 0, 6], [20, 1, 0, 60])
    c.compact()
    c.free([2, 0])
    c.compact()
    c.fork([6, 6], [0, 2])
    assert c.bits() == 0


def rows(g, n, hi, count):
    return [int(x) for x in torch.randint(n, hi, (count,), generator=g)]


@pytest.mark.parametrize("n", [300, 2048, 2049, 5000])
def test_long_lists(n):
    """Growth and forks whose pages come from several shares; rows repeat in the lists."""
    g = torch.Generator().manual_seed(n)
    lens = rows(g, 0, 90, n)
    used = sum(pages_of(x) for x in lens)
    c = Cache(lens + [0] * n, 8, max(LARGE + 1, 2 * used), hkv=1, d=32, seed=n)
    # the first shares are mostly full, so that even a short list reaches past them
    full = np.flatnonzero(c.model.refs[:9000] == 0)[100:]
    c.refs[torch.from_numpy(full).cuda()] = 1
    c.model.refs[full] = 1
    c.extend(rows(g, 0, n, n), rows(g, 0, 40, n))
    assert int(torch.nonzero(c.refs).max()) > 9000
    c.fork(rows(g, 0, n, n), list(range(n, 2 * n)))
    c.free(rows(g, 0, 2 * n, n))
    c.fork(rows(g, 0, 2 * n, n), rows(g, 0, 2 * n, n))
    c.compact()


@pytest.mark.parametrize("n", [300, 2048, 2049, 5000])
@pytest.mark.parametrize("fork", [False, True])
def test_too_few_pages(n, fork):
    """The pages run out within the list, in a share that is not the first."""
    g = torch.Generator().manual_seed(2 * n + fork)
    lens = [15 + 16 * x for x in rows(g, 0, 2, n)]     # (a fork takes a page)
    c = Cache(lens + [0] * n, 6, LARGE + 999, hkv=1, d=32, seed=n)
    left = 2 * n // 3
    free = np.flatnonzero(c.model.refs == 0)
    keep = np.sort(np.random.default_rng(n).permutation(free)[:left])
    take = np.setdiff1d(free, keep)
    c.refs[torch.from_numpy(take).cuda()] = 1
    c.model.refs[take] = 1
    if fork:
        c.fork(list(range(n)), list(range(n, 2 * n)))
        assert int((c.lens[n:] > 0).sum()) == left
    else:
        c.extend(list(range(n)), rows(g, 0, 40, n))
    assert c.bits() == vt.VT_DEV_NO_PAGE


@pytest.mark.parametrize("n", [1500, 2048, 2049, 5000])
def test_long_lists_in_a_small_pool(n):
    g = torch.Generator().manual_seed(3 * n)
    lens = [x * (i < 1200) for i, x in enumerate(rows(g, 0, 40, n))]
    c = Cache(lens + [0] * n, 6, 4096, hkv=1, d=32, seed=n)
    c.extend(rows(g, 0, n, n), rows(g, 0, 5, n))
    c.fork(rows(g, 0, n, n), list(range(n, 2 * n)))
    c.free(rows(g, 0, 2 * n, n))
    c.compact()
