"""The page operations against the numpy model of the books, to the bit."""
import numpy as np
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import make_pools
from cache_ref import Books, pages_of

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Cache:
    """The books and pools on the device, with the model beside them."""

    def __init__(self, lens, width, pages, hkv=2, d=64, layout="phd", seed=0, mla=False):
        rng = np.random.default_rng(seed)
        perm = rng.permutation(pages)
        table = np.full((len(lens), width), -1, dtype=np.int32)
        refs, at = np.zeros(pages, dtype=np.int32), 0
        for b, l in enumerate(lens):
            n = pages_of(l)
            table[b, :n] = perm[at:at + n]
            at += n
        refs[perm[:at]] = 1
        self.k, self.v = make_pools(pages, hkv, d, seed, layout)
        if mla:
            self.v = self.k[..., :512]
        self.cent = torch.randn((pages, hkv, d), device="cuda")
        self.mla = mla
        self.table, self.lens, self.refs = (torch.from_numpy(np.array(x, dtype=np.int32)).cuda()
                                            for x in (table, lens, refs))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.model = Books(table, lens, refs, self.host(self.k), self.host(self.v),
                           self.cent.cpu().numpy())

    @staticmethod
    def host(pool):
        return pool.contiguous().view(torch.int16).cpu().numpy()

    def fork(self, parents, children):
        vt.vt_fork_requests(self.k, self.v, self.table, self.lens, self.refs, i32(parents),
                            i32(children), status=self.status)
        cent = self.model.pools[2].copy()
        self.model.fork(parents, children)
        self.model.pools[2] = cent          # a fork copies no centroid
        self.check()

    def extend(self, requests, tokens):
        vt.vt_extend_requests(self.table, self.lens, self.refs, i32(requests), i32(tokens),
                              status=self.status)
        self.model.extend(requests, tokens)
        self.check()

    def free(self, requests):
        vt.vt_free_requests(self.table, self.lens, self.refs, i32(requests), status=self.status)
        self.model.free(requests)
        self.check()

    def compact(self):
        n = vt.vt_compact_pages(self.k, self.v, self.table, self.lens, self.refs,
                                centroids=self.cent, status=self.status)
        assert int(n.item()) == self.model.compact()
        self.check()

    def check(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), self.model.table)
        assert np.array_equal(self.lens.cpu().numpy(), self.model.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.model.refs)
        assert np.array_equal(self.host(self.k), self.model.pools[0])
        assert np.array_equal(self.host(self.v), self.model.pools[1])
        assert np.array_equal(self.cent.cpu().numpy(), self.model.pools[2])

    def bits(self):
        b = int(self.status.item())
        self.status.zero_()
        return b


@pytest.mark.parametrize("kw", [dict(), dict(layout="hpd"), dict(layout="shard", d=128),
                                dict(layout="pad", hkv=1), dict(mla=True, hkv=1, d=576),
                                dict(hkv=8, d=128)])
def test_a_life_of_the_cache(kw):
    c = Cache([33, 16, 100, 1, 0, 0, 0, 0], 10, 60, **kw)
    c.fork([0, 1, 2, 0], [4, 5, 6, 7])
    c.extend([4, 5, 0, 6], [20, 1, 0, 60])
    c.free([2, 0])
    c.compact()
    c.fork([6, 6], [0, 2])
    assert c.bits() == 0
    c.extend([0, 2, 3], [15, 16, 40])            # rows 0 and 2 fill their table rows already
    assert c.bits() == vt.VT_DEV_BAD_LEN and c.lens[[0, 2, 3]].tolist() == [160, 160, 41]
    c.free([6, 1, 3])
    c.compact()
    c.compact()                                  # nothing left to move
    c.free([0, 2, 4, 5, 7])
    c.compact()                                  # an empty cache
    assert c.bits() == 0


def test_entries_that_are_left_out():
    c = Cache([20, 40, 0, 0, 5], 4, 12)
    c.fork([0, 0, 1, 7, -1, 0, 0, 2], [2, 2, 0, 3, 3, 9, -1, 3])
    assert c.bits() == vt.VT_DEV_BAD_REQ and int(c.lens[3]) == 0
    c.extend([4, 4, 11, -2, 1], [3, 8, 1, 1, 8])
    assert c.bits() == vt.VT_DEV_BAD_REQ
    c.extend([0, 1, 4], [60, -1, 2**31 - 1])
    assert c.bits() == vt.VT_DEV_BAD_LEN
    c.free([3, 40, -1, 0, 0])                    # empty, out of range, twice
    assert c.bits() == vt.VT_DEV_BAD_REQ


def test_too_few_pages():
    c = Cache([20, 40, 17, 0, 0, 0, 0], 8, 12)   # 5 pages are free
    c.extend([3, 4, 5, 6], [33, 40, 16, 0])      # 3, then 3 (not there), then 1 (past them), then 0
    assert c.bits() == vt.VT_DEV_NO_PAGE
    assert c.lens.tolist() == [20, 40, 17, 33, 0, 0, 0]
    c.fork([0, 1, 3, 2], [4, 5, 6, 4])
    assert c.bits() == vt.VT_DEV_NO_PAGE | vt.VT_DEV_BAD_REQ
    assert c.lens.tolist() == [20, 40, 17, 33, 20, 40, 0]
    c.extend([0], [12])                          # fits its last page: needs none
    assert c.bits() == 0


def test_bad_books_are_reported_and_survived():
    c = Cache([40, 33, 0, 20], 4, 20)
    c.table[0, 1] = 99
    c.table[1, 0] = -3
    c.model.table[0, 1], c.model.table[1, 0] = 99, -3
    c.fork([0], [2])
    assert c.bits() == vt.VT_DEV_BAD_PAGE
    c.free([0])
    assert c.bits() == vt.VT_DEV_BAD_PAGE
    c.compact()
    assert c.bits() == vt.VT_DEV_BAD_PAGE
    lost = int(c.table[3, 0])
    c.refs[lost] = 0
    c.model.refs[lost] = 0
    c.free([3])
    assert c.bits() == vt.VT_DEV_BAD_REF
    c.lens[1] = 16 * 4 + 1
    c.model.lens[1] = 16 * 4 + 1
    c.free([1])
    assert c.bits() & vt.VT_DEV_BAD_LEN
    c.lens[2] = 2**31 - 1
    c.model.lens[2] = 2**31 - 1
    c.fork([2], [0])
    assert c.bits() == vt.VT_DEV_BAD_LEN and int(c.lens[0]) == 0
    c.extend([2], [1])
    assert c.bits() == vt.VT_DEV_BAD_LEN


def test_a_page_above_the_cut_without_a_reference_stays():
    c = Cache([16, 16, 16], 2, 9, seed=3)
    c.refs.zero_()
    c.model.refs[:] = 0
    c.compact()                                  # no page is in use: every entry stays
    assert c.bits() == vt.VT_DEV_BAD_REF


@pytest.mark.parametrize("n", [1500, 2048, 2049, 5000])
def test_long_lists(n):
    """Lists longer than a block, and than what a block keeps to itself; rows repeat in them."""
    g = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(0, 30, (n,), generator=g)]
    c = Cache(lens + [0] * n, 4, int(sum(pages_of(x) for x in lens) * 1.6) + 900, hkv=1)
    rows = [int(x) for x in torch.randint(0, n, (n,), generator=g)]
    c.extend(rows, [int(x) for x in torch.randint(0, 20, (n,), generator=g)])
    c.fork([int(x) for x in torch.randint(0, n, (n,), generator=g)], list(range(n, 2 * n)))
    c.free([int(x) for x in torch.randint(0, 2 * n, (n,), generator=g)])
    c.compact()


def test_copy_pages():
    for kw in (dict(), dict(layout="hpd"), dict(mla=True, hkv=1, d=576)):
        c = Cache([16], 1, 40, **kw)
        src, dst = [3, 3, 7, 39, 50, 3], [4, 5, 0, 1, 6, -1]
        vt.vt_copy_pages(c.k, c.v, i32(src), i32(dst), centroids=c.cent, status=c.status)
        for pool in c.model.pools:
            pool[[4, 5, 0, 1]] = pool[[3, 3, 7, 39]]
        c.check()
        assert c.bits() == vt.VT_DEV_BAD_PAGE
        vt.vt_copy_pages(c.k, c.v, i32([]), i32([]))
        vt.vt_copy_pages(c.k, c.v, i32([1]), i32([20]))   # no centroids
        for pool in c.model.pools[:2]:
            pool[20] = pool[1]
        c.check()


@pytest.mark.parametrize("pages", [1, 3, 4095, 4096, 4097, 32768, 32769, 70001])
def test_pools_around_the_scan_shares(pages):
    """Counts alone: the scan's shares and tiles, full, ragged and empty."""
    g = torch.Generator().manual_seed(pages)
    width = 2000
    used = torch.rand(pages, generator=g) < 0.6
    refs = used.int().cuda()
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    free = torch.nonzero(~used).view(-1)
    want = min(width, int(free.numel()))
    vt.vt_extend_requests(table, lens, refs, i32([1, 0]), i32([16 * want, 1]))
    assert torch.equal(table[1, :want].cpu(), free[:want].int())
    assert int(lens[1]) == 16 * want
    assert int(lens[0]) == (1 if free.numel() > want else 0)
    k = torch.arange(pages, device="cuda").to(torch.int32).view(pages, 1, 1, 1)
    k = k.expand(pages, 16, 1, 32).contiguous().view(torch.bfloat16)     # the page's id, as bits
    n = vt.vt_compact_pages(k, k, table, lens, refs)
    ids = k.view(torch.int32)[:, 0, 0, 0]
    n = int(n.item())
    now = (refs > 0).cpu()
    assert n == int(now.sum()) and bool(now[:n].all())
    assert torch.equal(ids[table[1, :want].long()].cpu(), free[:want].int())


def test_a_captured_cycle():
    """Fork, growth, end and compaction in one graph, on one workspace."""
    c = Cache([33, 50, 0, 0], 8, 30)
    parents, children, grow = i32([0, 1]), i32([2, 3]), i32([20, 3])
    ws = vt.page_workspace(30, 2, "cuda")
    ws.fill_(255)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")

    def cycle():
        vt.vt_fork_requests(c.k, c.v, c.table, c.lens, c.refs, parents, children, workspace=ws)
        vt.vt_extend_requests(c.table, c.lens, c.refs, children, grow, workspace=ws)
        vt.vt_compact_pages(c.k, c.v, c.table, c.lens, c.refs, centroids=c.cent, n_used=n,
                            workspace=ws)
        vt.vt_free_requests(c.table, c.lens, c.refs, children)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cycle()
    for _ in range(3):
        g.replay()
        cent = c.model.pools[2].copy()
        c.model.fork([0, 1], [2, 3])
        c.model.pools[2] = cent
        c.model.extend([2, 3], [20, 3])
        assert c.model.compact() == int(n.item())
        c.model.free([2, 3])
        c.check()


def test_random_lives():
    rng = np.random.default_rng(5)
    for seed in range(6):
        c = Cache([int(rng.integers(0, 70)) for _ in range(12)], 8, 70, seed=seed)
        for _ in range(12):
            op = rng.integers(0, 4)
            n = int(rng.integers(1, 9))
            rows = [int(x) for x in rng.integers(-1, 13, n)]
            if op == 0:
                c.fork([int(x) for x in rng.integers(-1, 13, n)], rows)
            elif op == 1:
                c.extend(rows, [int(x) for x in rng.integers(-1, 60, n)])
            elif op == 2:
                c.free(rows[:3])
            else:
                c.compact()


def test_binding_refusals():
    c = Cache([20, 0], 4, 12)
    one = i32([0])
    for call in (
            lambda: vt.vt_fork_requests(c.k, c.v, c.table, c.lens, c.refs, one, i32([0, 1])),
            lambda: vt.vt_fork_requests(c.k, c.v, c.table, c.lens, c.refs[:5], one, i32([1])),
            lambda: vt.vt_extend_requests(c.table, c.lens[:1], c.refs, one, one),
            lambda: vt.vt_extend_requests(c.table, c.lens, c.refs, one.long(), one),
            lambda: vt.vt_free_requests(c.table.t(), c.lens, c.refs, one),
            lambda: vt.vt_copy_pages(c.k, c.v, one, i32([1, 2])),
            lambda: vt.vt_copy_pages(c.k, c.v[:5], one, i32([1])),
            lambda: vt.vt_compact_pages(c.k, c.v, c.table, c.lens, c.refs, centroids=c.cent[:3]),
            lambda: vt.vt_compact_pages(c.k, c.v, c.table, c.lens, c.refs,
                                        workspace=torch.empty(0, dtype=torch.uint8,
                                                              device="cuda"))):
        with pytest.raises(vt.VtError):
            call()
    c.check()
