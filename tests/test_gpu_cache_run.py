"""The serving-cache calls together, as a server uses them: prompts are admitted and attended,
their pages summarised, samples fork off, everyone decodes token by token (dense over the shared
prompt, and block-sparse beside it), some leave, the pool is compacted, and the rest go on.  What
each call computes is held against the definition in 64 bits over the tokens that each request
really has, which the test keeps in plain lists."""
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_cases import scale_of
from cache_ref import PAGE, check_attend, pages_of

pytestmark = pytest.mark.gpu

P, ROWS, WIDTH, HKV, G, D = 160, 10, 24, 2, 3, 64
HQ, SCALE = HKV * G, scale_of(D)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Server:
    def __init__(self):
        self.gen = torch.Generator(device="cuda").manual_seed(3)
        nan = dict(fill_value=float("nan"), dtype=torch.bfloat16, device="cuda")
        self.k, self.v = (torch.full((P, PAGE, HKV, D), **nan) for _ in range(2))
        self.cent = torch.full((P, HKV, D), float("nan"), device="cuda")
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs = i32([0] * ROWS), i32([0] * P)
        self.status = i32([0])
        self.tokens = {}            # row -> (keys, values) of its tokens, [n, Hkv, D]

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.bfloat16)

    def grow(self, rows, counts):
        """Tokens for these rows: room, then their keys and values, then full pages' centroids."""
        vt.vt_extend_requests(self.table, self.lens, self.refs, i32(rows), i32(counts),
                              status=self.status)
        full = []
        for r, n in zip(rows, counts):
            new = self.randn(n, HKV, D), self.randn(n, HKV, D)
            old = self.tokens.get(r, (new[0][:0], new[1][:0]))
            begin = old[0].shape[0]
            pos = torch.arange(begin, begin + n, device="cuda")
            page = self.table[r].long()[pos // PAGE]
            self.k[page, pos % PAGE], self.v[page, pos % PAGE] = new
            self.tokens[r] = tuple(torch.cat(x) for x in zip(old, new))
            full += self.table[r, begin // PAGE:(begin + n) // PAGE].tolist()
        if full:
            vt.vt_build_centroids(self.k, i32(full), self.cent, status=self.status)

    def reference(self, q, rows, counts):
        """The last ``counts`` tokens of each row over the tokens that the test knows."""
        from cache_ref import attend_ref
        pools, table, at = [[], []], [], 0
        for r in rows:
            n = pages_of(self.tokens[r][0].shape[0])
            for pool, x in zip(pools, self.tokens[r]):
                pad = x.new_zeros((n * PAGE - x.shape[0], HKV, D))
                pool.append(torch.cat([x, pad]).view(n, PAGE, HKV, D))
            table.append(list(range(at, at + n)) + [0] * (WIDTH - n))
            at += n
        lens = [self.tokens[r][0].shape[0] for r in rows]
        return attend_ref(q, torch.cat(pools[0]), torch.cat(pools[1]),
                          torch.tensor(table, device="cuda"), lens, counts, SCALE)

    def prefill(self, rows, counts):
        q = self.randn(sum(counts), HQ, D)
        start = i32([sum(counts[:i]) for i in range(len(rows) + 1)])
        out, lse = vt.vt_prefill(q, self.k, self.v, self.table[rows].contiguous(),
                                 self.lens[rows].contiguous(), start, SCALE, status=self.status)
        check_attend(out, lse, self.reference(q, rows, counts), label=("prefill", rows))

    def decode(self, groups, prefix_pages):
        """One token more for each row of the groups; dense, and the sparse step with a top-k that
        covers every page, which must agree with it."""
        rows = [r for g in groups for r in g]
        self.grow(rows, [1] * len(rows))
        q = self.randn(len(rows), HQ, D)
        table, lens = self.table[rows].contiguous(), self.lens[rows].contiguous()
        start = i32([sum(len(g) for g in groups[:i]) for i in range(len(groups) + 1)])
        out, lse = vt.vt_shared_prefix_decode(q, self.k, self.v, table, lens, start,
                                              i32(prefix_pages), SCALE, status=self.status)
        check_attend(out, lse, self.reference(q, rows, [1] * len(rows)), label=("decode", groups))
        sparse, sparse_lse, _, _ = vt.vt_sparse_decode_fused(
            q, self.k, self.v, table, lens, self.cent, WIDTH, 1, 1, SCALE, status=self.status)
        # (the sparse calls' own tolerances against 64 bits are 1e-2 and 1e-3; twice that)
        assert float((sparse.float() - out.float()).abs().max()) <= 2e-2
        assert float((sparse_lse - lse).abs().max()) <= 2e-3
        # and really sparse: it needs the centroids of middle pages only, moved or not
        few, _, sel, n_sel = vt.vt_sparse_decode_fused(
            q, self.k, self.v, table, lens, self.cent, 2, 1, 1, SCALE, status=self.status,
            sel=torch.empty((len(rows), HKV, 4), dtype=torch.int32, device="cuda"),
            n_sel=torch.empty((len(rows), HKV), dtype=torch.int32, device="cuda"))
        assert bool(torch.isfinite(few).all())
        for i, r in enumerate(rows):
            n = pages_of(self.tokens[r][0].shape[0])
            assert n_sel[i].tolist() == [min(n, 4)] * HKV

    def fork(self, parents, children):
        vt.vt_fork_requests(self.k, self.v, self.table, self.lens, self.refs, i32(parents),
                            i32(children), status=self.status)
        for p, c in zip(parents, children):
            self.tokens[c] = tuple(x.clone() for x in self.tokens[p])

    def free(self, rows):
        vt.vt_free_requests(self.table, self.lens, self.refs, i32(rows), status=self.status)
        for r in rows:
            del self.tokens[r]


def test_a_serving_run():
    s = Server()
    s.grow([0, 1, 2], [130, 33, 48])
    s.prefill([0, 1, 2], [130, 33, 48])
    s.grow([1], [70])                                # a second chunk of prompt 1
    s.prefill([1], [70])
    s.fork([0, 0, 1, 0], [3, 4, 5, 6])               # samples; row 0 goes on as one of them
    for _ in range(3):
        s.decode([[0, 3, 4, 6], [1, 5], [2]], [8, 6, 0])
    s.free([0, 2])                                   # the first sample and a prompt are done
    n = vt.vt_compact_pages(s.k, s.v, s.table, s.lens, s.refs, centroids=s.cent, status=s.status)
    used = int(n.item())
    assert used == int((s.refs > 0).sum()) and bool((s.refs[:used] > 0).all())
    s.k[used:], s.v[used:], s.cent[used:] = (float("nan"),) * 3
    for _ in range(2):
        s.decode([[3, 4, 6], [1, 5]], [8, 6])
    s.grow([0, 2], [40, 17])                         # new requests in the rows that came free
    s.prefill([0, 2], [40, 17])
    s.grow([3], [5])
    s.prefill([3], [5])                              # five drafted tokens of a sample
    s.fork([3, 2], [7, 8])
    s.decode([[3, 7], [4, 6], [1, 5], [2, 8], [0]], [8, 8, 6, 1, 0])
    s.free(list(s.tokens))
    assert int(s.refs.abs().sum()) == 0 and int(s.lens.abs().sum()) == 0
    assert int(s.status.item()) == 0


def test_a_decode_step_of_a_fork_in_one_graph():
    """Growth, the dense decode and the bookkeeping's end captured once and replayed."""
    s = Server()
    s.grow([0], [100])
    rows, ones = i32([1, 2, 3]), i32([1, 1, 1])
    start, prefix = i32([0, 3]), i32([6])
    q = s.randn(3, HQ, D)
    out, lse = torch.empty_like(q), torch.empty(3, HQ, device="cuda")
    table, lens = s.table[1:4], s.lens[1:4]
    ws = vt.page_workspace(P, 3, "cuda")
    attend_ws = vt.shared_prefix_workspace(q, s.k, s.v, table, lens, start, prefix)
    parents = i32([0, 0, 0])
    key = torch.ones((3, HKV, D), dtype=torch.bfloat16, device="cuda")
    value = 2 * key

    def step():
        vt.vt_fork_requests(s.k, s.v, s.table, s.lens, s.refs, parents, rows, status=s.status,
                            workspace=ws)
        vt.vt_extend_requests(s.table, s.lens, s.refs, rows, ones, status=s.status, workspace=ws)
        pos = (lens - 1).long()
        page = table.gather(1, (pos // PAGE)[:, None]).squeeze(1).long()
        s.k[page, pos % PAGE] = key
        s.v[page, pos % PAGE] = value
        vt.vt_shared_prefix_decode(q, s.k, s.v, table, lens, start, prefix, SCALE, out=out,
                                   lse=lse, status=s.status, workspace=attend_ws)
        vt.vt_free_requests(s.table, s.lens, s.refs, rows, status=s.status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    base = s.tokens[0]
    for r in (1, 2, 3):
        s.tokens[r] = torch.cat([base[0], key[:1]]), torch.cat([base[1], value[:1]])
    for _ in range(3):
        q.copy_(s.randn(3, HQ, D))
        g.replay()
        torch.cuda.synchronize()
        check_attend(out, lse, s.reference(q, [1, 2, 3], [1, 1, 1]))
        assert s.refs.sum().item() == pages_of(100) and s.lens.tolist()[1:4] == [0, 0, 0]
    assert int(s.status.item()) == 0
