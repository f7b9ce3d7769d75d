"""Plain 64-bit forms of the serving-cache operators, and the error bounds the tests hold the
kernels to.  Attention by its definition, one request and KV head at a time (torch fp64, on the
inputs' device); the page operations as a numpy model of the books.

The bounds count the roundings there are: the weights and the output are rounded once to bf16
(half a step, 2^-8 relative each), everything else is fp32.
"""
import math

import numpy as np
import torch

PAGE = 16


def pages_of(n):
    return (n + PAGE - 1) // PAGE


def attend_ref(q, k_pool, v_pool, page_table, seq_lens, q_lens, scale, bad_pages=()):
    """Row i of the q_lens[b] rows of request b sees tokens 0 .. seq_lens[b] - q_lens[b] + i, but
    for those on a page of ``bad_pages[b]`` (logical indices).

    Returns (out, lse, out_bound, lse_bound) in fp64, rows packed.  With z = scale q.k computed
    in fp32 (D products and sums: |dz| <= eps := scale (D + 8) 2^-24 sum_d |q_d k_d|), weights
    w = exp(z) off by 2 eps relative to their sum, exponentials and sums good to 2^-16:
      |d out| <= 2^-8 |out| + (2^-8 + 2 eps + 2^-15) sum_j w_j |V_j|,
      |d lse| <= eps + 2^-16 + 2^-22 |lse|.
    """
    hq, d = q.shape[1:]
    hkv = k_pool.shape[2]
    g = hq // hkv
    n_rows = sum(q_lens)
    f64 = dict(dtype=torch.float64, device=q.device)
    out, bound = torch.zeros((n_rows, hq, d), **f64), torch.zeros((n_rows, hq, d), **f64)
    lse, lbound = torch.full((n_rows, hq), -math.inf, **f64), torch.zeros((n_rows, hq), **f64)
    row = 0
    for b, n in enumerate(q_lens):
        length = int(seq_lens[b])
        idx = page_table[b, :pages_of(length)].long()
        bad = list(bad_pages[b]) if bad_pages else []
        idx[bad] = 0
        gone = torch.zeros(length, dtype=torch.bool, device=q.device)
        for i in bad:
            gone[PAGE * i:PAGE * (i + 1)] = True
        for h in range(hkv if n else 0):
            k = k_pool[idx, :, h].reshape(-1, d)[:length].double()
            v = v_pool[idx, :, h].reshape(-1, d)[:length].double()
            v[gone] = 0.0
            for r0 in range(0, n, 512):
                rows = slice(row + r0, row + min(n, r0 + 512))
                x = q[rows, h * g:(h + 1) * g].double()
                z = torch.einsum("rgd,kd->rgk", x, k) * scale
                pos = length - n + r0 + torch.arange(x.shape[0], device=q.device)
                hide = (torch.arange(length, device=q.device)[None] > pos[:, None]) | gone[None]
                z.masked_fill_(hide[:, None], -math.inf)
                eps = torch.einsum("rgd,kd->rgk", x.abs(), k.abs()).masked_fill_(
                    hide[:, None], 0.0).amax(-1) * scale * (d + 8) * 2.0 ** -24
                m = z.amax(-1, keepdim=True)
                p = (z - torch.where(m == -math.inf, 0.0, m)).exp()
                total = p.sum(-1, keepdim=True)
                p = p / torch.where(total == 0, 1.0, total)
                o = torch.einsum("rgk,kd->rgd", p, v)
                mass = torch.einsum("rgk,kd->rgd", p, v.abs())
                heads = slice(h * g, (h + 1) * g)
                out[rows, heads] = o
                lse[rows, heads] = torch.where(total == 0, -math.inf, m + total.log()).squeeze(-1)
                bound[rows, heads] = 2.0 ** -8 * o.abs() + mass * (
                    2.0 ** -8 + 2.0 ** -15 + 2 * eps[..., None])
                lbound[rows, heads] = eps + 2.0 ** -16 + 2.0 ** -22 * torch.where(
                    total == 0, 0.0, m + total.log()).squeeze(-1).abs()
        row += n
    return out, lse, bound, lbound


def check_attend(got_out, got_lse, ref, label=""):
    out, lse, bound, lbound = ref
    o = got_out.double()
    assert torch.isfinite(o).all(), label
    over = (o - out).abs() - bound
    assert (over <= 1e-30).all(), (label, "out", float(over.max()), int((over > 0).sum()))
    if got_lse is not None:
        empty = lse == -math.inf
        x = got_lse.double()
        assert torch.equal(x == -math.inf, empty), (label, "empty rows")
        over = ((x - lse).abs() - lbound)[~empty]
        assert over.numel() == 0 or (over <= 0).all(), (label, "lse", float(over.max()))


class Books:
    """The page operations by their rules, one entry after the other, on numpy arrays; ``pools``
    are arrays [P, ...] whose rows are copied with the pages."""

    def __init__(self, table, lens, refs, *pools):
        self.table, self.lens, self.refs = (np.array(x, dtype=np.int32) for x in (table, lens, refs))
        self.pools = [np.array(x) for x in pools]
        self.width = self.table.shape[1]

    def free_pages(self):
        return list(np.flatnonzero(self.refs <= 0))

    def _take(self, targets, valid, need):
        """The pages of each entry: None where it is left out."""
        free = self.free_pages()
        taken, seen, at = [], set(), 0
        for t, ok, n in zip(targets, valid, need):
            if not ok or t in seen:
                taken.append(None)
                continue
            seen.add(t)
            # the running count goes on over the entries that found too little
            taken.append(free[at:at + n] if n == 0 or at + n <= len(free) else None)
            at += n
        return taken

    def fork(self, parents, children):
        lens, rows = self.lens.copy(), len(self.lens)
        valid = [0 <= p < rows and 0 <= c < rows and lens[c] == 0 and lens[p] > 0 and
                 pages_of(int(lens[p])) <= self.width for p, c in zip(parents, children)]
        need = [int(ok and lens[p] % PAGE != 0) for ok, p in zip(valid, parents)]
        for p, c, pages in zip(parents, children, self._take(children, valid, need)):
            if pages is None:
                continue
            full = int(lens[p]) // PAGE
            self.table[c, :full] = self.table[p, :full]
            for x in self.table[p, :full]:
                if 0 <= x < len(self.refs):
                    self.refs[x] += 1
            for x in pages:
                old = self.table[p, full]
                self.table[c, full] = x
                self.refs[x] = 1
                for pool in self.pools:
                    if 0 <= old < len(self.refs):
                        pool[x] = pool[old]
            self.lens[c] = lens[p]

    def extend(self, requests, tokens):
        lens, rows = self.lens.copy(), len(self.lens)
        valid = [0 <= r < rows and lens[r] >= 0 and t >= 0 and
                 int(lens[r]) + t <= PAGE * self.width for r, t in zip(requests, tokens)]
        need = [pages_of(int(lens[r]) + t) - pages_of(int(lens[r])) if ok else 0
                for ok, r, t in zip(valid, requests, tokens)]
        for r, t, pages in zip(requests, tokens, self._take(requests, valid, need)):
            if pages is None:
                continue
            have = pages_of(int(lens[r]))
            self.table[r, have:have + len(pages)] = pages
            self.refs[pages] = 1
            self.lens[r] += t

    def free(self, requests):
        for r in requests:
            if 0 <= r < len(self.lens) and self.lens[r] > 0:
                for x in self.table[r, :min(self.width, pages_of(int(self.lens[r])))]:
                    if 0 <= x < len(self.refs) and self.refs[x] > 0:
                        self.refs[x] -= 1
                self.lens[r] = 0

    def compact(self):
        used = int((self.refs > 0).sum())
        src = [x for x in range(used, len(self.refs)) if self.refs[x] > 0]
        dst = [x for x in range(used) if self.refs[x] <= 0]
        for pool in self.pools:
            pool[dst] = pool[src]
        to = dict(zip(src, dst))
        for b, n in enumerate(self.lens):
            for i in range(min(self.width, pages_of(max(0, int(n))))):
                self.table[b, i] = to.get(int(self.table[b, i]), self.table[b, i])
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0
        return used
