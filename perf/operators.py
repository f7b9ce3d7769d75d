"""What the operators of a serving cache are measured on: attention over packed prompts in a
paged K/V cache, decode attention for requests that share a prefix of pages, and the cache's
page operations (fork, extend, free, compact).

Every case is a dict of plain sizes; lengths follow from its ``len_seed``, values from the seed
given to ``prepare``.  ``run`` computes the plain form (elementary torch operations in fp32), or,
with ``own`` set, makes the framework's calls.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
CAP = 9.0e12     # flops of the largest listed case; a drawn one stays below it
CAP_BYTES = 3.0e9


def listed():
    return [
        # one short prompt of a small model (the 64-dim head shape): latency
        dict(name="prefill-tiny", op="prefill", B=1, Hq=2, Hkv=1, D=64, q_lo=37, q_hi=37,
             c_lo=0, c_hi=0, len_seed=1),
        # a batch of prompts of very different lengths, packed, as a server admits them
        dict(name="prefill-packed", op="prefill", B=32, Hq=16, Hkv=8, D=128, q_lo=61, q_hi=4096,
             c_lo=0, c_hi=0, len_seed=2),
        # one long document, whole
        dict(name="prefill-long", op="prefill", B=1, Hq=32, Hkv=8, D=128, q_lo=32768, q_hi=32768,
             c_lo=0, c_hi=0, len_seed=3),
        # chunked prompts and a few drafted tokens in one batch, over contexts already cached
        dict(name="prefill-chunked", op="prefill", B=24, Hq=48, Hkv=8, D=128, q_lo=1, q_hi=1024,
             c_lo=1000, c_hi=32768, len_seed=4),
        # four samples of one short prompt on a small model
        dict(name="shared-tiny", op="shared", B=4, Hq=2, Hkv=1, D=64, groups=1, p_lo=20, p_hi=20,
             s_lo=3, s_hi=90, len_seed=5),
        # 32 samples of one prompt, each some hundred tokens along
        dict(name="shared-samples", op="shared", B=32, Hq=16, Hkv=8, D=128, groups=1, p_lo=512,
             p_hi=512, s_lo=64, s_hi=1024, len_seed=6),
        # several system prompts, each with its own users
        dict(name="shared-groups", op="shared", B=128, Hq=32, Hkv=8, D=128, groups=5, p_lo=200,
             p_hi=2048, s_lo=100, s_hi=4096, len_seed=7),
        # a large batch of short questions over one long document
        dict(name="shared-document", op="shared", B=256, Hq=48, Hkv=8, D=128, groups=1, p_lo=4096,
             p_hi=4096, s_lo=17, s_hi=300, len_seed=8),
        # a few samples branch off, grow, and end: bookkeeping and partial pages
        dict(name="fork-few", op="fork", R=16, n=4, pages=1000, Hkv=8, D=128, l_lo=300, l_hi=4000,
             ext_hi=40, len_seed=9),
        # every request of a large batch branches off at once
        dict(name="fork-many", op="fork", R=512, n=256, pages=12000, Hkv=8, D=128, l_lo=100,
             l_hi=1500, ext_hi=100, len_seed=10),
        # a small pool after some requests have left
        dict(name="compact-small", op="compact", R=12, pages=500, Hkv=2, D=64, l_lo=100, l_hi=900,
             len_seed=11),
        # a large pool, half empty, squeezed together
        dict(name="compact-large", op="compact", R=256, pages=24000, Hkv=8, D=128, l_lo=64,
             l_hi=4096, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["prefill", "shared", "fork", "compact"])
    while True:
        hkv = rng.choice([1, 2, 4, 8])
        head = dict(Hq=hkv * rng.randint(1, 8), Hkv=hkv, D=rng.choice([64, 128]))
        seed = rng.randrange(1 << 20)
        if op == "prefill":
            q_hi = _log_int(rng, 1, 32768)
            c_hi = rng.choice([0, _log_int(rng, 1, 32768)])
            case = dict(op=op, B=_log_int(rng, 1, 64), **head, q_lo=max(1, _log_int(rng, 1, q_hi)),
                        q_hi=q_hi, c_lo=min(c_hi, 1), c_hi=c_hi, len_seed=seed)
        elif op == "shared":
            B = _log_int(rng, 1, 256)
            p_hi = _log_int(rng, 1, 4096)
            s_hi = _log_int(rng, 1, 4096)
            case = dict(op=op, B=B, **head, groups=rng.randint(1, min(B, 6)),
                        p_lo=_log_int(rng, 1, p_hi), p_hi=p_hi, s_lo=_log_int(rng, 1, s_hi),
                        s_hi=s_hi, len_seed=seed)
        elif op == "fork":
            R = _log_int(rng, 4, 512)
            l_hi = _log_int(rng, 16, 4000)
            case = dict(op=op, R=R, n=rng.randint(1, R // 2), Hkv=hkv, D=head["D"],
                        l_lo=_log_int(rng, 1, l_hi), l_hi=l_hi, ext_hi=_log_int(rng, 1, 100),
                        len_seed=seed)
            case["pages"] = _fork_pages(case) + rng.randint(0, 300)
        else:
            R = _log_int(rng, 4, 256)
            l_hi = _log_int(rng, 16, 4096)
            case = dict(op=op, R=R, pages=0, Hkv=hkv, D=head["D"], l_lo=_log_int(rng, 1, l_hi),
                        l_hi=l_hi, len_seed=seed)
            case["pages"] = 2 + int(sum(_pages(l) for l in _cache_lens(case, R)) * rng.uniform(1, 2))
        w = work(case)
        if w["flops"] <= CAP and w["bytes"] <= CAP_BYTES:
            return case


# ---- sizes ---------------------------------------------------------------------------------------


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _prefill_lens(case):
    rng = random.Random(case["len_seed"])
    q = [_log_int(rng, case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    c = [_log_int(rng, max(1, case["c_lo"]), case["c_hi"]) if case["c_hi"] else 0 for _ in q]
    return q, c


def _shared_lens(case):
    """(requests, prefix pages) of each group, and each request's own tokens after the prefix."""
    rng = random.Random(case["len_seed"])
    cuts = sorted(rng.sample(range(1, case["B"]), case["groups"] - 1))
    start = [0] + cuts + [case["B"]]
    prefix = [_log_int(rng, case["p_lo"], case["p_hi"]) for _ in range(case["groups"])]
    own_tokens = [_log_int(rng, case["s_lo"], case["s_hi"]) for _ in range(case["B"])]
    return start, prefix, own_tokens


def _cache_lens(case, n):
    rng = random.Random(case["len_seed"])
    return [_log_int(rng, case["l_lo"], case["l_hi"]) for _ in range(n)]


def _fork_lens(case):
    """Lengths of the R - n requests there are, the n parents (repeats among them), the growth."""
    n = case["n"]
    lens = _cache_lens(case, case["R"] - n)
    rng = random.Random(case["len_seed"] + 1)
    parents = [rng.randrange(len(lens)) for _ in range(n)]
    return lens, parents, [rng.randint(1, case["ext_hi"]) for _ in range(n)]


def _fork_pages(case):
    """Pages in use at the peak of a fork case."""
    lens, parents, grow = _fork_lens(case)
    return sum(_pages(l) for l in lens) + sum(
        _pages(lens[p] + g) - lens[p] // PAGE for p, g in zip(parents, grow))


def work(case):
    """What one pass cannot do without."""
    if case["op"] == "prefill":
        q, c = _prefill_lens(case)
        rows = sum(q)
        keys = sum(l * x + l * (l + 1) // 2 for l, x in zip(q, c))
        kv = sum(l + x for l, x in zip(q, c)) * case["Hkv"] * case["D"] * 4
        return dict(bytes=kv + rows * case["Hq"] * (case["D"] * 4 + 4),
                    flops=4 * keys * case["Hq"] * case["D"])
    if case["op"] == "shared":
        start, prefix, tail = _shared_lens(case)
        kv = (sum(prefix) * PAGE + sum(tail)) * case["Hkv"] * case["D"] * 4
        keys = sum((start[g + 1] - start[g]) * p * PAGE for g, p in enumerate(prefix)) + sum(tail)
        return dict(bytes=kv + case["B"] * case["Hq"] * (case["D"] * 4 + 4),
                    flops=4 * keys * case["Hq"] * case["D"])
    page = PAGE * case["Hkv"] * case["D"] * 4
    if case["op"] == "fork":
        lens, parents, grow = _fork_lens(case)
        copied = sum(lens[p] % PAGE != 0 for p in parents)
        entries = sum(_pages(lens[p]) + _pages(lens[p] + g) for p, g in zip(parents, grow))
        return dict(bytes=2 * copied * page + 8 * entries + 4 * case["pages"], flops=entries)
    lens = _cache_lens(case, case["R"])
    used = sum(_pages(l) for l in lens)
    moved = used * (case["pages"] - used) / case["pages"]  # of a random placement
    cent = case["Hkv"] * case["D"] * 4
    return dict(bytes=int(2 * moved * (page + cent)) + 8 * case["pages"] + 8 * used,
                flops=case["pages"])


# ---- inputs --------------------------------------------------------------------------------------


def _pools(pages, hkv, d, gen):
    """K and V pools: N(0, 1) plus an offset for each page and head, as cached keys cluster."""
    pools = []
    for _ in range(2):
        x = torch.randn((pages, PAGE, hkv, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        x += 0.5 * torch.randn((pages, 1, hkv, d), generator=gen, device="cuda",
                               dtype=torch.bfloat16)
        pools.append(x)
    return pools


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case=case, scale=1.0 / math.sqrt(case["D"]))
    hkv, d = case["Hkv"], case["D"]
    if case["op"] in ("prefill", "shared"):
        if case["op"] == "prefill":
            q_lens, ctx = _prefill_lens(case)
            seq = [a + b for a, b in zip(q_lens, ctx)]
            shared = [0] * len(seq)
            owner = list(range(len(seq)))
            s["q_lens"] = q_lens
            s["q_start"] = _ints(np.concatenate([[0], np.cumsum(q_lens)]).tolist())
            rows = sum(q_lens)
        else:
            start, prefix, tail = _shared_lens(case)
            owner = [g for g in range(len(prefix)) for _ in range(start[g + 1] - start[g])]
            shared = [prefix[g] for g in owner]
            seq = [shared[b] * PAGE + t for b, t in enumerate(tail)]
            s.update(start=start, prefix=prefix, tail=tail, group_start=_ints(start),
                     prefix_pages=_ints(prefix))
            rows = case["B"]
        # scattered pages: each owner's shared pages once, then every request's own
        need = sum(s.get("prefix", [])) + sum(_pages(l) - p for l, p in zip(seq, shared))
        P = need + need // 8 + 2
        perm = rng.permutation(P).astype(np.int32)
        at, first = 0, {}
        table = np.full((len(seq), max(_pages(l) for l in seq)), perm[-1], dtype=np.int32)
        for b, l in enumerate(seq):
            if owner[b] not in first:
                first[owner[b]] = perm[at:at + shared[b]]
                at += shared[b]
            mine = _pages(l) - shared[b]
            table[b, :shared[b]] = first[owner[b]]
            table[b, shared[b]:shared[b] + mine] = perm[at:at + mine]
            at += mine
        s["k"], s["v"] = _pools(P, hkv, d, gen)
        s["q"] = 1.5 * torch.randn((rows, case["Hq"], d), generator=gen, device="cuda",
                                   dtype=torch.bfloat16)
        s.update(seq=seq, table=torch.from_numpy(table).cuda(), seq_lens=_ints(seq))
        return s
    # a cache of R rows: some in use, their pages scattered
    P, R = case["pages"], case["R"]
    if case["op"] == "fork":
        lens, parents, grow = _fork_lens(case)
        lens = lens + [0] * case["n"]
        s["parents"], s["grow"] = _ints(parents), _ints(grow)
        s["children"] = _ints(list(range(R - case["n"], R)))
        width = max(_pages(lens[p] + g) for p, g in zip(parents, grow))
        width = max(width, max(_pages(l) for l in lens))
    else:
        lens = _cache_lens(case, R)
        width = max(_pages(l) for l in lens)
    perm = rng.permutation(P).astype(np.int32)
    table = np.full((R, width), -1, dtype=np.int32)
    refs = np.zeros(P, dtype=np.int32)
    at = 0
    for b, l in enumerate(lens):
        n = _pages(l)
        table[b, :n] = perm[at:at + n]
        at += n
    refs[perm[:at]] = 1
    s["k"], s["v"] = _pools(P, hkv, d, gen)
    # what the bookkeeping holds, in one buffer: page table, lengths, reference counts
    s["width"] = width
    s["books0"] = torch.from_numpy(np.concatenate(
        [table.reshape(-1), np.array(lens, dtype=np.int32), refs])).cuda()
    s["books"] = s["books0"].clone()
    if case["op"] == "compact":
        s["cent"] = torch.randn((P, hkv, d), generator=gen, device="cuda")
    return s


def _books(s, buf):
    R, W = s["case"]["R"], s["width"]
    return buf[:R * W].view(R, W), buf[R * W:R * W + R], buf[R * W + R:]


# ---- one pass ------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if op == "prefill":
        if own:
            import paged_block_sparse_vt_b200 as vt
            return vt.vt_prefill(state["q"], state["k"], state["v"], state["table"],
                                 state["seq_lens"], state["q_start"], state["scale"])
        return _plain_prefill(state)
    if op == "shared":
        if own:
            import paged_block_sparse_vt_b200 as vt
            return vt.vt_shared_prefix_decode(
                state["q"], state["k"], state["v"], state["table"], state["seq_lens"],
                state["group_start"], state["prefix_pages"], state["scale"])
        return _plain_shared(state)
    # every pass starts from the same books; what it copies goes to the same pages again
    state["books"].copy_(state["books0"])
    table, lens, refs = _books(state, state["books"])
    if op == "fork":
        if own:
            import paged_block_sparse_vt_b200 as vt
            vt.vt_fork_requests(state["k"], state["v"], table, lens, refs, state["parents"],
                                state["children"])
            vt.vt_extend_requests(table, lens, refs, state["children"], state["grow"])
            grown = lens.clone()
            vt.vt_free_requests(table, lens, refs, state["parents"])
        else:
            _plain_fork(state["k"], state["v"], table, lens, refs, state["parents"],
                        state["children"])
            _plain_extend(table, lens, refs, state["children"], state["grow"])
            grown = lens.clone()
            _plain_free(table, lens, refs, state["parents"])
        return state["k"], state["v"], table, grown, lens, refs
    if own:
        import paged_block_sparse_vt_b200 as vt
        used = vt.vt_compact_pages(state["k"], state["v"], table, lens, refs,
                                   centroids=state["cent"])
    else:
        used = _plain_compact(state["k"], state["v"], table, lens, refs, state["cent"])
    return state["k"], state["v"], state["cent"], table, refs, used


def _attend(q, k, v, visible, scale):
    """q [n, Hkv, G, D], k / v [m, Hkv, D], visible [n, m] or None: the unnormalised fp32 parts
    (row maximum, row sum, weighted values) with rows [Hkv, n, G]."""
    n, hkv, g, d = q.shape
    z = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, n * g, d), k.permute(1, 2, 0)) * scale
    z = z.view(hkv, n, g, -1)
    if visible is not None:
        z.masked_fill_(~visible[None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m).exp_()
    o = torch.matmul(p.view(hkv, n * g, -1), v.permute(1, 0, 2)).view(hkv, n, g, -1)
    return m, p.sum(-1, keepdim=True), o


def _plain_prefill(s):
    c = s["case"]
    hkv, g, d = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    row = 0
    for b, (n, l) in enumerate(zip(s["q_lens"], s["seq"])):
        pages = s["table"][b, :_pages(l)].long()
        k = s["k"][pages].reshape(-1, hkv, d).float()
        v = s["v"][pages].reshape(-1, hkv, d).float()
        step = max(16, (1 << 28) // (c["Hq"] * l))
        for i in range(0, n, step):
            j = min(n, i + step)
            end = l - n + j
            pos = torch.arange(l - n + i, end, device="cuda")
            seen = torch.arange(end, device="cuda")[None, :] <= pos[:, None]
            q = s["q"][row + i:row + j].float().view(j - i, hkv, g, d)
            m, t, o = _attend(q, k[:end], v[:end], seen, s["scale"])
            out[row + i:row + j] = (o / t).permute(1, 0, 2, 3).reshape(j - i, -1, d)
            lse[row + i:row + j] = (m + t.log()).squeeze(-1).permute(1, 0, 2).reshape(j - i, -1)
        row += n
    return out, lse


def _plain_shared(s):
    """The prefix of a group once for all its rows; the requests' own tokens as one padded batch."""
    c = s["case"]
    hkv, g, d = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    q = s["q"].float().view(-1, hkv, g, d)
    parts = []
    for i, p in enumerate(s["prefix"]):
        pages = s["table"][s["start"][i], :p].long()
        parts.append(_attend(q[s["start"][i]:s["start"][i + 1]],
                             s["k"][pages].reshape(-1, hkv, d).float(),
                             s["v"][pages].reshape(-1, hkv, d).float(), None, s["scale"]))
    m1, t1, o1 = (torch.cat(x, 1).transpose(0, 1) for x in zip(*parts))   # [B, Hkv, G, ...]
    most = max(_pages(t) for t in s["tail"])
    span = torch.arange(most, device="cuda")
    first = torch.repeat_interleave(s["prefix_pages"], s["group_start"].diff(),
                                    output_size=c["B"]).long()
    outs, lses = [], []
    step = max(1, (1 << 27) // (most * PAGE * hkv * d))
    for i in range(0, c["B"], step):
        j = min(c["B"], i + step)
        at = (first[i:j, None] + span).clamp_(max=s["table"].shape[1] - 1)
        pages = s["table"][i:j].gather(1, at).long()
        k = s["k"][pages].reshape(j - i, -1, hkv, d).float()
        v = s["v"][pages].reshape(j - i, -1, hkv, d).float()
        z = torch.matmul(q[i:j], k.permute(0, 2, 3, 1)) * s["scale"]
        left = s["seq_lens"][i:j] - first[i:j] * PAGE
        z.masked_fill_((torch.arange(z.shape[-1], device="cuda") >= left[:, None])[:, None, None],
                       -math.inf)
        m = torch.maximum(m1[i:j], z.amax(-1, keepdim=True))
        p = (z - m).exp()
        a = (m1[i:j] - m).exp()
        t = p.sum(-1, keepdim=True) + a * t1[i:j]
        o = torch.matmul(p, v.transpose(1, 2)) + a * o1[i:j]
        outs.append((o / t).reshape(j - i, -1, d))
        lses.append((m + t.log()).reshape(j - i, -1))
    return torch.cat(outs).to(torch.bfloat16), torch.cat(lses)


def _lowest_free(refs, count):
    """The ids of the ``count`` lowest pages that nothing refers to."""
    rank = torch.cumsum(refs == 0, 0)
    return torch.searchsorted(rank, torch.arange(1, count + 1, device="cuda"))


def _plain_fork(k, v, table, lens, refs, parents, children):
    p, c = parents.long(), children.long()
    l = lens[p]
    at = torch.arange(table.shape[1], device="cuda")
    table[c] = torch.where(at < ((l + PAGE - 1) // PAGE)[:, None], table[p], table[c])
    lens[c] = l
    full = at < (l // PAGE)[:, None]
    refs.index_add_(0, torch.where(full, table[p], 0).long().view(-1), full.int().view(-1))
    # a partly filled last page is copied to a page of its own; a full one has no copy to make
    part = l % PAGE != 0
    rank = (torch.cumsum(part, 0) - 1).clamp_(min=0)
    fresh = _lowest_free(refs, p.numel()).clamp_(max=refs.numel() - 1)[rank]
    last = ((l - 1) // PAGE).long()[:, None]
    old = table[p].gather(1, last).squeeze(1).long()
    new = torch.where(part, fresh, old)
    table[c] = table[c].scatter(1, last, new.int()[:, None])
    refs.index_add_(0, new, part.int())
    k[new] = k[old]
    v[new] = v[old]


def _plain_extend(table, lens, refs, requests, tokens):
    r = requests.long()
    l = lens[r]
    have, want = (l + PAGE - 1) // PAGE, (l + tokens + PAGE - 1) // PAGE
    base = torch.cumsum(want - have, 0) - (want - have)
    at = torch.arange(table.shape[1], device="cuda")
    new = (at >= have[:, None]) & (at < want[:, None])
    rank = (base[:, None] + at - have[:, None]).clamp_(0, refs.numel() - 1).long()
    free = _lowest_free(refs, refs.numel()).clamp_(max=refs.numel() - 1)
    page = free[rank]
    table[r] = torch.where(new, page.int(), table[r])
    refs.index_add_(0, torch.where(new, page, 0).view(-1), new.int().view(-1))
    lens[r] = l + tokens


def _plain_free(table, lens, refs, requests):
    # a request that is listed twice is freed once
    hit = torch.zeros_like(lens).index_fill_(0, requests.long(), 1)
    at = torch.arange(table.shape[1], device="cuda")
    gone = (at < (hit * ((lens + PAGE - 1) // PAGE))[:, None])
    refs.index_add_(0, torch.where(gone, table, 0).long().view(-1), -gone.int().view(-1))
    lens.mul_(1 - hit)


def _plain_compact(k, v, table, lens, refs, cent):
    """The used pages above the count of used pages go, in order, to the free ones below it."""
    P = refs.numel()
    used = (refs > 0)
    n = used.sum()
    ids = torch.arange(P, device="cuda")
    high, low = used & (ids >= n), ~used & (ids < n)
    rank = torch.arange(1, P + 1, device="cuda")
    src = torch.searchsorted(torch.cumsum(high, 0), rank)
    dst = torch.searchsorted(torch.cumsum(low, 0), rank)
    moves = rank <= high.sum()
    src = torch.where(moves, src, P)   # entry P stands for "no move"
    dst = torch.where(moves, dst, P)
    new_id = torch.arange(P + 1, device="cuda").scatter_(0, src, dst)[:P]
    old_id = torch.arange(P + 1, device="cuda").scatter_(0, dst, src)[:P]
    for pool in (k, v, cent):
        pool.copy_(pool[old_id])
    count = torch.where(ids < n, refs[old_id], 0)
    refs.copy_(count)
    at = torch.arange(table.shape[1], device="cuda")
    live = at < ((lens + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(live, new_id[table.clamp(min=0).long()].int(), table))
    return n.int().view(1)


# ---- the definition in 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_rows(s, s["q_lens"])
    if case["op"] == "shared":
        return _exact_rows(s, [1] * case["B"])
    return _exact_fork(s) if case["op"] == "fork" else _exact_compact(s)


def _exact_rows(s, q_lens):
    """Every request by itself, one KV head after the other: its q_lens[b] rows are its last."""
    hq, hkv = s["case"]["Hq"], s["case"]["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device="cuda")
    begin = 0
    for b, (n, length) in enumerate(zip(q_lens, s["seq"])):
        used = s["table"][b].long()[:_pages(length)]
        for h in range(hkv):
            keys = s["k"][used, :, h].flatten(0, 1)[:length].double()
            values = s["v"][used, :, h].flatten(0, 1)[:length].double()
            heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
            for i in range(0, n, 1024):
                rows = slice(begin + i, begin + min(n, i + 1024))
                x = torch.einsum("ngd,md->gnm", s["q"][rows, heads].double(), keys) * s["scale"]
                if n > 1:
                    hide = torch.ones(x.shape[1:], dtype=torch.bool, device="cuda")
                    x.masked_fill_(hide.triu(length - n + i + 1), -math.inf)
                lse[rows, heads] = torch.logsumexp(x, -1).t()
                x = torch.softmax(x, -1)
                out[rows, heads] = torch.einsum("gnm,md->ngd", x, values)
        begin += n
    return out, lse


def _host_books(s):
    return [x.cpu().numpy().copy() for x in _books(s, s["books0"])]


def _exact_fork(s):
    table, lens, refs = _host_books(s)
    k, v = s["k"], s["v"]
    old, new = [], []
    for p, c in zip(s["parents"].tolist(), s["children"].tolist()):
        full, rest = divmod(int(lens[p]), PAGE)
        table[c, :full] = table[p, :full]
        np.add.at(refs, table[p, :full], 1)
        if rest:
            page = int(np.argmin(refs != 0))
            old.append(int(table[p, full]))
            new.append(page)
            table[c, full] = page
            refs[page] = 1
        lens[c] = lens[p]
    for pool in (k, v):
        pool[new] = pool[old].clone()
    for r, t in zip(s["children"].tolist(), s["grow"].tolist()):
        for slot in range(_pages(int(lens[r])), _pages(int(lens[r]) + t)):
            table[r, slot] = np.argmin(refs != 0)
            refs[table[r, slot]] = 1
        lens[r] += t
    grown = lens.copy()
    for r in sorted(set(s["parents"].tolist())):
        np.add.at(refs, table[r, :_pages(int(lens[r]))], -1)
        lens[r] = 0
    return (k, v) + tuple(torch.from_numpy(x).cuda() for x in (table, grown, lens, refs))


def _exact_compact(s):
    table, lens, refs = _host_books(s)
    n = int((refs > 0).sum())
    src = [p for p in range(n, refs.size) if refs[p] > 0]
    dst = [p for p in range(n) if refs[p] == 0]
    for pool in (s["k"], s["v"], s["cent"]):
        pool[dst] = pool[src].clone()
    moved = dict(zip(src, dst))
    for b, l in enumerate(lens):
        for i in range(_pages(int(l))):
            table[b, i] = moved.get(int(table[b, i]), table[b, i])
    refs[dst] = refs[src]
    refs[src] = 0
    return (s["k"], s["v"], s["cent"]) + tuple(
        torch.from_numpy(x).cuda() for x in (table, refs, np.array([n], dtype=np.int32)))
