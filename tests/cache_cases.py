"""Small seeded caches for the serving-cache tests."""
import math

import torch

from cache_ref import PAGE, pages_of


def make_pools(pages, hkv, d, seed=0, layout="phd", device="cuda"):
    """K and V pools [P, 16, Hkv, D].  layout "phd": contiguous; "hpd": heads before tokens in
    memory; "shard": a view of every second head of a wider pool; "pad": rows with a gap."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g, device=device, dtype=torch.bfloat16)

    pools = []
    for _ in range(2):
        if layout == "phd":
            pools.append(draw(pages, PAGE, hkv, d))
        elif layout == "hpd":
            pools.append(draw(pages, hkv, PAGE, d).transpose(1, 2))
        elif layout == "shard":
            pools.append(draw(pages, PAGE, 2 * hkv, d)[:, :, ::2])
        else:
            pools.append(draw(pages, PAGE, hkv, d + 8)[..., :d])
    return pools


def make_cache(seq_lens, hkv, d, seed=0, layout="phd", poison=True, shared=None, width=None):
    """Scattered pages for requests of these lengths.  ``shared``: (group_start, prefix_pages),
    whose requests have their group's first pages in common.  ``poison``: NaN and infinities in
    every pool slot that belongs to no token."""
    owner = list(range(len(seq_lens)))
    lead = [0] * len(seq_lens)
    if shared:
        for g, n in enumerate(shared[1]):
            for b in range(shared[0][g], shared[0][g + 1]):
                owner[b], lead[b] = shared[0][g], n
    need = sum(pages_of(l) for l in seq_lens) + 3
    gen = torch.Generator().manual_seed(seed + 1)
    perm = torch.randperm(need, generator=gen).to(torch.int32)
    width = width or max(1, max(pages_of(l) for l in seq_lens))
    table = torch.full((len(seq_lens), width), int(perm[-1]), dtype=torch.int32)
    at = 0
    for b, l in enumerate(seq_lens):
        n = pages_of(l)
        first = lead[b] if owner[b] != b else 0
        table[b, :first] = table[owner[b], :first]
        table[b, first:n] = perm[at:at + n - first]
        at += n - first
    k, v = make_pools(need, hkv, d, seed, layout)
    if poison:
        live = torch.zeros((need, PAGE), dtype=torch.bool)
        for b, l in enumerate(seq_lens):
            n = pages_of(l)
            for i in range(n):
                live[int(table[b, i]), :min(PAGE, l - PAGE * i)] = True
        k[~live.cuda()] = float("nan")
        v[~live.cuda()] = float("inf")
    return k, v, table.cuda(), torch.tensor(seq_lens, dtype=torch.int32, device="cuda")


def make_q(rows, hq, d, seed=0, gain=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    return gain * torch.randn((rows, hq, d), generator=g, device="cuda", dtype=torch.bfloat16)


def starts(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)) if len(lens) else [0],
                        dtype=torch.int32, device="cuda")


def scale_of(d):
    return 1.0 / math.sqrt(d)
