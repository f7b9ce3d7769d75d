"""The binding's rules for workspaces are those of the C side."""
import ctypes
import os
import random
import re

import pytest

import paged_block_sparse_vt_b200 as vt
from paged_block_sparse_vt_b200 import binding
from paged_block_sparse_vt_b200.build import build
from test_cache_abi import BIG, FAKE, INV, _books, _kv

CSRC = os.path.join(os.path.dirname(os.path.abspath(binding.__file__)), "csrc")


@pytest.fixture(scope="module")
def lib():
    build()
    return vt.load_library()


def test_lists_in_shared_memory(lib):
    with open(os.path.join(CSRC, "pages.cuh")) as f:
        (n,) = re.findall(r"constexpr int kListSmem = (\d+);", f.read())
    assert int(n) == binding.LIST_SMEM
    b = ctypes.byref(_books())
    assert lib.vt_extend_requests(b, 1000, FAKE, FAKE, int(n) + 1, None, 0, None) == INV
    assert b"workspace" in lib.vt_last_error_detail()


def _need(lib, tokens, batch, hkv, group, d, pt_stride, max_pages=0):
    row = hkv * group * d
    kv = _kv(num_kv_heads=hkv, head_dim=d, head_dim_v=d, sk_h=d, sv_h=d, sk_t=hkv * d,
             sv_t=hkv * d, sk_p=16 * hkv * d, sv_p=16 * hkv * d)
    a = binding.PrefillArgs(batch=batch, num_q_heads=hkv * group, num_tokens=tokens, q=FAKE,
                            sq_t=row, q_start=FAKE, page_table=FAKE, pt_stride=pt_stride,
                            seq_lens=FAKE, sm_scale=0.1, status=None, max_pages=max_pages)
    n = lib.vt_prefill_workspace_size(ctypes.byref(kv), ctypes.byref(a))
    rc = lib.vt_prefill(ctypes.byref(kv), ctypes.byref(a), None, None, FAKE, BIG, None)
    assert rc == INV and b"out is NULL" in lib.vt_last_error_detail()  # (sizes that are accepted)
    return n


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_from_there_on_need_the_same(lib, d):
    rng = random.Random(d)
    least = binding.PREFILL_SAME_WS
    sizes = {_need(lib, least, 1, 1, 1, d, 1), _need(lib, least, 1, 1, 1, d, 64, 1),
             _need(lib, 1 << 30, 65536, 8, 8, d, 32768)}
    for _ in range(300):
        pages = rng.randint(1, 32768)
        sizes.add(_need(lib, rng.choice([least, least + rng.randint(0, 5000), 1 << 20]),
                        rng.randint(1, 5000), rng.randint(1, 8), rng.randint(1, 8), d, pages,
                        rng.randint(0, pages)))
    assert len(sizes) == 1 and sizes.pop() > 0
