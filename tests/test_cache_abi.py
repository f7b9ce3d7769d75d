"""Refusals of the serving-cache calls on the host: fake, aligned addresses that must never be
touched, because every call here ends in its argument checks (or has nothing to do)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from cache_ref import Books
from paged_block_sparse_vt_b200 import binding
from paged_block_sparse_vt_b200.build import build

OK, INV, UNS = 0, 1, 2
FAKE = 0x7F0000000000
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    build()
    return vt.load_library()


def _kv(**over):
    f = dict(k_pool=FAKE, v_pool=FAKE + 0x100000, num_pages=1000, page_size=16, num_kv_heads=8,
             head_dim=128, head_dim_v=128, sk_p=16 * 8 * 128, sk_t=8 * 128, sk_h=128,
             sv_p=16 * 8 * 128, sv_t=8 * 128, sv_h=128)
    f.update(over)
    return binding.PagedKV(**f)


_MLA = dict(num_kv_heads=1, head_dim=576, head_dim_v=512, v_pool=FAKE, sk_h=576, sv_h=576,
            sk_p=16 * 576, sv_p=16 * 576, sk_t=576, sv_t=576)
# faults that both attention calls refuse
_COMMON = [
    (dict(page_size=8), {}, UNS),
    (dict(k_pool=None), {}, INV),
    (dict(num_pages=0), {}, INV),
    (dict(v_pool=FAKE + 8), {}, UNS),
    (dict(head_dim=96, head_dim_v=96), {}, UNS),
    (dict(head_dim=128, head_dim_v=64), {}, UNS),
    (_MLA, dict(num_q_heads=32), UNS),
    (dict(sk_t=8 * 128 + 4), {}, UNS),
    (dict(sk_p=0), {}, UNS),                    # one page repeated
    (dict(sv_h=0), {}, UNS),                    # one head repeated
    (dict(sk_p=1 << 39), {}, UNS),
    ({}, dict(num_q_heads=30), INV),
    ({}, dict(num_q_heads=72), UNS),
    (dict(num_kv_heads=32768, sk_h=128, sv_h=128), dict(num_q_heads=32768, sq_t=1 << 23), UNS),
    ({}, dict(batch=-1), INV),
    ({}, dict(batch=65537), UNS),
    ({}, dict(batch=0), OK),
    ({}, dict(pt_stride=0), UNS),
    ({}, dict(pt_stride=40000), UNS),
    ({}, dict(sm_scale=0.0), INV),
    ({}, dict(sm_scale=-0.1), INV),
    ({}, dict(sm_scale=float("inf")), INV),
    ({}, dict(sm_scale=float("nan")), INV),
    ({}, dict(sm_scale=3e38), INV),             # times log2 e it leaves fp32
    ({}, dict(q=None), INV),
    ({}, dict(q=FAKE + 0x200008), UNS),
    ({}, dict(page_table=None), INV),
    ({}, dict(seq_lens=None), INV),
]


def _prefill(lib, kv, over, out=FAKE + 0x600000, ws=FAKE + 0x8000000, ws_bytes=BIG):
    f = dict(batch=4, num_q_heads=32, num_tokens=100, q=FAKE + 0x200000, sq_t=32 * 128,
             q_start=FAKE + 0x300000, page_table=FAKE + 0x310000, pt_stride=64,
             seq_lens=FAKE + 0x400000, sm_scale=0.088, status=None)
    f.update(over)
    a = binding.PrefillArgs(**f)
    need = lib.vt_prefill_workspace_size(ctypes.byref(kv), ctypes.byref(a))
    return lib.vt_prefill(ctypes.byref(kv), ctypes.byref(a), out, None, ws, ws_bytes, None), need


def _shared(lib, kv, over, out=FAKE + 0x600000, ws=FAKE + 0x8000000, ws_bytes=BIG):
    f = dict(batch=4, num_q_heads=32, num_groups=2, q=FAKE + 0x200000, group_start=FAKE + 0x300000,
             prefix_pages=FAKE + 0x305000, page_table=FAKE + 0x310000, pt_stride=64,
             seq_lens=FAKE + 0x400000, sm_scale=0.088, status=None)
    f.update(over)
    f.pop("sq_t", None)
    a = binding.SharedPrefixArgs(**f)
    need = lib.vt_shared_prefix_workspace_size(ctypes.byref(kv), ctypes.byref(a))
    return lib.vt_shared_prefix_decode(ctypes.byref(kv), ctypes.byref(a), out, None, ws, ws_bytes,
                                       None), need


@pytest.mark.parametrize("kv_over,over,code", _COMMON + [
    ({}, dict(num_tokens=-1), INV),
    ({}, dict(num_tokens=(1 << 30) + 1), UNS),
    ({}, dict(num_tokens=0), OK),
    ({}, dict(sq_t=32 * 128 - 8), UNS),
    ({}, dict(sq_t=32 * 128 + 4), UNS),
    ({}, dict(sq_t=1 << 39), UNS),
    ({}, dict(q_start=None), INV),
])
def test_prefill_refusals(lib, kv_over, over, code):
    rc, need = _prefill(lib, _kv(**kv_over), over)
    assert rc == code and need == 0
    assert (code == OK) or lib.vt_last_error_detail()


@pytest.mark.parametrize("kv_over,over,code", _COMMON + [
    ({}, dict(num_groups=-1), INV),
    ({}, dict(num_groups=65537), UNS),
    ({}, dict(num_groups=0), OK),
    ({}, dict(group_start=None), INV),
    ({}, dict(prefix_pages=None), INV),
])
def test_shared_prefix_refusals(lib, kv_over, over, code):
    rc, need = _shared(lib, _kv(**kv_over), over)
    assert rc == code and need == 0
    assert (code == OK) or lib.vt_last_error_detail()


@pytest.mark.parametrize("call", [_prefill, _shared])
def test_attention_output_and_workspace_refusals(lib, call):
    _, need = call(lib, _kv(), {}, out=None)
    assert need > 0
    assert call(lib, _kv(), {}, out=None)[0] == INV
    assert call(lib, _kv(), {}, out=FAKE + 8)[0] == UNS
    assert call(lib, _kv(), {}, ws=None)[0] == INV
    assert call(lib, _kv(), {}, ws_bytes=need - 1)[0] == INV
    assert b"workspace" in lib.vt_last_error_detail()
    assert call(lib, _kv(), {}, ws=FAKE + 16)[0] == INV
    # one CTA's work needs none
    assert _prefill(lib, _kv(num_kv_heads=1), dict(num_q_heads=2, batch=1, num_tokens=7, sq_t=256,
                                                   pt_stride=4), out=None) == (INV, 0)
    assert lib.vt_prefill(ctypes.byref(_kv()), None, FAKE, None, FAKE, BIG, None) == INV
    assert lib.vt_shared_prefix_decode(None, None, FAKE, None, FAKE, BIG, None) == INV


def _books(**over):
    f = dict(rows=10, page_table=FAKE, pt_stride=64, seq_lens=FAKE + 0x1000, refs=FAKE + 0x2000,
             status=None)
    f.update(over)
    return binding.PageBooks(**f)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INV), (dict(page_table=None), INV), (dict(seq_lens=None), INV),
    (dict(refs=None), INV), (dict(pt_stride=0), UNS), (dict(pt_stride=40000), UNS)])
def test_page_books_refusals(lib, over, code):
    kv, b = ctypes.byref(_kv()), ctypes.byref(_books(**over))
    assert lib.vt_fork_requests(kv, b, FAKE, FAKE, 3, FAKE, BIG, None) == code
    assert lib.vt_extend_requests(b, 1000, FAKE, FAKE, 3, FAKE, BIG, None) == code
    assert lib.vt_free_requests(b, 1000, FAKE, 3, None) == code
    assert lib.vt_compact_pages(kv, b, None, FAKE, FAKE, BIG, None) == code


def test_page_call_refusals(lib):
    kv, b = ctypes.byref(_kv()), ctypes.byref(_books())
    need = lib.vt_page_workspace_size(1000, 3)
    assert need >= 4 * 3 * 1000 and need % 256 == 0
    assert lib.vt_page_workspace_size(0, 3) == 0 and lib.vt_page_workspace_size(1000, -1) == 0
    for ws, size in ((None, BIG), (FAKE, need - 1), (FAKE + 16, BIG)):
        assert lib.vt_fork_requests(kv, b, FAKE, FAKE, 3, ws, size, None) == INV
        # (up to 2048 rows grow without a workspace)
        assert lib.vt_extend_requests(b, 1000, FAKE, FAKE, 2049, ws, size, None) == INV
    assert lib.vt_compact_pages(kv, b, None, FAKE, None, BIG, None) == INV
    assert lib.vt_compact_pages(kv, b, None, None, FAKE, BIG, None) == INV
    assert lib.vt_compact_pages(kv, b, FAKE + 4, FAKE, FAKE, BIG, None) == UNS
    for n, code in ((-1, INV), (0, OK)):
        assert lib.vt_fork_requests(kv, b, None, None, n, None, 0, None) == code
        assert lib.vt_extend_requests(b, 1000, None, None, n, None, 0, None) == code
        assert lib.vt_free_requests(b, 1000, None, n, None) == code
        assert lib.vt_copy_pages(kv, None, None, n, None, None, None) == code
    assert lib.vt_fork_requests(kv, b, None, FAKE, 3, FAKE, BIG, None) == INV
    assert lib.vt_extend_requests(b, 1000, FAKE, None, 3, FAKE, BIG, None) == INV
    assert lib.vt_extend_requests(b, 0, FAKE, FAKE, 3, FAKE, BIG, None) == INV
    assert lib.vt_extend_requests(b, 1 << 31, FAKE, FAKE, 3, FAKE, BIG, None) == UNS
    assert lib.vt_free_requests(b, 1000, None, 3, None) == INV
    assert lib.vt_copy_pages(kv, None, FAKE, 3, None, None, None) == INV
    assert lib.vt_copy_pages(kv, FAKE, FAKE, 3, FAKE + 8, None, None) == UNS
    odd = ctypes.byref(_kv(head_dim=100, head_dim_v=100))
    assert lib.vt_copy_pages(odd, FAKE, FAKE, 3, None, None, None) == UNS


def test_binding_refuses_cpu_tensors():
    i32 = dict(dtype=torch.int32)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    table, one = torch.zeros(1, 2, **i32), torch.ones(1, **i32)
    start, refs = torch.zeros(2, **i32), torch.zeros(4, **i32)
    for call in (lambda: vt.vt_prefill(q, pool, pool, table, one, start, 0.1),
                 lambda: vt.vt_shared_prefix_decode(q[:1], pool, pool, table, one, start, one, 0.1),
                 lambda: vt.vt_copy_pages(pool, pool, one, one),
                 lambda: vt.vt_fork_requests(pool, pool, table, one, refs, one, one),
                 lambda: vt.vt_extend_requests(table, one, refs, one, one),
                 lambda: vt.vt_free_requests(table, one, refs, one),
                 lambda: vt.vt_compact_pages(pool, pool, table, one, refs)):
        with pytest.raises(vt.VtError):
            call()


def test_model_of_the_books_by_hand():
    """The numpy model itself, on a cache small enough to follow by hand."""
    pool = np.arange(8)[:, None] * 10.0
    b = Books([[5, 2, 7], [0, -1, -1], [-1] * 3, [-1] * 3], [40, 16, 0, 0],
              [1, 0, 1, 0, 0, 1, 0, 1], pool)
    b.fork([0, 1, 0, 3], [2, 3, 2, 0])        # row 2 once; row 3 was empty, row 0 in use
    assert b.table.tolist() == [[5, 2, 7], [0, -1, -1], [5, 2, 1], [0, -1, -1]]
    assert b.lens.tolist() == [40, 16, 40, 16]
    assert b.refs.tolist() == [2, 1, 2, 0, 0, 2, 0, 1] and b.pools[0][1, 0] == 70
    b.extend([3, 1], [17, 40])                # 2 pages, then 3 wanted of 1 left
    assert b.table[3].tolist() == [0, 3, 4] and b.lens.tolist() == [40, 16, 40, 33]
    b.free([0, 3, 0])
    assert b.lens.tolist() == [0, 16, 40, 0] and b.refs.tolist() == [1, 1, 1, 0, 0, 1, 0, 0]
    assert b.compact() == 4
    assert b.table[2].tolist() == [3, 2, 1] and b.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert b.pools[0][3, 0] == 50
