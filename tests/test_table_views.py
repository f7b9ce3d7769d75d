"""A page table that is some columns of a wider one: its rows have the view's entries, not those of
the stride.  On the host: what the binding hands over, and what the C calls refuse."""
import ctypes

import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from paged_block_sparse_vt_b200 import binding
from paged_block_sparse_vt_b200.build import build
from test_cache_abi import BIG, FAKE, INV, _books, _kv, _prefill, _shared


@pytest.fixture(scope="module")
def lib():
    build()
    return vt.load_library()


@pytest.mark.parametrize("view,want", [
    (lambda t: t, (4, 50, 50)),
    (lambda t: t[:, :40], (4, 50, 40)),
    (lambda t: t[:, 10:], (4, 50, 40)),
    (lambda t: t[::2, 3:4], (2, 100, 1)),
    (lambda t: t[1:2, :40], (1, 40, 40)),          # one row: the stride is nobody's
    (lambda t: t.as_strided((4, 50), (30, 1)), (4, 30, 30)),
])
def test_rows_stride_and_entries(view, want):
    table = torch.zeros((4, 50), dtype=torch.int32)
    assert binding._table(view(table), -1) == want  # (-1: a CPU tensor's device index)


@pytest.mark.parametrize("max_pages", [-1, 65, 1 << 40])
def test_refusals(lib, max_pages):
    for call in (_prefill, _shared):
        rc, need = call(lib, _kv(), dict(max_pages=max_pages))
        assert rc == INV and need == 0 and b"max_pages" in lib.vt_last_error_detail()
    kv, b = ctypes.byref(_kv()), ctypes.byref(_books(max_pages=max_pages))
    assert lib.vt_fork_requests(kv, b, FAKE, FAKE, 3, FAKE, BIG, None) == INV
    assert lib.vt_extend_requests(b, 1000, FAKE, FAKE, 3, FAKE, BIG, None) == INV
    assert lib.vt_free_requests(b, 1000, FAKE, 3, None) == INV
    assert lib.vt_compact_pages(kv, b, None, FAKE, FAKE, BIG, None) == INV


def test_no_entries_given_means_the_stride(lib):
    """0 (what C's initializers leave) and the stride itself: the same call."""
    for call in (_prefill, _shared):
        sizes = {call(lib, _kv(), dict(max_pages=m), out=None)[1] for m in (0, 64)}
        assert len(sizes) == 1 and sizes.pop() > 0
