"""Compaction of books in which a live entry's page has no reference: the entry stays and is
reported, wherever its page is."""
import numpy as np
import pytest
import torch

import paged_block_sparse_vt_b200 as vt
from test_gpu_pages import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [40, 20000])   # one CTA's plan, and a cluster's
@pytest.mark.parametrize("where", ["below", "above"])
def test_an_entry_without_a_reference_stays_and_is_reported(where, pages):
    c = Cache([16 * 6, 16 * 3, 0, 16 * 2], 7, pages, hkv=1, seed=pages)
    used = c.table[c.table >= 0].cpu().numpy()
    # every used page but one counts; the cut is then at 10
    c.table[0, :6] = torch.arange(0, 12, 2, dtype=torch.int32, device="cuda")
    c.table[1, :3] = torch.tensor([pages - 1, 5, pages - 9], dtype=torch.int32, device="cuda")
    c.table[3, :2] = torch.tensor([1, pages - 3], dtype=torch.int32, device="cuda")
    c.refs.zero_()
    live = c.table[c.table >= 0].long()
    assert live.numel() == used.size == 11 and live.unique().numel() == 11
    c.refs[live] = 1
    lost = 4 if where == "below" else pages - 9
    c.refs[lost] = 0
    c.model.table[:] = c.table.cpu().numpy()
    c.model.refs[:] = c.refs.cpu().numpy()
    c.compact()
    assert c.bits() == vt.VT_DEV_BAD_REF
    assert int((c.table == lost).sum()) == (2 if where == "below" else 1)
    c.refs[lost] = 1              # (below the cut it is the place of a page that moved)
    c.model.refs[lost] = 1
    c.compact()
    assert c.bits() == 0 and np.array_equal(c.table.cpu().numpy(), c.model.table)
