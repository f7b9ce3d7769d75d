"""Page copies where K and V are views of one pool: every row of either is copied, and nothing
else of the pool."""
import pytest
import torch

import paged_block_sparse_vt_b200 as vt

pytestmark = pytest.mark.gpu

SIDES = {  # dims of a pool's rows of 128 that are K's, and V's
    "v_within_k": (slice(0, 128), slice(0, 64)),
    "k_within_v": (slice(0, 64), slice(0, 128)),
    "the_same": (slice(0, 96), slice(0, 96)),
    "side_by_side": (slice(0, 64), slice(64, 128)),
    "overlapping": (slice(0, 80), slice(40, 104)),
}


@pytest.mark.parametrize("name", list(SIDES))
@pytest.mark.parametrize("heads", [1, 3])
def test_rows_of_one_pool(name, heads):
    kd, vd = SIDES[name]
    pool = torch.randn((12, 16, heads, 128), device="cuda", dtype=torch.bfloat16)
    want = pool.clone()
    for d in (kd, vd):
        want[[2, 9], :, :, d] = pool[[5, 0], :, :, d]
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([5, 0], [2, 9]))
    vt.vt_copy_pages(pool[..., kd], pool[..., vd], src, dst)
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
