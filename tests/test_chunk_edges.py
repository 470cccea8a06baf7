"""Ragged chunks at the edges of what their calls allow: maps that are part of a wider matrix."""
import pytest
import torch

import paged_kv_mla_create_b200 as mla
from test_chunk import Batch, gpu


def as_columns(batch, first, cols, behind):
    """The batch's req_to_token as columns [first, first + cols) of a wider matrix of -7; returns that matrix."""
    rows = batch.r2t.shape[0]
    big = torch.full((rows, first + cols + behind), -7, dtype=torch.int32, device="cuda")
    have = min(cols, batch.r2t.shape[1])
    big[:, first:first + have] = batch.r2t[:, :have]
    batch.r2t = big[:, first:first + cols]
    return big


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("first,behind", [(0, 100), (512, 0), (64, 7)])
def test_metadata_on_some_columns_of_a_wider_map(first, behind, given):
    """A view whose columns hold every position gives the same maps, and its neighbours keep their entries."""
    b = Batch([500, 0, 64], [60, 130, 1], seed=3, pad=2, given=given)
    big = as_columns(b, first, b.width * 64, behind)
    b.check(b.maps())
    inside = torch.zeros_like(big, dtype=torch.bool)
    inside[:, first:first + b.width * 64] = True
    assert bool((big[~inside] == -7).all())


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("cols", [512, 500, 540, 1])
def test_positions_past_a_views_columns_have_no_slot(cols, given):
    """Requests longer than the view (the matrix's last row among them): reported, slot -1, nothing written outside."""
    b = Batch([500, 20, 30], [60, 600, 3], seed=4, given=given, width=12)
    b.rpi = torch.tensor([2, 5, 0], device="cuda")   # 5: the last row
    for r in range(3):   # the map's rows follow the requests'
        keep = b.L[r] if given else b.prefix[r]
        b.r2t[int(b.rpi[r])] = -7
        b.r2t[int(b.rpi[r]), :keep] = torch.tensor(b.slots[r][:keep], dtype=torch.int32, device="cuda")
    big = as_columns(b, 256, cols, 0)
    before = big.clone()
    bt, seqlens, cu, pos, loc, plan, taken = b.maps()
    assert mla.read_device_error() == 4
    assert seqlens.tolist() == b.L and cu.tolist() == [0, 60, 660, 663]
    got, table, at = loc.tolist(), bt.tolist(), 0
    for r in range(3):
        pages = min(-(-b.L[r] // 64), -(-cols // 64))
        assert [x >= 0 for x in table[r]] == [p < pages for p in range(b.width)], r
        for i in range(b.chunk[r]):
            p = b.prefix[r] + i
            slot = got[at + i]
            assert slot == (table[r][p // 64] * 64 + p % 64 if p < cols else -1), (r, p)
            if p < cols:
                assert int(big[int(b.rpi[r]), 256 + p]) == slot
                before[int(b.rpi[r]), 256 + p] = slot
        at += b.chunk[r]
    assert torch.equal(big, before)


def test_view_validation_happens_before_any_launch():
    f = mla.library().mla_build_chunk_metadata_view
    args = [1 << 20, 5, 192, 64, 1 << 21, 3, 1 << 22, 1 << 23, 2, 2, 9, None, 0, 16, 1, 74, 1 << 24, 3, 3, 64, 1, -1, 1 << 25, 1 << 26,
            1 << 27, 1 << 28, 1 << 29, None, None]
    for at, value in ((1, 0), (2, 0), (3, -1), (4, None), (14, 2), (17, 2)):
        assert f(*args[:at], value, *args[at + 1:]) == 1, at
