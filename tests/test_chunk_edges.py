"""Ragged chunks at the edges of what their calls allow: maps that are part of a wider matrix, lengths other than the
plan's, more new tokens than rows, buffers that do not fit."""
import os
import subprocess
import sys
import types

import pytest
import torch

import paged_kv_mla_create_b200 as mla
from test_chunk import SCALE, Batch, assert_attention, gpu, make_cache, reference


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


@gpu
@pytest.mark.parametrize("cols", [512, 540])
def test_table_builders_read_a_views_own_columns_alone(cols):
    """The decode calls' tables of a map that is part of a wider matrix: a length past its columns is reported and
    cut off there, in the last row too; lengths within them give what a copy of the view gives."""
    big = torch.full((5, 200 + cols), 640, dtype=torch.int32, device="cuda")   # a page that is no request's
    view = big[:, 200:]
    view[:] = 64 * (torch.arange(5, device="cuda")[:, None] * 9 + torch.arange(cols, device="cuda") // 64) + torch.arange(
        cols, device="cuda") % 64
    rpi = torch.tensor([4, 0, 2], device="cuda")
    width, reach = 11, -(-cols // 64)
    for lens, code in (([cols, 1, 130], 0), ([700, 700, 64], 4)):
        sl = torch.tensor(lens, device="cuda")
        want = [[9 * r + p if p < min(reach, -(-n // 64)) else -1 for p in range(width)] for r, n in zip([4, 0, 2], lens)]
        assert mla.build_block_table(view, rpi, sl, width).tolist() == want and mla.read_device_error() == code
        bt, seqlens, _, _ = mla.build_decode_metadata(view, rpi, sl, width, 16)
        assert bt.tolist() == want and seqlens.tolist() == lens and mla.read_device_error() == code
        kept = torch.full((3, width), 77, dtype=torch.int32, device="cuda")
        mla.build_block_table(view, rpi, sl, width, out=kept, fill_tail=False)
        assert kept.tolist() == [[77 if x < 0 else x for x in row] for row in want] and mla.read_device_error() == code
    cache = torch.randn(45, 64, 576, device="cuda").bfloat16()
    q, k_new = torch.randn(3, 2, 16, 576, device="cuda").bfloat16(), torch.randn(3, 2, 576, device="cuda").bfloat16()
    sl = torch.tensor([cols, 1, 130], dtype=torch.int32, device="cuda")
    got = mla.extend_paged_prefix(q, k_new, cache, view, rpi, sl, width, SCALE)
    same = mla.extend_paged_prefix(q, k_new, cache, view.contiguous(), rpi, sl, reach, SCALE)
    assert mla.read_device_error() == 0 and torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    mla.extend_paged_prefix(q, k_new, cache, view, rpi, sl + 200, width, SCALE)
    assert mla.read_device_error() & 4


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cut,width", [
    ([500, 9030, 103], None), ([0, 20, 1], None), ([129, 640, 0], None), ([39000, 8000, 103], None), ([40001, 9040, 103], 5),
    ([384, 385, 64], 9),
])
def test_lengths_below_those_of_the_plan(cut, width, causal, kv):
    """A plan that cuts long requests over many parts, used with shorter lengths or a narrower table: cuts past a
    unit's last key leave nothing to merge.  The workspace is NaN: a piece that this call did not write shows."""
    b = Batch([40000, 9000, 100], [1, 40, 3], seed=3)
    h = 128
    bt, _, cu, _, _, plan, _ = b.maps(h, causal=causal)
    cache, scale, values = make_cache(b, kv, 5)
    q = torch.randn(b.rows, h, 576, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    ws = torch.full((mla.chunk_workspace_bytes(mla.num_chunk_parts()),), 255, dtype=torch.uint8, device="cuda")
    lens = torch.tensor(cut, dtype=torch.int32, device="cuda")
    table = bt if width is None else bt[:, :width]
    o, lse = mla.mla_chunk_paged(q, cache, table, lens, cu, 512, plan, SCALE, causal, descale_k=scale, workspace=ws)
    assert mla.read_device_error() == 0
    at = 0
    for r, n in enumerate(b.chunk):
        L = cut[r]
        cap = L if width is None else min(L, 64 * width)
        keys = values[torch.tensor(b.slots[r][:cap], device="cuda", dtype=torch.long)]
        for i in range(n):   # a token at a time: its limit may lie past the table
            lim = max(0, min(cap, L - n + i + 1 if causal else L))
            ro, rl, pv, ds = reference(q[at + i:at + i + 1], keys[:lim], False)
            assert_attention(o[at + i:at + i + 1], lse[at + i:at + i + 1], ro, rl, pv, ds, lim, kv, float(values.abs().max()))
        at += n


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("rows", [0, 3, 20, 62, 63, 64, 150, 254])
def test_tokens_past_the_batchs_rows_do_not_count(rows, given):
    """More new tokens than rows: reported, and the maps, lengths and pages are those of the tokens that have one."""
    b = Batch([10, 100, 64, 0], [3, 60, 1, 191], seed=5, given=given)
    whole = b.chunk
    b.rows = rows
    bt, seqlens, cu, pos, loc, plan, taken = out = b.maps()
    assert mla.read_device_error() == 4
    kept, left = [], rows
    for n in whole:
        kept.append(min(n, left))
        left -= kept[-1]
    L = [p + n for p, n in zip(b.prefix, kept)]
    assert seqlens.tolist() == L and cu.tolist() == [sum(kept[:i]) for i in range(5)]
    total = [-(-x // 64) for x in L]
    assert bt.tolist() == [[b.slots[r][64 * p] // 64 for p in range(total[r])] + [-1] * (b.width - total[r]) for r in range(4)]
    assert loc.tolist() == [s for r in range(4) for s in b.slots[r][b.prefix[r]:L[r]]]
    assert pos.tolist() == [p for r in range(4) for p in range(b.prefix[r], L[r])]
    assert given or int(taken) == sum(t - -(-p // 64) for t, p in zip(total, b.prefix))
    for r in range(4):
        row = b.r2t[int(b.rpi[r])].tolist()
        assert row[:L[r]] == b.slots[r][:L[r]] and (given or set(row[L[r]:]) <= {-7})
    if rows == 0:
        assert bool((plan == torch.tensor([4, 0, 0, 4, 0, 0, 0, 0], device="cuda")).all())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_of_a_batch_whose_tokens_were_cut_off(kv):
    """The rows that are there see the keys up to their own; rows of the dropped tokens hold NaN."""
    b = Batch([3000, 500, 64], [40, 300, 9], seed=6)
    h, rows = 64, 200
    b.rows = rows
    bt, seqlens, cu, _, _, plan, _ = b.maps(h)
    assert mla.read_device_error() == 4
    kept = [40, 160, 0]
    b.slots = [s[:p + n] for s, p, n in zip(b.slots, b.prefix, kept)]   # the others are no request's: NaN
    cache, scale, values = make_cache(b, kv, 7)
    q = torch.randn(rows, h, 576, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    assert mla.read_device_error() == 0
    at = 0
    for r, n in enumerate(kept):
        if n:
            keys = values[torch.tensor(b.slots[r], device="cuda")]
            ro, rl, pv, ds = reference(q[at:at + n], keys, True)
            assert_attention(o[at:at + n], lse[at:at + n], ro, rl, pv, ds, keys.shape[0], kv, float(keys.abs().max()))
        at += n


@gpu
def test_a_plan_buffer_of_other_rows_is_refused():
    """A plan has a row for each part: rows behind the last would be run as parts by the attention."""
    b = Batch([30, 0], [5, 7], seed=3)
    parts = mla.num_chunk_parts()
    out = list(b.maps())
    for rows, kw in ((parts + 1, {}), (100, {}), (parts - 1, {}), (parts, dict(num_parts=3)), (3, {})):
        out[5] = torch.zeros(rows, 8, dtype=torch.int32, device="cuda")
        with pytest.raises(ValueError, match="chunk_plan"):
            b.maps(out=tuple(out), **kw)
    out[5] = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    assert b.maps(out=tuple(out), num_parts=3)[5] is out[5]
    assert mla.read_device_error() == 0


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("parts", [1, 74])
def test_a_bad_page_reads_as_zeros(parts, kv):
    """A page outside the pool is reported and counts as 64 rows of zeros (scores and values), wherever it lies."""
    b = Batch([1300, 100], [5, 40], seed=3)
    h = 16
    bt, seqlens, cu, _, _, plan, _ = b.maps(h, num_parts=parts)
    cache, scale, values = make_cache(b, kv, 1)
    q = torch.randn(b.rows, h, 576, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    for bad, pages in ((-1, [1]), (b.pool, [0, 7]), (2**31 - 1, [20]), (-2**31, [2, 3])):
        t = bt.clone()
        t[0, pages] = bad
        o, lse = mla.mla_chunk_paged(q, cache, t, seqlens, cu, 512, plan, SCALE, descale_k=scale)
        assert mla.read_device_error() == 1
        at = 0
        for r, n in enumerate(b.chunk):
            keys = values[torch.tensor(b.slots[r], device="cuda")]
            if r == 0:
                for p in pages:
                    keys[64 * p:64 * p + 64] = 0
            ro, rl, pv, ds = reference(q[at:at + n], keys, True)
            assert_attention(o[at:at + n], lse[at:at + n], ro, rl, pv, ds, b.L[r], kv, float(keys.abs().max()))
            at += n


@gpu
@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
def test_8_bit_pages_past_four_gigabytes(kv):
    """Byte offsets past 32 bits in an 8-bit pool, whose rows come by other loads than a bf16 one's."""
    b = Batch([500, 70], [20, 3], seed=4)
    shift = 120000   # pages of 36,864 bytes
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, scale, _ = make_cache(b, kv, 5)
    big = torch.full((shift + b.pool, 64, 576), 0x7F, dtype=torch.uint8, device="cuda")   # NaN
    big[shift:] = cache.view(torch.uint8)
    q = torch.randn(b.rows, 16, 576, device="cuda").bfloat16()
    table = torch.where(bt >= 0, bt + shift, bt)
    o, lse = mla.mla_chunk_paged(q, big.view(cache.dtype), table, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    o2, lse2 = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    assert mla.read_device_error() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    assert bool(torch.isfinite(o).all())


@gpu
@pytest.mark.parametrize("n", [1, 5, 70])
def test_agrees_with_the_extend_call(n):
    """A uniform chunk gives what extend_paged_prefix gives.  With u, ds, pv as for the 64-bit tests, the ragged call is
    off by (u + 2 ds) pv + 2^-8 |o|.  The extend call's two parts are off by as much each, weighted to one, with
    |o_part| <= pv_part (so 2^-8 pv for their roundings), their weights by a relative 2 ds and 2^-18 for the
    exponentials, and its result by 2^-8 |o|.  The extend call takes finite pools only, the ragged one any tail rows."""
    b = Batch([1000, 63, 2500, 0], [n] * 4, seed=6)
    h = 16
    bt, seqlens, cu, _, _, plan, _ = b.maps(h)
    cache, _, values = make_cache(b, "bf16", 7)
    q = torch.randn(b.rows, h, 576, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE)
    new = torch.stack([cache.view(-1, 576)[torch.tensor(s[p:], device="cuda")] for s, p in zip(b.slots, b.prefix)])
    finite = torch.nan_to_num(cache, nan=3.0)
    o2, lse2 = mla.extend_paged_prefix(q.view(4, n, h, 576), new, finite, b.r2t, b.rpi, b.prefix_t, 40, SCALE)
    assert mla.read_device_error() == 0
    for r in range(4):
        at = r * n
        ro, rl, pv, ds = reference(q[at:at + n], values[torch.tensor(b.slots[r], device="cuda")], True)
        u = 2.0**-8
        tol = 2 * (u + 2 * ds) * pv + (u + 2 * ds + 2.0**-18) * pv + 2 * u * ro.abs()
        assert bool(((o[at:at + n].double() - o2[r].double()).abs() <= tol).all())
        assert bool(((lse[at:at + n] - lse2[r]).abs() <= 2 * (ds + b.L[r] * 2.0**-24) + 2.0**-20 * (1 + rl.abs())).all())


@gpu
def test_a_workspace_that_is_not_memory_of_its_size_is_refused():
    b = Batch([300, 70], [5, 40], seed=3)
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, _, _ = make_cache(b, "bf16", 1)
    q = torch.randn(b.rows, 16, 576, device="cuda").bfloat16()
    need = mla.chunk_workspace_bytes(mla.num_chunk_parts())
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need), torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, workspace=ws)
    assert mla.read_device_error() == 0


def test_view_validation_happens_before_any_launch():
    f = mla.library().mla_build_chunk_metadata_view
    args = [1 << 20, 5, 192, 64, 1 << 21, 3, 1 << 22, 1 << 23, 2, 2, 9, None, 0, 16, 1, 74, 1 << 24, 3, 3, 64, 1, -1, 1 << 25, 1 << 26,
            1 << 27, 1 << 28, 1 << 29, None, None]
    for at, value in ((1, 0), (2, 0), (3, -1), (4, None), (14, 2), (17, 2)):
        assert f(*args[:at], value, *args[at + 1:]) == 1, at


@gpu
def test_a_device_by_any_of_its_names():
    for device in (None, 0, "cuda", "cuda:0", torch.device("cuda"), torch.device("cuda", 0)):
        assert mla.read_device_error(device) == 0


def test_the_current_stream_is_found_by_any_name_of_the_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(mla, "_raw_stream", lambda index: 1000 + index)
    for device, index in ((0, 0), (2, 2), ("cuda:1", 1), ("cuda", 3), (torch.device("cuda"), 3), (torch.device("cuda", 2), 2)):
        assert mla._stream(device).value == 1000 + index


def test_the_current_stream_without_the_private_call():
    """A torch without the private name: the public call takes its place."""
    code = ("import types, torch; torch._C.__dict__.pop('_cuda_getCurrentRawStream', None)\n"
            "torch.cuda.current_stream = lambda index: types.SimpleNamespace(cuda_stream=500 + index)\n"
            "import paged_kv_mla_create_b200 as mla; assert mla._stream(7).value == 507")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_device_zero_is_not_the_current_device(monkeypatch):
    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "get_device_properties",
                        lambda d: asked.append(d) or types.SimpleNamespace(multi_processor_count=148 if d == 0 else 20))
    mla._device_parts.cache_clear()
    assert mla._device_parts(0) == 74 and mla._device_parts(3) == 10 and mla.sm_count() == 20
    assert asked == [0, 3, 3]
    mla._device_parts.cache_clear()
