"""Ragged chunks over the paged cache: build_chunk_metadata (page table, lengths, offsets, positions,
slots, split plan) against its definition, entry by entry, and mla_chunk_paged against attention
computed in 64 bits from the same rows.

Tolerances.  Let p be the probabilities, v the value rows, u = finfo(P's type).eps / 2 (bf16 2^-8,
f16 2^-11 for 8-bit caches).  The kernel rounds each p once to P's type (relative u) and o once to
bf16 (2^-8); a score is a sum of 576 exact products in fp32, off by at most 576 * 2^-24 * sum |q k| *
scale =: ds (plus 2^-22 for exp2, 2^-24 a step in the sums, counted in ds), which moves a probability
by a relative 2 ds (numerator and sum).  So |o - ref| <= (u + 2 ds) sum_j p_j |v_j| + 2^-8 |o|; an f16
P below 2^-14 is off by up to 2^-25 instead, at most L 2^-25 max|v| over a row.  lse is off by at
most ds + L 2^-24 + 2^-22 |lse|."""
import math
import random

import pytest
import torch

import paged_kv_mla_create_b200 as mla

SCALE = 1.0 / math.sqrt(192.0)
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
gpu = pytest.mark.gpu


def cdiv(a, b):
    return -(-a // b)


class Batch:
    """A ragged batch: request b has prefix[b] cached tokens on pages of a shuffled pool and brings
    chunk[b] new ones; slots[b] are the slots its tokens must get (new pages in free-list order)."""

    def __init__(self, prefix, chunk, seed=0, pad=0, index=torch.int64, lens=torch.int64, width=None, extra_cols=0,
                 given=False):
        g = torch.Generator().manual_seed(seed)
        self.prefix, self.chunk, self.pad = list(prefix), list(chunk), pad
        self.bs = len(prefix)
        self.L = [p + n for p, n in zip(prefix, chunk)]
        self.total, have = [cdiv(x, 64) for x in self.L], [cdiv(p, 64) for p in prefix]
        self.width = width or max([1] + self.total)
        self.pool = max(4, sum(self.total) + 3)
        perm = torch.randperm(self.pool, generator=g)
        rows = self.bs + 3
        rpi = torch.randperm(rows, generator=g)[:self.bs]
        r2t = torch.full((rows, self.width * 64 + extra_cols), -7, dtype=torch.int32)
        own = self.total if given else have
        at, self.slots = 0, []
        for b in range(self.bs):
            pages = perm[at:at + own[b]]
            at += own[b]
            self.slots.append((pages[:, None] * 64 + torch.arange(64)).reshape(-1)[:self.L[b] if given else prefix[b]].tolist())
        free = perm[at:].tolist()
        for b in range(self.bs):
            r2t[rpi[b], :len(self.slots[b])] = torch.tensor(self.slots[b], dtype=torch.int32)
        self.taken = 0
        if not given:
            for b in range(self.bs):
                for pos in range(prefix[b], self.L[b]):
                    if pos % 64 == 0:
                        self.slots[b].append(free[self.taken] * 64)
                        self.taken += 1
                    else:
                        self.slots[b].append(self.slots[b][-1] + 1)
        self.r2t, self.rpi = r2t.cuda(), rpi.to(index).cuda()
        self.free = None if given else torch.tensor(free, dtype=index).cuda()
        self.prefix_t = torch.tensor(self.prefix, dtype=lens).cuda()
        self.chunk_t = torch.tensor(self.chunk, dtype=lens).cuda()
        self.tokens = sum(chunk)
        self.rows = self.tokens + pad

    def maps(self, h=16, **kw):
        return mla.build_chunk_metadata(self.r2t, self.rpi, self.prefix_t, self.chunk_t, self.rows, self.width, h,
                                        free_pages=self.free, **kw)

    def check(self, out, pad_slot=-1):
        bt, seqlens, cu, pos, loc, plan, taken = out
        assert mla.read_device_error() == 0
        assert seqlens.tolist() == self.L
        assert cu.tolist() == [sum(self.chunk[:b]) for b in range(self.bs + 1)]
        table = bt.cpu()
        for b in range(self.bs):
            want = [self.slots[b][64 * p] // 64 for p in range(self.total[b])]
            assert table[b, :self.width].tolist() == want + [-1] * (self.width - self.total[b]), b
        assert loc.tolist() == [s for b in range(self.bs) for s in self.slots[b][self.prefix[b]:]] + [pad_slot] * self.pad
        assert pos.tolist() == [p for b in range(self.bs) for p in range(self.prefix[b], self.L[b])] + [0] * self.pad
        r2t = self.r2t.cpu()
        for b in range(self.bs):
            row = r2t[int(self.rpi[b])]
            assert row[:self.L[b]].tolist() == self.slots[b] and bool((row[self.L[b]:] == -7).all())
        assert (taken is None) if self.free is None else int(taken) == self.taken


def make_cache(batch, kv, seed, poison=True):
    """The pool (every row that no request owns NaN) and the rows' values in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(batch.pool * 64, 576, generator=g, device="cuda")
    scale = None
    if kv == "bf16":
        cache = x.bfloat16()
        values = cache.double()
    else:
        scale = (x.abs().max() / TOP[kv]).reshape(1)
        cache = (x / scale).clamp(-TOP[kv], TOP[kv]).to(DTYPE[kv])
        values = cache.double() * scale.double()
    if poison:
        dead = torch.ones(batch.pool * 64, dtype=torch.bool)
        for s in batch.slots:
            dead[torch.tensor(s, dtype=torch.long)] = False
        if kv == "bf16":
            cache[dead.cuda()] = float("nan")
        else:
            cache.view(torch.uint8)[dead.cuda()] = 0x7F
    return cache.view(batch.pool, 64, 576), scale, values


def reference(q, keys, causal):
    """o, lse, sum_j p_j |v_j| and the score error ds of n tokens, the last of keys' rows, in 64 bits."""
    n, L = q.shape[0], keys.shape[0]
    q = q.double()
    s = torch.einsum("nhd,kd->nhk", q, keys) * SCALE
    ds = 576 * 2.0**-24 * float((q.abs().reshape(-1, 576) @ keys.abs().t()).max()) * SCALE + 2.0**-20 if L else 0.0
    if causal:
        lim = L - n + torch.arange(n, device=q.device) + 1
        s = s.masked_fill((torch.arange(L, device=q.device)[None] >= lim[:, None])[:, None], -math.inf)
    lse = torch.logsumexp(s, -1) if L else torch.full(q.shape[:2], -math.inf, device=q.device, dtype=torch.double)
    p = torch.nan_to_num(torch.exp(s - lse[..., None]), nan=0.0)
    v = keys[:, :512]
    return torch.einsum("nhk,kd->nhd", p, v), lse, torch.einsum("nhk,kd->nhd", p, v.abs()), ds


def assert_attention(o, lse, ro, rl, pv, ds, L, kv, vmax):
    u = 2.0**-8 if kv == "bf16" else 2.0**-11
    tol = (u + 2 * ds) * pv + 2.0**-8 * ro.abs() + (0.0 if kv == "bf16" else L * 2.0**-25 * vmax) + 1e-9
    assert bool(((o.double() - ro).abs() <= tol).all()), float(((o.double() - ro).abs() / tol).max())
    dead = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), dead)
    err = (lse.double() - rl).abs()[~dead]
    assert bool((err <= (ds + L * 2.0**-24 + 2.0**-22 * rl.abs()[~dead])).all()), float(err.max())


def run_attention(batch, h, kv="bf16", causal=True, parts=None, seed=0, workspace=None):
    maps = batch.maps(h, causal=causal, num_parts=parts)
    cache, scale, values = make_cache(batch, kv, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(batch.rows, h, 576, generator=g, device="cuda").bfloat16()
    q[batch.tokens:] = float("nan")
    o = torch.full((batch.rows, h, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.rows, h), 7.0, device="cuda")
    bt, seqlens, cu, _, _, plan, _ = maps
    mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, causal, descale_k=scale, out=o, lse=lse,
                        workspace=workspace)
    assert mla.read_device_error() == 0
    return q, values, o, lse


def check_attention(batch, h, kv="bf16", causal=True, parts=None, seed=0, workspace=None):
    q, values, o, lse = run_attention(batch, h, kv, causal, parts, seed, workspace)
    vmax = float(values.abs().max())
    at = 0
    for b, n in enumerate(batch.chunk):
        if n:
            keys = values[torch.tensor(batch.slots[b], device="cuda")]
            for i in range(0, n, 256):   # blocks of tokens bound the reference's scores
                m = min(256, n - i)
                qi = q[at + i:at + i + m]
                ks = keys[:batch.L[b] - n + i + m] if causal else keys
                ro, rl, pv, ds = reference(qi, ks, causal)
                assert_attention(o[at + i:at + i + m], lse[at + i:at + i + m], ro, rl, pv, ds, batch.L[b], kv, vmax)
        at += n
    # rows of no request stay as they were
    assert bool((o[at:] == 7).all()) and bool((lse[at:] == 7).all())
    return o, lse


# ------------------------------------------------------------------------------- metadata
METADATA = [
    ([0], [1]), ([0], [64]), ([64], [1]), ([63], [1]), ([65], [0]), ([0, 0], [0, 0]), ([1, 127, 128, 129], [0, 1, 64, 65]),
    ([30, 0, 64, 63, 0, 500, 1], [5, 130, 0, 2, 0, 1, 63]), ([2000] * 40, [1] * 40), ([100], [5000]),
]


@gpu
@pytest.mark.parametrize("prefix,chunk", METADATA)
@pytest.mark.parametrize("given", [False, True])
def test_metadata_matches_its_definition(prefix, chunk, given):
    for index, lens in ((torch.int32, torch.int64), (torch.int64, torch.int32)):
        b = Batch(prefix, chunk, seed=len(prefix), pad=3, index=index, lens=lens, extra_cols=13, given=given)
        b.check(b.maps(pad_slot=-1))


@gpu
def test_metadata_random_batches():
    rng = random.Random(5)
    for s in range(40):
        bs = rng.choice([1, 2, 9, 33, 300])
        top = rng.choice([10, 300, 3000])
        prefix = [rng.choice([0, 1, 63, 64, 65, rng.randrange(top)]) for _ in range(bs)]
        chunk = [rng.choice([0, 1, 1, 64, rng.randrange(1, 200)]) for _ in range(bs)]
        b = Batch(prefix, chunk, seed=s, pad=rng.choice([0, 1, 1500]), given=rng.random() < 0.4)
        b.check(b.maps(h=rng.choice([1, 16, 128]), pad_slot=5), pad_slot=5)


@gpu
def test_metadata_of_the_largest_batch_and_of_none():
    rng = random.Random(6)
    b = Batch([rng.randrange(200) for _ in range(4096)], [rng.choice([0, 1, 2, 70]) for _ in range(4096)], seed=7)
    b.check(b.maps())
    e = Batch([], [], pad=4, width=2)
    bt, seqlens, cu, pos, loc, plan, taken = e.maps(h=128)
    assert cu.tolist() == [0] and loc.tolist() == [-1] * 4 and int(taken) == 0 and bt.shape == (0, 2)
    assert bool((plan == 0).all())
    with pytest.raises(mla.MlaError) as err:
        big = torch.zeros(4097, dtype=torch.int64, device="cuda")
        mla.build_chunk_metadata(b.r2t, big, big, big, 1, 1, 16)
    assert err.value.status == 2


@gpu
def test_metadata_leaves_the_tail_alone_on_request():
    b = Batch([10, 100], [3, 60], pad=5, width=6)
    new = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
    table = new(3, 9)
    out = (table[:, :6], new(2), new(3), new(b.rows), new(b.rows), new(mla.num_chunk_parts(), 8), new(1))
    got = b.maps(fill_tail=False, out=out)
    assert got[0].data_ptr() == table.data_ptr()
    assert table[0].tolist() == [b.slots[0][0] // 64] + [77] * 8
    assert table[1, 3:].tolist() == [77] * 6 and table[2].tolist() == [77] * 9
    assert got[4].tolist()[b.tokens:] == [77] * 5 and got[3].tolist()[b.tokens:] == [77] * 5
    assert mla.read_device_error() == 0


@gpu
def test_metadata_reports_what_only_the_device_sees():
    def err(batch, **change):
        for k, v in change.items():
            setattr(batch, k, v)
        out = batch.maps()
        torch.cuda.synchronize()
        return mla.read_device_error(), out

    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, rpi=torch.tensor([0, 99, -1], device="cuda"))
    assert code & 2 and bool((out[0][1:] == -1).all()) and out[4].tolist()[3:] == [-1] * 61
    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, free=b.free[:1])     # two pages are needed: the second request's and the third's
    assert code == 512 and int(out[6]) == 1 and out[4].tolist()[-1] == -1
    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, free=b.free[:0])
    assert code == 512 and int(out[6]) == 0
    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, width=2)            # the second request's third page has no column
    assert code == 4 and out[4].tolist()[3 + 28:3 + 60] == [-1] * 32 and out[1].tolist() == b.L
    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, rows=20)            # more new tokens than rows
    assert code == 4 and out[2].tolist() == [0, 3, 20, 20]
    b = Batch([10, 100, 64], [3, 60, 1])
    code, out = err(b, prefix_t=torch.tensor([-5, 100, 64], device="cuda"), chunk_t=torch.tensor([3, 60, -1], device="cuda"))
    assert code == 0 and out[1].tolist() == [3, 160, 64] and out[2].tolist() == [0, 3, 63, 63]
    b = Batch([10, 100, 64], [3, 60, 1])
    b.r2t[int(b.rpi[1]), 64] += 3          # a page that does not begin on a page's first slot
    assert err(b)[0] == 64
    b = Batch([10, 100, 64], [3, 60, 1])
    assert err(b, free=torch.full_like(b.free, -2))[0] == 64


def units_of(batch, h, causal, b):
    """Key tiles of request b's row tiles."""
    n, L = batch.chunk[b], batch.L[b]
    out = []
    for m in range(cdiv(n * h, 128)):
        last = min(n * h - 1, 128 * m + 127) // h
        out.append(cdiv(max(0, min(L, L - n + last + 1) if causal else L), 128))
    return out


@gpu
@pytest.mark.parametrize("causal", [True, False])
def test_plan_covers_every_key_tile_once_and_evenly(causal):
    rng = random.Random(8)
    for s in range(30):
        bs = rng.choice([1, 3, 64, 300])
        prefix = [rng.randrange(rng.choice([2, 500, 6000])) for _ in range(bs)]
        chunk = [rng.choice([0, 1, rng.randrange(1, 100)]) for _ in range(bs)]
        h = rng.choice([1, 16, 24, 128, 130])
        parts = rng.choice([1, 2, 74, 200])
        b = Batch(prefix, chunk, seed=s)
        plan = b.maps(h, causal=causal, num_parts=parts)[5].tolist()
        units = [units_of(b, h, causal, i) for i in range(bs)]
        assert all(row[6:] == [0, 0] for row in plan)
        # one cut after another: a part begins where the part before it ends, the last ends at the end
        ends = [tuple(row[3:6]) for row in plan]
        begins = [tuple(row[:3]) for row in plan]
        assert begins[1:] == ends[:-1] and ends[-1] == (bs, 0, 0) and begins == sorted(begins)
        assert all(sum(len(x) for x in units[:begins[0][0]]) == 0 for _ in [0]) and begins[0][1:] == (0, 0)
        for r, m, t in ends:
            assert r == bs or (m == t == 0) or (m < len(units[r]) and (t == 0 or 2 <= t <= units[r][m] - 2))
        # no part does much more than its share (a cut is off by at most a short piece and the rounding of its units)
        cost = lambda c: sum(sum(t + 3 for t in u) for u in units[:c[0]]) + (
            sum(t + 3 for t in units[c[0]][:c[1]]) + c[2] if c[0] < bs else 0)
        total = cost((bs, 0, 0))
        count = sum(len(u) for u in units)
        worst = max((cost(e) - cost(s0) for s0, e in zip(begins, ends)), default=0)
        assert worst <= max(total / parts, 7) * 1.35 + 10, (worst, total, parts, count)


# ------------------------------------------------------------------------------ attention
@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("prefix,chunk,h", [
    ([0], [1], 1), ([0], [1], 128), ([30, 0], [5, 1], 16), ([0, 37, 64, 63, 130], [5, 1, 0, 2, 100], 16),
    ([4000, 20], [1, 200], 128), ([127, 128, 129, 0], [1, 1, 1, 129], 128), ([900, 100, 0], [33, 7, 50], 24),
    ([300], [70], 129), ([65] * 30, [1] * 30, 64), ([0, 0, 700], [64, 63, 3], 200), ([5], [300], 3),
])
def test_attention_matches_64_bits(prefix, chunk, h, kv):
    check_attention(Batch(prefix, chunk, seed=h, pad=2), h, kv, seed=h)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("parts", [1, 2, 5, 74, 130])
def test_attention_with_forced_part_counts(parts, kv):
    """Every way of cutting the same batch (few parts, many, more than SM pairs: CTAs in waves)."""
    check_attention(Batch([1000, 0, 3000, 10, 5000], [37, 129, 1, 0, 2], seed=3), 64, kv, parts=parts, seed=4)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e5m2"])
def test_attention_without_the_causal_limit(kv):
    check_attention(Batch([100, 0, 900, 3000], [7, 50, 33, 1], seed=5, pad=1), 40, kv, causal=False, seed=6)


@gpu
def test_attention_random_batches():
    rng = random.Random(9)
    for s in range(25):
        bs = rng.choice([1, 2, 5, 20])
        prefix = [rng.choice([0, 1, 63, 64, 65, rng.randrange(3000)]) for _ in range(bs)]
        chunk = [rng.choice([0, 1, 1, rng.randrange(1, 160)]) for _ in range(bs)]
        check_attention(Batch(prefix, chunk, seed=s, pad=rng.choice([0, 5])), rng.choice([1, 8, 16, 128, rng.randrange(1, 150)]),
                        rng.choice(["bf16", "bf16", "e4m3", "e5m2"]), parts=rng.choice([None, rng.randrange(1, 120)]), seed=s)


@gpu
def test_attention_of_one_long_request_cut_over_every_part():
    check_attention(Batch([40000], [1], seed=1), 128, seed=2)
    check_attention(Batch([20000], [3], seed=1), 16, "e4m3", seed=2)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rows_without_any_key(kv):
    """Lengths below the chunk's own (a caller's cut-off cache): the first rows see no key; a length of 0: none does."""
    b = Batch([0, 0, 0], [40, 20, 9], seed=2)
    cut = [25, 0, 9]
    h = 16
    bt, _, cu, _, _, plan, _ = b.maps(h)
    cache, scale, values = make_cache(b, kv, 3)
    q = torch.randn(b.rows, h, 576, device="cuda").bfloat16()
    lens = torch.tensor(cut, dtype=torch.int32, device="cuda")
    o, lse = mla.mla_chunk_paged(q, cache, bt, lens, cu, 512, plan, SCALE, descale_k=scale)
    assert mla.read_device_error() == 0
    at = 0
    for r, n in enumerate(b.chunk):
        keys = values[torch.tensor(b.slots[r][:cut[r]], device="cuda", dtype=torch.long)]
        ro, rl, pv, ds = reference(q[at:at + n], keys, True)
        assert_attention(o[at:at + n], lse[at:at + n], ro, rl, pv, ds, cut[r], kv, 8.0)
        at += n
    assert bool((o[:15] == 0).all()) and bool(torch.isneginf(lse[:15]).all()) and bool((o[40:60] == 0).all())


@gpu
def test_scores_of_any_magnitude():
    """Large scores (one key takes all) and rows whose maximum grows from tile to tile."""
    b = Batch([1000], [4], seed=2)
    bt, seqlens, cu, _, _, plan, _ = b.maps(32)
    cache, _, values = make_cache(b, "bf16", 3)
    flat = cache.view(-1, 576)
    slots = torch.tensor(b.slots[0], device="cuda")
    ramp = torch.linspace(0.01, 4.0, len(b.slots[0]), device="cuda")[:, None]
    flat[slots] = (flat[slots].float() * ramp).bfloat16()
    keys = flat[slots].double()
    q = (8 * torch.randn(4, 32, 576, device="cuda")).bfloat16()
    o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE)
    ro, rl, pv, ds = reference(q, keys, True)
    assert_attention(o, lse, ro, rl, pv, ds, 1004, "bf16", 0.0)


@gpu
def test_equal_bits_whatever_the_workspace_holds():
    b = Batch([1000, 0, 3000, 10], [37, 129, 1, 30], seed=3, pad=2)
    ws = torch.full((mla.chunk_workspace_bytes(74),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    first = run_attention(b, 128, seed=1, parts=74, workspace=ws)
    for _ in range(5):
        again = run_attention(b, 128, seed=1, parts=74, workspace=ws)
        assert torch.equal(first[2], again[2]) and torch.equal(first[3], again[3])


@gpu
def test_pages_past_four_gigabytes():
    """Row offsets that do not fit 32 bits: the requests' pages at the far end of a 4.7 GB pool."""
    b = Batch([500, 70], [20, 3], seed=4)
    shift = 64000
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, _, values = make_cache(b, "bf16", 5)
    big = torch.empty((shift + b.pool, 64, 576), dtype=torch.bfloat16, device="cuda")
    big[shift:] = cache
    q = torch.randn(b.rows, 16, 576, device="cuda").bfloat16()
    table = torch.where(bt >= 0, bt + shift, bt)
    o, lse = mla.mla_chunk_paged(q, big, table, seqlens, cu, 512, plan, SCALE)
    o2, lse2 = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE)
    assert mla.read_device_error() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    assert bool(torch.isfinite(o).all())


@gpu
def test_agrees_with_the_decode_and_extend_calls():
    """Single tokens give what mla_decode_paged gives, a uniform chunk what its causal form gives, up to the
    roundings of P (2^-8 of sum p |v|, itself at most max |v|) and o (2^-8) on either side."""
    for n in (1, 4):
        b = Batch([1000, 63, 2500, 0], [n] * 4, seed=6)
        bt, seqlens, cu, _, _, plan, _ = b.maps(128)
        cache, _, values = make_cache(b, "bf16", 7, poison=False)
        q = torch.randn(b.rows, 128, 576, device="cuda").bfloat16()
        o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE)
        md, ns = mla.get_mla_metadata(seqlens, n * 128)
        o2, lse2 = mla.mla_decode_paged(q.view(4, n, 128, 576), cache, bt, seqlens, 512, md, ns, SCALE, True)
        at = 0
        for r in range(4):
            ro, rl, pv, ds = reference(q[at:at + n], values[torch.tensor(b.slots[r], device="cuda")], True)
            tol = 2 * ((2.0**-8 + 2 * ds) * pv + 2.0**-8 * ro.abs())
            assert bool(((o[at:at + n].double() - o2[r].double()).abs() <= tol).all())
            assert bool(((lse[at:at + n] - lse2[r]).abs() <= 2 * (ds + b.L[r] * 2.0**-24) + 2.0**-21 * rl.abs()).all())
            at += n


# --------------------------------------------------------------- as a server runs them together
@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_chunked_prefill_then_decode_through_the_pool(kv):
    """Prompts brought in chunks of other sizes, then decoded: metadata (pages from the free list),
    KV write, attention, step after step on one pool and one req_to_token.  Each step's rows are
    compared with attention in 64 bits over the rows written so far."""
    h, pool, bs = 16, 40, 3
    g = torch.Generator(device="cuda").manual_seed(11)
    scale = None if kv == "bf16" else torch.tensor([0.02], device="cuda")
    cache = torch.full((pool, 64, 576), float("nan"), device="cuda").to(DTYPE[kv])
    r2t = torch.zeros((bs + 1, 640), dtype=torch.int32, device="cuda")
    rpi = torch.tensor([2, 0, 3], device="cuda")
    free = torch.randperm(pool, device="cuda", generator=g)
    lens = torch.zeros(bs, dtype=torch.int64, device="cuda")
    rows = [torch.zeros(0, 576, dtype=torch.double, device="cuda") for _ in range(bs)]
    for chunk in ([100, 0, 7], [28, 300, 1], [64, 64, 120], [1, 1, 1], [1, 0, 1], [1, 1, 1]):
        tokens = sum(chunk)
        new = torch.tensor(chunk, device="cuda")
        bt, seqlens, cu, pos, loc, plan, taken = mla.build_chunk_metadata(r2t, rpi, lens, new, tokens, 10, h, free_pages=free)
        k = torch.randn(tokens, 576, device="cuda", generator=g).bfloat16()
        q = torch.randn(tokens, h, 576, device="cuda", generator=g).bfloat16()
        mla.set_kv_buffer(cache, loc, k, scale)
        o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
        assert mla.read_device_error() == 0
        stored = k.double() if scale is None else (k.float() / scale).clamp(-TOP[kv], TOP[kv]).to(DTYPE[kv]).double() * scale.double()
        at = 0
        for r, n in enumerate(chunk):
            rows[r] = torch.cat([rows[r], stored[at:at + n]])
            if n:
                ro, rl, pv, ds = reference(q[at:at + n], rows[r], True)
                assert_attention(o[at:at + n], lse[at:at + n], ro, rl, pv, ds, rows[r].shape[0], kv, float(rows[r].abs().max()))
                assert pos[at:at + n].tolist() == list(range(rows[r].shape[0] - n, rows[r].shape[0]))
            at += n
        lens = lens + new
        free = free[int(taken):]
    assert sum(cdiv(int(x), 64) for x in lens) == pool - free.shape[0]


@gpu
def test_one_graph_replayed_with_other_lengths_on_another_stream():
    """Metadata, KV write and attention captured once for a padded batch; lengths, queries and rows change
    between replays.  The padded rows' slot is a scratch row of the pool."""
    h, pad_rows = 128, 300
    b0 = Batch([700, 0, 64, 900], [40, 130, 1, 1], seed=1)
    width, pool = 20, 80
    r2t0 = torch.full((7, width * 64), -7, dtype=torch.int32, device="cuda")
    first_pages = [[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14], [], [20], list(range(30, 45))]
    rpi = torch.tensor([1, 4, 0, 6], device="cuda")
    for r, pages in zip(rpi.tolist(), first_pages):
        for i, p in enumerate(pages):
            r2t0[r, 64 * i:64 * i + 64] = torch.arange(64 * p, 64 * p + 64, dtype=torch.int32)
    r2t = r2t0.clone()
    free = torch.arange(50, 78, device="cuda")
    prefix, chunk = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    cache = torch.randn(pool, 64, 576, device="cuda").bfloat16()
    k, q = (torch.zeros(pad_rows, *s, 576, dtype=torch.bfloat16, device="cuda") for s in ((), (h,)))
    out, lse = torch.zeros(pad_rows, h, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(pad_rows, h, device="cuda")
    ws = torch.empty(mla.chunk_workspace_bytes(mla.num_chunk_parts()), dtype=torch.uint8, device="cuda")

    def step():
        maps = mla.build_chunk_metadata(r2t, rpi, prefix, chunk, pad_rows, width, h, free_pages=free, pad_slot=79 * 64)
        mla.set_kv_buffer(cache, maps[4], k)
        mla.mla_chunk_paged(q, cache, maps[0], maps[1], maps[2], 512, maps[5], SCALE, out=out, lse=lse, workspace=ws)
        return maps

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        prefix.copy_(torch.tensor([700, 0, 64, 900]))
        chunk.copy_(torch.tensor([40, 130, 1, 1]))
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            maps = step()
        for p, n in (([700, 0, 64, 900], [40, 130, 1, 1]), ([3, 0, 63, 960], [1, 1, 1, 1]), ([900, 0, 0, 100], [60, 0, 200, 40]),
                     ([0, 0, 0, 0], [0, 0, 0, 0]), ([64, 0, 10, 0], [150, 150, 0, 0])):
            r2t.copy_(r2t0)
            prefix.copy_(torch.tensor(p))
            chunk.copy_(torch.tensor(n))
            k.copy_(torch.randn(pad_rows, 576, device="cuda"))
            q.copy_(torch.randn(pad_rows, h, 576, device="cuda"))
            out.fill_(7.0)
            lse.fill_(7.0)
            graph.replay()
            stream.synchronize()
            assert mla.read_device_error() == 0
            at = 0
            for r in range(4):
                L = p[r] + n[r]
                if n[r]:
                    slots = r2t[int(rpi[r]), :L].long()
                    assert torch.equal(maps[4][at:at + n[r]].long(), slots[p[r]:])
                    keys = cache.view(-1, 576)[slots].double()
                    assert torch.equal(keys[p[r]:], k[at:at + n[r]].double())
                    ro, rl, pv, ds = reference(q[at:at + n[r]], keys, True)
                    assert_attention(out[at:at + n[r]], lse[at:at + n[r]], ro, rl, pv, ds, L, "bf16", 0.0)
                at += n[r]
            assert bool((out[at:] == 7).all()) and bool((lse[at:] == 7).all())


@gpu
def test_two_streams_at_once():
    """Overlapping calls, each with its own workspace."""
    b = Batch([1000, 0, 3000], [37, 129, 1], seed=3)
    alone = run_attention(b, 64, seed=1)
    bt, seqlens, cu, _, _, plan, _ = b.maps(64)
    cache, _, _ = make_cache(b, "bf16", 1)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(mla.mla_chunk_paged(alone[0], cache, bt, seqlens, cu, 512, plan, SCALE))
    torch.cuda.synchronize()
    assert mla.read_device_error() == 0
    for o, lse in got:
        assert torch.equal(o[:b.tokens], alone[2][:b.tokens]) and torch.equal(lse[:b.tokens], alone[3][:b.tokens])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("parts", [1, 74])
def test_nan_queries_give_nan_in_their_rows_alone(parts, kv):
    """A row whose query holds NaN gets NaN (o and lse) whether or not the plan cuts its unit; a length below a
    softmax thread's 32 keys among them.  The other rows keep their bits."""
    b = Batch([4000, 3, 200], [2, 1, 40], seed=4)
    h = 64
    bt, seqlens, cu, _, _, plan, _ = b.maps(h, num_parts=parts)
    cache, scale, _ = make_cache(b, kv, 5)
    q = torch.randn(b.rows, h, 576, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    call = lambda x: mla.mla_chunk_paged(x, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    o0, lse0 = call(q)
    assert mla.read_device_error() == 0
    bad = torch.zeros(b.rows, h, dtype=torch.bool, device="cuda")
    bad[0, 5] = bad[1, 63] = bad[2, 0] = bad[30, 33] = bad[42, 40] = True
    nan = q.clone()
    nan[bad, 100] = float("nan")
    o, lse = call(nan)
    assert mla.read_device_error() == (0 if kv == "bf16" else 32)
    assert bool(lse[bad].isnan().all()) and bool(o[bad].isnan().all())
    assert torch.equal(o[~bad], o0[~bad]) and torch.equal(lse[~bad], lse0[~bad])


@gpu
def test_query_scale_and_a_strided_table():
    """descale_q of a power of two undoes q's; a table that is part of a wider one; no rows at all."""
    b = Batch([300, 70], [5, 40], seed=3)
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, scale, values = make_cache(b, "e5m2", 1)
    q = torch.randn(b.rows, 16, 576, device="cuda").bfloat16()
    o, lse = mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    wide = torch.full((bt.shape[0], bt.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + bt.shape[1]] = bt
    half = torch.full((1,), 0.5, device="cuda")
    o2, lse2 = mla.mla_chunk_paged(2 * q, cache, wide[:, 4:4 + bt.shape[1]], seqlens, cu, 512, plan, SCALE, descale_q=half,
                                   descale_k=scale)
    # q becomes f16 here: exact, and so the same bits, but for values below 2^-17, whose bits end below
    # f16's smallest step, 2^-24.  Those round by at most 2^-25 in q and, halved again, 2^-26 in 2 q, so a
    # row's scores differ by ds <= SCALE sum_d |k_d| (2^-25 + 2^-26) at most, lse by ds (and fp32's rounding
    # of it), o by 2 ds sum_j p_j |v_j|, p's two roundings to f16 and its own two to bf16.
    exact = (2 * q.half() == (2 * q).half()).all(-1)
    assert torch.equal(o[exact], o2[exact]) and torch.equal(lse[exact], lse2[exact])
    vmax = float(values.abs().max())
    ds = SCALE * 576 * vmax * 1.5 * 2.0**-25
    assert bool(((lse - lse2).abs() <= ds + 2.0**-22 * lse.abs()).all())
    assert bool(((o.double() - o2.double()).abs() <= (2 * ds + 2 * 2.0**-11) * vmax + 2 * 2.0**-8 * o.double().abs()).all())
    none, _ = mla.mla_chunk_paged(q[:0], cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    assert none.shape == (0, 16, 512) and mla.read_device_error() == 0


# ------------------------------------------------------------------------- errors and refusals
@gpu
def test_bad_pages_and_offsets_are_reported_or_clamped():
    b = Batch([300, 100], [5, 40], seed=3)
    h = 16
    bt, seqlens, cu, _, _, plan, _ = b.maps(h)
    cache, _, values = make_cache(b, "bf16", 1)
    q = torch.randn(b.rows, h, 576, device="cuda").bfloat16()
    for bad in (-1, b.pool, 2**31 - 1):
        t = bt.clone()
        t[0, 1] = bad
        o, _ = mla.mla_chunk_paged(q, cache, t, seqlens, cu, 512, plan, SCALE)
        assert mla.read_device_error() == 1 and bool(torch.isfinite(o).all())
    # offsets beyond the rows are clamped: the second request's rows are cut to those that exist
    o, lse = torch.zeros(b.rows, h, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(b.rows, h, device="cuda")
    far = torch.tensor([0, 5, 10**6], dtype=torch.int32, device="cuda")
    mla.mla_chunk_paged(q, cache, bt, seqlens, far, 512, plan, SCALE, out=o, lse=lse)
    assert mla.read_device_error() == 0
    ro, rl, pv, ds = reference(q[5:], values[torch.tensor(b.slots[1], device="cuda")], True)
    assert_attention(o[5:], lse[5:], ro, rl, pv, ds, 140, "bf16", 0.0)
    # a plan whose rows end before they begin: those parts do nothing, and say so
    wrong = plan.clone()
    wrong[:, 0], wrong[:, 3] = 2, 0
    mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, wrong, SCALE)
    assert mla.read_device_error() == 8


@gpu
def test_queries_outside_the_range_of_an_8_bit_cache_are_reported():
    b = Batch([30], [5], seed=3)
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, scale, _ = make_cache(b, "e4m3", 1)
    q = torch.randn(5, 16, 576, device="cuda").bfloat16()
    q[2, 3, 500] = 1e6
    mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
    assert mla.read_device_error() == 32


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_wait_that_runs_out_returns_with_an_error(kv):
    """Every pair's leader withholds one tile's page (host-side test hook, 2 ms budget): the call returns and
    reports, and the next call is right again."""
    b = Batch([1000, 600], [1, 40], seed=3)
    bt, seqlens, cu, _, _, plan, _ = b.maps(128)
    cache, scale, _ = make_cache(b, kv, 1)
    q = torch.randn(b.rows, 128, 576, device="cuda").bfloat16()
    try:
        mla.set_test_hooks(wait_budget_ns=2_000_000, withhold_tile=1)
        mla.mla_chunk_paged(q, cache, bt, seqlens, cu, 512, plan, SCALE, descale_k=scale)
        assert mla.read_device_error() == 16
    finally:
        mla.set_test_hooks()
    check_attention(Batch([1000, 600], [1, 40], seed=3), 128, kv, seed=2)


@gpu
def test_binding_refusals():
    b = Batch([30, 0], [5, 7], seed=3)
    bt, seqlens, cu, _, _, plan, _ = b.maps(16)
    cache, scale, _ = make_cache(b, "bf16", 1)
    q = torch.randn(12, 16, 576, device="cuda").bfloat16()
    call = lambda **kw: mla.mla_chunk_paged(**{**dict(q=q, k_cache=cache, block_table=bt, cache_seqlens=seqlens, cu_seqlens=cu,
                                                      head_dim_v=512, chunk_plan=plan, softmax_scale=SCALE), **kw})
    call()
    for kw in (dict(q=q.float()), dict(q=q[:, ::2]), dict(q=q.view(2, 6, 16, 576)), dict(k_cache=cache.float()),
               dict(k_cache=cache[:, :63]), dict(block_table=bt.long()), dict(cache_seqlens=seqlens.long()),
               dict(cache_seqlens=seqlens[:1]), dict(cu_seqlens=cu[:2]), dict(chunk_plan=plan[:, :4]), dict(chunk_plan=plan.long()),
               dict(out=torch.empty(12, 16, 512, device="cuda")), dict(out=torch.empty(11, 16, 512, dtype=torch.bfloat16, device="cuda")),
               dict(lse=torch.empty(12, 15, device="cuda")), dict(descale_k=torch.ones(1, dtype=torch.double, device="cuda")),
               dict(cu_seqlens=cu.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw, status in ((dict(descale_k=torch.ones(1, device="cuda")), 1), (dict(head_dim_v=256), 2), (dict(softmax_scale=math.inf), 1),
                       (dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")), 5)):
        with pytest.raises(mla.MlaError) as err:
            call(**kw)
        assert err.value.status == status
    meta = lambda **kw: mla.build_chunk_metadata(**{**dict(req_to_token=b.r2t, req_pool_indices=b.rpi, prefix_lens=b.prefix_t,
                                                           chunk_lens=b.chunk_t, num_tokens=12, max_seqlen_pad=1, num_heads=16,
                                                           free_pages=b.free), **kw})
    for kw in (dict(req_to_token=b.r2t.long()), dict(req_pool_indices=b.rpi[:1]), dict(prefix_lens=b.prefix_t.int()),
               dict(prefix_lens=b.prefix_t.float(), chunk_lens=b.chunk_t.float()), dict(free_pages=b.free.int()), dict(num_tokens=-1),
               dict(num_heads=0), dict(free_pages=b.free.cpu())):
        with pytest.raises(ValueError):
            meta(**kw)
    assert mla.read_device_error() == 0


@gpu
def test_numbers_past_32_bits_are_refused():
    b = Batch([30, 0], [5, 7], seed=3)
    args = dict(req_to_token=b.r2t, req_pool_indices=b.rpi, prefix_lens=b.prefix_t, chunk_lens=b.chunk_t, num_tokens=12,
                max_seqlen_pad=1, num_heads=16, free_pages=b.free)
    out = mla.build_chunk_metadata(**args)
    for kw in (dict(num_tokens=2**32 + 12), dict(max_seqlen_pad=2**32 + 1), dict(num_heads=2**32 + 16), dict(pad_slot=2**31),
               dict(num_parts=2**32 + 74)):
        with pytest.raises(ValueError):
            mla.build_chunk_metadata(**{**args, "out": out, **kw})
    assert mla.read_device_error() == 0


# ----------------------------------------------------------------------------- without a GPU
def test_chunk_sizes():
    lib = mla.library()
    assert [lib.mla_num_chunk_parts(n) for n in (148, 1, 2, 0, -3, 5000)] == [74, 1, 1, -1, -1, 1024]
    a256 = lambda x: -(-x // 256) * 256
    for parts in (1, 74, 1024):
        assert lib.mla_chunk_workspace_bytes(parts) == a256(parts * 2 * 128 * 512 * 4) + a256(parts * 2 * 128 * 4)
    assert lib.mla_chunk_workspace_bytes(0) == lib.mla_chunk_workspace_bytes(1025) == 0
    with pytest.raises(ValueError):
        mla.chunk_workspace_bytes(0)


def test_chunk_attention_validation_happens_before_any_launch():
    f = mla.library().mla_chunk_paged
    ok = dict(q=1 << 20, q_dtype=0, tokens=9, h=16, d=576, dv=512, k=1 << 21, kv=0, pages=8, page=64, bt=1 << 22, stride=3,
              max_pages=3, lens=1 << 23, cu=1 << 24, bs=2, plan=1 << 25, parts=74, scale=0.07, causal=1, dq=None, dk=None,
              out=1 << 26, lse=1 << 27, ws=1 << 28, ws_bytes=16, stream=None)
    bad = lambda **kw: f(*{**ok, **kw}.values())
    assert bad() == 5 and bad(ws=None) == 5 and bad(ws=(1 << 28) + 128, ws_bytes=1 << 30) == 5
    assert bad(bs=0) == 0 and bad(tokens=0) == 0                 # nothing to do
    for kw in (dict(bs=-1), dict(tokens=-1), dict(h=0), dict(parts=0), dict(parts=1025), dict(q_dtype=3), dict(kv=7), dict(causal=2),
               dict(scale=float("nan")), dict(dk=1 << 29), dict(pages=0), dict(pages=1 << 25), dict(max_pages=4), dict(max_pages=0),
               dict(q=(1 << 20) + 8), dict(plan=(1 << 25) + 8), dict(out=(1 << 26) + 2), *[{x: None} for x in ("q", "k", "bt", "lens",
               "cu", "plan", "out", "lse")]):
        assert bad(**kw) == 1, kw
    for kw in (dict(d=512), dict(dv=576), dict(page=32), dict(q_dtype=1), dict(tokens=1 << 27)):
        assert bad(**kw) == 2, kw


def test_chunk_metadata_validation_happens_before_any_launch():
    f = mla.library().mla_build_chunk_metadata
    ok = dict(r2t=1 << 20, rows=5, stride=192, rpi=1 << 21, idx=3, prefix=1 << 22, chunk=1 << 23, lens=2, bs=2, tokens=9, free=None,
              nfree=0, heads=16, causal=1, parts=74, bt=1 << 24, bt_stride=3, max_pages=3, page=64, fill=1, pad=-1, seqlens=1 << 25,
              cu=1 << 26, pos=1 << 27, loc=1 << 28, plan=1 << 29, taken=None, stream=None)
    bad = lambda **kw: f(*{**ok, **kw}.values())
    for kw in (dict(bs=-1), dict(tokens=-1), dict(heads=0), dict(page=16), dict(parts=0), dict(parts=1025), dict(causal=3), dict(idx=0),
               dict(lens=0), dict(nfree=-1), dict(max_pages=-1), dict(bt_stride=2), dict(rows=0), dict(stride=0), dict(plan=(1 << 29) + 4),
               *[{x: None} for x in ("r2t", "rpi", "prefix", "chunk", "bt", "seqlens", "cu", "pos", "loc", "plan")]):
        assert bad(**kw) == 1, kw
    assert bad(bs=4097) == 2 and bad(tokens=1 << 27) == 2
    # the lengths that are read may not be the ones that are written
    assert bad(seqlens=1 << 22) == 1 and bad(seqlens=1 << 23) == 1


def test_chunk_calls_refuse_cpu_tensors():
    z = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        mla.build_chunk_metadata(torch.zeros(2, 64, dtype=torch.int32), z, z, z, 0, 1, 16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_chunk_paged(torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(1, 64, 576, dtype=torch.bfloat16),
                            i[:2].view(2, 1), i[:2], i, 512, torch.zeros(74, 8, dtype=torch.int32), SCALE)
