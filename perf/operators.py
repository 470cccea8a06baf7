"""The operators of ragged chunks over the paged MLA cache, as they are measured.

Two operators, and a step that runs them together with the KV write:

* ``metadata``  — block table, slot map, positions and offsets of a ragged batch, built on the
  GPU from the requests' lengths, with new pages taken from a free list (or slots that the
  caller has already entered into ``req_to_token``);
* ``attention`` — the new tokens' queries of every request over its rows of the paged latent
  cache, causally: chunked prefill, whole prompts, single tokens, and batches that mix them;
* ``step``      — metadata, KV write and attention of one layer, in the order a model runs them.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits); with
``own`` true it makes the framework's calls.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

PAGE, D_QK, D_V = 64, 576, 512
SCALE = 1.0 / math.sqrt(192.0)
KV = {"bf16": (torch.bfloat16, 2, None), "e4m3": (torch.float8_e4m3fn, 1, 448.0),
      "e5m2": (torch.float8_e5m2, 1, 57344.0)}


# ------------------------------------------------------------------------------- the cases
def _case(name, kind, bs, chunk, prefix, singles=0, empties=0, h=128, kv="bf16", pad=0, alloc=True,
          index="int32", lens=1):
    """chunk / prefix: (lowest, highest) of a request's new / cached tokens; `singles` of the
    requests bring one token instead and `empties` none; `pad` rows lie behind the last request."""
    return dict(name=name, kind=kind, bs=bs, chunk_lo=chunk[0], chunk_hi=chunk[1], prefix_lo=prefix[0],
                prefix_hi=prefix[1], singles=singles, empties=empties, h=h, kv=kv, pad=pad, alloc=alloc,
                index=index, lens=lens)


def listed():
    return [
        # a decode batch in the DeepSeek-V3 shape: one new token a request, most without a new page
        _case("metadata, 64 single tokens", "metadata", 64, (1, 1), (1024, 4096)),
        # a serving batch: decodes and a few prefill chunks, padded for a captured graph
        _case("metadata, 250 decodes and 6 chunks", "metadata", 256, (200, 2000), (0, 16384), singles=250,
              pad=77, index="int64", lens=2),
        # many long requests whose slots the caller's allocator has entered already
        _case("metadata, 96 chunks of long requests, slots given", "metadata", 96, (256, 1024), (4096, 131072),
              alloc=False, lens=3),
        # the smallest call: two short prompts' tails on one of eight tensor-parallel ranks (16 heads)
        _case("attention, 2 requests of 5 and fewer tokens, 16 heads", "attention", 2, (1, 5), (30, 130), h=16, lens=4),
        # decode through the ragged call: one token a request, the cache read once
        _case("attention, 64 single tokens", "attention", 64, (1, 1), (1024, 4096), lens=5),
        # decode over an 8-bit cache
        _case("attention, 128 single tokens, e4m3", "attention", 128, (1, 1), (4000, 4200), kv="e4m3", lens=6),
        # whole prompts without a cached prefix, 16 heads: query tiles that span several tokens, e5m2 cache
        _case("attention, 24 prompts, 16 heads, e5m2", "attention", 24, (33, 900), (0, 0), h=16, kv="e5m2", pad=13, lens=7),
        # chunked prefill in the middle of prompts
        _case("attention, 4 chunks", "attention", 4, (384, 640), (1024, 8192), lens=8),
        # the same over an e4m3 cache
        _case("attention, 3 chunks, e4m3", "attention", 3, (256, 512), (2048, 8192), kv="e4m3", lens=9),
        # the largest: one chunk of a long document
        _case("attention, a chunk of 2000 tokens at 32768", "attention", 1, (2000, 2000), (32768, 32768), lens=10),
        # a serving step: decodes with two prefill chunks, requests without new tokens among them
        _case("step, 40 decodes and 2 chunks", "step", 44, (200, 500), (100, 6000), singles=40, empties=2, lens=11),
        # a decode step of few requests, one token each, 128 heads
        _case("step, 8 single tokens", "step", 8, (1, 1), (500, 9000), lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["metadata", "metadata", "attention", "attention", "attention", "step"])
    lens = rng.randrange(1 << 30)
    index = rng.choice(["int32", "int64"])
    if kind == "metadata":
        bs = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, max(1, 65536 // bs))
        top = _log_int(rng, 1, 131072 if bs <= 96 else 16384)
        singles = rng.randrange(bs + 1) if rng.random() < 0.5 else 0
        empties = rng.randrange(bs - singles + 1) // 4
        return _case("", kind, bs, (rng.randrange(hi // 3 + 1) + 1 if hi > 1 else 1, max(hi, hi // 3 + 1)),
                     (rng.randrange(top + 1) // 2, top), singles, empties, pad=rng.choice([0, 0, rng.randrange(200)]),
                     alloc=rng.random() < 0.7, index=index, lens=lens)
    most = work(listed()[9])["flops"]
    while True:
        bs = _log_int(rng, 1, 128)
        h = rng.choice([16, 32, 64, 128, 128, 128, rng.randrange(1, 129)])
        hi = _log_int(rng, 1, 2000)
        top = _log_int(rng, 16, 32768)
        singles = bs if rng.random() < 0.25 else (rng.randrange(bs + 1) if rng.random() < 0.5 else 0)
        empties = min(bs - singles, rng.choice([0, 0, 1, 2]))
        c = _case("", kind, bs, (max(1, hi // 3), hi), (rng.choice([0, top // 2]), top), singles, empties, h,
                  "bf16" if kind == "step" else rng.choice(["bf16", "bf16", "e4m3", "e5m2"]), 0 if kind == "step" else rng.choice([0, 0, rng.randrange(40)]),
                  True, index, lens)
        chunks, prefix = _lengths(c)
        if sum(chunks) and sum(chunks) * h <= 2000 * 128 and sum(chunks) + sum(prefix) <= 600000 and work(c)["flops"] <= most:
            return c


def _lengths(case):
    """The requests' new and cached tokens: they go by the case alone, so that its work is the same for every seed."""
    rng = random.Random(case["lens"])
    bs = case["bs"]
    chunks = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(bs)]
    prefix = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(bs)]
    order = list(range(bs))
    rng.shuffle(order)
    for b in order[:case["singles"]]:
        chunks[b] = 1
    for b in order[case["singles"]:case["singles"] + case["empties"]]:
        chunks[b] = 0
    return chunks, prefix


def _pages(n):
    return -(-n // PAGE)


def work(case):
    """Bytes that are read or written once, and the flops of the attended pairs."""
    chunks, prefix = _lengths(case)
    tokens, h, size = sum(chunks), case["h"], KV[case["kv"]][1]
    lens = [p + n for p, n in zip(prefix, chunks)]
    width = max(1, _pages(max(lens)))
    out = {"bytes": 0, "flops": 0}
    if case["kind"] != "attention":
        idx = 8 if case["index"] == "int64" else 4
        new_pages = sum(_pages(L) - _pages(p) for L, p in zip(lens, prefix))
        table_reads = sum(_pages(p) for p in prefix) if case["alloc"] else sum(_pages(L) for L in lens)
        out["bytes"] += case["bs"] * (3 * idx + 4 * width + 8) + 4 * table_reads + 8 * (tokens + case["pad"])
        out["bytes"] += (idx * new_pages + 4 * tokens) if case["alloc"] else 4 * tokens
    if case["kind"] == "step":
        out["bytes"] += tokens * D_QK * (2 + size)
    if case["kind"] != "metadata":
        pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(prefix, chunks))
        out["flops"] = 2 * h * (D_QK + D_V) * pairs
        out["bytes"] += tokens * h * (2 * D_QK + 2 * D_V + 4) + sum(L * D_QK * size for L, n in zip(lens, chunks) if n)
    return out


# ------------------------------------------------------------------------------ the inputs
def _inputs(case, seed):
    """What a server holds when the batch arrives: the request-to-token map with the cached
    tokens' slots, a shuffled free list, the lengths, and for attention queries and the pool."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    chunks, prefix = _lengths(case)
    bs, h, tokens = case["bs"], case["h"], sum(chunks)
    lens = [p + n for p, n in zip(prefix, chunks)]
    have, total = [_pages(p) for p in prefix], [_pages(L) for L in lens]
    width = max(1, max(total))
    need = sum(total)
    pool = max(8, math.ceil(1.25 * need))
    idx = torch.int64 if case["index"] == "int64" else torch.int32
    rows = bs + 3
    perm = torch.randperm(pool, generator=cpu)
    rpi = torch.randperm(rows, generator=cpu)[:bs]
    # pages of the cached tokens, one after another from the shuffled pool; with slots given, of all tokens
    owned = have if case["alloc"] else total
    starts = [0]
    for n in owned:
        starts.append(starts[-1] + n)
    r2t = torch.zeros(rows, width * PAGE, dtype=torch.int32)
    in_page = torch.arange(PAGE)
    for b in range(bs):
        keep = prefix[b] if case["alloc"] else lens[b]
        slots = (perm[starts[b]:starts[b + 1], None] * PAGE + in_page).reshape(-1)[:keep]
        r2t[rpi[b], :keep] = slots.to(torch.int32)
    st = dict(kind=case["kind"], h=h, kv=case["kv"], chunks=chunks, prefix=prefix, width=width, rows_out=tokens + case["pad"],
              req_to_token=r2t.cuda(), rpi=rpi.to(idx).cuda(), prefix_lens=torch.tensor(prefix, dtype=idx).cuda(),
              chunk_lens=torch.tensor(chunks, dtype=idx).cuda(),
              free_pages=perm[starts[-1]:].to(idx).cuda() if case["alloc"] else None)
    if case["kind"] == "metadata":
        return st
    dtype, _, top = KV[case["kv"]]
    st["q"] = torch.randn(tokens + case["pad"], h, D_QK, generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn(pool, PAGE, D_QK, generator=gen, device="cuda")
    st["k_scale"] = None
    if top:
        scale = (x.abs().max() / top).reshape(1)
        x = (x / scale).clamp_(-top, top)
        st["k_scale"] = scale
    st["k_cache"] = x.to(dtype)
    st["k_new"] = torch.randn(tokens, D_QK, generator=gen, device="cuda").to(torch.bfloat16) if case["kind"] == "step" else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    out = st["rows_out"]
    if case["kind"] != "metadata":
        # rows behind the last request stay as the caller left them
        st["out"] = torch.zeros(out, st["h"], D_V, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros(out, st["h"], dtype=torch.float32, device="cuda")
    if case["kind"] == "attention":
        maps = _plain_maps(st)
        st["maps"] = (maps["block_table"], maps["cache_seqlens"], maps["cu_seqlens"])
    if own:
        import paged_kv_mla_create_b200 as mla
        if case["kind"] == "attention":
            st["plan"] = mla.build_chunk_metadata(st["req_to_token"], st["rpi"], st["prefix_lens"], st["chunk_lens"], out,
                                                  st["width"], st["h"], free_pages=st["free_pages"])[5]
        if case["kind"] != "metadata":
            st["workspace"] = torch.zeros(mla.chunk_workspace_bytes(mla.num_chunk_parts()), dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------------- the plain forms
def _plain_maps(st):
    """Block table, lengths, offsets, positions and slots; the new tokens' slots go into req_to_token."""
    r2t, rpi = st["req_to_token"], st["rpi"].long()
    prefix, chunk = st["prefix_lens"].long(), st["chunk_lens"].long()
    bs, dev, width = rpi.shape[0], rpi.device, st["width"]
    total = prefix + chunk
    ends = chunk.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    have, pages = (prefix + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    p = torch.arange(width, device=dev)
    table = r2t[rpi][:, ::PAGE].long().div(PAGE, rounding_mode="floor")
    taken = None
    if st["free_pages"] is not None:
        need = pages - have
        off = need.cumsum(0) - need
        at = (off[:, None] + p - have[:, None]).clamp(0, st["free_pages"].shape[0] - 1)
        table = torch.where(p >= have[:, None], st["free_pages"].long()[at], table)
        taken = need.sum().reshape(1).int()
    table = torch.where(p < pages[:, None], table, -1)
    t = torch.arange(st["rows_out"], device=dev)
    b = torch.searchsorted(ends, t, right=True)
    valid = b < bs
    last = torch.searchsorted(ends, (ends[-1:] - 1).clamp(min=0), right=True).clamp(max=bs - 1)
    bb = torch.where(valid, b, last)
    i = torch.where(valid, t, (ends[-1] - 1).clamp(min=0)) - cu[bb]
    pos = prefix[bb] + i
    slot = table[bb, (pos // PAGE).clamp(max=width - 1)] * PAGE + pos % PAGE
    if st["free_pages"] is not None:
        # the rows behind the last token write its slot once more
        r2t[rpi[bb], pos.clamp(max=r2t.shape[1] - 1)] = slot.int()
    else:
        slot = r2t[rpi[bb], pos.clamp(max=r2t.shape[1] - 1)].long()
    return dict(block_table=table.int(), cache_seqlens=total.int(), cu_seqlens=cu.int(),
                positions=torch.where(valid, pos, 0).int(), cache_loc=torch.where(valid, slot, -1).int(),
                req_to_token=r2t, pages_taken=taken)


def _take(pool, index):
    """Rows of a pool of any type (an 8-bit one is indexed as bytes)."""
    return pool[index] if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)[index].view(pool.dtype)


def _plain_attention(st, table, out, lse):
    """softmax(scale q k^T) v in 32 bits: the requests as one padded batch where its scores fit,
    else one after another, in blocks of rows."""
    chunks, prefix, h = st["chunks"], st["prefix"], st["h"]
    n_max, tokens, bs = max(chunks), sum(chunks), len(chunks)
    scale = SCALE if st["k_scale"] is None else SCALE * st["k_scale"]
    vscale = 1.0 if st["k_scale"] is None else st["k_scale"]
    keys = table.shape[1] * PAGE
    if bs * n_max * h * keys <= 1 << 29 and bs * keys * D_QK <= 1 << 30:
        ends = st["chunk_lens"].long().cumsum(0)
        first = ends - st["chunk_lens"].long()
        i = torch.arange(n_max, device=out.device)
        row = (first[:, None] + i).clamp(max=out.shape[0] - 1)
        k = _take(st["k_cache"], table.clamp(min=0).long()).reshape(bs, keys, D_QK).float()
        q = st["q"][row].float().reshape(bs, n_max * h, D_QK)
        s = (q @ k.transpose(1, 2)).reshape(bs, n_max, h, keys) * scale
        seen = st["prefix_lens"].long()[:, None] + i + 1
        s = s.masked_fill(torch.arange(keys, device=out.device) >= seen[:, :, None, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        w = (s - m).exp()
        z = w.sum(-1, keepdim=True)
        o = (w.reshape(bs, n_max * h, keys) @ k[:, :, :D_V]).reshape(bs, n_max, h, D_V) / z * vscale
        t = torch.arange(tokens, device=out.device)
        b = torch.searchsorted(ends, t, right=True)
        out[:tokens] = o[b, t - first[b]].to(out.dtype)
        lse[:tokens] = (m + z.log())[b, t - first[b], :, 0]
        return
    at = 0
    for b in range(bs):
        n, p = chunks[b], prefix[b]
        if n == 0:
            continue
        L = p + n
        k = _take(st["k_cache"], table[b, :_pages(L)].long()).reshape(-1, D_QK)[:L].float()
        step = max(1, (1 << 29) // (h * L))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            s = (st["q"][at + i0:at + i1].float().reshape(-1, D_QK) @ k.t()).reshape(i1 - i0, h, L) * scale
            seen = p + 1 + torch.arange(i0, i1, device=out.device)
            s = s.masked_fill(torch.arange(L, device=out.device) >= seen[:, None, None], -math.inf)
            m = s.amax(-1, keepdim=True)
            w = (s - m).exp_()
            z = w.sum(-1, keepdim=True)
            o = (w.reshape(-1, L) @ k[:, :D_V]).reshape(i1 - i0, h, D_V) / z * vscale
            out[at + i0:at + i1] = o.to(out.dtype)
            lse[at + i0:at + i1] = (m + z.log())[:, :, 0]
        at += n


def _plain_write(st, loc):
    """The new rows into the (bf16) pool."""
    st["k_cache"].view(-1, D_QK)[loc.long()] = st["k_new"]


# ------------------------------------------------------------------------------ one pass
def run(state):
    st = state
    kind = st["kind"]
    if own:
        import paged_kv_mla_create_b200 as mla
        maps = {}
        if kind != "attention":
            table, seqlens, cu, positions, loc, plan, taken = mla.build_chunk_metadata(
                st["req_to_token"], st["rpi"], st["prefix_lens"], st["chunk_lens"], st["rows_out"], st["width"], st["h"],
                free_pages=st["free_pages"])
            maps = dict(block_table=table, cache_seqlens=seqlens, cu_seqlens=cu, positions=positions, cache_loc=loc,
                        req_to_token=st["req_to_token"], pages_taken=taken)
            if kind == "metadata":
                return {k: v for k, v in maps.items() if v is not None}
            mla.set_kv_buffer(st["k_cache"], loc, st["k_new"])
        else:
            (table, seqlens, cu), plan = st["maps"], st["plan"]
        o, lse = mla.mla_chunk_paged(st["q"], st["k_cache"], table, seqlens, cu, D_V, plan, SCALE, True,
                                     descale_k=st["k_scale"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
    else:
        maps = {}
        if kind != "attention":
            maps = _plain_maps(st)
            if kind == "metadata":
                return {k: v for k, v in maps.items() if v is not None}
            _plain_write(st, maps["cache_loc"])
            table = maps["block_table"]
        else:
            table = st["maps"][0]
        o, lse = st["out"], st["lse"]
        _plain_attention(st, table, o, lse)
    if kind == "attention":
        return {"o": o, "lse": lse}
    return {"o": o, "lse": lse, "cache_loc": maps["cache_loc"], "block_table": maps["block_table"],
            "pool": st["k_cache"]}


# ------------------------------------------------------------------------- the definition
def exact(case, seed):
    """o and lse from the definition in 64 bits, key rows looked up one slot at a time."""
    if case["kind"] == "metadata":
        return None
    st = _inputs(case, seed)
    chunks, prefix, h = st["chunks"], st["prefix"], st["h"]
    o = torch.zeros(st["rows_out"], h, D_V, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["rows_out"], h, dtype=torch.float64, device="cuda")
    r2t, rpi = st["req_to_token"].cpu(), st["rpi"].tolist()
    free = st["free_pages"].tolist()
    factor = 1.0 if st["k_scale"] is None else float(st["k_scale"].double())
    flat = st["k_cache"].view(-1, D_QK)
    at = taken = 0
    for n, p, row in zip(chunks, prefix, rpi):
        slots = r2t[row, :p].tolist()
        for pos in range(p, p + n):
            if pos % PAGE == 0:
                slots.append(free[taken] * PAGE)
                taken += 1
            else:
                slots.append(slots[-1] + 1)
        if n == 0:
            continue
        keys = flat.view(torch.uint8 if case["kv"] != "bf16" else flat.dtype)[torch.tensor(slots, device="cuda")].view(flat.dtype)
        keys = keys.double() * factor
        if case["kind"] == "step":
            keys[p:] = st["k_new"][at:at + n].double()
        values = keys[:, :D_V]
        block = max(1, (1 << 28) // (h * (p + n)))
        for a in range(0, n, block):
            z = min(n, a + block)
            logits = torch.einsum("thd,kd->thk", st["q"][at + a:at + z].double(), keys) * SCALE
            hidden = torch.arange(p + n, device="cuda")[None, :] > torch.arange(p + a, p + z, device="cuda")[:, None]
            logits.masked_fill_(hidden[:, None, :], float("-inf"))
            norm = torch.logsumexp(logits, -1)
            lse[at + a:at + z] = norm
            o[at + a:at + z] = torch.einsum("thk,kd->thd", torch.exp(logits - norm[..., None]), values)
        at += n
    if case["kind"] == "attention":
        return {"o": o, "lse": lse}
    return {"o": o, "lse": lse, "cache_loc": None, "block_table": None, "pool": None}
