"""Measured cases of the operators over a paged K/V cache that is held in 8 bits, and of
eviction from a paged cache by accumulated attention weight.

The operators: writing new K/V rows into the cache ("write": written, then the tiles they
fall into read back as bf16), decode attention ("decode"), attention of many query rows
per request ("extend"), the attention weight that keys receive ("weigh": with a decode
step, or from given query rows), and the eviction of the pages that received least
("evict").

The cache.  Slots lie in tiles of t = min(page size, 64) consecutive ones.  A tile's K rows
of one kv head share a scale, and its V rows another: a power of two s = 2^(E - 127), held as
the byte E (1 .. 247), the least one with max |x| <= 448 s.  Each element is an e4m3 float:

    code = e4m3(x / s) (to nearest, ties to even),   value = code s

A tile is uint8: for each kv head K codes [t, D] and V codes [t, D], then for each kv head its
two bytes (E of K, E of V), padded to whole 32 bytes (128 from 16 slots on).  Rows that a call
writes share one maximum per tile.  Where they hold the tile's first slot its scale is theirs;
else it is the larger of theirs and the tile's, and codes of other slots follow a scale that
grows, rounded again.

Weights.  acc has a column for each column of the token table: a key's weight is the sum of
exp(score - lse) over the query rows that see it and all query heads.

Eviction.  A request of n pages keeps max(1, budget // page size) of them: those with one of the
first `keep_first` or the last `keep_last` tokens and its last page in any case, and of the others
those whose keys' weights sum to most (in 64 bits, rounded to 32; of equal ones the earlier).
Kept columns of the table and of acc move together, acc's columns that fall free become 0, and the
evicted pages go to the front of the free list, request after request, in the order of their
columns.

With ``own`` false, ``run`` computes the plain form in fp32 torch operations; with ``own``
true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new rows of a small batch, appended to tiles in use: latency
        dict(name="append_step_b32", op="write", batch=32, hkv=8, d=128, ps=16, lo=1, hi=4096, new_lo=1, new_hi=1, pad=0),
        # a chunked prefill's new rows (8 requests x 1024 tokens), some of them padding
        dict(name="write_chunk_8x1024", op="write", batch=8, hkv=8, d=128, ps=64, lo=1024, hi=5120, new_lo=1024, new_hi=1024,
             pad=37),
        # four short requests on pages of one token: the latency floor of a decode step
        dict(name="decode_tiny_ps1", op="decode", batch=4, hq=16, hkv=8, d=128, ps=1, lo=17, hi=255, layout="csr"),
        # one head per kv head at 64 dims: an encoder-decoder's cross-attention
        dict(name="decode_mha_d64", op="decode", batch=64, hq=20, hkv=20, d=64, ps=16, lo=1500, hi=1500, layout="block"),
        # a large batch of uneven lengths: the cache's bandwidth
        dict(name="decode_b128", op="decode", batch=128, hq=32, hkv=8, d=128, ps=64, lo=128, hi=16384, layout="table"),
        # a drafted step of uneven lengths: four query rows per request
        dict(name="verify_b64x4", op="extend", batch=64, hq=32, hkv=8, d=128, ps=64, lo=132, hi=16384, rows_lo=4, rows_hi=4,
             bounds="causal", layout="table"),
        # a chunked prefill over cached prefixes
        dict(name="prefill_8x1024", op="extend", batch=8, hq=16, hkv=8, d=128, ps=16, lo=1024, hi=5120, rows_lo=1024,
             rows_hi=1024, bounds="causal", layout="table"),
        # one long prompt's second half, and the largest case
        dict(name="prefill_1x8192", op="extend", batch=1, hq=32, hkv=8, d=128, ps=64, lo=16384, hi=16384, rows_lo=8192,
             rows_hi=8192, bounds="causal", layout="csr"),
        # a decode step that keeps count of what each key receives
        dict(name="weigh_step_b32", op="weigh", batch=32, hq=32, hkv=8, d=128, ps=16, lo=128, hi=8192, rows_lo=0, rows_hi=0,
             bounds="causal", layout="table"),
        # the last rows of prompts, from which a prefill chooses what to keep
        dict(name="weigh_window_8x32", op="weigh", batch=8, hq=32, hkv=8, d=128, ps=64, lo=2048, hi=32768, rows_lo=32, rows_hi=32,
             bounds="causal", layout="table"),
        # a small batch that outgrew its budget, pages of 16: latency
        dict(name="evict_b32_ps16", op="evict", batch=32, ps=16, lo=64, hi=4096, budget=1024, first=4, last=256),
        # token by token out of a large batch of long requests
        dict(name="evict_b128_ps1", op="evict", batch=128, ps=1, lo=8192, hi=16384, budget=8192, first=4, last=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "extend", "weigh", "evict"])
    ps = rng.choice([1, 4, 16, 32, 64, 128])
    if op == "evict":
        case = dict(op=op, ps=ps, batch=_log(rng, 1, 256))
        case["hi"] = min(_log(rng, 1, 131072), (1 << 21) // case["batch"])
        case["lo"] = rng.choice([case["hi"], max(1, case["hi"] // 2), min(case["hi"], 1 + rng.randrange(64))])
        case["budget"] = _log(rng, 1, 2 * case["hi"])
        case["first"] = rng.choice([0, 4, rng.randrange(0, 200)])
        case["last"] = rng.choice([0, 1, rng.randrange(0, 2000)])
        return case
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 20])
    case = dict(op=op, hkv=hkv, d=d, ps=ps)
    case["batch"] = _log(rng, 1, 128)
    room = max(1, (1 << 28) // (case["batch"] * hkv * d))   # key elements of the padded batch
    hi = min(_log(rng, 1, 65536), room)
    lo = rng.choice([hi, max(1, hi // 2), min(hi, 1 + rng.randrange(64))])
    case["lo"], case["hi"] = min(lo, hi), hi
    if op == "write":
        case["new_hi"] = min(hi, rng.choice([1, _log(rng, 1, 64), _log(rng, 64, 2048)]))
        case["new_lo"] = rng.choice([1, case["new_hi"]])
        case["pad"] = rng.choice([0, rng.randrange(1, 100)])
        return case
    case["hq"] = hkv * rng.choice([1, 2, 4, 7, 8, 16])
    case["layout"] = rng.choice(["csr", "block", "table"])
    if op == "decode":
        return case
    cap = max(1, min(hi, (1 << 33) // (case["batch"] * case["hq"] * hi * 4)))
    if op == "extend":
        rows = min(cap, _log(rng, 1, 12) if rng.random() < 0.5 else _log(rng, 12, 2048))
    else:
        case["layout"] = "table"
        rows = rng.choice([0, min(cap, _log(rng, 1, 128))])
    case["rows_hi"] = rows
    case["rows_lo"] = rng.choice([rows, max(1, rows // 2), 1]) if rows else 0
    case["bounds"] = rng.choice(["causal", "given"]) if rows else "causal"
    case["hi"] = max(hi, rows)
    case["lo"] = max(case["lo"], rows)
    return case


def _lens(case):
    """The requests' key counts: the case's own (log-uniform between lo and hi, shuffled)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    u = (np.arange(b) + 0.5) / b
    n = np.clip(np.round(np.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))), lo, hi).astype(np.int64)
    return np.random.RandomState(b * 7919 + hi).permutation(n)


def _rows(case):
    """Query rows of each request (a decode step: one)."""
    b, lo, hi = case["batch"], case.get("rows_lo", 0), case.get("rows_hi", 0)
    if not hi:
        return np.ones(b, dtype=np.int64)
    n = np.random.RandomState(b * 104729 + hi).randint(lo, hi + 1, b)
    return np.minimum(n, _lens(case)).astype(np.int64)


def _bounds(case):
    """Key bound of every query row: causal, or given ones, some of them 0."""
    lens, rows = _lens(case), _rows(case)
    if case.get("bounds", "causal") == "causal":
        return np.concatenate([np.arange(l - n + 1, l + 1) for l, n in zip(lens, rows)])
    r = np.random.RandomState(case["batch"] * 31 + case["hi"])
    ends = np.concatenate([r.randint(0, l + 1, n) for l, n in zip(lens, rows)])
    ends[::7] = 0
    return ends


def _new(case):
    """New tokens of each request (its last ones)."""
    b = case["batch"]
    n = np.random.RandomState(b * 613 + case["hi"]).randint(case["new_lo"], case["new_hi"] + 1, b)
    return np.minimum(n, _lens(case)).astype(np.int64)


def _tile(case):
    return min(case["ps"], 64)


def _evicted(case):
    """Pages that each request loses."""
    lens, ps = _lens(case), case["ps"]
    n = -(-lens // ps)
    head = np.minimum(-(-min(case["first"], 1 << 30) // ps), n)
    tail = np.minimum(np.maximum(lens - case["last"], 0) // ps, n - 1)      # from here on pages stay
    return np.minimum(np.maximum(n - max(1, case["budget"] // ps), 0), np.maximum(tail - head, 0))


def work(case):
    lens = _lens(case)
    if case["op"] == "evict":
        kept = lens - _evicted(case) * case["ps"]
        return {"bytes": int((8 * lens + 8 * kept + 4 * _evicted(case)).sum()), "flops": int(lens.sum())}
    hkv, d, t = case["hkv"], case["d"], _tile(case)
    if case["op"] == "write":
        new = _new(case)
        back = lens - (lens - new) // t * t                                # rows read back
        return {"bytes": int(new.sum()) * (6 * hkv * d + 4) + int(back.sum()) * (6 * hkv * d + 4),
                "flops": int((new + back).sum()) * 2 * hkv * d}
    hq, tokens = case["hq"], int(lens.sum())
    pages, tiles = int((-(-lens // case["ps"])).sum()), int((-(-lens // t)).sum())
    ends, n = _bounds(case), _rows(case)
    at = np.concatenate([[0], np.cumsum(n)])
    seen = tokens if case["op"] == "decode" else sum(int(ends[at[b]:at[b + 1]].max()) for b in range(case["batch"]) if n[b])
    q = int(n.sum()) * hq
    pairs = hq * int(ends.sum())
    if case["op"] == "weigh":
        decode = not case["rows_hi"]
        held = hkv * d * (2 if decode else 1)
        return {"bytes": seen * held + 2 * hkv * tiles + q * (d * (4 if decode else 2) + 4) + 4 * pages + 8 * tokens,
                "flops": (4 if decode else 2) * d * pairs}
    return {"bytes": seen * 2 * hkv * d + 2 * hkv * tiles + q * (4 * d + 4) + 4 * pages, "flops": 4 * d * pairs}


# ------------------------------------------------------------------------- inputs
def _tile_bytes(case):
    pad = 128 if _tile(case) >= 16 else 32
    return case["hkv"] * 2 * _tile(case) * case["d"] + -(-2 * case["hkv"] // pad) * pad


def _power(e):
    """2^(E - 127) in fp32, from its bits (E 1 .. 254)."""
    return (e.int() << 23).view(torch.float32)


def _to_e4m3(x):
    """fp32 rounded to the nearest e4m3 value (ties to even, at most 448)."""
    a = x.abs().clamp(max=448.0)
    step = _power(torch.frexp(a)[1].clamp(min=-5) + 123)         # a < 2^e: steps of 2^(e - 4), of 2^-9 at least
    return torch.copysign(torch.round(a / step) * step, x)


def _scale_byte(top):
    """E of a block with largest magnitude `top` (fp32 from bf16 values)."""
    m, e = torch.frexp(top)                                      # top = m 2^e, 0.5 <= m < 1
    return torch.where(top > 0, e - 9 + (m > 0.875) + 127, 1).clamp(min=1)


def _values(gen, shape, spread):
    """Rows [..., heads, d] as a projection gives them: normal, with a few channels several times larger."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    ch = torch.rand(shape[-2:], generator=gen, device="cuda")
    return (x * torch.where(ch < 0.05, 4.0, 1.0) * spread).to(torch.bfloat16)


def _pages(case, rng, lens):
    """Shuffled pages (page 0 unused), the table's rows, and the slots of all tokens in order."""
    ps, batch = case["ps"], case["batch"]
    npages = -(-lens // ps)
    pages = int(npages.sum()) + int(npages.sum()) // 8 + 2
    order = rng.permutation(pages - 1)[:int(npages.sum())] + 1
    at = np.concatenate([[0], np.cumsum(npages)])
    width = int(-(-(lens.max() + 1) // 32) * 32)
    width = -(-width // ps) * ps
    table = np.zeros((batch + 1, width), dtype=np.int32)
    row = (rng.permutation(batch) + 1).astype(np.int32)
    for b in range(batch):
        table[row[b], :lens[b]] = (order[at[b]:at[b + 1]].astype(np.int64)[:, None] * ps + np.arange(ps)).reshape(-1)[:lens[b]]
    flat = np.concatenate([table[row[b], :lens[b]] for b in range(batch)]).astype(np.int64)
    return npages, pages, order, at, table, row, flat


def _fill(st, gen, held, spread_k=1.0, spread_v=0.3):
    """The pool's rows at the first held[b] positions of each request; everything else stays 0xFF."""
    case = st["case"]
    t, hkv, d, ps = _tile(case), case["hkv"], case["d"], case["ps"]
    per = max(1, ps // t)
    tiles, valid = [], []
    for b in range(case["batch"]):
        n = -(-int(held[b]) // t)
        first = st["table_host"][st["row_host"][b], np.arange(n) * t].astype(np.int64)
        tiles.append(first // t)
        valid.append(np.minimum(int(held[b]) - np.arange(n) * t, t))
    assert per >= 1
    tiles = torch.from_numpy(np.concatenate(tiles)).cuda()
    valid = torch.from_numpy(np.concatenate(valid)).cuda()
    pool, entry = st["pool"], torch.arange(t, device="cuda")
    step = max(1, (1 << 25) // (t * hkv * d))
    for i in range(0, tiles.numel(), step):
        at, live = tiles[i:i + step], (entry < valid[i:i + step, None])[:, None, :, None]
        for part, spread in ((0, spread_k), (1, spread_v)):
            x = _values(gen, (at.numel(), t, hkv, d), spread).permute(0, 2, 1, 3).float()
            e = _scale_byte((x * live).abs().amax((2, 3)))
            c = _to_e4m3(x / _power(e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            c = torch.where(live, c, torch.full_like(c, 0xFF))
            codes, scales = _parts(case, pool)
            codes[at, :, part] = c
            scales[at, :, part] = e.to(torch.uint8)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    rng = np.random.RandomState(seed % (1 << 31))
    lens, ps = _lens(case), case["ps"]
    batch, total = case["batch"], int(lens.sum())
    npages, pages, order, at, table, row, flat = _pages(case, rng, lens)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
    st = dict(case=case, lens_host=lens, batch=batch, total=total, max_len=int(lens.max()), table_host=table, row_host=row)
    st["table"], st["row"], st["lens"] = up(table), up(row), up(lens.astype(np.int32))
    st["flat"] = up(flat)
    st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if case["op"] == "evict":
        return _prepare_evict(st, gen, rng, pages)
    hkv, d, t = case["hkv"], case["d"], _tile(case)
    # slots that nobody wrote hold whatever was there
    st["pool"] = torch.full((pages * ps // t, _tile_bytes(case)), 0xFF, dtype=torch.uint8, device=dev)
    if case["op"] == "write":
        new = _new(case)
        _fill(st, gen, lens - new)
        n = int(new.sum()) + case["pad"]
        # every third request's new rows are larger than what its tile holds so far
        grow = np.repeat(np.where(np.arange(batch) % 3 == 0, 6.0, 1.0), new)
        keep = np.sort(rng.permutation(n)[:int(new.sum())])      # padded tokens lie anywhere between the real ones
        slot = np.full(n, -1, dtype=np.int32)
        slot[keep] = np.concatenate([table[row[b], lens[b] - new[b]:lens[b]] for b in range(batch)])
        big = np.ones(n, dtype=np.float32)
        big[keep] = grow
        big = up(big).view(-1, 1, 1)
        st["k_new"], st["v_new"] = ((_values(gen, (n, hkv, d), s) * big).to(torch.bfloat16) for s in (1.0, 0.3))
        st["slot"] = up(slot)
        # read back: from the first slot of the tile that each request's new rows begin in
        start = (lens - new) // t * t
        back = lens - start
        st["start"], st["back"], st["back_max"] = up(start.astype(np.int32)), up(back.astype(np.int32)), int(back.max())
        st["flat"] = up(np.concatenate([table[row[b], start[b]:lens[b]] for b in range(batch)]).astype(np.int64))
        st["rows_back"] = int(back.sum())
        # room for a few rows more than come back: those stay as they are
        st["k_out"] = torch.zeros((st["rows_back"] + 5, hkv, d), dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.zeros_like(st["k_out"])
        st["cu"] = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
        if own:
            from paged_kv_cache_req_gb300 import _binding as B
            st["workspace"] = torch.empty(B.pkv_q8_store_workspace_size(st["pool"].shape[0], ps), dtype=torch.uint8, device=dev)
        return st
    _fill(st, gen, lens)
    rows = _rows(case)
    st["rows"] = rows
    nq = int(rows.sum())
    st["q"] = _values(gen, (nq, case["hq"], d), 1.0)
    st["out"] = torch.zeros((nq, case["hq"], d), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros((nq, case["hq"]), dtype=torch.float32, device=dev)
    st["sm_scale"] = d ** -0.5
    st["qo_indptr"] = up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
    ends = lens if case["op"] == "decode" else _bounds(case)
    st["ends"] = up(ends.astype(np.int32))
    # where each query row stands in a padded [batch, rows] array
    st["q_at"] = up(np.concatenate([b * int(rows.max()) + np.arange(n) for b, n in enumerate(rows)]))
    if case["layout"] == "csr":
        st["indptr"] = up(at.astype(np.int32))
        st["indices"] = up(order.astype(np.int32))
        st["last"] = up((lens - (npages - 1) * ps).astype(np.int32))
    elif case["layout"] == "block":
        bt = np.full((batch, int(npages.max())), -1, dtype=np.int32)
        for b in range(batch):
            bt[b, :npages[b]] = order[at[b]:at[b + 1]]
        st["block_table"] = up(bt)
    if case["op"] == "weigh":
        # weight received so far: a few keys have most of it
        st["acc"] = torch.exp(3.0 * torch.randn(st["table"].shape, generator=gen, device=dev))
        st["acc_out"] = torch.zeros_like(st["acc"])
        if case["rows_hi"]:
            st["lse"] = _plain_attention(st, values=False)["lse"]
    if own:      # the argument block and the workspace, which a serving loop builds once
        from paged_kv_cache_req_gb300 import _binding as B
        kw = dict(page_size=ps, num_kv_heads=hkv, sm_scale=st["sm_scale"], max_seq_len=st["max_len"], lse=st["lse"])
        if case["layout"] == "csr":
            layout = B.PKV_LAYOUT_CSR
            kw.update(kv_indptr=st["indptr"], kv_indices=st["indices"], kv_last_page_len=st["last"])
        elif case["layout"] == "block":
            layout = B.PKV_LAYOUT_BLOCK_TABLE
            kw.update(block_table=st["block_table"], seq_lens=st["lens"])
        else:
            layout = B.PKV_LAYOUT_REQ_TO_TOKEN
            kw.update(req_to_token=st["table"], req_pool_idx=st["row"], seq_lens=st["lens"])
        kw.update(total_kv=total)
        if case["op"] == "weigh":
            kw.update(acc_in=st["acc"], acc_out=st["acc_out"])
        if case["op"] == "extend" or case.get("rows_hi"):
            kw.update(qo_indptr=st["qo_indptr"], max_q_len=int(rows.max()))
            if case["bounds"] == "given":
                kw.update(kv_end=st["ends"])
        size = {"decode": B.pkv_q8_decode_workspace_size, "extend": B.pkv_q8_extend_workspace_size,
                "weigh": B.pkv_q8_weights_workspace_size if case.get("rows_hi") else B.pkv_q8_decode_workspace_size}[case["op"]]
        st["args"] = B.make_q8_args(layout, st["q"], st["pool"], st["out"], **kw)
        st["workspace"] = torch.empty(size(st["args"]), dtype=torch.uint8, device=dev)
    return st


def _prepare_evict(st, gen, rng, pages):
    case, dev = st["case"], "cuda"
    # weights as keys receive them: heavy-tailed, many of them none at all or the same
    acc = torch.exp(2.0 * torch.randn(st["table"].shape, generator=gen, device=dev))
    kind = torch.rand(st["table"].shape, generator=gen, device=dev)
    st["acc"] = torch.where(kind < 0.1, 0.0, torch.where(kind < 0.2, torch.exp2(torch.floor(torch.log2(acc))), acc))
    full = lambda v: torch.full((st["batch"],), v, dtype=torch.int32, device=dev)  # noqa: E731
    st["budget"], st["first"], st["last"] = full(case["budget"]), full(case["first"]), full(case["last"])
    # the free list: `used` entries were taken from its front, the rest is free
    used = int((-(-st["lens_host"] // case["ps"])).sum())
    st["pages"] = pages
    st["free"] = torch.from_numpy(rng.permutation(pages).astype(np.int32)).to(dev)
    st["free_state"] = torch.tensor([used, pages - used], dtype=torch.int32, device=dev)
    st["table_out"], st["acc_out"] = torch.zeros_like(st["table"]), torch.zeros_like(st["acc"])
    st["lens_out"], st["state_out"] = torch.zeros_like(st["lens"]), torch.zeros_like(st["free_state"])
    if own:
        from paged_kv_cache_req_gb300 import _binding as B
        st["workspace"] = torch.empty(B.pkv_evict_workspace_size(st["batch"], st["max_len"], case["ps"]), dtype=torch.uint8,
                                      device=dev)
    return st


# ------------------------------------------------------------------------- plain form
def _parts(case, pool):
    """Codes [tiles, hkv, 2, t, d] and scale bytes [tiles, hkv, 2] of the pool, as views."""
    t, d, hkv = _tile(case), case["d"], case["hkv"]
    n = hkv * 2 * t * d
    return pool[:, :n].unflatten(-1, (hkv, 2, t, d)), pool[:, n:n + 2 * hkv].unflatten(-1, (hkv, 2))


def _held(st, slots, part):
    """fp32 values of the K (0) or V (1) rows at `slots` [...]: [..., hkv, d]."""
    codes, scales = _parts(st["case"], st["pool"])
    t = _tile(st["case"])
    c = codes[slots // t, :, part, slots % t].view(torch.float8_e4m3fn).float()
    return c.mul_(_power(scales[slots // t, :, part]).unsqueeze(-1))


def _plain_attention(st, values=True):
    case = st["case"]
    hq, hkv, d, batch, m = case["hq"], case["hkv"], case["d"], st["batch"], st["max_len"]
    g, nmax = hq // hkv, int(st["rows"].max())
    pos = torch.arange(m, device="cuda")
    live = pos < st["lens"][:, None]                                               # [B, M]
    slots = torch.where(live, st["table"][st["row"].long()][:, :m].long(), 0)
    k = torch.where(live[..., None, None], _held(st, slots, 0), 0.0)               # [B, M, hkv, d]
    q = torch.zeros((batch * nmax, hq, d), device="cuda")
    q[st["q_at"]] = st["q"].float()
    q = q.view(batch, nmax, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nmax * g, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["sm_scale"]                     # [B, hkv, nmax g, M]
    del k
    end = torch.zeros(batch * nmax, dtype=torch.int32, device="cuda")
    end[st["q_at"]] = st["ends"]
    seen = (pos < end.view(batch, 1, nmax, 1, 1)).expand(batch, 1, nmax, g, m).reshape(batch, 1, nmax * g, m)
    s = s.masked_fill_(~seen, -math.inf)
    if case["op"] == "weigh" and values and case["rows_hi"]:       # the rows' lse is known
        lse = torch.full((batch * nmax, hq), math.inf, device="cuda")
        lse[st["q_at"]] = torch.where(st["lse"] == -math.inf, math.inf, st["lse"])
        lse = lse.view(batch, nmax, hkv, g).permute(0, 2, 1, 3).reshape(batch, hkv, nmax * g, 1)
        return {"acc": _add_weights(st, s.sub_(lse).exp_().sum((1, 2)), live)}
    top = s.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(base).exp_()
    den = p.sum(-1, keepdim=True)
    res = {}
    if values:
        v = torch.where(live[..., None, None], _held(st, slots, 1), 0.0)
        o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(den > 0, den, 1.0)
        res["out"] = o.view(batch, hkv, nmax, g, d).permute(0, 2, 1, 3, 4).reshape(batch * nmax, hq, d)[st["q_at"]].to(torch.bfloat16)
    lse = torch.where(den > 0, torch.log(den) + base, -math.inf)
    res["lse"] = lse.view(batch, hkv, nmax, g).permute(0, 2, 1, 3).reshape(batch * nmax, hq)[st["q_at"]]
    if case["op"] == "weigh" and values:
        res["acc"] = _add_weights(st, (p / torch.where(den > 0, den, 1.0)).sum((1, 2)), live)
    return res


def _add_weights(st, w, live):
    """acc_out: acc plus the weights w [B, M] in the requests' columns."""
    out, m, row = st["acc_out"].clone(), st["max_len"], st["row"].long()
    out[row, :m] = torch.where(live, st["acc"][row, :m] + w, out[row, :m])
    return out


def _plain_write(st):
    case = st["case"]
    t = _tile(case)
    codes, scales = _parts(case, st["pool"])
    tiles, n = st["pool"].shape[0], st["slot"].numel()
    slot = torch.where(st["slot"] >= 0, st["slot"], tiles * t).long()              # padded tokens: one tile past the last
    touched = torch.zeros(tiles + 1, dtype=torch.bool, device="cuda")
    touched[slot // t] = True
    fresh = torch.zeros_like(touched)
    fresh[torch.where(slot % t == 0, slot // t, tiles)] = True
    who = torch.full((tiles * t + 1,), -1, dtype=torch.int64, device="cuda")
    who[slot] = torch.arange(n, device="cuda")
    f = st["flat"]
    mine = who[f]
    is_new, at = (mine >= 0)[:, None, None], mine.clamp(min=0)
    got = {}
    for part, name in enumerate("kv"):
        x = st[name + "_new"].float()
        need = torch.zeros((tiles + 1, case["hkv"]), dtype=torch.float32, device="cuda")
        need.scatter_reduce_(0, (slot // t)[:, None].expand(-1, case["hkv"]), x.abs().amax(-1), "amax")
        old = scales[f // t, :, part].int()                                        # [R, hkv]
        e = _scale_byte(need[f // t]).int()
        e = torch.where(fresh[f // t, None], e, torch.maximum(e, old))
        e = torch.where(touched[f // t, None], e, old)
        s = _power(e).unsqueeze(-1)
        before = codes[f // t, :, part, f % t].view(torch.float8_e4m3fn).float() * _power(old).unsqueeze(-1)
        value = _to_e4m3(torch.where(is_new, x[at], before) / s) * s
        out = torch.zeros_like(st["k_out"])
        out[:st["rows_back"]] = value.to(torch.bfloat16)
        got[name] = out
    got["cu"] = torch.zeros(st["batch"] + 1, dtype=torch.int32, device="cuda")
    got["cu"][1:] = torch.cumsum(st["back"], 0)
    return got


def _plain_evict(st):
    case = st["case"]
    ps, batch, lens = case["ps"], st["batch"], st["lens"].long()
    row = st["row"].long()
    width = st["table"].shape[1]
    table, acc = st["table"][row], st["acc"][row]                                  # [B, width]
    n = (lens + ps - 1) // ps
    pages = width // ps
    page = torch.arange(pages, device="cuda")
    col = torch.arange(width, device="cuda")
    live = col < lens[:, None]
    score = torch.where(live, acc.double(), 0.0).view(batch, pages, ps).sum(-1).float()
    head = ((st["first"].long() + ps - 1) // ps)[:, None]
    tail = torch.minimum((lens - st["last"]).clamp(min=0) // ps, n - 1)[:, None]
    free = (page >= head) & (page < tail)                                          # pages that may go
    keep_n = (st["budget"].long() // ps).clamp(min=1)
    gone_n = torch.minimum((n - keep_n).clamp(min=0), free.sum(1))
    order = torch.sort(torch.where(free, score, math.inf), dim=1, stable=True, descending=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, page.expand(batch, -1).contiguous())
    gone = free & (rank >= (pages - gone_n)[:, None])
    # (free pages are the last in the order: of infinite scores those that may not go come first or are never reached)
    keep = (~gone).repeat_interleave(ps, 1) & live
    to = torch.cumsum(keep, 1) - 1
    lens_new = lens - gone_n * ps
    table_out, acc_out = st["table_out"].clone(), st["acc_out"].clone()
    b_at = row[:, None].expand(-1, width)[keep]
    table_out[b_at, to[keep]] = table[keep]
    clear = live & (col >= lens_new[:, None])
    acc_out[row[:, None].expand(-1, width)[clear], col.expand(batch, -1)[clear]] = 0.0
    acc_out[b_at, to[keep]] = acc[keep]
    total = gone_n.sum()
    free_out = st["free"].clone()
    at = st["free_state"][0] - total + torch.arange(free_out.numel(), device="cuda")
    ids = (table[:, ::ps] // ps)[gone]
    free_out[at[:ids.numel()]] = ids
    state = st["free_state"] + torch.stack([-total, total]).int()
    return {"table": table_out, "acc": acc_out, "lens": lens_new.int(), "free": free_out, "state": state}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return _plain_write(state) if op == "write" else _plain_evict(state) if op == "evict" else _plain_attention(state)
    from paged_kv_cache_req_gb300 import _binding as B
    if op == "decode":
        B.pkv_q8_decode(state["args"], state["workspace"], state["err"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "extend":
        B.pkv_q8_extend(state["args"], state["workspace"], state["err"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "weigh":
        if case["rows_hi"]:
            B.pkv_q8_weights(state["args"], state["workspace"], state["err"])
            return {"acc": state["acc_out"]}
        B.pkv_q8_decode(state["args"], state["workspace"], state["err"])
        return {"out": state["out"], "lse": state["lse"], "acc": state["acc_out"]}
    if op == "evict":
        B.pkv_evict(state["table"], state["row"], state["lens"], state["acc"], state["budget"], state["free"],
                    state["free_state"], state["workspace"], state["err"], page_size=case["ps"],
                    num_pool_pages=state["pages"], max_seq_len=state["max_len"], keep_first=state["first"],
                    keep_last=state["last"], req_to_token_out=state["table_out"], acc_out=state["acc_out"],
                    seq_lens_out=state["lens_out"], free_state_out=state["state_out"])
        return {"table": state["table_out"], "acc": state["acc_out"], "lens": state["lens_out"], "free": state["free"],
                "state": state["state_out"]}
    B.pkv_q8_store(state["pool"], state["k_new"], state["v_new"], state["slot"], state["workspace"], state["err"],
                   page_size=case["ps"])
    B.pkv_q8_gather(state["pool"], state["table"], state["row"], state["back"], state["back_max"], state["k_out"],
                    state["v_out"], state["cu"], state["err"], page_size=case["ps"], kv_start=state["start"])
    return {"k": state["k_out"], "v": state["v_out"], "cu": state["cu"]}


# ------------------------------------------------------------------------- definition in 64 bits
def _power64(e):
    """2^e in fp64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _code64(byte):
    """fp64 value of e4m3 bytes."""
    byte = byte.long()
    e, m = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * _power64(e - 7))
    return torch.where(byte >= 128, -mag, mag)


def _byte64(st, slots, part):
    """Code bytes [n, hkv, d] and scale exponents [n, hkv] of the rows at `slots`, by the tile's byte positions."""
    case = st["case"]
    t, d, hkv = _tile(case), case["d"], case["hkv"]
    h = torch.arange(hkv, device="cuda").view(1, -1, 1)
    at = (slots % t).view(-1, 1, 1)
    where = ((2 * h + part) * t + at) * d + torch.arange(d, device="cuda")
    tile = st["pool"][slots // t]
    codes = torch.gather(tile, 1, where.flatten(1)).view(-1, hkv, d)
    e = tile[:, hkv * 2 * t * d + 2 * torch.arange(hkv, device="cuda") + part]
    return codes, e.long() - 127


def _read64(st, slots, part):
    codes, e = _byte64(st, slots, part)
    return _code64(codes) * _power64(e).unsqueeze(-1)


def _round64(x):
    """x to e4m3: three fraction bits, smallest exponent -6, ties to even, at most 448."""
    unit = _power64((torch.frexp(x.abs())[1] - 1).clamp(min=-6) - 3)
    return torch.sign(x) * (torch.round(x.abs() / unit) * unit).clamp(max=448.0)


def _exact_write(st):
    case = st["case"]
    t, hkv = _tile(case), case["hkv"]
    slot = st["slot"].cpu().numpy().astype(np.int64)
    live = np.flatnonzero(slot >= 0)
    tile_of = slot[live] // t
    names, which = np.unique(tile_of, return_inverse=True)
    fresh = np.zeros(len(names), dtype=bool)
    fresh[which[slot[live] % t == 0]] = True
    flat = st["flat"].cpu().numpy()
    place = np.searchsorted(names, flat // t)
    hit = (place < len(names)) & (names[np.minimum(place, len(names) - 1)] == flat // t)
    new_of = {int(s): int(i) for s, i in zip(slot[live], live)}
    src = np.array([new_of.get(int(s), -1) for s in flat], dtype=np.int64)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    which, fresh, place, hit, src, rows = up(which), up(fresh), up(np.where(hit, place, 0)), up(hit), up(src), up(live)
    got = []
    for part, name in enumerate("kv"):
        x = st[name + "_new"].double()
        top = torch.zeros((len(names), hkv), dtype=torch.float64, device="cuda")
        top.index_reduce_(0, which, x[rows].abs().amax(-1), "amax")
        need = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -126))).long()   # least e with top <= 448 2^e, made sure of below
        need = torch.where(448 * _power64(need - 1) >= top, need - 1, need)
        need = torch.where(448 * _power64(need) < top, need + 1, need).clamp(min=-126)
        out = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 24) // (hkv * case["d"]))
        for i in range(0, st["rows_back"], step):
            at = slice(i, min(st["rows_back"], i + step))
            codes, old = _byte64(st, st["flat"][at], part)
            e = torch.where(fresh[place[at], None], need[place[at]], torch.maximum(need[place[at]], old))
            e = _power64(torch.where(hit[at, None], e, old)).unsqueeze(-1)
            is_new = (src[at] >= 0)[:, None, None]
            value = torch.where(is_new, x[src[at].clamp(min=0)], _code64(codes) * _power64(old).unsqueeze(-1))
            out[at] = _round64(value / e) * e
        got.append(out)
    return {"k": got[0], "v": got[1], "cu": None}


def _exact_evict(st):
    """Request after request on the host; acc's values are only moved."""
    case = st["case"]
    ps, first, last = case["ps"], case["first"], case["last"]
    table, acc = st["table_host"], st["acc"].double().cpu().numpy()
    table_out, acc_out = np.zeros_like(table), np.zeros_like(acc)
    lens_out, gone_ids = [], []
    for r, length in zip(st["row_host"], st["lens_host"]):
        n = -(-length // ps)
        may_go = [p for p in range(n - 1) if p * ps >= first and (p + 1) * ps <= length - last]
        score = [np.float32(acc[r, p * ps:(p + 1) * ps].sum()) for p in may_go]
        drop = min(len(may_go), max(0, n - max(1, case["budget"] // ps)))
        worst = sorted(zip(score, [-p for p in may_go]))[:drop]                    # the later of equal ones first
        gone = sorted(-p for _, p in worst)
        gone_ids += [table[r, p * ps] // ps for p in gone]
        keep = np.delete(np.arange(length), np.concatenate([np.arange(p * ps, (p + 1) * ps) for p in gone] + [[]]).astype(int))
        lens_out.append(len(keep))
        table_out[r, :len(keep)] = table[r, keep]
        acc_out[r, :len(keep)] = acc[r, keep]
    free = st["free"].cpu().numpy().copy()
    head, count = st["free_state"].tolist()
    free[head - len(gone_ids):head] = gone_ids
    up = lambda x, like: torch.from_numpy(np.asarray(x)).to(like.device, like.dtype)  # noqa: E731
    return {"table": up(table_out, st["table"]), "acc": torch.from_numpy(acc_out).cuda(), "lens": up(lens_out, st["lens"]),
            "free": up(free, st["free"]), "state": up([head - len(gone_ids), count + len(gone_ids)], st["free_state"])}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(st)
    if case["op"] == "evict":
        return _exact_evict(st)
    hq, hkv = case["hq"], case["hkv"]
    g, rows = hq // hkv, st["rows"]
    given = case["op"] == "weigh" and case["rows_hi"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((st["q"].shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    acc = st["acc_out"].double() if case["op"] == "weigh" else None
    q0 = k0 = 0
    for b in range(case["batch"]):
        n, length = int(rows[b]), int(st["lens_host"][b])
        slots = st["flat"][k0:k0 + length]
        k, v = _read64(st, slots, 0), _read64(st, slots, 1)
        end = st["ends"][q0:q0 + n].view(-1, 1)
        pos = torch.arange(length, device="cuda")
        part = max(1, (1 << 28) // max(1, length))
        weight = torch.zeros(length, dtype=torch.float64, device="cuda")
        for h in range(hq):
            for r in range(0, n, part):
                at = slice(q0 + r, q0 + min(n, r + part))
                s = st["q"][at, h].double() @ k[:, h // g].T * st["sm_scale"]
                s = s.masked_fill(pos >= end[r:r + part], -math.inf)
                z = st["lse"][at, h:h + 1].double() if given else torch.logsumexp(s, -1, keepdim=True)
                lse[at, h] = z[:, 0]
                p = torch.exp(s - torch.where(z == -math.inf, 0.0, z))
                if not given:
                    out[at, h] = p @ v[:, h // g]
                weight += p.sum(0)
        if acc is not None:
            r = int(st["row_host"][b])
            acc[r, :length] = st["acc"][r, :length].double() + weight
        q0, k0 = q0 + n, k0 + length
    if given:
        return {"acc": acc}
    res = {"out": out, "lse": lse}
    return res if acc is None else dict(res, acc=acc)
