"""Measured cases of the operators over a paged K/V cache that is held in 4 bits.

Four operators: writing new K/V rows into the cache ("roundtrip": written, then read
back), reading a batch's rows back as bf16 ("readback"), decode attention over the cache
("decode") and attention of many query rows per request ("extend").

The cache.  A block of 16 consecutive head dims of one key (or value) row is held as 16
4-bit floats (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one 8-bit scale
(e4m3); a kv head has an fp32 scale g besides:

    s = e4m3(amax / (6 g)),   code_i = e2m1(x_i / (s g)),   value_i = code_i s g

with both roundings to nearest, ties to even, and saturating.  The pool is uint8
[tiles, kv heads, tile bytes]; a tile is t = min(page size, 64) consecutive slots of one
kv head: K codes [t, D/2], V codes [t, D/2], K scales [t, D/16], V scales [t, D/16] (two
codes per byte, the even dim in the low half), padded to a multiple of 16 bytes.

With ``own`` false, ``run`` computes the plain form in fp32 torch operations; with ``own``
true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

_BLOCK = 16


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new rows of a small batch: latency of two launches
        dict(name="write_step_b32", op="roundtrip", batch=32, hq=16, hkv=8, d=128, ps=16, lo=1, hi=1, pad=0),
        # a chunked prefill's new rows (8 requests x 1024 tokens), some of them padding
        dict(name="write_chunk_8x1024", op="roundtrip", batch=8, hq=32, hkv=8, d=128, ps=64, lo=1024, hi=1024, pad=37),
        # an encoder's output written once per request: many heads of 64 dims, ragged lengths
        dict(name="write_encoder_d64", op="roundtrip", batch=64, hq=20, hkv=20, d=64, ps=16, lo=1201, hi=1500, pad=0),
        # cached prefixes read back as bf16 before a long prefill
        dict(name="read_prefix_b32", op="readback", batch=32, hq=16, hkv=8, d=128, ps=16, lo=1, hi=4096),
        # an encoder region read back for a contiguous cross-attention
        dict(name="read_encoder_d64", op="readback", batch=64, hq=20, hkv=20, d=64, ps=16, lo=1500, hi=1500),
        # four short requests on pages of one token: the latency floor of a decode step
        dict(name="decode_tiny_ps1", op="decode", batch=4, hq=16, hkv=8, d=128, ps=1, lo=17, hi=255, layout="csr"),
        # a small model's decode step
        dict(name="decode_b32", op="decode", batch=32, hq=16, hkv=8, d=128, ps=16, lo=1, hi=4096, layout="table"),
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
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["roundtrip", "readback", "decode", "extend"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 20])
    g = rng.choice([1, 2, 4, 7, 8, 16])
    ps = rng.choice([1, 4, 16, 32, 64, 128])
    case = dict(op=op, hq=hkv * g, hkv=hkv, d=d, ps=ps)
    elems = 1 << 28                      # key elements of the padded batch
    case["batch"] = _log(rng, 1, 128)
    room = max(1, elems // (case["batch"] * hkv * d))
    hi = min(_log(rng, 1, 65536), room)
    lo = rng.choice([hi, max(1, hi // 2), min(hi, 1 + rng.randrange(64))])
    case["lo"], case["hi"] = min(lo, hi), hi
    if op == "roundtrip":
        case["pad"] = rng.choice([0, rng.randrange(1, 100)])
    if op in ("decode", "extend"):
        case["layout"] = rng.choice(["csr", "block", "table"])
    if op == "extend":
        few = rng.random() < 0.5
        cap = max(1, min(hi, (1 << 33) // (case["batch"] * case["hq"] * hi * 4)))
        rows = min(cap, _log(rng, 1, 12) if few else _log(rng, 12, 2048))
        case["rows_hi"] = rows
        case["rows_lo"] = rng.choice([rows, max(1, rows // 2), 1])
        case["bounds"] = rng.choice(["causal", "given"])
        case["hi"] = hi = max(hi, rows)
        case["lo"] = max(case["lo"], rows)
    return case


def _lens(case):
    """The requests' key counts: the case's own (log-uniform between lo and hi, shuffled)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    u = (np.arange(b) + 0.5) / b
    n = np.clip(np.round(np.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))), lo, hi).astype(np.int64)
    return np.random.RandomState(b * 7919 + hi).permutation(n)


def _rows(case):
    b, lo, hi = case["batch"], case["rows_lo"], case["rows_hi"]
    n = np.random.RandomState(b * 104729 + hi).randint(lo, hi + 1, b)
    return np.minimum(n, _lens(case)).astype(np.int64)


def _bounds(case):
    """Key bound of every query row: causal, or given ones, some of them 0."""
    lens, rows = _lens(case), _rows(case)
    if case["bounds"] == "causal":
        return np.concatenate([np.arange(l - n + 1, l + 1) for l, n in zip(lens, rows)])
    r = np.random.RandomState(case["batch"] * 31 + case["hi"])
    ends = np.concatenate([r.randint(0, l + 1, n) for l, n in zip(lens, rows)])
    ends[::7] = 0
    return ends


def work(case):
    lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
    held, plain = hkv * d * 2 * 9 // 16, hkv * d * 2 * 2      # bytes of a token's K and V, in 4 bits and in bf16
    tokens = int(lens.sum())
    if case["op"] == "roundtrip":
        return {"bytes": tokens * (2 * plain + 2 * held + 8), "flops": tokens * hkv * d * 2 * 8}
    if case["op"] == "readback":
        return {"bytes": tokens * (held + plain + 4), "flops": tokens * hkv * d * 2 * 2}
    pages = int((-(-lens // case["ps"])).sum())
    if case["op"] == "decode":
        q = case["batch"] * hq
        return {"bytes": tokens * held + q * (4 * d + 4) + 4 * pages, "flops": 4 * d * hq * tokens}
    ends, n = _bounds(case), _rows(case)
    at = np.concatenate([[0], np.cumsum(n)])
    seen = sum(int(ends[at[b]:at[b + 1]].max()) for b in range(case["batch"]) if n[b])
    q = int(n.sum()) * hq
    return {"bytes": seen * held + q * (4 * d + 4) + 4 * pages, "flops": 4 * d * hq * int(ends.sum())}


# ------------------------------------------------------------------------- inputs
def _tile(case):
    return min(case["ps"], 64)


def _tile_bytes(case):
    return -(-_tile(case) * case["d"] * 9 // 8 // 16) * 16


def _to_e4m3(x):
    """Non-negative fp32 rounded to the nearest e4m3 value (ties to even, at most 448)."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(torch.exp2(e + 1) <= x, e + 1, e)            # log2 may land just beside a power of two
    e = torch.where((torch.exp2(e) > x) & (e > -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _to_e2m1(x):
    """fp32 rounded to the nearest e2m1 value (ties to even, at most 6)."""
    a = x.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), x)


def _quantise(x, g):
    """(block scales, codes as values) of x [..., hkv, d] with head scales g [hkv], in fp32."""
    x = x.float()
    b = x.view(*x.shape[:-1], x.shape[-1] // _BLOCK, _BLOCK)
    g = g.view(-1, 1)
    s = _to_e4m3(b.abs().amax(-1) / (6.0 * g))
    den = (s * g).unsqueeze(-1)
    return s, torch.where(den > 0, _to_e2m1(b / torch.where(den > 0, den, 1.0)), torch.zeros_like(b))


def _pack(s, c):
    """Bytes [..., hkv, d/2] and [..., hkv, d/16] of scales and codes."""
    a = c.abs().flatten(-2)
    n = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    n = n | ((c.flatten(-2) < 0).to(torch.uint8) << 3)
    return n[..., 0::2] | (n[..., 1::2] << 4), s.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(gen, n, hkv, d, spread):
    """n rows as a projection gives them: normal, with a few channels several times larger."""
    x = torch.randn((n, hkv, d), generator=gen, device="cuda", dtype=torch.float32)
    ch = torch.rand((hkv, d), generator=gen, device="cuda")
    return (x * torch.where(ch < 0.05, 4.0, 1.0) * spread).to(torch.bfloat16)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    rng = np.random.RandomState(seed % (1 << 31))
    lens, ps, hkv, d, tile = _lens(case), case["ps"], case["hkv"], case["d"], _tile(case)
    batch, total = case["batch"], int(lens.sum())
    # pages: shuffled, page 0 unused
    npages = -(-lens // ps)
    pages = int(npages.sum()) + int(npages.sum()) // 8 + 2
    order = rng.permutation(pages - 1)[:int(npages.sum())] + 1
    at = np.concatenate([[0], np.cumsum(npages)])
    width = int(-(-(lens.max() + 1) // 32) * 32)
    width = -(-width // ps) * ps
    table = np.zeros((batch + 1, width), dtype=np.int32)
    row = (rng.permutation(batch) + 1).astype(np.int32)
    for b in range(batch):
        slots = (order[at[b]:at[b + 1]].astype(np.int64)[:, None] * ps + np.arange(ps)).reshape(-1)[:lens[b]]
        table[row[b], :lens[b]] = slots
    flat = np.concatenate([table[row[b], :lens[b]] for b in range(batch)]).astype(np.int64)
    st = dict(case=case, lens_host=lens, batch=batch, total=total, max_len=int(lens.max()))
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
    st["table"], st["row"], st["lens"] = up(table), up(row), up(lens.astype(np.int32))
    st["flat"] = up(flat)
    st["k_scale"] = 0.25 + torch.rand(hkv, generator=gen, device=dev)
    st["v_scale"] = 0.05 + 0.1 * torch.rand(hkv, generator=gen, device=dev)
    tiles = pages * ps // tile
    # slots that nobody wrote hold whatever was there
    st["pool"] = torch.full((tiles, hkv, _tile_bytes(case)), 0xFF, dtype=torch.uint8, device=dev)
    st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if case["op"] == "roundtrip":
        n = total + case["pad"]
        st["k_new"], st["v_new"] = _values(gen, n, hkv, d, 1.0), _values(gen, n, hkv, d, 0.3)
        slot = np.full(n, -1, dtype=np.int32)
        keep = np.sort(rng.permutation(n)[:total])           # padded tokens lie anywhere between the real ones
        slot[keep] = flat
        st["slot"], st["keep"] = up(slot), up(keep)
    else:
        kc, ks, vc, vs = _parts(case, st["pool"])
        step = max(1, (1 << 25) // (hkv * d))
        for i in range(0, total, step):
            f = st["flat"][i:i + step]
            for codes, scales, g, spread in ((kc, ks, st["k_scale"], 1.0), (vc, vs, st["v_scale"], 0.3)):
                cb, sb = _pack(*_quantise(_values(gen, f.numel(), hkv, d, spread), g))
                codes[f // tile, :, f % tile] = cb
                scales[f // tile, :, f % tile] = sb
    if case["op"] in ("roundtrip", "readback"):
        # room for a few rows more than the batch holds: those stay as they are
        st["k_out"] = torch.zeros((total + 5, hkv, d), dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.zeros_like(st["k_out"])
        st["cu"] = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
        return st
    rows = np.ones(batch, dtype=np.int64) if case["op"] == "decode" else _rows(case)
    st["rows"] = rows
    nq = int(rows.sum())
    st["q"] = _values(gen, nq, case["hq"], d, 1.0)
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
    if own:      # the argument block and the workspace, which a serving loop builds once
        from paged_kv_cache_req_gb300 import _binding as B
        kw = dict(page_size=ps, sm_scale=st["sm_scale"], max_seq_len=st["max_len"], k_scale=st["k_scale"],
                  v_scale=st["v_scale"], lse=st["lse"])
        if case["layout"] == "csr":
            layout = B.PKV_LAYOUT_CSR
            kw.update(kv_indptr=st["indptr"], kv_indices=st["indices"], kv_last_page_len=st["last"])
        elif case["layout"] == "block":
            layout = B.PKV_LAYOUT_BLOCK_TABLE
            kw.update(block_table=st["block_table"], seq_lens=st["lens"])
        else:
            layout = B.PKV_LAYOUT_REQ_TO_TOKEN
            kw.update(req_to_token=st["table"], req_pool_idx=st["row"], seq_lens=st["lens"])
        if case["op"] == "extend":
            kw.update(qo_indptr=st["qo_indptr"], total_kv=total)
            if case["bounds"] == "given":
                kw.update(kv_end=st["ends"])
        st["args"] = B.make_quant_args(layout, st["q"], st["pool"], st["out"], **kw)
        size = B.pkv_quant_decode_workspace_size if case["op"] == "decode" else B.pkv_quant_extend_workspace_size
        st["workspace"] = torch.empty(max(size(st["args"]), 256), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------------- plain form
def _parts(case, pool):
    """K codes, K scales, V codes, V scales of the pool's tiles, as views [tiles, hkv, t, ...]."""
    t, d = _tile(case), case["d"]
    n, h = pool.shape[:2]
    cut = lambda a, w: pool[:, :, a:a + t * w].unflatten(-1, (t, w))  # noqa: E731
    return cut(0, d // 2), cut(t * d, d // 16), cut(t * d // 2, d // 2), cut(t * d + t * d // 16, d // 16)


def _held(codes, scales, slots, tile):
    """fp32 code x block scale of the rows at `slots` [...]: [..., hkv, d]."""
    c = codes[slots // tile, :, slots % tile]
    s = scales[slots // tile, :, slots % tile].view(torch.float8_e4m3fn).float()
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=c.device)
    table = torch.cat([table, -table])
    v = table[torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, _BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _plain_attention(st):
    case = st["case"]
    hq, hkv, d, batch, m = case["hq"], case["hkv"], case["d"], st["batch"], st["max_len"]
    g, nmax = hq // hkv, int(st["rows"].max())
    kc, ks, vc, vs = _parts(case, st["pool"])
    pos = torch.arange(m, device="cuda")
    live = pos < st["lens"][:, None]                                               # [B, M]
    slots = torch.where(live, st["table"][st["row"].long()][:, :m].long(), 0)
    k = torch.where(live[..., None, None], _held(kc, ks, slots, _tile(case)), 0.0)  # [B, M, hkv, d]
    k = k * st["k_scale"].view(-1, 1)
    q = torch.zeros((batch * nmax, hq, d), device="cuda")
    q[st["q_at"]] = st["q"].float()
    q = q.view(batch, nmax, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nmax * g, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["sm_scale"]                     # [B, hkv, nmax g, M]
    del k
    end = torch.zeros(batch * nmax, dtype=torch.int32, device="cuda")
    end[st["q_at"]] = st["ends"]
    seen = (pos < end.view(batch, 1, nmax, 1, 1)).expand(batch, 1, nmax, g, m).reshape(batch, 1, nmax * g, m)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(base).exp_()
    den = p.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], _held(vc, vs, slots, _tile(case)), 0.0)
    v = v * st["v_scale"].view(-1, 1)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(den > 0, den, 1.0)
    lse = torch.where(den > 0, torch.log(den) + base, -math.inf)
    o = o.view(batch, hkv, nmax, g, d).permute(0, 2, 1, 3, 4).reshape(batch * nmax, hq, d)[st["q_at"]]
    lse = lse.view(batch, hkv, nmax, g).permute(0, 2, 1, 3).reshape(batch * nmax, hq)[st["q_at"]]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain(st):
    case = st["case"]
    if case["op"] in ("decode", "extend"):
        return _plain_attention(st)
    got = []
    parts = _parts(case, st["pool"])
    for i, (name, g) in enumerate((("k", st["k_scale"]), ("v", st["v_scale"]))):
        if case["op"] == "roundtrip":
            s, c = _quantise(st[name + "_new"][st["keep"]], g)
            x = (c * s.unsqueeze(-1)).flatten(-2)
        else:
            x = _held(parts[2 * i], parts[2 * i + 1], st["flat"], _tile(case))
        out = torch.zeros_like(st["k_out"])
        out[:st["total"]] = (x * g.view(-1, 1)).to(torch.bfloat16)
        got.append(out)
    cu = torch.zeros(st["batch"] + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(st["lens"], 0)
    return {"k": got[0], "v": got[1], "cu": cu}


def run(state):
    case = state["case"]
    if not own:
        return _plain(state)
    from paged_kv_cache_req_gb300 import _binding as B
    if case["op"] == "decode":
        B.pkv_quant_decode(state["args"], state["workspace"], state["err"])
        return {"out": state["out"], "lse": state["lse"]}
    if case["op"] == "extend":
        B.pkv_quant_extend(state["args"], state["workspace"], state["err"])
        return {"out": state["out"], "lse": state["lse"]}
    if case["op"] == "roundtrip":
        B.pkv_quant_store(state["pool"], state["k_new"], state["v_new"], state["slot"], state["err"],
                          page_size=case["ps"], k_scale=state["k_scale"], v_scale=state["v_scale"])
    B.pkv_quant_gather(state["pool"], state["table"], state["row"], state["lens"], state["max_len"], state["k_out"],
                       state["v_out"], state["cu"], state["err"], page_size=case["ps"], k_scale=state["k_scale"],
                       v_scale=state["v_scale"])
    return {"k": state["k_out"], "v": state["v_out"], "cu": state["cu"]}


# ------------------------------------------------------------------------- definition in 64 bits
def _round_to(x, mantissa, least, most):
    """x to `mantissa` fraction bits with smallest exponent `least`, ties to even, at most `most`."""
    e = (torch.frexp(x.abs())[1] - 1).clamp(min=least).double()
    unit = 2.0 ** (e - mantissa)
    return torch.sign(x) * (torch.round(x.abs() / unit) * unit).clamp(max=most)


def _read64(st, slots, part):
    """fp64 K (part 0) or V (part 1) rows at `slots`, decoded from the pool's bytes one field at a time."""
    case = st["case"]
    t, d = _tile(case), case["d"]
    tiles = st["pool"][slots // t]                                      # [n, hkv, bytes]
    at = (slots % t).view(-1, 1, 1)
    i = torch.arange(d, device=slots.device).view(1, 1, -1)
    byte = torch.gather(tiles, 2, (part * t * d // 2 + at * (d // 2) + i // 2).expand(-1, case["hkv"], -1)).long()
    code = (byte >> (4 * (i % 2))) & 15
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double())
    byte = torch.gather(tiles, 2, (t * d + part * t * d // 16 + at * (d // 16) + i // 16).expand(-1, case["hkv"], -1)).long()
    e, m = (byte >> 3) & 15, (byte & 7).double()
    s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7).double())
    g = st["v_scale" if part else "k_scale"].double().view(1, -1, 1)
    return torch.where(code >= 8, -mag, mag) * s * g


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("roundtrip", "readback"):
        got = []
        for part, name in enumerate("kv"):
            out = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            step = max(1, (1 << 24) // (case["hkv"] * case["d"]))
            for i in range(0, st["total"], step):
                if case["op"] == "readback":
                    out[i:i + step][:st["total"] - i] = _read64(st, st["flat"][i:i + step], part)
                    continue
                x = st[name + "_new"][st["keep"][i:i + step]].double()
                g = st[name + "_scale"].double().view(1, -1, 1)
                b = x.view(x.shape[0], x.shape[1], -1, _BLOCK)
                s = _round_to(b.abs().amax(-1) / (6 * g), 3, -6, 448.0)
                den = (s * g).unsqueeze(-1)
                c = _round_to(b / torch.where(den > 0, den, 1.0), 1, 0, 6.0)
                out[i:i + step][:st["total"] - i] = torch.where(den > 0, c * den, 0.0).flatten(-2)
            got.append(out)
        return {"k": got[0], "v": got[1], "cu": None}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, rows = hq // hkv, st["rows"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b in range(case["batch"]):
        n, length = int(rows[b]), int(st["lens_host"][b])
        slots = st["flat"][k0:k0 + length]
        k, v = _read64(st, slots, 0), _read64(st, slots, 1)
        end = st["ends"][q0:q0 + n].view(-1, 1)
        pos = torch.arange(length, device="cuda")
        part = max(1, (1 << 28) // max(1, length))
        for h in range(hq):
            for r in range(0, n, part):
                at = slice(q0 + r, q0 + min(n, r + part))
                s = st["q"][at, h].double() @ k[:, h // g].T * st["sm_scale"]
                s = s.masked_fill(pos >= end[r:r + part], -math.inf)
                z = torch.logsumexp(s, -1, keepdim=True)
                lse[at, h] = z[:, 0]
                out[at, h] = torch.exp(s - torch.where(z == -math.inf, 0.0, z)) @ v[:, h // g]
        q0, k0 = q0 + n, k0 + length
    return {"out": out, "lse": lse}
