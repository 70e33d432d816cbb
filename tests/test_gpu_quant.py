"""The 4-bit K/V pool on the GPU: writing, reading back, decode and multi-query attention,
against the plain fp64 reference (bounds derived in _quant_ref), at the sizes, layouts and
masks where they can go wrong."""
import numpy as np
import pytest
import torch

import _quant_ref as R
from _harness import paged_table

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def values(rng, shape, spread=1.0):
    """bf16 normals (as fp32), some channels larger."""
    x = rng.standard_normal(shape) * spread * np.where(rng.random(shape[-1]) < 0.05, 5.0, 1.0)
    return R.bf16(x)


def head_scales(rng, H):
    return rng.uniform(0.2, 1.5, H).astype(np.float32), rng.uniform(0.02, 0.2, H).astype(np.float32)


def to_bf16(x):
    return up(x).to(torch.bfloat16)


def host(t):
    return t.detach().float().cpu().numpy()


# --------------------------------------------------------------------------- store
@pytest.mark.parametrize("D,ps,H,n", [(128, 16, 8, 33), (128, 64, 2, 130), (64, 1, 3, 17), (128, 1, 1, 5), (64, 4, 20, 9),
                                      (64, 128, 1, 64), (128, 1024, 2, 7), (64, 2, 5, 1)])
@pytest.mark.parametrize("form", ["plain", "slice", "odd"])
def test_store_bytes(B, D, ps, H, n, form):
    rng = np.random.default_rng(D * 1000 + ps + H + n)
    t, nb = R.tile_of(ps), R.tile_bytes(ps, D)
    tiles = max(4, -(-2 * n // t) + 2)
    k, v = values(rng, (n, H, D)), values(rng, (n, H, D), 0.1)
    # exact ties, zeros, a block of one value, tiny and large values
    k[0, 0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0]
    k[0, 0, 16:32] = 0.0
    v[0, 0, :16] = R.bf16(np.full(16, 1e-30))
    v[0, 0, 16:32] = R.bf16(np.full(16, 3e38))
    k[-1, -1, 32:48] = R.bf16(np.float32(2.0) ** np.arange(-12, 4))
    k[-1, -1, 48] = np.inf
    v[-1, -1, 50] = np.nan
    ks, vs = head_scales(rng, H)
    ks[0] = 1.0
    slots = rng.permutation(tiles * t)[:n].astype(np.int32)
    pad = rng.random(n) < 0.2
    pad[[0, -1]] = False
    mapping = np.where(pad, -1 - rng.integers(0, 5, n), slots).astype(np.int32)
    before = rng.integers(0, 256, (tiles, H, nb)).astype(np.uint8)
    want = before.copy()
    for part, x, g in ((0, k, ks), (1, v, vs)):
        c, s = R.quantise(x[~pad], g)
        R.write(want, ps, slots[~pad], part, c, s)
    if form == "plain":
        kd, vd = to_bf16(k), to_bf16(v)
    else:       # K and V as slices of one wider row; `odd` also 2 bytes off any alignment
        off = 1 if form == "odd" else 8
        wide = torch.zeros((n, off + 2 * H * D + 7 + (1 if form == "slice" else 0)), dtype=torch.bfloat16, device=DEV)
        wide[:, off:off + H * D] = to_bf16(k).view(n, -1)
        wide[:, off + H * D:off + 2 * H * D] = to_bf16(v).view(n, -1)
        kd = wide[:, off:off + H * D].unflatten(1, (H, D))
        vd = wide[:, off + H * D:off + 2 * H * D].unflatten(1, (H, D))
    store = torch.zeros((tiles, H + 1, nb), dtype=torch.uint8, device=DEV)     # tiles further apart than they are long
    pool = store[:, :H]
    pool.copy_(up(before))
    err = err_word()
    B.pkv_quant_store(pool, kd, vd, up(mapping), err, page_size=ps, k_scale=up(ks), v_scale=up(vs))
    assert err.item() == 0
    got = pool.cpu().numpy()
    assert (got == want).all(), "%d bytes differ" % (got != want).sum()
    assert not store[:, H:].any()


@pytest.mark.parametrize("e", [-126, -100, -85, -60, -20, 20, 100, 125])
def test_store_with_any_head_scale(B, e):
    """g = 2^e against magnitudes from 2^-120 to 2^127: saturated, vanishing and far quotients."""
    rng = np.random.default_rng(300 + e)
    n, H, D, ps = 64, 1, 64, 16
    x = values(rng, (n, H, D))
    x = R.bf16(np.clip(x, -3, 3) * np.float32(2.0) ** np.linspace(-120, 126, n).astype(np.int64)[:, None, None])
    x[::5, :, ::7] = 0.0
    g = np.array([2.0 ** e], dtype=np.float32)
    pool = torch.zeros((n // ps, H, R.tile_bytes(ps, D)), dtype=torch.uint8, device=DEV)
    want = pool.cpu().numpy()
    for part in (0, 1):
        R.write(want, ps, np.arange(n), part, *R.quantise(x, g))
    err = err_word()
    B.pkv_quant_store(pool, to_bf16(x), to_bf16(x), up(np.arange(n, dtype=np.int32)), err, page_size=ps, k_scale=up(g), v_scale=up(g))
    assert err.item() == 0
    got = pool.cpu().numpy()
    assert (got == want).all(), "%d bytes differ" % (got != want).sum()


def test_store_flags(B):
    rng = np.random.default_rng(3)
    k = values(rng, (4, 2, 128))
    for mapping, ks, bit in (([0, 64, 1, -1], [1, 1], 1), ([0, 1, 2, 3], [1, 0], 1), ([0, 1, 2, 3], [np.nan, 1], 1),
                             ([0, 1, 2, 3], [-1, 1], 1), ([0, 1, 2, 3], [np.inf, 1], 1), ([0, 1, 2, 63], [1, 1], 0)):
        pool = torch.full((4, 2, R.tile_bytes(16, 128)), 7, dtype=torch.uint8, device=DEV)
        err = err_word()
        g = np.asarray(ks, dtype=np.float32)
        B.pkv_quant_store(pool, to_bf16(k), to_bf16(k), up(np.asarray(mapping, dtype=np.int32)), err, page_size=16,
                          k_scale=up(g))
        assert err.item() == bit
        want = np.full(tuple(pool.shape), 7, dtype=np.uint8)
        live = [i for i, s in enumerate(mapping) if 0 <= s < 64]
        for part in (0, 1):
            c, s = R.quantise(k[live], np.where(np.isfinite(g) & (g > 0), g, 1) if part == 0 else np.ones(2, np.float32))
            R.write(want, 16, [mapping[i] for i in live], part, c, s)
        bad = [h for h in range(2) if not (np.isfinite(g[h]) and g[h] > 0)]
        got = pool.cpu().numpy()
        if not bad:
            assert (got == want).all()
        for h in bad:      # that head's K is left alone, its V written
            assert (got[:, h, :16 * 64] == 7).all()
            assert (got[:, 1 - h] == want[:, 1 - h]).all()


# --------------------------------------------------------------------------- gather
@pytest.mark.parametrize("D,ps,H,lens", [(128, 16, 8, [0, 1, 17, 300, 16]), (64, 1, 3, [5, 0, 0, 70]), (128, 64, 1, [64, 65, 63, 1000]),
                                         (64, 128, 20, [129, 3]), (128, 4, 2, [2000]), (64, 16, 4, [0, 0])])
def test_gather_bits(B, D, ps, H, lens):
    rng = np.random.default_rng(D + ps + H)
    starts = np.array([(b % 3) * 5 for b in range(len(lens))], dtype=np.int32)
    pages = sum(-(-(l + 20) // ps) + 1 for l in lens) + 3
    r2t, rpi = paged_table(rng, [l + s for l, s in zip(lens, starts)], ps, pages)
    t = R.tile_of(ps)
    pool = rng.integers(0, 256, (-(-pages * ps // t), H, R.tile_bytes(ps, D))).astype(np.uint8)
    ks, vs = head_scales(rng, H)
    total = sum(lens)
    flat = np.concatenate([r2t[rpi[b], starts[b]:starts[b] + l] for b, l in enumerate(lens)] + [np.zeros(0, np.int32)])
    k_out = torch.full((total + 3, H, D), 5.0, dtype=torch.bfloat16, device=DEV)
    v_out = torch.full((total + 3, H, D), 6.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.full((len(lens) + 1,), -7, dtype=torch.int32, device=DEV)
    err = err_word()
    B.pkv_quant_gather(up(pool), up(r2t), up(rpi), up(np.array(lens, dtype=np.int32)), max(lens), k_out, v_out, cu, err,
                       page_size=ps, k_scale=up(ks), v_scale=up(vs), kv_start=up(starts))
    assert err.item() == 0
    assert cu.tolist() == np.concatenate([[0], np.cumsum(lens)]).tolist()
    for part, out, g, fill in ((0, k_out, ks, 5.0), (1, v_out, vs, 6.0)):
        got = host(out)
        assert (got[total:] == fill).all()
        # (scale x g) rounded to fp32, x code rounded to fp32, rounded to bf16
        code = R.read(pool, ps, D, flat, part)
        with np.errstate(invalid="ignore"):
            want = code.astype(np.float32) * g.reshape(1, H, 1)
            tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -22)
            R.assert_within(got[:total], want, tol, "gather")
    # without head scales every value is exact
    B.pkv_quant_gather(up(pool), up(r2t), up(rpi), up(np.array(lens, dtype=np.int32)), max(lens), k_out, v_out, cu, err,
                       page_size=ps, kv_start=up(starts))
    for part, out in ((0, k_out), (1, v_out)):
        want = R.read(pool, ps, D, flat, part)
        got = host(out)[:total].astype(np.float64)
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()


def test_gather_flags(B):
    rng = np.random.default_rng(5)
    lens = [20, 40, 10]
    r2t, rpi = paged_table(rng, lens, 16, 12)
    pool = up(rng.integers(0, 100, (12, 2, R.tile_bytes(16, 128))).astype(np.uint8))

    def call(table=r2t, rows=rpi, sl=lens, cap=80, scale=None):
        k = torch.full((80, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        v = torch.full_like(k, 9.0)
        cu, err = torch.zeros(4, dtype=torch.int32, device=DEV), err_word()
        B.pkv_quant_gather(pool, up(table), up(rows), up(np.array(sl, dtype=np.int32)), 40, k[:cap], v[:cap], cu, err,
                           page_size=16, v_scale=scale)
        return host(k), cu.tolist(), err.item()

    good, cu, e = call()
    assert e == 0 and cu == [0, 20, 60, 70] and (good[70:] == 9).all()
    bad = r2t.copy()
    bad[rpi[1], 3], bad[rpi[1], 4] = 12 * 16, -1
    k, cu, e = call(table=bad)
    assert e == 1 and (k[23:25] == 0).all() and (np.delete(k, [23, 24], 0) == np.delete(good, [23, 24], 0)).all()
    rows = rpi.copy()
    rows[0] = 99
    k, cu, e = call(rows=rows)
    assert e == 1 and (k[:20] == 0).all() and (k[20:] == good[20:]).all()
    k, cu, e = call(cap=50)
    assert e == 4 and cu == [0, 20, 60, 70] and (k[:50] == good[:50]).all() and (k[50:] == 9).all()
    k, cu, e = call(sl=[20, -4, 10])
    assert e == 1 and cu == [0, 20, 20, 30] and (k[20:30] == good[60:70]).all()
    assert call(scale=up(np.array([0.0, 1.0], dtype=np.float32)))[2] == 1


# --------------------------------------------------------------------------- attention
class Cache:
    """A 4-bit pool holding the given lengths on shuffled pages; every byte that no key owns
    is a NaN scale or an all-ones code."""

    def __init__(self, rng, lens, ps, H, D, spread=1.0, starts=None):
        self.lens, self.ps, self.H, self.D = list(lens), ps, H, D
        starts = [0] * len(lens) if starts is None else starts
        self.starts = np.array(starts, dtype=np.int32)
        pages = sum(-(-l // ps) for l in lens) + 3
        self.r2t, self.rpi = paged_table(rng, lens, ps, pages, kv_start=starts)
        self.pages = pages
        t = R.tile_of(ps)
        self.pool = np.full((-(-pages * ps // t), H, R.tile_bytes(ps, D)), 0xFF, dtype=np.uint8)
        self.ks, self.vs = head_scales(rng, H)
        self.slots = [self.r2t[self.rpi[b], s:s + l].astype(np.int64) for b, (l, s) in enumerate(zip(lens, starts))]
        flat = np.concatenate(self.slots + [np.zeros(0, np.int64)])
        for part, g, sp in ((0, self.ks, spread), (1, self.vs, 0.3)):
            R.write(self.pool, ps, flat, part, *R.quantise(values(rng, (len(flat), H, D), sp), g))

    def kv(self, b):
        return (R.read(self.pool, self.ps, self.D, self.slots[b], 0, self.ks),
                R.read(self.pool, self.ps, self.D, self.slots[b], 1, self.vs))

    def layout(self, B, name):
        npg = [-(-l // self.ps) for l in self.lens]
        lists = [s[::self.ps] // self.ps for s in self.slots]
        lens = up(np.array(self.lens, dtype=np.int32))
        if name == "csr":
            last = np.array([l - (n - 1) * self.ps if n else 0 for l, n in zip(self.lens, npg)], dtype=np.int32)
            idx = np.concatenate(lists + [np.zeros(0, np.int64)]).astype(np.int32)
            return B.PKV_LAYOUT_CSR, dict(kv_indptr=up(np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)),
                                          kv_indices=up(idx) if len(idx) else torch.zeros(1, dtype=torch.int32, device=DEV),
                                          kv_last_page_len=up(last))
        if name == "block":
            bt = np.full((len(npg), max(npg + [1])), -1, dtype=np.int32)
            for b, x in enumerate(lists):
                bt[b, :len(x)] = x
            return B.PKV_LAYOUT_BLOCK_TABLE, dict(block_table=up(bt), seq_lens=lens)
        return B.PKV_LAYOUT_REQ_TO_TOKEN, dict(req_to_token=up(self.r2t), req_pool_idx=up(self.rpi), seq_lens=lens,
                                               kv_start=up(self.starts))

    def args(self, B, layout, q, out, **kw):
        lay, fields = self.layout(B, layout)
        fields.update(page_size=self.ps, sm_scale=self.D ** -0.5, max_seq_len=max(self.lens + [1]), k_scale=up(self.ks),
                      v_scale=up(self.vs))
        fields.update(kw)
        return B.make_quant_args(lay, q, fields.pop("pool", None) if "pool" in fields else up(self.pool), out, **fields)


def decode(B, cache, q, layout="table", **kw):
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device=DEV)
    err = err_word()
    a = cache.args(B, layout, q, out, lse=lse, **kw)
    ws = torch.full((B.pkv_quant_decode_workspace_size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_quant_decode(a, ws, err)
    return out, lse, err.item()


def extend(B, cache, q, rows, layout="table", kv_end=None, **kw):
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device=DEV)
    err = err_word()
    kw.setdefault("qo_indptr", up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)))
    a = cache.args(B, layout, q, out, lse=lse, kv_end=None if kv_end is None else up(np.asarray(kv_end, dtype=np.int32)), **kw)
    ws = torch.full((B.pkv_quant_extend_workspace_size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_quant_extend(a, ws, err)
    return out, lse, err.item()


def check(cache, q, out, lse, rows=None, kv_end=None, only=None, sm_scale=None):
    """Every (or only the named) request's rows against the reference."""
    n = [1] * len(cache.lens) if rows is None else list(rows)
    at = np.concatenate([[0], np.cumsum(n)])
    qh, oh, lh = host(q).astype(np.float64), host(out), host(lse)
    for b, L in enumerate(cache.lens):
        if n[b] == 0 or (only is not None and b not in only):
            continue
        sl = slice(at[b], at[b + 1])
        if kv_end is not None:
            ends = np.asarray(kv_end)[sl]
        else:
            ends = [L] if rows is None else np.arange(L - n[b] + 1, L + 1)
        k, v = cache.kv(b)
        ref, rl, tol, lt = R.attention(qh[sl], k, v, ends, cache.D ** -0.5 if sm_scale is None else sm_scale)
        R.assert_within(oh[sl], ref, tol, "request %d (L %d) out" % (b, L))
        R.assert_within(lh[sl], rl, lt, "request %d (L %d) lse" % (b, L))


DECODE = [  # D, ps, H, g, lens, layout, kv_chunk
    (128, 16, 8, 2, [17, 64, 100, 255], "table", 0),
    (128, 1, 8, 2, [17, 64, 100, 255], "csr", 0),
    (128, 64, 2, 4, [0, 1, 63, 64, 65, 128, 700], "block", 0),
    (64, 16, 5, 1, [448, 1, 0, 33], "table", 64),
    (64, 1, 1, 16, [5, 130, 1], "csr", 64),
    (64, 2, 3, 3, [90, 2, 7], "block", 0),
    (128, 4, 2, 7, [257, 31], "csr", 128),
    (128, 8, 1, 8, [1000], "table", 64),
    (128, 256, 2, 5, [300, 256, 10], "block", 0),
    (64, 1024, 2, 12, [1500, 1024], "csr", 0),
    (128, 32, 4, 16, [4099, 3], "table", 0),
    (64, 64, 1, 1, [1], "block", 0),
    (128, 16, 1, 4, [12345], "csr", 0),
]


@pytest.mark.parametrize("D,ps,H,g,lens,layout,chunk", DECODE)
def test_decode(B, D, ps, H, g, lens, layout, chunk):
    rng = np.random.default_rng(D + ps * 3 + H * 7 + g)
    cache = Cache(rng, lens, ps, H, D, starts=[(b % 2) * ps for b in range(len(lens))] if layout == "table" else None)
    q = to_bf16(values(rng, (len(lens), H * g, D)))
    out, lse, e = decode(B, cache, q, layout, kv_chunk=chunk)
    assert e == 0
    check(cache, q, out, lse)


def test_decode_many_requests_all_layouts_agree(B):
    """A batch larger than the grid: uneven lengths, and the three layouts bit for bit the same."""
    rng = np.random.default_rng(11)
    lens = np.exp(rng.uniform(0, np.log(600), 700)).astype(int).tolist()
    cache = Cache(rng, lens, 16, 2, 128)
    q = to_bf16(values(rng, (700, 8, 128)))
    out, lse, e = decode(B, cache, q, "csr")
    assert e == 0
    check(cache, q, out, lse, only=list(range(0, 700, 37)) + [int(np.argmax(lens))])
    for layout in ("block", "table"):
        o2, l2, e = decode(B, cache, q, layout)
        assert e == 0 and torch.equal(out, o2) and torch.equal(lse, l2)


def test_decode_same_result_every_time(B):
    rng = np.random.default_rng(12)
    cache = Cache(rng, [3000, 5, 900], 16, 4, 128)
    q = to_bf16(values(rng, (3, 16, 128)))
    first = decode(B, cache, q)
    for _ in range(5):
        again = decode(B, cache, q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("qs", [1e-30, 1e-4, 1.0, 200.0, 3e4, 1e30])
def test_query_magnitudes(B, qs):
    """Queries far from 1 (fp16's range included): scores scale exactly with them."""
    rng = np.random.default_rng(13)
    cache = Cache(rng, [130, 64], 16, 2, 128, spread=0.02)
    x = values(rng, (2, 8, 128)).astype(np.float64) * qs
    x[0, 0, :64] *= 2.0 ** -30                     # one row of very uneven magnitudes
    x[1, 3] = 0.0
    q = to_bf16(R.bf16(x))
    sm = float(np.float32(0.05 / qs))
    out, lse, e = decode(B, cache, q, sm_scale=sm)
    assert e == 0
    check(cache, q, out, lse, sm_scale=sm)


def test_peaked_and_equal_weights(B):
    """One key far above the rest, in the first, the last and a middle tile; and all keys equal."""
    rng = np.random.default_rng(14)
    cache = Cache(rng, [500, 500, 500, 500], 16, 1, 64)
    one = np.zeros((1, 1, 64))
    one[..., :] = 40.0
    for b, t in ((0, 0), (1, 499), (2, 250)):
        R.write(cache.pool, 16, cache.slots[b][t:t + 1], 0, *R.quantise(one.astype(np.float32), cache.ks))
    same = np.broadcast_to(R.bf16(rng.standard_normal((1, 1, 64))), (500, 1, 64))
    R.write(cache.pool, 16, cache.slots[3], 0, *R.quantise(same, cache.ks))
    q = to_bf16(np.abs(values(rng, (4, 4, 64))))
    out, lse, e = decode(B, cache, q)
    assert e == 0
    check(cache, q, out, lse)


def test_a_poisoned_key_reaches_only_who_sees_it(B):
    """A NaN in a stored row makes the outputs that see it NaN (their head, their rows), and no others."""
    rng = np.random.default_rng(15)
    for rows in ([1, 1], [6, 3], [150, 40]):
        cache = Cache(rng, [200, 90], 16, 2, 128)
        bad = values(rng, (1, 2, 128))
        c, s = R.quantise(bad, cache.ks)
        s[0, 1, 3] = 0x7f
        R.write(cache.pool, 16, cache.slots[0][199:200], 0, c, s)
        q = to_bf16(values(rng, (sum(rows), 4, 128)))
        if rows == [1, 1]:
            out, lse, e = decode(B, cache, q)
        else:
            out, lse, e = extend(B, cache, q, rows)
        assert e == 0
        o, l = host(out), host(lse)
        seen = np.zeros(o.shape[:2], dtype=bool)
        seen[rows[0] - 1, 2:] = True                      # the last row of request 0, heads of kv head 1
        assert np.isnan(l[seen]).all() and np.isnan(o[seen]).all()
        assert np.isfinite(l[~seen]).all() and np.isfinite(o[~seen]).all()


EXTEND = [  # D, ps, H, g, lens, rows, layout, kv_chunk
    (128, 16, 8, 2, [40, 300, 5], [4, 4, 4], "table", 0),
    (128, 64, 2, 4, [1000, 64, 65, 9], [1, 7, 0, 9], "csr", 0),
    (64, 1, 2, 1, [100, 33], [33, 33], "block", 64),
    (64, 16, 1, 16, [400], [77], "table", 128),
    (128, 8, 2, 3, [260, 12], [50, 12], "csr", 0),
    (128, 32, 1, 7, [700], [129], "block", 256),
    (64, 256, 4, 5, [513, 200], [100, 200], "csr", 0),
    (128, 16, 2, 2, [1100, 1024], [600, 513], "table", 0),
    (128, 2, 1, 4, [3], [3], "table", 0),
    (64, 4, 3, 1, [600, 0, 300], [300, 0, 1], "table", 0),
    (128, 64, 1, 8, [2048], [300], "block", 512),
    (128, 16, 1, 1, [1], [1], "csr", 0),
]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("D,ps,H,g,lens,rows,layout,chunk", EXTEND)
def test_extend(B, D, ps, H, g, lens, rows, layout, chunk, given):
    rng = np.random.default_rng(D + ps * 3 + H * 7 + g)
    cache = Cache(rng, lens, ps, H, D, starts=[((b + 1) % 2) * ps for b in range(len(lens))] if layout == "table" else None)
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    ends = None
    if given:       # bounds in any order, rows without keys among them
        ends = np.concatenate([rng.integers(0, l + 1, n) for l, n in zip(lens, rows)]).astype(np.int32)
        ends[::5] = 0
    out, lse, e = extend(B, cache, q, rows, layout, ends, kv_chunk=chunk, total_kv=sum(lens))
    assert e == 0
    check(cache, q, out, lse, rows, ends)


def test_extend_mixed_steps(B):
    """One prompt chunk among single-token rows (and requests without rows), strided queries."""
    rng = np.random.default_rng(21)
    lens = [900] + [int(x) for x in rng.integers(1, 500, 60)]
    rows = [800] + [1] * 50 + [0] * 10
    cache = Cache(rng, lens, 16, 2, 128)
    wide = torch.zeros((sum(rows), 3, 8, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 1] = to_bf16(values(rng, (sum(rows), 8, 128)))
    q = wide[:, 1]
    out, lse, e = extend(B, cache, q, rows)
    assert e == 0
    check(cache, q, out, lse, rows, only=[0, 1, 2, 30, 50])


def test_extend_of_one_row_equals_decode_within_rounding(B):
    rng = np.random.default_rng(22)
    cache = Cache(rng, [100, 2000], 16, 2, 128)
    q = to_bf16(values(rng, (2, 8, 128)))
    o1, l1, _ = decode(B, cache, q)
    o2, l2, _ = extend(B, cache, q, [1, 1])
    check(cache, q, o1, l1)
    check(cache, q, o2, l2)


# --------------------------------------------------------------------------- flags
def test_attention_flags(B):
    rng = np.random.default_rng(31)
    cache = Cache(rng, [100, 70, 50], 16, 2, 128)
    q = to_bf16(values(rng, (3, 4, 128)))

    def one(layout="csr", **kw):
        """The output and flags; the requests that nothing is wrong with hold the right values."""
        out, lse, e = decode(B, cache, q, layout, **kw)
        if "k_scale" not in kw and "v_scale" not in kw and "kv_indptr" not in kw and "kv_last_page_len" not in kw:
            check(cache, q, out, lse, only=[1, 2])
        return out, e

    assert one()[1] == 0

    _, f = cache.layout(B, "csr")
    idx = f["kv_indices"].cpu().numpy()
    for page in (-1, cache.pages + 100, 2 ** 31 - 1):
        bad = idx.copy()
        bad[2] = page
        out, e = one(kv_indices=up(bad))
        assert e == 1
        assert torch.isfinite(out[0].float()).all()
    for bad in ([0, 999, 11, 15], [-3, 7, 12, 16], [0, 12, 7, 16]):
        out, e = one(kv_indptr=up(np.array(bad, dtype=np.int32)))
        assert e & 1
    for bad in ([0, 6, 2], [4, 17, 2], [4, -1, 2]):
        out, e = one(kv_last_page_len=up(np.array(bad, dtype=np.int32)))
        assert e & 1
    out, e = one(max_seq_len=80)
    assert e == 4
    # token table: rows and regions outside it, a page start off its page
    for kw in (dict(req_pool_idx=up(np.array([99, cache.rpi[1], cache.rpi[2]], dtype=np.int32))),
               dict(kv_start=up(np.array([8, 0, 0], dtype=np.int32))), dict(kv_start=up(np.array([-16, 0, 0], dtype=np.int32))),
               dict(seq_lens=up(np.array([-5, 70, 50], dtype=np.int32))),
               dict(kv_start=up(np.array([16 * 1000, 0, 0], dtype=np.int32)))):
        out, e = one("table", **kw)
        assert e == 1 and (out[0] == 0).all()
    bad = cache.r2t.copy()
    bad[cache.rpi[0], 32] += 1
    out, e = one("table", req_to_token=up(bad))
    assert e == 2
    bad[cache.rpi[0], 32] = -4
    assert one("table", req_to_token=up(bad))[1] == 1
    assert one(k_scale=up(np.array([1.0, -1.0], dtype=np.float32)))[1] == 1
    assert one(v_scale=up(np.array([np.nan, 1.0], dtype=np.float32)))[1] == 1


@pytest.mark.parametrize("rows", [[5, 3], [300, 200]])
def test_extend_flags(B, rows):
    rng = np.random.default_rng(32)
    lens = [400, 300]
    cache = Cache(rng, lens, 16, 2, 128)
    q = to_bf16(values(rng, (sum(rows), 8, 128)))
    out, lse, e = extend(B, cache, q, rows)
    assert e == 0
    check(cache, q, out, lse, rows)
    ends = np.concatenate([np.arange(l - n + 1, l + 1) for l, n in zip(lens, rows)])
    bad = ends.copy()
    bad[1], bad[rows[0] - 1] = -1, 401
    out, lse, e = extend(B, cache, q, rows, kv_end=bad)
    assert e == 1 and (out[1] == 0).all() and (out[rows[0] - 1] == 0).all()
    check(cache, q, out, lse, rows, only=[1])
    # more causal rows than keys: the request has no rows
    cache.lens[0] = rows[0] - 1
    out, lse, e = extend(B, cache, q, rows)
    assert e == 1 and (out[:rows[0]] == 3).all()
    check(cache, q, out, lse, rows, only=[1])
    cache.lens[0] = 400
    out, lse, e = extend(B, cache, q, rows, max_seq_len=350)
    assert e == 4
    check(cache, q, out, lse, rows, only=[1])


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("ps,D", [(16, 128), (1, 64), (64, 128)])
def test_a_serving_loop(B, ps, D):
    """Allocate, lay out, quantise, attend, step by step: a chunk of each prompt, then single
    tokens, then everything read back; no page list in between."""
    rng = np.random.default_rng(41)
    H, g, nreq, pages = 2, 4, 5, 400 if ps == 1 else 64
    plan = [[70, 1, 33, 100, 17]] + [[1] * 5] * 3
    t = R.tile_of(ps)
    cap = pages * ps
    pool = torch.full((-(-cap // t), H, B.pkv_quant_tile_bytes(ps, D)), 0xFF, dtype=torch.uint8, device=DEV)
    ref = np.full(tuple(pool.shape), 0xFF, dtype=np.uint8)
    r2t = torch.zeros((nreq + 1, 128), dtype=torch.int32, device=DEV)
    rpi = up((rng.permutation(nreq) + 1).astype(np.int32))
    free = up((rng.permutation(pages - 1) + 1).astype(np.int32))
    state = up(np.array([0, pages - 1], dtype=np.int32))
    ks, vs = head_scales(rng, H)
    ksd, vsd = up(ks), up(vs)
    err = err_word()
    lens = np.zeros(nreq, dtype=np.int32)
    last = np.full(nreq, -1, dtype=np.int32)
    for new in plan:
        prefix, lens = lens.copy(), lens + np.array(new, dtype=np.int32)
        loc = torch.zeros(sum(new), dtype=torch.int32, device=DEV)
        B.pkv_alloc_extend(up(prefix), up(lens), up(last), ps, pages, free, state, loc, err)
        B.pkv_write_req_to_token(r2t, rpi, up(prefix), up(lens), loc, err)
        k, v = values(rng, (sum(new), H, D)), values(rng, (sum(new), H, D), 0.2)
        B.pkv_quant_store(pool, to_bf16(k), to_bf16(v), loc, err, page_size=ps, k_scale=ksd, v_scale=vsd)
        slots = loc.cpu().numpy()
        last = slots[np.cumsum(new) - 1]
        R.write(ref, ps, slots, 0, *R.quantise(k, ks))
        R.write(ref, ps, slots, 1, *R.quantise(v, vs))
        q = to_bf16(values(rng, (sum(new), H * g, D)))
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        kw = dict(page_size=ps, sm_scale=D ** -0.5, max_seq_len=int(lens.max()), k_scale=ksd, v_scale=vsd, lse=lse,
                  req_to_token=r2t, req_pool_idx=rpi, seq_lens=up(lens))
        single = max(new) == 1
        if not single:
            kw["qo_indptr"] = up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        a = B.make_quant_args(B.PKV_LAYOUT_REQ_TO_TOKEN, q, pool, out, **kw)
        size, call = ((B.pkv_quant_decode_workspace_size, B.pkv_quant_decode) if single
                      else (B.pkv_quant_extend_workspace_size, B.pkv_quant_extend))
        call(a, torch.empty(size(a), dtype=torch.uint8, device=DEV), err)
        assert err.item() == 0
        assert (pool.cpu().numpy() == ref).all()
        table, row = r2t.cpu().numpy(), rpi.cpu().numpy()
        at = np.concatenate([[0], np.cumsum(new)])
        for b in range(nreq):
            sl = table[row[b], :lens[b]]
            kk, vv = R.read(ref, ps, D, sl, 0, ks), R.read(ref, ps, D, sl, 1, vs)
            o, l, tol, lt = R.attention(host(q)[at[b]:at[b + 1]].astype(np.float64), kk, vv,
                                        np.arange(prefix[b] + 1, lens[b] + 1), D ** -0.5)
            R.assert_within(host(out)[at[b]:at[b + 1]], o, tol, "out")
            R.assert_within(host(lse)[at[b]:at[b + 1]], l, lt, "lse")
    total = int(lens.sum())
    ko, vo = (torch.zeros((total, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cu = torch.zeros(nreq + 1, dtype=torch.int32, device=DEV)
    B.pkv_quant_gather(pool, r2t, rpi, up(lens), int(lens.max()), ko, vo, cu, err, page_size=ps, k_scale=ksd, v_scale=vsd)
    assert err.item() == 0
    sl = np.concatenate([table[row[b], :lens[b]] for b in range(nreq)])
    for part, x, s in ((0, ko, ks), (1, vo, vs)):
        want = R.read(ref, ps, D, sl, part, s)
        R.assert_within(host(x), want, np.abs(want) * (2.0 ** -8 + 2.0 ** -22), "read back")


def test_captured_steps(B):
    """A step (write, decode, extend, read back) captured once and replayed on new contents, while
    another stream runs its own step with its own workspace."""
    rng = np.random.default_rng(42)
    caches, graphs, data = [], [], []
    for s in range(2):
        cache = Cache(rng, [300, 45], 16, 2, 128)
        pool = up(cache.pool)
        q1, q2 = to_bf16(values(rng, (2, 8, 128))), to_bf16(values(rng, (90, 8, 128)))
        o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
        l1, l2 = (torch.empty(x.shape[:2], dtype=torch.float32, device=DEV) for x in (q1, q2))
        a1 = cache.args(B, "table", q1, o1, lse=l1, pool=pool)
        a2 = cache.args(B, "csr", q2, o2, lse=l2, pool=pool, qo_indptr=up(np.array([0, 60, 90], dtype=np.int32)))
        w1 = torch.empty(B.pkv_quant_decode_workspace_size(a1), dtype=torch.uint8, device=DEV)
        w2 = torch.empty(B.pkv_quant_extend_workspace_size(a2), dtype=torch.uint8, device=DEV)
        new = [to_bf16(values(rng, (2, 2, 128))) for _ in range(2)]
        slot = up(np.array([cache.slots[0][-1], cache.slots[1][-1]], dtype=np.int32))
        ko, vo = (torch.zeros((345, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        cu, err, ks, vs = torch.zeros(3, dtype=torch.int32, device=DEV), err_word(), up(cache.ks), up(cache.vs)
        r2t, rpi, lens = up(cache.r2t), up(cache.rpi), up(np.array(cache.lens, dtype=np.int32))

        def step():
            B.pkv_quant_store(pool, new[0], new[1], slot, err, page_size=16, k_scale=ks, v_scale=vs)
            B.pkv_quant_decode(a1, w1, err)
            B.pkv_quant_extend(a2, w2, err)
            B.pkv_quant_gather(pool, r2t, rpi, lens, 300, ko, vo, cu, err, page_size=16, k_scale=ks, v_scale=vs)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        caches.append(cache)
        graphs.append(graph)
        data.append((new, slot, q1, q2, o1, l1, o2, l2, ko, err, (pool, a1, a2, w1, w2, cu, vo, ks, vs, r2t, rpi, lens)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        for s in range(2):
            new, slot, q1, q2 = data[s][:4]
            fresh = [values(rng, (2, 2, 128)) for _ in range(2)]
            for x, y in zip(new, fresh):
                x.copy_(to_bf16(y))
            q1.copy_(to_bf16(values(rng, (2, 8, 128))))
            q2.copy_(to_bf16(values(rng, (90, 8, 128))))
            for part, x, g in ((0, fresh[0], caches[s].ks), (1, fresh[1], caches[s].vs)):
                R.write(caches[s].pool, 16, slot.cpu().numpy(), part, *R.quantise(x, g))
        torch.cuda.synchronize()
        for _ in range(4):
            for s in range(2):
                with torch.cuda.stream(streams[s]):
                    graphs[s].replay()
        torch.cuda.synchronize()
        for s in range(2):
            new, slot, q1, q2, o1, l1, o2, l2, ko, err, _ = data[s]
            assert err.item() == 0
            check(caches[s], q1, o1, l1)
            check(caches[s], q2, o2, l2, rows=[60, 30])
            want = R.read(caches[s].pool, 16, 128, np.concatenate(caches[s].slots), 0, caches[s].ks)
            R.assert_within(host(ko), want, np.abs(want) * (2.0 ** -8 + 2.0 ** -22), "read back")


def test_slots_past_two_gigabytes(B):
    """Pool offsets past 2^32 bytes: the last pages of a 4.5 GB pool."""
    H, D, ps = 8, 128, 64
    nb = R.tile_bytes(ps, D)
    tiles = (9 << 29) // (H * nb) + 2
    pool = torch.empty((tiles, H, nb), dtype=torch.uint8, device=DEV)
    pool[0].fill_(0xFF)
    rng = np.random.default_rng(51)
    n = 130
    pages = np.array([tiles - 1, 0, tiles - 2], dtype=np.int32)
    slots = (pages[:, None].astype(np.int64) * ps + np.arange(ps)).reshape(-1)[:n]
    k, v = values(rng, (n, H, D)), values(rng, (n, H, D), 0.2)
    err = err_word()
    B.pkv_quant_store(pool, to_bf16(k), to_bf16(v), up(slots.astype(np.int32)), err, page_size=ps)
    small = np.full((3, H, nb), 0xFF, dtype=np.uint8)
    one = np.ones(H, dtype=np.float32)
    R.write(small, ps, np.arange(n), 0, *R.quantise(k, one))
    R.write(small, ps, np.arange(n), 1, *R.quantise(v, one))
    for i, p in enumerate(pages):
        got = pool[int(p)].cpu().numpy()
        own = np.zeros(nb, dtype=bool)
        rows = min(ps, n - i * ps)
        for base, w in ((0, D // 2), (ps * D // 2, D // 2), (ps * D, D // 16), (ps * D + ps * D // 16, D // 16)):
            own[base:base + rows * w] = True
        assert (got[:, own] == small[i][:, own]).all()
    q = to_bf16(values(rng, (1, 32, D)))
    out, lse = torch.empty_like(q), torch.empty((1, 32), dtype=torch.float32, device=DEV)
    a = B.make_quant_args(B.PKV_LAYOUT_BLOCK_TABLE, q, pool, out, page_size=ps, sm_scale=D ** -0.5, max_seq_len=n, lse=lse,
                          block_table=up(pages[None]), seq_lens=up(np.array([n], dtype=np.int32)))
    B.pkv_quant_decode(a, torch.empty(B.pkv_quant_decode_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == 0
    o, l, tol, lt = R.attention(host(q).astype(np.float64), R.read(small, ps, D, np.arange(n), 0),
                                R.read(small, ps, D, np.arange(n), 1), [n], D ** -0.5)
    R.assert_within(host(out), o, tol, "out")
    R.assert_within(host(lse), l, lt, "lse")
