"""The 8-bit K/V pool on the GPU: writing, reading back, decode and multi-query attention, and
the weights that keys receive, against the plain reference (bounds derived in _byte_ref), at the
sizes, layouts and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import _byte_ref as R
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


def i32(x):
    return up(np.asarray(x, dtype=np.int32))


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def values(rng, shape, spread=1.0):
    """bf16 normals (as fp32), some channels larger."""
    return R.bf16(rng.standard_normal(shape) * spread * np.where(rng.random(shape[-1]) < 0.05, 5.0, 1.0))


def to_bf16(x):
    return up(x).to(torch.bfloat16)


def host(t):
    return t.detach().float().cpu().numpy()


def random_pool(rng, tiles, ps, D, H, lo=100, hi=150):
    """Any bytes, with scales in a range that values of either side of them meet."""
    data = rng.integers(0, 256, (tiles, R.tile_bytes(ps, D, H))).astype(np.uint8)
    pool = R.Pool(data, ps, D, H)
    pool.E[:] = rng.integers(lo, hi, pool.E.shape)
    return pool


def store(B, pool, k, v, slots, ps, n_ws=None):
    ws = torch.full((B.pkv_byte_store_workspace_size(pool.shape[0], ps),), 0xAB, dtype=torch.uint8, device=DEV)
    err = err_word()
    B.pkv_byte_store(pool, k, v, i32(slots), ws, err, page_size=ps)
    return err.item()


# --------------------------------------------------------------------------- store
@pytest.mark.parametrize("D,ps,H,n", [(128, 16, 8, 33), (128, 64, 2, 130), (64, 1, 3, 17), (128, 1, 1, 5), (64, 4, 20, 9),
                                      (64, 128, 1, 64), (128, 1024, 2, 7), (64, 2, 5, 1), (64, 64, 1, 500), (128, 32, 3, 200),
                                      (128, 8, 1, 3000)])
@pytest.mark.parametrize("form", ["plain", "slice", "odd"])
def test_store_bytes(B, D, ps, H, n, form):
    """Rows in any order and number per tile, over a pool that holds others, padding between them."""
    rng = np.random.default_rng(D * 1000 + ps + H + n)
    t = R.tile_of(ps)
    tiles = max(4, -(-2 * n // t) + 2)
    spread = 2.0 ** rng.integers(-8, 9, (n, H, 1))
    k, v = values(rng, (n, H, D)) * spread.astype(np.float32), values(rng, (n, H, D), 0.1)
    k[0, 0, :16] = [0.0, -0.0, 1e-30, -1e-30, 3, 5, 7, 9, 11, 13, 15, 17, 19, 21, -23, 1e-38]
    k[-1, -1, 5], k[-1, -1, 6] = np.inf, -np.inf
    v[-1, -1, 50] = np.nan
    v[0, -1] = 0.0
    v[0, 0] = R.bf16(np.full(D, 3e38))
    k[n // 2, 0] = R.bf16(np.full(D, 1e-39))
    slots = rng.permutation(tiles * t)[:n].astype(np.int32)
    pad = rng.random(n) < 0.2
    pad[[0, -1]] = False
    mapping = np.where(pad, -1 - rng.integers(0, 5, n), slots).astype(np.int32)
    want = random_pool(rng, tiles, ps, D, H)
    wide = torch.zeros((tiles, want.data.shape[1] + 48), dtype=torch.uint8, device=DEV)      # tiles further apart than they are long
    pool = wide[:, :want.data.shape[1]]
    pool.copy_(up(want.data))
    want.store(k, v, mapping)
    if form == "plain":
        kd, vd = to_bf16(k), to_bf16(v)
    else:       # K and V as slices of one wider row; `odd` also 2 bytes off any alignment
        off = 1 if form == "odd" else 16
        row = torch.zeros((n, off + 2 * H * D + 16 - off % 16), dtype=torch.bfloat16, device=DEV)
        row[:, off:off + H * D] = to_bf16(k).view(n, -1)
        row[:, off + H * D:off + 2 * H * D] = to_bf16(v).view(n, -1)
        kd = row[:, off:off + H * D].unflatten(1, (H, D))
        vd = row[:, off + H * D:off + 2 * H * D].unflatten(1, (H, D))
    assert store(B, pool, kd, vd, mapping, ps) == 0
    got = pool.cpu().numpy()
    assert (got == want.data).all(), "%d bytes differ" % (got != want.data).sum()
    assert not wide[:, want.data.shape[1]:].any()


@pytest.mark.parametrize("ps,D,H", [(16, 128, 2), (64, 64, 3), (4, 128, 1), (128, 64, 1)])
def test_store_step_after_step(B, ps, D, H):
    """Requests that grow by a few rows at a time, ever larger or smaller ones: scales grow with a tile, and
    begin anew with the next."""
    rng = np.random.default_rng(ps + D)
    t = R.tile_of(ps)
    want = random_pool(rng, 48, ps, D, H, 0, 256)
    pool = up(want.data)
    starts, at = [0, 16 * t, 32 * t], [0, 0, 0]
    for step, n in enumerate([1, 1, 3, t - 2, 1, 2, t, 1, 5]):
        k = values(rng, (3 * n, H, D)) * np.float32(2.0 ** (3 * step if step < 5 else -2 * step))
        slots = np.concatenate([starts[b] + at[b] + np.arange(n) for b in range(3)])
        order = rng.permutation(3 * n)
        want.store(k, k * np.float32(0.25), slots[order])
        assert store(B, pool, to_bf16(k), to_bf16(k * np.float32(0.25)), slots[order], ps) == 0
        assert (pool.cpu().numpy() == want.data).all(), step
        at = [a + n for a in at]


def test_store_same_slot_twice(B):
    """One of the two rows is stored, whole, and the other counts for nothing."""
    rng = np.random.default_rng(7)
    for ps, slots in ((16, [3, 4, 3]), (1, [5, 5, 6]), (64, [0, 1, 0])):
        k = values(rng, (3, 2, 64))
        twice = [i for i in range(3) if slots.count(slots[i]) == 2]
        k[twice[1]] *= 1024
        base = random_pool(rng, 8, ps, 64, 2)
        pool = up(base.data)
        assert store(B, pool, to_bf16(k), to_bf16(k), slots, ps) == 0
        got = pool.cpu().numpy()
        wants = []
        for drop in twice:
            w = R.Pool(base.data.copy(), ps, 64, 2)
            w.store(k, k, [-1 if i == drop else s for i, s in enumerate(slots)])
            wants.append(w.data)
        assert any((got == w).all() for w in wants)


@pytest.mark.parametrize("n", [256, 257, 2500])
@pytest.mark.parametrize("D,ps,H,order", [(128, 8, 8, "rising"), (64, 16, 8, "any"), (128, 64, 8, "falling"), (64, 1, 8, "any"),
                                          (128, 4, 1, "rising")])
def test_store_around_the_sizes_that_change_the_kernel(B, D, ps, H, order, n):
    """Whole tiles and parts of them, slots named twice (by rows that hold the same), padding, slots outside."""
    rng = np.random.default_rng(D + ps + n)
    t = R.tile_of(ps)
    tiles = -(-n // t) + 3
    k, v = values(rng, (n, H, D)), values(rng, (n, H, D), 3.0)
    slots = 3 + np.arange(n, dtype=np.int32) if order == "rising" else rng.permutation(n).astype(np.int32) + t
    if order == "falling":
        slots = np.sort(slots)[::-1].copy()
    for a, b in ((5, 200), (0, n - 1), (n // 2, 17)):
        slots[b], k[b], v[b] = slots[a], k[a], v[a]
    alone = slots.copy()
    alone[[200, n - 1, 17]] = -1
    for where, what in ((40, -1), (41, -7), (n - 2, tiles * t), (90, 2 ** 31 - 1)):
        slots[where], alone[where] = what, -1
    want = random_pool(rng, tiles, ps, D, H)
    pool = up(want.data)
    want.store(k, v, alone)
    assert store(B, pool, to_bf16(k), to_bf16(v), slots, ps) == 1
    got = pool.cpu().numpy()
    assert (got == want.data).all(), "%d bytes differ" % (got != want.data).sum()


def test_pool_of_more_than_4_gb(B):
    """Rows stored, read, attended and weighed at both ends of a large pool."""
    rng = np.random.default_rng(8)
    H, D, ps, L = 8, 128, 64, 200
    tiles = 2 ** 32 // R.tile_bytes(ps, D, H) + 40
    pool = torch.empty((tiles, R.tile_bytes(ps, D, H)), dtype=torch.uint8, device=DEV)
    pages = np.concatenate([np.arange(4), tiles - 1 - np.arange(4)]).reshape(2, 4)
    table = (pages[:, :, None] * ps + np.arange(ps)).reshape(2, -1)[:, :L].astype(np.int32)
    k, v = values(rng, (2 * L, H, D)), values(rng, (2 * L, H, D))
    assert store(B, pool, to_bf16(k), to_bf16(v), table.reshape(-1), ps) == 0
    small = R.Pool(np.zeros((8, R.tile_bytes(ps, D, H)), dtype=np.uint8), ps, D, H)
    near = (np.arange(8).reshape(2, 4, 1) * ps + np.arange(ps)).reshape(2, -1)[:, :L]
    small.store(k, v, near.reshape(-1))
    assert (pool[torch.from_numpy(pages.reshape(-1)).to(DEV)].cpu().numpy()[:, :2 * ps * D * H].reshape(8, H, 2, ps, D)[[0, 1, 2, 4, 5, 6]] ==
            small.codes[[0, 1, 2, 4, 5, 6]]).all()
    rows, lens, err = i32([0, 1]), i32([L, L]), err_word()
    ko, vo = [torch.empty((2 * L, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    B.pkv_byte_gather(pool, up(table), rows, lens, L, ko, vo, i32([0, 0, 0]), err, page_size=ps)
    assert (host(ko) == small.read(near.reshape(-1), 0)).all() and (host(vo) == small.read(near.reshape(-1), 1)).all()
    n = 40
    q = to_bf16(values(rng, (2 * n, H, D)))
    acc = torch.zeros((2, L), device=DEV)
    for one in (True, False):       # a decode that counts, and rows whose weights follow
        x = q[:2] if one else q
        out, lse = torch.empty_like(x), torch.empty(x.shape[:2], device=DEV)
        kw = dict(page_size=ps, num_kv_heads=H, sm_scale=D ** -0.5, max_seq_len=L, lse=lse, req_to_token=up(table), req_pool_idx=rows,
                  seq_lens=lens, qo_indptr=None if one else i32([0, n, 2 * n]))
        acc.zero_()
        a = B.make_byte_args(B.PKV_LAYOUT_REQ_TO_TOKEN, x, pool, out, acc_out=acc if one else None, **kw)
        size, call = ((B.pkv_byte_decode_workspace_size, B.pkv_byte_decode) if one else
                      (B.pkv_byte_extend_workspace_size, B.pkv_byte_extend))
        call(a, torch.empty(size(a), dtype=torch.uint8, device=DEV), err)
        if not one:
            for total in (0, 1 << 22):
                acc.zero_()
                a = B.make_byte_args(B.PKV_LAYOUT_REQ_TO_TOKEN, x, pool, None, acc_out=acc, total_kv=total, **kw)
                B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
                assert err.item() == 0
        for b in range(2):
            sl = slice(b, b + 1) if one else slice(b * n, (b + 1) * n)
            ref, rl, w, tol, lt, wt = R.attention(host(x)[sl].astype(np.float64), small.read(near[b], 0), small.read(near[b], 1),
                                                  [L] if one else np.arange(L - n + 1, L + 1), D ** -0.5, small.largest(near[b]))
            R.assert_within(host(out)[sl], ref, tol, "out")
            R.assert_within(host(lse)[sl], rl, lt, "lse")
            want = w.sum((0, 1))
            R.assert_within(host(acc)[b], want, wt.sum((0, 1)) + (len(ref) * H + 1) * 2.0 ** -23 * want, "weights")
    assert err.item() == 0


def test_store_flags_and_small_calls(B):
    rng = np.random.default_rng(3)
    k = values(rng, (4, 2, 128))
    for mapping, bit in (([0, 64, 1, -1], 1), ([-1, -2, -3, -4], 0), ([2 ** 31 - 1, 63, 62, 61], 1)):
        base = random_pool(rng, 4, 16, 128, 2)
        pool = up(base.data)
        assert store(B, pool, to_bf16(k), to_bf16(k), mapping, 16) == bit
        base.store(k, k, [s if s < 64 else -1 for s in mapping])
        assert (pool.cpu().numpy() == base.data).all()
    with pytest.raises(ValueError):
        store(B, pool, to_bf16(k), to_bf16(k)[:3], mapping, 16)
    with pytest.raises(ValueError):
        store(B, pool[:, 1:], to_bf16(k), to_bf16(k), mapping, 16)
    with pytest.raises(ValueError):
        store(B, pool.cpu(), to_bf16(k), to_bf16(k), mapping, 16)
    with pytest.raises(B.PkvError):
        store(B, pool, to_bf16(k), to_bf16(k), mapping, 24)


# --------------------------------------------------------------------------- gather
@pytest.mark.parametrize("D,ps,H,lens", [(128, 16, 8, [0, 1, 17, 300, 16]), (64, 1, 3, [5, 0, 0, 70]), (128, 64, 1, [64, 65, 63, 1000]),
                                         (64, 128, 20, [129, 3]), (128, 4, 2, [2000]), (64, 16, 4, [0, 0])])
def test_gather_bits(B, D, ps, H, lens):
    rng = np.random.default_rng(D + ps + H)
    starts = np.array([(b % 3) * 5 for b in range(len(lens))], dtype=np.int32)
    pages = sum(-(-(l + 20) // ps) + 1 for l in lens) + 3
    r2t, rpi = paged_table(rng, [l + s for l, s in zip(lens, starts)], ps, pages)
    pool = random_pool(rng, -(-pages * ps // R.tile_of(ps)), ps, D, H, 1, 248)
    total = sum(lens)
    flat = np.concatenate([r2t[rpi[b], starts[b]:starts[b] + l] for b, l in enumerate(lens)] + [np.zeros(0, np.int32)])
    k_out = torch.full((total + 3, H, D), 5.0, dtype=torch.bfloat16, device=DEV)
    v_out = torch.full((total + 3, H, D), 6.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.full((len(lens) + 1,), -7, dtype=torch.int32, device=DEV)
    err = err_word()
    B.pkv_byte_gather(up(pool.data), up(r2t), up(rpi), i32(lens), max(lens), k_out, v_out, cu, err, page_size=ps,
                      kv_start=up(starts))
    assert err.item() == 0
    assert cu.tolist() == np.concatenate([[0], np.cumsum(lens)]).tolist()
    for part, out, fill in ((0, k_out, 5.0), (1, v_out, 6.0)):
        got = host(out)
        assert (got[total:] == fill).all()
        with np.errstate(over="ignore"):
            want = R.bf16(pool.read(flat, part).astype(np.float32))
        assert ((got[:total] == want) | (np.isnan(got[:total]) & np.isnan(want))).all()


def test_gather_flags(B):
    rng = np.random.default_rng(5)
    lens = [20, 40, 10]
    r2t, rpi = paged_table(rng, lens, 16, 12)
    pool = up(random_pool(rng, 12, 16, 128, 2).data)

    def call(table=r2t, rows=rpi, sl=lens, cap=80):
        k = torch.full((80, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        v = torch.full_like(k, 9.0)
        cu, err = torch.zeros(4, dtype=torch.int32, device=DEV), err_word()
        B.pkv_byte_gather(pool, up(table), up(rows), i32(sl), 40, k[:cap], v[:cap], cu, err, page_size=16)
        return np.nan_to_num(host(k), nan=77), cu.tolist(), err.item()

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


# --------------------------------------------------------------------------- attention
class Cache:
    """An 8-bit pool holding the given lengths on shuffled pages; every byte that no key owns is
    0xFF: NaN codes, and scale bytes of tiles without keys."""

    def __init__(self, rng, lens, ps, H, D, spread=1.0, starts=None, v_scale=None):
        self.lens, self.ps, self.H, self.D = list(lens), ps, H, D
        starts = [0] * len(lens) if starts is None else starts
        self.starts = np.array(starts, dtype=np.int32)
        pages = sum(-(-l // ps) for l in lens) + 3
        self.r2t, self.rpi = paged_table(rng, lens, ps, pages, kv_start=starts)
        self.pages = pages
        self.pool = R.Pool(np.full((-(-pages * ps // R.tile_of(ps)), R.tile_bytes(ps, D, H)), 0xFF, dtype=np.uint8), ps, D, H)
        self.slots = [self.r2t[self.rpi[b], s:s + l].astype(np.int64) for b, (l, s) in enumerate(zip(lens, starts))]
        flat = np.concatenate(self.slots + [np.zeros(0, np.int64)])
        n = len(flat)
        v = values(rng, (n, H, D), 0.3)
        if v_scale is not None:
            v = R.bf16(v * v_scale(np.concatenate([np.arange(l) for l in lens] + [np.zeros(0)])).reshape(n, 1, 1))
        self.pool.store(values(rng, (n, H, D), spread), v, flat)

    def layout(self, B, name):
        npg = [-(-l // self.ps) for l in self.lens]
        lists = [s[::self.ps] // self.ps for s in self.slots]
        if name == "csr":
            last = [l - (n - 1) * self.ps if n else 0 for l, n in zip(self.lens, npg)]
            idx = np.concatenate(lists + [np.zeros(0, np.int64)])
            return B.PKV_LAYOUT_CSR, dict(kv_indptr=i32(np.concatenate([[0], np.cumsum(npg)])),
                                          kv_indices=i32(idx) if len(idx) else torch.zeros(1, dtype=torch.int32, device=DEV),
                                          kv_last_page_len=i32(last))
        if name == "block":
            bt = np.full((len(npg), max(npg + [1])), -1, dtype=np.int32)
            for b, x in enumerate(lists):
                bt[b, :len(x)] = x
            return B.PKV_LAYOUT_BLOCK_TABLE, dict(block_table=up(bt), seq_lens=i32(self.lens))
        return B.PKV_LAYOUT_REQ_TO_TOKEN, dict(req_to_token=up(self.r2t), req_pool_idx=up(self.rpi), seq_lens=i32(self.lens),
                                               kv_start=up(self.starts))

    def args(self, B, layout, q, out, **kw):
        lay, fields = self.layout(B, layout)
        fields.update(page_size=self.ps, sm_scale=self.D ** -0.5, max_seq_len=max(self.lens + [1]), num_kv_heads=self.H)
        fields.update(kw)
        pool = fields.pop("pool", None)
        return B.make_byte_args(lay, q, up(self.pool.data) if pool is None else pool, out, **fields)


def decode(B, cache, q, layout="table", stream=None, **kw):
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device=DEV)
    err = err_word()
    a = cache.args(B, layout, q, out, lse=lse, **kw)
    ws = torch.full((B.pkv_byte_decode_workspace_size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_byte_decode(a, ws, err)
    return out, lse, err.item()


def extend(B, cache, q, rows, layout="table", kv_end=None, **kw):
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device=DEV)
    err = err_word()
    kw.setdefault("qo_indptr", i32(np.concatenate([[0], np.cumsum(rows)])))
    a = cache.args(B, layout, q, out, lse=lse, kv_end=None if kv_end is None else i32(kv_end), **kw)
    ws = torch.full((B.pkv_byte_extend_workspace_size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_byte_extend(a, ws, err)
    return out, lse, err.item()


def check(cache, q, out, lse, rows=None, kv_end=None, only=None, sm_scale=None, held=False, acc=None, acc_in=None):
    """Every (or only the named) request's rows against the reference; acc: the weights' table after the call."""
    n = [1] * len(cache.lens) if rows is None else list(rows)
    at = np.concatenate([[0], np.cumsum(n)])
    qh = host(q).astype(np.float64)
    for b, L in enumerate(cache.lens):
        if only is not None and b not in only:
            continue
        sl = slice(at[b], at[b + 1])
        if kv_end is not None:
            ends = np.asarray(kv_end)[sl]
        else:
            ends = [L] * n[b] if rows is None else np.arange(L - n[b] + 1, L + 1)
        k, v = cache.pool.read(cache.slots[b], 0), cache.pool.read(cache.slots[b], 1)
        ref, rl, w, tol, lt, wt = R.attention(qh[sl], k, v, ends, cache.D ** -0.5 if sm_scale is None else sm_scale,
                                              cache.pool.largest(cache.slots[b]), held)
        if out is not None and n[b]:
            R.assert_within(host(out)[sl], ref, tol, "request %d (L %d) out" % (b, L))
            R.assert_within(host(lse)[sl], rl, lt, "request %d (L %d) lse" % (b, L))
        if acc is not None:
            s = cache.starts[b]
            before = 0.0 if acc_in is None else host(acc_in)[cache.rpi[b], s:s + L].astype(np.float64)
            want = before + w.sum((0, 1))
            terms = n[b] * q.shape[1] + 1
            R.assert_within(host(acc)[cache.rpi[b], s:s + L], want, wt.sum((0, 1)) + terms * 2.0 ** -23 * np.abs(want),
                            "request %d (L %d) weights" % (b, L))


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
    (64, 32, 20, 1, [600, 31, 33], "block", 64),
    (64, 64, 1, 1, [1], "block", 0),
    (128, 16, 1, 4, [12345], "csr", 0),
    (128, 1, 20, 2, [200, 70], "table", 64),
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
    lens = [int(x) for x in rng.integers(0, 400, 300)]
    cache = Cache(rng, lens, 16, 2, 64)
    q = to_bf16(values(rng, (300, 8, 64)))
    res = [decode(B, cache, q, lay) for lay in ("table", "csr", "block")]
    assert all(r[2] == 0 for r in res)
    assert all(torch.equal(r[0], res[0][0]) and torch.equal(r[1], res[0][1]) for r in res)
    check(cache, q, *res[0][:2], only=range(0, 300, 17))


def test_decode_large_batch_takes_the_table_launch(B):
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    cache = Cache(rng, lens, 4, 1, 64)
    q = to_bf16(values(rng, (1500, 2, 64)))
    out, lse, e = decode(B, cache, q, "csr")
    assert e == 0
    check(cache, q, out, lse, only=list(range(0, 1500, 97)) + [1499])


@pytest.mark.parametrize("ps,chunk", [(1, 0), (1, 64), (4, 0), (16, 64), (64, 0), (64, 64)])
@pytest.mark.parametrize("octaves", [20, 100])
def test_values_whose_scales_lie_far_apart(B, ps, chunk, octaves):
    """V grows and shrinks by 2^20 or 2^100 along a request."""
    rng = np.random.default_rng(ps + chunk + octaves)
    cache = Cache(rng, [700, 130, 65], ps, 2, 128, v_scale=lambda t: np.float32(2.0) ** np.round((octaves / 2 * np.sin(t / 50))).astype(np.int64))
    q = to_bf16(values(rng, (3, 4, 128)))
    out, lse, e = decode(B, cache, q, "table", kv_chunk=chunk)
    assert e == 0
    check(cache, q, out, lse)


@pytest.mark.parametrize("big", [2.0 ** 118, 2.0 ** -125])
def test_extreme_values(B, big):
    """Keys against queries that bring them back, and values near the ends of bf16's range."""
    rng = np.random.default_rng(5)
    lens = [300, 7]
    cache = Cache(rng, lens, 16, 2, 64, spread=big, v_scale=lambda t: np.full(len(t), np.float32(big)))
    q = to_bf16(R.bf16(values(rng, (2, 4, 64)) / np.float32(big)))
    out, lse, e = decode(B, cache, q, "table")
    assert e == 0
    check(cache, q, out, lse)


def test_scores_far_apart(B):
    rng = np.random.default_rng(6)
    cache = Cache(rng, [2000, 90], 64, 2, 128, spread=8.0)
    q = to_bf16(values(rng, (2, 8, 128), 8.0))
    out, lse, e = decode(B, cache, q, "block")
    assert e == 0
    check(cache, q, out, lse)


def test_nan_and_inf_in_the_pool(B):
    """A NaN in K makes its row NaN, one in V its dim; requests that do not hold it are untouched."""
    rng = np.random.default_rng(8)
    for ps in (64, 16, 2):
        cache = Cache(rng, [100, 100, 40], ps, 2, 64)
        q = to_bf16(values(rng, (3, 4, 64)))
        s = cache.slots
        t = R.tile_of(ps)
        cache.pool.codes[s[0][70] // t, 0, 0, s[0][70] % t, 3] = 0x7f
        cache.pool.codes[s[1][99] // t, 1, 1, s[1][99] % t, 9] = 0xff
        out, lse, e = decode(B, cache, q)
        o, l = host(out), host(lse)
        assert e == 0 and np.isnan(o[0, :2]).all() and np.isnan(l[0, :2]).all()
        assert np.isnan(o[1, 2:, 9]).all() and np.isfinite(np.delete(o[1, 2:], 9, 1)).all() and np.isfinite(l[1]).all()
        check(cache, q, out, lse, only=[2])
        assert np.isfinite(o[0, 2:]).all() and np.isfinite(o[1, :2]).all()


def test_strided_queries_and_tiles_and_no_lse(B):
    rng = np.random.default_rng(9)
    cache = Cache(rng, [77, 300], 16, 3, 128)
    wide = torch.zeros((2, 6 * 128 + 40), dtype=torch.bfloat16, device=DEV)
    q = wide[:, 8:8 + 6 * 128].unflatten(1, (6, 128))
    q.copy_(to_bf16(values(rng, (2, 6, 128))))
    store_ = torch.zeros((len(cache.pool.data), cache.pool.data.shape[1] + 112), dtype=torch.uint8, device=DEV)
    pool = store_[:, :cache.pool.data.shape[1]]
    pool.copy_(up(cache.pool.data))
    out, lse, e = decode(B, cache, q, "table", pool=pool)
    assert e == 0
    check(cache, q, out, lse)
    out2 = torch.zeros_like(out)
    a = cache.args(B, "table", q, out2, pool=pool)
    err = err_word()
    B.pkv_byte_decode(a, torch.empty(B.pkv_byte_decode_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert torch.equal(out, out2) and err.item() == 0


def test_bad_pages_and_lengths(B):
    rng = np.random.default_rng(10)
    for ps in (16, 64, 2):
        cache = Cache(rng, [100, 90, 80], ps, 1, 64)
        q = to_bf16(values(rng, (3, 2, 64)))
        good = decode(B, cache, q, "table")
        table = cache.r2t.copy()
        cache.r2t[cache.rpi[1], 64:64 + ps] = cache.pages * ps + 5 * ps
        bad = decode(B, cache, q, "table")
        assert bad[2] == 1
        for b in (0, 2):
            assert torch.equal(bad[0][b], good[0][b])
        assert torch.isfinite(bad[0]).all()
        if ps > 1:
            cache.r2t = table.copy()
            cache.r2t[cache.rpi[1], 64] += 1
            assert decode(B, cache, q, "table")[2] == 2
        cache.r2t = table
        assert decode(B, cache, q, "table", max_seq_len=85)[2] == 4
        assert decode(B, cache, q, "table", req_pool_idx=i32([cache.rpi[0], 99, cache.rpi[2]]))[2] == 1


# --------------------------------------------------------------------------- many rows
EXTEND = [  # D, ps, H, g, lens, rows, layout, bounds
    (128, 16, 2, 4, [100, 37, 5], [4, 4, 4], "table", None),
    (128, 64, 2, 4, [100, 64, 5], [4, 1, 0], "csr", None),
    (64, 1, 1, 7, [70, 9], [9, 3], "block", None),
    (128, 16, 2, 2, [300, 200], [200, 20], "table", None),         # one request's keys held, the other's not
    (64, 64, 1, 1, [700], [700], "csr", None),
    (128, 4, 1, 16, [130, 129, 3], [100, 5, 3], "block", "given"),
    (64, 32, 3, 3, [90, 500], [60, 110], "table", "given"),
    (128, 128, 1, 12, [400], [33], "csr", None),
    (64, 16, 2, 8, [33, 0, 1, 200], [5, 0, 1, 16], "block", "given"),
]


@pytest.mark.parametrize("D,ps,H,g,lens,rows,layout,bounds", EXTEND)
@pytest.mark.parametrize("hints", [False, True])
def test_extend(B, D, ps, H, g, lens, rows, layout, bounds, hints):
    rng = np.random.default_rng(D + ps + H + g + sum(lens))
    cache = Cache(rng, lens, ps, H, D)
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    ends = None
    if bounds:
        ends = np.concatenate([rng.integers(0, l + 1, n) for l, n in zip(lens, rows)])
        ends[::3] = 0
    kw = dict(total_kv=sum(lens), max_q_len=max(rows)) if hints else {}
    out, lse, e = extend(B, cache, q, rows, layout, ends, **kw)
    assert e == 0
    for b in range(len(lens)):
        check(cache, q, out, lse, rows, ends, only=[b], held=rows[b] * g > 128 or max(rows) * g > 128)


def test_extend_nan_in_values_that_some_rows_do_not_see(B):
    rng = np.random.default_rng(20)
    for ps in (64, 16, 4):
        cache = Cache(rng, [90], ps, 1, 64)
        s = cache.slots[0]
        t = R.tile_of(ps)
        cache.pool.codes[s[87] // t, 0, 1, s[87] % t, 5] = 0x7f
        q = to_bf16(values(rng, (6, 2, 64)))
        out, lse, e = extend(B, cache, q, [6])
        o = host(out)
        assert e == 0 and np.isfinite(o[:3]).all() and np.isnan(o[3:, :, 5]).all()
        assert np.isfinite(np.delete(o[3:], 5, 2)).all() and np.isfinite(host(lse)).all()


def test_extend_rows_behind_the_last_stay(B):
    rng = np.random.default_rng(21)
    cache = Cache(rng, [50, 60], 16, 1, 64)
    q = to_bf16(values(rng, (9, 2, 64)))
    out, lse, e = extend(B, cache, q, [3, 4], qo_indptr=i32([0, 3, 7]))
    assert e == 0 and (host(out)[7:] == 3).all() and (host(lse)[7:] == 3).all()
    check(cache, q, out, lse, [3, 4])


# --------------------------------------------------------------------------- weights
def table_of(cache, rng, fill=None):
    x = np.exp(rng.standard_normal(cache.r2t.shape)).astype(np.float32) if fill is None else np.full(cache.r2t.shape, fill, np.float32)
    return up(x)


@pytest.mark.parametrize("D,ps,H,g,lens,layout,chunk", [x for x in DECODE if x[5] == "table"] + [
    (128, 16, 8, 4, [3000, 5, 0, 1023], "table", 0), (64, 64, 4, 5, [513, 2000], "table", 64), (128, 64, 1, 13, [9000], "table", 0)])
@pytest.mark.parametrize("form", ["new", "added", "in place"])
def test_decode_weights(B, D, ps, H, g, lens, layout, chunk, form):
    rng = np.random.default_rng(D + ps * 3 + H * 7 + g)
    cache = Cache(rng, lens, ps, H, D, starts=[(b % 2) * ps for b in range(len(lens))])
    q = to_bf16(values(rng, (len(lens), H * g, D)))
    plain = decode(B, cache, q, "table", kv_chunk=chunk)
    acc_in = None if form == "new" else table_of(cache, rng)
    acc = acc_in.clone() if form == "in place" else table_of(cache, rng, 7.0)
    out, lse, e = decode(B, cache, q, "table", kv_chunk=chunk, acc_in=acc if form == "in place" else acc_in, acc_out=acc)
    assert e == 0 and torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    check(cache, q, out, lse, acc=acc, acc_in=acc_in)
    rest = np.ones(acc.shape, bool)
    for b, L in enumerate(lens):
        rest[cache.rpi[b], cache.starts[b]:cache.starts[b] + L] = False
    assert (host(acc)[rest] == (host(acc_in)[rest] if form == "in place" else 7.0)).all()


WEIGHTS = [  # D, ps, H, g, lens, rows, bounds
    (128, 16, 2, 4, [100, 37, 5], [4, 4, 4], None),
    (128, 64, 2, 4, [600, 64, 5], [32, 1, 0], None),
    (64, 1, 1, 7, [70, 9, 0], [9, 3, 0], None),
    (64, 4, 5, 16, [1300], [31], "given"),
    (128, 32, 1, 3, [513, 512, 511], [40, 7, 1], "given"),
    (64, 128, 2, 1, [200, 90], [150, 90], None),
]


@pytest.mark.parametrize("D,ps,H,g,lens,rows,bounds", WEIGHTS)
def test_weights_of_rows(B, D, ps, H, g, lens, rows, bounds):
    rng = np.random.default_rng(D + ps + H + g + sum(lens))
    cache = Cache(rng, lens, ps, H, D, starts=[(b % 2) * ps for b in range(len(lens))])
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    ends = None
    if bounds:
        ends = np.concatenate([rng.integers(0, l + 1, n) for l, n in zip(lens, rows)])
        ends[::3] = 0
    out, lse, e = extend(B, cache, q, rows, "table", ends)
    assert e == 0
    acc_in, acc, err = table_of(cache, rng), table_of(cache, rng, 7.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])),
                   kv_end=None if ends is None else i32(ends), acc_in=acc_in, acc_out=acc)
    ws = torch.full((B.pkv_byte_weights_workspace_size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_byte_weights(a, ws, err)
    assert err.item() == 0
    check(cache, q, None, None, rows, ends, acc=acc, acc_in=acc_in)
    rest = np.ones(acc.shape, bool)
    for b, L in enumerate(lens):
        rest[cache.rpi[b], cache.starts[b]:cache.starts[b] + L] = False
    assert (host(acc)[rest] == 7.0).all()
    # once more: the same to the bit
    again = table_of(cache, rng, 7.0)
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])),
                   kv_end=None if ends is None else i32(ends), acc_in=acc_in, acc_out=again)
    B.pkv_byte_weights(a, ws, err)
    assert torch.equal(acc, again)


@pytest.mark.parametrize("total", [0, 1 << 22])
@pytest.mark.parametrize("D,ps,H,g,lens,rows", [
    (128, 64, 2, 1, [300, 1, 0, 129], [1, 1, 1, 1]),
    (64, 16, 1, 4, [128, 127, 700], [0, 0, 3]),
    (128, 1, 1, 2, [260], [2]),
    (64, 4, 3, 5, [90, 513, 64], [9, 1, 4]),
    (128, 256, 1, 8, [2000, 31], [7, 7]),
])
def test_weights_of_few_rows_of_many_keys(B, D, ps, H, g, lens, rows, total):
    """The bound on the keys decides which kernel runs, not what comes out."""
    rng = np.random.default_rng(33 + D + ps + sum(lens))
    cache = Cache(rng, lens, ps, H, D)
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    out, lse, e = extend(B, cache, q, rows)
    acc, err = table_of(cache, rng, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])), acc_out=acc, total_kv=total)
    B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == any(n > L for n, L in zip(rows, lens))   # (causal rows of a request without keys are flagged)
    check(cache, q, None, None, rows, acc=acc)


@pytest.mark.parametrize("batch", [1024, 1025])
def test_weights_of_the_largest_batches(B, batch):
    """As many requests as are numbered in shared memory, and one more; some without keys or rows."""
    rng = np.random.default_rng(34)
    lens = rng.integers(0, 200, batch)
    lens[[0, 7, 8, batch - 1]] = [130, 0, 0, 129]
    rows = np.minimum(rng.integers(0, 4, batch), lens)
    cache = Cache(rng, [int(x) for x in lens], 16, 1, 64)
    q = to_bf16(values(rng, (int(rows.sum()), 2, 64)))
    rows = [int(x) for x in rows]
    out, lse, e = extend(B, cache, q, rows)
    assert e == 0
    acc, err = table_of(cache, rng, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])), acc_out=acc, total_kv=1 << 22)
    B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == 0
    check(cache, q, None, None, rows, acc=acc, only=set(range(0, batch, 9)) | {0, 7, 8, 1023, batch - 1})


@pytest.mark.parametrize("more", [0, 60])
@pytest.mark.parametrize("tiny", [2.0 ** -4, 2.0 ** -100])
def test_weights_of_extreme_rows(B, more, tiny):
    """Rows without keys, rows of zeros, a row of large and one of tiny values; alone and among many."""
    rng = np.random.default_rng(30)
    cache = Cache(rng, [700], 16, 1, 64)
    n = 5 + more
    x = values(rng, (n, 2, 64))
    x[1] = 0
    x[2] *= np.float32(tiny)
    x[3] *= 16
    q = to_bf16(x)
    ends = [0, 200, 150, 199, 1] + [700 - i for i in range(more)]
    out, lse, e = extend(B, cache, q, [n], "table", ends)
    acc, err = table_of(cache, rng, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32([0, n]), kv_end=i32(ends), acc_out=acc)
    B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == 0
    check(cache, q, out, lse, [n], ends, acc=acc, held=n * 2 > 128)


@pytest.mark.parametrize("D,rows", [(128, 5), (128, 40), (64, 40)])
def test_weights_over_strided_tiles(B, D, rows):
    """Tiles a multiple of 16 bytes apart, and of no more; more rows than one pass takes."""
    rng = np.random.default_rng(32 + D + rows)
    cache = Cache(rng, [300, 129], 64, 2, D)
    q = to_bf16(values(rng, (2 * rows, 8, D)))
    out, lse, e = extend(B, cache, q, [rows, rows])
    nbytes = cache.pool.data.shape[1]
    pool = torch.zeros((len(cache.pool.data), nbytes + 16), dtype=torch.uint8, device=DEV)[:, :nbytes]
    pool.copy_(up(cache.pool.data))
    acc, err = table_of(cache, rng, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32([0, rows, 2 * rows]), acc_out=acc, pool=pool)
    B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == 0
    check(cache, q, out, lse, [rows, rows], acc=acc, held=rows * 4 > 128)


def test_weights_flags(B):
    rng = np.random.default_rng(31)
    cache = Cache(rng, [40, 50], 16, 1, 64)
    q = to_bf16(values(rng, (4, 2, 64)))
    out, lse, e = extend(B, cache, q, [2, 2])

    def call(**kw):
        acc, err = table_of(cache, rng, 7.0), err_word()
        fields = dict(lse=lse, qo_indptr=i32([0, 2, 4]), acc_out=acc)
        fields.update(kw)
        a = cache.args(B, "table", q, None, **fields)
        B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
        return host(acc), err.item()

    good, e = call()
    assert e == 0
    acc, e = call(kv_end=i32([40, 99, 50, 50]))
    assert e == 1
    acc, e = call(req_pool_idx=i32([cache.rpi[0], 55]))
    assert e == 1 and (acc[cache.rpi[0]] == good[cache.rpi[0]]).all() and (acc[cache.rpi[1]] == 7).all()
    acc, e = call(max_seq_len=45)
    assert e == 4
    acc, e = call(qo_indptr=i32([0, 2, 9]))
    assert e == 1 and (acc[cache.rpi[0]] == good[cache.rpi[0]]).all()


# --------------------------------------------------------------------------- streams and graphs
def test_two_calls_at_once_and_a_replayed_graph(B):
    rng = np.random.default_rng(40)
    caches = [Cache(rng, [500, 33], 16, 2, 128), Cache(rng, [64, 700], 16, 2, 128)]
    qs = [to_bf16(values(rng, (2, 8, 128))) for _ in caches]
    want = [decode(B, c, q, acc_out=table_of(c, rng, 0.0)) for c, q in zip(caches, qs)]
    calls = []
    for c, q in zip(caches, qs):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        acc = table_of(c, rng, 0.0)
        a = c.args(B, "table", q, out, lse=lse, acc_out=acc)
        calls.append((a, torch.empty(B.pkv_byte_decode_workspace_size(a), dtype=torch.uint8, device=DEV), err_word(), out, acc))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (a, ws, err, out, acc) in zip(streams, calls):
            B.pkv_byte_decode(a, ws, err, stream=s)
    torch.cuda.synchronize()
    for (a, ws, err, out, acc), w in zip(calls, want):
        assert torch.equal(out, w[0]) and err.item() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, ws, err, out, acc in calls:
            B.pkv_byte_decode(a, ws, err)
    for a, ws, err, out, acc in calls:
        out.zero_()
        acc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for (a, ws, err, out, acc), w, c, q in zip(calls, want, caches, qs):
        assert torch.equal(out, w[0])
        check(c, q, out, None if out is None else a._keep and w[1], acc=acc)


@pytest.mark.parametrize("D,ps,rows", [(128, 64, 40), (64, 4, 300)])
def test_weights_whose_wait_runs_out(B, D, ps, rows):
    """With a limit of 1 ns the call gives up, says so, and the next one is right."""
    rng = np.random.default_rng(42)
    cache = Cache(rng, [2000, 700], ps, 2, D)
    q = to_bf16(values(rng, (2 * rows, 4, D)))
    out, lse, e = extend(B, cache, q, [rows, rows])
    acc, err = table_of(cache, rng, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32([0, rows, 2 * rows]), acc_out=acc)
    ws = torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV)
    B.pkv_set_wait_limit(1)
    try:
        B.pkv_byte_weights(a, ws, err)
        assert err.item() in (0, 8)
    finally:
        B.pkv_set_wait_limit(0)
    err.zero_()
    B.pkv_byte_weights(a, ws, err)
    assert err.item() == 0
    check(cache, q, out, lse, [rows, rows], acc=acc, held=True)


@pytest.mark.parametrize("ps", [64, 16, 4, 1])
def test_weights_bad_pages(B, ps):
    """A page outside the pool, and one that is not aligned, in a call of many rows."""
    rng = np.random.default_rng(43)
    cache = Cache(rng, [300, 200], ps, 1, 128)
    q = to_bf16(values(rng, (100, 2, 128)))
    out, lse, e = extend(B, cache, q, [50, 50])
    table = cache.r2t.copy()
    for bad, bit in ((cache.pages * ps + 5 * ps, 1), (-1, 1)) + (((table[cache.rpi[0], 64] + 1), 2),) * (ps > 1):
        cache.r2t = table.copy()
        cache.r2t[cache.rpi[0], 64] = bad
        acc, err = table_of(cache, rng, 0.0), err_word()
        a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32([0, 50, 100]), acc_out=acc)
        B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
        assert err.item() == bit
        got = host(acc)
        cache.r2t = table
        n = host(q).astype(np.float64)[50:]
        k, v = cache.pool.read(cache.slots[1], 0), cache.pool.read(cache.slots[1], 1)
        w, wt = R.attention(n, k, v, np.arange(151, 201), 128 ** -0.5, cache.pool.largest(cache.slots[1]))[2::3]
        want = w.sum((0, 1))
        R.assert_within(got[cache.rpi[1], :200], want, wt.sum((0, 1)) + 101 * 2.0 ** -23 * want, "the other request")
        assert np.isfinite(got[cache.rpi[0], :300]).all()


@pytest.mark.parametrize("batch,hi", [(3, 200), (40, 3000)])
def test_a_wait_that_runs_out(B, batch, hi):
    """With a limit of 1 ns the call gives up, says so, and the next one is right."""
    rng = np.random.default_rng(41)
    cache = Cache(rng, [int(x) for x in rng.integers(1, hi, batch)], 16, 2, 64)
    q = to_bf16(values(rng, (batch, 4, 64)))
    B.pkv_set_wait_limit(1)
    try:
        out, lse, e = decode(B, cache, q)
    finally:
        B.pkv_set_wait_limit(0)
    assert e in (0, 8)
    out, lse, e = decode(B, cache, q)
    assert e == 0
    check(cache, q, out, lse, only=range(3))
