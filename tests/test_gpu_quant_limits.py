"""The 4-bit attention calls at the ends of what they allow: many short segments per warp, weights
and scales far apart, first calls from several threads, large batches."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _quant_ref as R
from test_gpu_quant import DEV, Cache, check, decode, extend, host, to_bf16, up, values  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


@pytest.mark.parametrize("D,H,g", [(128, 8, 4), (64, 20, 1)])
def test_short_segments_follow_one_another(B, D, H, g):
    """Pages of 64 and requests of one to three tiles, several to a warp: each segment's query rows are
    fetched while the tile before it is worked on."""
    rng = np.random.default_rng(90 + D)
    lens = rng.integers(1, 190, 500).tolist()
    cache = Cache(rng, lens, 64, H, D)
    q = to_bf16(values(rng, (len(lens), H * g, D)))
    out, lse, e = decode(B, cache, q, kv_chunk=256)
    assert e == 0
    check(cache, q, out, lse, only=list(range(0, 500, 9)) + [499])
    for _ in range(10):
        o2, l2, e = decode(B, cache, q, kv_chunk=256)
        assert e == 0 and torch.equal(out, o2) and torch.equal(lse, l2)


FIRST_CALLS = """
import sys, threading
import torch
from paged_kv_cache_req_gb300 import _binding as B

dev = "cuda"
failed = []
barrier = threading.Barrier(2)


def make(D, Hq, ps, batch):
    # one key per request, all on page 0
    pool = torch.zeros((16, 1, B.pkv_quant_tile_bytes(ps, D)), dtype=torch.uint8, device=dev)
    q = torch.ones((batch, Hq, D), dtype=torch.bfloat16, device=dev)
    ones = torch.ones(batch, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    a = B.make_quant_args(B.PKV_LAYOUT_BLOCK_TABLE, q, pool, out, page_size=ps, sm_scale=1.0, max_seq_len=64, kv_chunk=64,
                          block_table=torch.zeros((batch, 64), dtype=torch.int32, device=dev), seq_lens=ones)
    ws = torch.empty(B.pkv_quant_decode_workspace_size(a), dtype=torch.uint8, device=dev)
    return a, ws, torch.zeros(1, dtype=torch.int32, device=dev), torch.cuda.Stream()


def work(batch):
    for a, ws, err, stream in calls[batch]:
        barrier.wait()
        for _ in range(3):
            try:
                B.pkv_quant_decode(a, ws, err, stream=stream)
            except B.PkvError as e:
                failed.append("batch %d, head_dim %d: %s" % (batch, a.head_dim, e))


calls = {n: [make(D, Hq, ps, n) for D in (64, 128) for Hq in (4, 16) for ps in (1, 16, 64)] for n in (2, 1000)}
torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(n,)) for n in calls]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert all(err.item() == 0 for n in calls for _, _, err, _ in calls[n])
sys.exit("\\n".join(failed) if failed else 0)
"""


def test_first_calls_from_two_threads(B):
    """A small and a large batch of each kernel, called for the first time in a process by two threads
    at once: neither takes back the shared memory that the other needs."""
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr


def test_many_rows_under_far_bounds(B):
    """More rows and a higher bound on the keys than the span kernel's sequence of tiles could count."""
    rng = np.random.default_rng(92)
    lens, rows = [500, 33, 70], [65000, 3, 2000]
    cache = Cache(rng, lens, 16, 8, 64)
    q = to_bf16(values(rng, (sum(rows), 16, 64)))
    ends = np.concatenate([rng.integers(0, n + 1, r) for n, r in zip(lens, rows)]).astype(np.int32)
    out, lse, e = extend(B, cache, q, rows, kv_end=ends, max_seq_len=1 << 20, total_kv=sum(lens))
    assert e == 0
    some = np.concatenate([[0, 1, 64999, 65000, 65001, 65002, 65003, 67002], rng.integers(0, sum(rows), 60)])
    req = np.searchsorted(np.cumsum(rows), some, side="right")
    for b in range(3):
        at = some[req == b]
        k, v = cache.kv(b)
        ref, rl, tol, lt = R.attention(host(q[up(at)]).astype(np.float64), k, v, ends[at], 64 ** -0.5)
        R.assert_within(host(out[up(at)]), ref, tol, "request %d out" % b)
        R.assert_within(host(lse[up(at)]), rl, lt, "request %d lse" % b)


def sink_bound(q, k, v, ends, sm_scale):
    """q [n, D], k / v [L, D] fp64 of one head -> (out, lse, bounds of both).

    As _quant_ref.attention (the sum that lse is the logarithm of has L terms in fp32, so L 2^-23
    relative: the largest weight is 2^7 there, and each of 16384 weights of 2^-14.6 is added to it
    with up to half of 128's last place, 2^-18, lost), but for the weights: one is rounded by 2^-11 relative, or, where it is
    subnormal in fp16, by 2^-25; the largest is held as 2^7 or more, so that is 2^-32 of it."""
    s = q @ k.T * sm_scale
    s[np.arange(k.shape[0])[None] >= np.asarray(ends)[:, None]] = -np.inf
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    den = p.sum(1, keepdims=True)
    out = p @ v / den
    ds = (np.abs(q) @ np.abs(k).T).max(1, keepdims=True) * sm_scale * k.shape[1] * 2.0 ** -23
    rel = 2.0 ** -11 + 2 * (ds + 2.0 ** -21 + k.shape[0] * 2.0 ** -23)
    tol = 2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * (rel * (p @ np.abs(v) / den) +
                                                       2.0 ** -32 * (np.isfinite(s) @ np.abs(v)) / den)
    lse = m + np.log(den)
    ltol = ds + 2.0 ** -21 + k.shape[0] * 2.0 ** -23 + 2.0 ** -22 * (np.abs(m) + np.abs(lse) + 1)
    return out, lse[:, 0], tol, ltol[:, 0]


@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("D,rows,chunk", [(128, 1, 1 << 20), (64, 1, 1 << 20), (128, 1, 0), (64, 9, 1 << 20), (128, 14, 1 << 20),
                                          (128, 200, 1 << 20), (64, 200, 1 << 20), (128, 200, 2048)])
def test_a_key_far_above_the_others(B, D, rows, chunk, spread):
    """One key 15 to 18 nats above 16384 others, with a value of 0: the output is what the others give."""
    rng = np.random.default_rng(94)
    L, nats = 16385, np.array([15.0, 17.0, 18.0])
    cache = Cache(rng, [L] * 3, 64, 1, D)
    cache.ks[:], cache.vs[:] = 1.0, 0.25
    for b in range(3):
        k = np.tile(spread * rng.standard_normal((L, 1, 1)), (1, 1, D)) * np.where(np.arange(D) % 2 == 0, 1, -1) / 8
        v = np.abs(values(rng, (L, 1, D), 0.3))
        k[:], v[5 * b] = R.bf16(k), 0.0
        k[5 * b, 0] = 6.0
        for part, x, g in ((0, k, cache.ks), (1, v, cache.vs)):
            R.write(cache.pool, 64, cache.slots[b], part, *R.quantise(x.astype(np.float32), g))
    q = np.repeat(nats / (6.0 * D * D ** -0.5), rows)[:, None, None] + np.zeros((1, 1, D))
    if spread:   # the even and odd dims' difference gives the other keys scores of some 0.5 nats
        q = q + np.where(np.arange(D) % 2 == 0, 1, -1) * (8 * D ** -0.5 / D) * D
    q = to_bf16(R.bf16(q))
    if rows == 1:
        out, lse, e = decode(B, cache, q, kv_chunk=chunk)
    else:
        out, lse, e = extend(B, cache, q, [rows] * 3, kv_chunk=chunk)
    assert e == 0
    for b in range(3):
        k, v = cache.kv(b)
        at = slice(b * rows, (b + 1) * rows)
        ref, rl, tol, lt = sink_bound(host(q)[at, 0].astype(np.float64), k[:, 0], v[:, 0], np.arange(L - rows + 1, L + 1),
                                      D ** -0.5)
        assert (tol < 0.06 * ref + 1e-9).all()
        R.assert_within(host(out)[at, 0], ref, tol, "%g nats" % nats[b])
        R.assert_within(host(lse)[at, 0], rl, lt, "lse")


@pytest.mark.parametrize("rows,chunk", [(1, 0), (1, 128), (7, 128), (200, 0), (200, 256)])
def test_a_vanishing_score_scale(B, rows, chunk):
    """sm_scale times K's head scale below fp32's range: equal weights, also beside masked keys."""
    rng = np.random.default_rng(95)
    cache = Cache(rng, [333, 260], 16, 2, 128)
    cache.ks[:] = 1e-20
    q = to_bf16(values(rng, (2 * rows, 8, 128)))
    if rows == 1:
        out, lse, e = decode(B, cache, q, sm_scale=5e-32, kv_chunk=chunk)
    else:
        out, lse, e = extend(B, cache, q, [rows] * 2, sm_scale=5e-32, kv_chunk=chunk)
    assert e == 0
    check(cache, q, out, lse, None if rows == 1 else [rows] * 2, sm_scale=5e-32)


@pytest.mark.parametrize("e", [-121, 100])
@pytest.mark.parametrize("rows,chunk", [(1, 0), (1, 1 << 20), (1, 256), (6, 1 << 20), (6, 256), (300, 1 << 20), (300, 1024)])
def test_far_head_scales_of_v(B, rows, chunk, e):
    """V's head scale near both ends of fp32 over thousands of equal keys: the output keeps its bits."""
    rng = np.random.default_rng(96)
    cache = Cache(rng, [4000, 700], 64, 1, 64, spread=0.1)
    cache.vs[:] = 2.0 ** e
    for b, L in enumerate(cache.lens):      # values of one sign: their mean is as large as they are
        R.write(cache.pool, 64, cache.slots[b], 1, *R.quantise(np.abs(values(rng, (L, 1, 64))), np.ones(1, np.float32)))
    q = to_bf16(values(rng, (2 * rows, 4, 64)))
    if rows == 1:
        out, lse, err = decode(B, cache, q, kv_chunk=chunk)
    else:
        out, lse, err = extend(B, cache, q, [rows] * 2, kv_chunk=chunk)
    assert err == 0
    out = torch.ldexp(out.double(), torch.tensor(-e))          # (exact: compared at a scale of 1)
    cache.vs[:] = 1.0
    check(cache, q, out, lse, None if rows == 1 else [rows] * 2)


@pytest.mark.parametrize("rows,chunk", [(1, 0), (1, 64), (3, 64)])
def test_far_queries_over_vanishing_scales(B, rows, chunk):
    """Queries near bf16's largest value, sm_scale and K's head scale so small that their product alone
    is 0 in fp32: the logits are not."""
    rng = np.random.default_rng(97)
    D, L = 128, 2 * rows
    cache = Cache(rng, [L], 16, 1, D)
    for part, x in ((0, 1.0), (1, 1.0)):      # every second key 6 x 448 in all dims, the others 0; values of both signs
        rowsx = np.full((L, 1, D), x, dtype=np.float32) * (np.arange(L) % 2 == 0 if part == 0 else 1 - 2 * (np.arange(L) % 2))[:, None, None]
        c, s = R.quantise(rowsx.astype(np.float32), np.array([1.0 / 2688], dtype=np.float32))
        R.write(cache.pool, 16, cache.slots[0], part, c, s)
    cache.ks[:], cache.vs[:] = 2.0 ** -75, 2.0 ** -11
    sm = 2.0 ** -76
    q = torch.full((rows, 1, D), 2.0 ** 127, dtype=torch.bfloat16, device=DEV)
    if rows == 1:
        out, lse, e = decode(B, cache, q, sm_scale=sm, kv_chunk=chunk)
    else:
        out, lse, e = extend(B, cache, q, [rows], sm_scale=sm, kv_chunk=chunk, kv_end=[L] * rows)
    assert e == 0
    assert (np.abs(host(out)) > 0.005).all()
    check(cache, q, out, lse, None if rows == 1 else [rows], kv_end=None if rows == 1 else [L] * rows, sm_scale=sm)


@pytest.mark.parametrize("D,H", [(128, 1), (64, 2), (128, 8), (64, 3)])
@pytest.mark.parametrize("batch", [2047, 2048, 2049, 5000])
def test_gather_of_thousands_of_requests(B, batch, D, H):
    """Requests past the 2048 whose offsets are scanned at a time: empty ones at the border, tokens of
    half a warp and whole ones; a capacity that ends inside the second part."""
    rng = np.random.default_rng(98 + batch + D + H)
    ps, slots, lens = 16, 640, rng.integers(0, 6, batch).astype(np.int32)
    lens[2040:2052] = 0
    lens[2050:2051] = 9
    lens[-1] = 4
    total = int(lens.sum())
    x = values(rng, (slots, H, D))
    g = (2.0 ** -rng.integers(0, 4, H)).astype(np.float32)      # (products with it are exact)
    pool = np.zeros((slots // ps, H, R.tile_bytes(ps, D)), dtype=np.uint8)
    for part in (0, 1):
        R.write(pool, ps, np.arange(slots), part, *R.quantise(x * (1 + part), g))
    table = rng.integers(0, slots, (batch + 3, 12)).astype(np.int32)
    rows = rng.permutation(batch + 3)[:batch].astype(np.int32)
    flat = np.concatenate([table[r, :n] for r, n in zip(rows, lens)]).astype(np.int64)
    want = [R.bf16(R.read(pool, ps, D, flat, part, g).astype(np.float32)) for part in (0, 1)]
    cu_want = np.concatenate([[0], np.cumsum(lens)])
    caps = [total + 7] + ([int(cu_want[2048]) + 1, int(cu_want[3000]) + 1] if batch == 5000 else [])
    for cap in caps:
        out = [torch.full((cap, H, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        B.pkv_quant_gather(up(pool), up(table), up(rows), up(lens), int(lens.max()), out[0], out[1], cu, err, page_size=ps,
                           k_scale=up(g), v_scale=up(g))
        assert err.item() == (0 if cap >= total else B.PKV_DEVERR_CAPACITY)
        assert cu.tolist() == cu_want.tolist()
        n = min(cap, total)
        for o, w in zip(out, want):
            assert (host(o[:n]) == w[:n]).all() and (o[n:] == 9).all()


PATHS = [([1, 1, 1], dict(kv_chunk=0)), ([1, 1, 1], dict(kv_chunk=128)), ([6, 3, 0], dict(kv_chunk=0)), ([6, 3, 5], dict(kv_chunk=128)),
         ([200, 150, 140], dict(kv_chunk=0)), ([200, 1, 140], dict(kv_chunk=256, max_q_len=200))]


def call(B, cache, q, rows, **kw):
    if rows == [1, 1, 1]:
        return decode(B, cache, q, **kw)
    return extend(B, cache, q, rows, **kw)


@pytest.mark.parametrize("rows,kw", PATHS)
@pytest.mark.parametrize("D,ps", [(128, 16), (64, 64), (128, 4)])
def test_a_poisoned_value_reaches_only_who_sees_it(B, D, ps, rows, kw):
    """A NaN in a stored value: the rows that see its key are NaN in that block, the others as without it."""
    rng = np.random.default_rng(99)
    cache = Cache(rng, [333, 200, 150], ps, 2, D)
    c, s = R.quantise(values(rng, (1, 2, D)), cache.vs)
    s[0, 1, 2] = 0x7f
    at = 331
    R.write(cache.pool, ps, cache.slots[0][at:at + 1], 1, c, s)
    q = to_bf16(values(rng, (sum(rows), 8, D)))
    out, lse, e = call(B, cache, q, rows, **kw)
    assert e == 0
    o = host(out)
    seen = np.zeros(o.shape[:2], dtype=bool)
    first = max(0, at + 1 - (333 - rows[0] + 1)) if rows != [1, 1, 1] else 0
    seen[first:rows[0], 4:] = True
    assert np.isnan(o[seen][:, 32:48]).all() and np.isfinite(o[~seen]).all()
    clean = c.copy(), s.copy()
    clean[1][0, 1, 2] = 0
    R.write(cache.pool, ps, cache.slots[0][at:at + 1], 1, *clean)
    o2, l2, e = call(B, cache, q, rows, **kw)
    assert e == 0 and (host(o2)[~seen] == o[~seen]).all()
    check(cache, q, o2, l2, None if rows == [1, 1, 1] else rows)


@pytest.mark.parametrize("rows,kw", PATHS)
def test_strided_queries_and_tiles(B, rows, kw):
    """Query rows as slices of wider rows, tiles further apart than they are long, rows past the last
    request's (left as they were), and a call without lse."""
    rng = np.random.default_rng(100)
    D, H, g = 64, 3, 4
    cache = Cache(rng, [333, 200, 150], 16, H, D)
    one, n = rows == [1, 1, 1], sum(rows)
    q = to_bf16(values(rng, (n, H * g, D)))
    out, lse, e = call(B, cache, q, rows, **kw)
    assert e == 0
    check(cache, q, out, lse, None if one else rows)
    offsets = {} if one else dict(qo_indptr=up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)))
    o2, err = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device=DEV)
    a = cache.args(B, "table", q, o2, **dict(kw, **offsets))
    size, fn = ((B.pkv_quant_decode_workspace_size, B.pkv_quant_decode) if one else
                (B.pkv_quant_extend_workspace_size, B.pkv_quant_extend))
    fn(a, torch.empty(size(a), dtype=torch.uint8, device=DEV), err)
    assert err.item() == 0 and torch.equal(o2, out)
    wide = torch.full((n + 5, H * g * D + 2 * H * D + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:n, 8:8 + H * g * D] = q.view(n, -1)
    sliced = wide[:n if one else n + 5, 8:8 + H * g * D].unflatten(1, (H * g, D))
    tiles = torch.full((cache.pool.shape[0], H + 2, cache.pool.shape[2]), 0xFF, dtype=torch.uint8, device=DEV)
    tiles[:, :H] = up(cache.pool)
    o2, l2, e = call(B, cache, sliced, rows, **dict(kw, pool=tiles[:, :H], **offsets))
    assert e == 0 and (o2[n:] == 3).all() and (l2[n:] == 3).all()
    check(cache, q, o2[:n], l2[:n], None if one else rows)


@pytest.mark.parametrize("batch,chunk", [(300, 0), (1100, 0), (300, 128)])
def test_copied_keys_of_hundreds_of_requests(B, batch, chunk):
    """Many requests of just more rows than the spans take, others of few rows or none between them."""
    rng = np.random.default_rng(101 + batch)
    rows = rng.choice([0, 1, 5, 32, 33, 40], batch, p=[0.1, 0.1, 0.1, 0.1, 0.4, 0.2])
    rows[[0, -1]] = 33, 40
    lens = np.maximum(rows, rng.integers(0, 200, batch)).tolist()
    cache = Cache(rng, lens, 16, 2, 64)
    q = to_bf16(values(rng, (int(rows.sum()), 8, 64)))
    out, lse, e = extend(B, cache, q, rows.tolist(), max_q_len=40, total_kv=sum(lens), kv_chunk=chunk)
    assert e == 0
    check(cache, q, out, lse, rows.tolist(), only=[0, 1, 255, 256, 257, batch - 2, batch - 1] + list(range(0, batch, batch // 20)))
