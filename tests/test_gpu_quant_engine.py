"""The engine's steps over a 4-bit pool: every sampled row against the plain fp64 reference of
what the pool holds after the step's store, the give-up path of bounded waits, and sizes that
only larger batches reach."""
import numpy as np
import pytest
import torch

import _quant_ref as R
from test_gpu_quant import DECODE, DEV, EXTEND, Cache, check, decode, extend, host, to_bf16, up, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    yield _binding
    _binding.pkv_set_wait_limit(0)


def stored(quant, slots):
    """fp64 K and V at `slots` of a _QuantPool, from the tiles that hold them."""
    slots = np.asarray(slots, dtype=np.int64)
    t, D = R.tile_of(quant.page_size), None
    tiles = np.unique(slots // t)
    pool = quant.pool[torch.from_numpy(tiles).to(quant.pool.device)].cpu().numpy()
    for D in (64, 128):
        if R.tile_bytes(quant.page_size, D) == pool.shape[2]:
            break
    at = np.searchsorted(tiles, slots // t) * t + slots % t
    return (R.read(pool, quant.page_size, D, at, 0, quant.k_scale.cpu().numpy()),
            R.read(pool, quant.page_size, D, at, 1, quant.v_scale.cpu().numpy()))


def check_decode(step, name, sample, varlen=False):
    wl, pb = step.wl, step.problems[name]
    r2t, rpi = step.r2t.cpu().numpy(), wl.req_pool_idx.numpy()
    lens, starts = pb.spec.seq_lens.numpy(), pb.spec.kv_start.numpy()
    for b in sample:
        slots = r2t[rpi[b], starts[b]:starts[b] + lens[b]]
        k, v = stored(step.quant, slots)
        if varlen:      # read back as bf16 first: the call's own rows (an element may lie on a tie), held to their bound
            at = int(lens[:b].sum())
            kr, vr = (host(x)[at:at + lens[b]].astype(np.float64) for x in (pb.k_rag, pb.v_rag))
            R.assert_within(kr, k, np.abs(k) * (2.0 ** -8 + 2.0 ** -22), "read back")
            R.assert_within(vr, v, np.abs(v) * (2.0 ** -8 + 2.0 ** -22), "read back")
            k, v = kr, vr
        q = host(pb.q)[b:b + 1].astype(np.float64)
        o, l, tol, lt = R.attention(q, k, v, [lens[b]], wl.sm_scale)
        if varlen:      # the bf16 decode rounds its weights to bf16 (2^-8), not fp16
            tol = tol + 2.0 ** -8 * np.einsum("hl,lhd->hd", _weights(q[0], k, wl.sm_scale), np.abs(np.repeat(v, q.shape[1] // v.shape[1], 1)))[None]
        R.assert_within(host(pb.out)[b:b + 1], o, tol, "%s request %d" % (name, b))
        R.assert_within(host(pb.lse)[b:b + 1], l, lt, "%s request %d lse" % (name, b))


def _weights(q, k, scale):
    g = q.shape[0] // k.shape[1]
    s = np.einsum("hd,lhd->hl", q, np.repeat(k, g, 1)) * scale
    p = np.exp(s - s.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


@pytest.mark.parametrize("name,batch,kw", [
    ("qwen3_0p6b", 6, {}), ("qwen3_0p6b", 6, dict(fused=True)), ("tiny_gqa", 4, dict(fused=True)),
    ("qwen3_0p6b", 6, dict(alloc=True, fused=True)), ("whisper_encdec", 5, {}),
    ("whisper_encdec", 5, dict(fused=True, cross_mode="gather")), ("llama3_8b", 20, dict(fused=True, kv_chunk=512))])
def test_decode_step(B, name, batch, kw):
    from paged_kv_cache_req_gb300.engine import DecodeStep
    from paged_kv_cache_req_gb300.workloads import make_workload
    wl = make_workload(name, batch=batch)
    step = DecodeStep(wl, quant=True, **kw)
    assert step.check_errors() == 0
    before = step.quant.pool.clone()
    step.run()
    assert step.check_errors() == 0
    for n, pb in step.problems.items():
        check_decode(step, n, range(0, batch, 3), varlen=pb.gather)
        if pb.spec.stores:
            # the step's rows, and nothing else, were written
            slots = pb.slot_mapping.cpu().numpy()
            t = R.tile_of(wl.page_size)
            tiles = np.unique(slots // t)
            want = before[torch.from_numpy(tiles).to(DEV)].cpu().numpy()
            at = np.searchsorted(tiles, slots // t) * t + slots % t
            for part, x, g in ((0, step.k_new, step.quant.k_scale), (1, step.v_new, step.quant.v_scale)):
                R.write(want, wl.page_size, at, part, *R.quantise(host(x), g.cpu().numpy()))
            assert (step.quant.pool[torch.from_numpy(tiles).to(DEV)].cpu().numpy() == want).all()
            rest = torch.ones(before.shape[0], dtype=torch.bool, device=DEV)
            rest[torch.from_numpy(tiles).to(DEV)] = False
            assert torch.equal(step.quant.pool[rest], before[rest])


def check_extend(step, sample, rows):
    ew = step.ew
    r2t, rpi, lens = step.r2t.cpu().numpy(), ew.req_pool_idx.numpy(), ew.seq_lens.numpy()
    qo = step.qo_indptr.cpu().numpy()
    ends = step.kv_end.cpu().numpy() if step.kv_end is not None else None
    for b in sample:
        n = qo[b + 1] - qo[b]
        k, v = stored(step.quant, r2t[rpi[b], :lens[b]])
        pick = np.array(rows(n))
        e = ends[qo[b] + pick] if ends is not None else lens[b] - n + pick + 1
        o, l, tol, lt = R.attention(host(step.q)[qo[b] + pick].astype(np.float64), k, v, e, ew.sm_scale)
        R.assert_within(host(step.out)[qo[b] + pick], o, tol, "request %d" % b)
        R.assert_within(host(step.lse)[qo[b] + pick], l, lt, "request %d lse" % b)


@pytest.mark.parametrize("name,batch,table", [("llama3_8b_verify", 6, True), ("llama3_8b_verify", 3, False),
                                              ("qwen3_0p6b_prefill", 3, True), ("qwen3_0p6b_prefill", 1, False),
                                              ("hunyuan_image_spans", 1, True)])
def test_extend_step(B, name, batch, table):
    from paged_kv_cache_req_gb300.engine import ExtendStep
    from paged_kv_cache_req_gb300.workloads import make_extend_workload
    step = ExtendStep(make_extend_workload(name, batch=batch), token_table=table, quant=True)
    step.run()
    assert step.check_errors() == 0
    check_extend(step, range(batch), lambda n: sorted({0, 1, n // 3, n // 2, n - 2, n - 1}) if n > 6 else range(n))


def _big(B, rows):
    """Arguments of a call that reads 184 MB of pool, so that warps do wait for their copies."""
    H, D, ps, tiles = 8, 128, 64, 2500
    nb, gen = R.tile_bytes(ps, D), torch.Generator(device=DEV)
    gen.manual_seed(7)
    pool = torch.randint(0, 256, (tiles, H, nb), generator=gen, dtype=torch.uint8, device=DEV)
    pool[:, :, ps * D:] = torch.randint(32, 64, (tiles, H, nb - ps * D), generator=gen, dtype=torch.uint8, device=DEV)
    lens = [100000, 5, 59000, 130]
    npg = [-(-x // ps) for x in lens]
    pages = np.random.default_rng(7).permutation(tiles)[:sum(npg)].astype(np.int32)
    ind = np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)
    n = sum(rows)
    q = torch.randn((n, 32, D), generator=gen, device=DEV).to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros((n, 32), dtype=torch.float32, device=DEV)
    kw = dict(qo_indptr=up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))) if rows != [1] * 4 else {}
    a = B.make_quant_args(B.PKV_LAYOUT_CSR, q, pool, out, page_size=ps, sm_scale=D ** -0.5, max_seq_len=max(lens), lse=lse,
                          kv_indptr=up(ind), kv_indices=up(pages),
                          kv_last_page_len=up(np.array([l - (k - 1) * ps for l, k in zip(lens, npg)], dtype=np.int32)), **kw)

    def right():
        for b in (1, 3):      # the short requests in full
            at = sum(rows[:b])
            slots = (pages[ind[b]:ind[b + 1], None].astype(np.int64) * ps + np.arange(ps)).reshape(-1)[:lens[b]]
            tl = np.unique(slots // ps)
            sub = pool[torch.from_numpy(tl).to(DEV)].cpu().numpy()
            loc = np.searchsorted(tl, slots // ps) * ps + slots % ps
            o, l, tol, lt = R.attention(host(q)[at:at + rows[b]].astype(np.float64), R.read(sub, ps, D, loc, 0),
                                        R.read(sub, ps, D, loc, 1), np.arange(lens[b] - rows[b] + 1, lens[b] + 1), D ** -0.5)
            R.assert_within(host(out)[at:at + rows[b]], o, tol, "out")
            R.assert_within(host(lse)[at:at + rows[b]], l, lt, "lse")
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()

    return a, right


@pytest.mark.parametrize("kv_chunk", [0, 1024])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [4, 2, 3, 4], [300, 5, 200, 100]])
def test_a_call_that_gives_up_ends_and_the_next_is_right(B, rows, kv_chunk):
    a, right = _big(B, rows)
    a.kv_chunk = kv_chunk
    size, call = ((B.pkv_quant_decode_workspace_size, B.pkv_quant_decode) if rows == [1] * 4
                  else (B.pkv_quant_extend_workspace_size, B.pkv_quant_extend))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((size(a),), 0xFF, dtype=torch.uint8, device=DEV)
    B.pkv_set_wait_limit(1)
    try:
        call(a, ws, err)
        torch.cuda.synchronize()      # the abandoned launch ends
    finally:
        B.pkv_set_wait_limit(0)
    # a decode waits for memory; with more rows the math may never have to
    assert err.item() == B.PKV_DEVERR_TIMEOUT or (err.item() == 0 and rows != [1] * 4)
    err.zero_()
    call(a, ws, err)
    assert err.item() == 0
    right()


@pytest.mark.parametrize("n", [129, 1024, 1025, 3000])
def test_large_batches(B, n):
    """Around the sizes at which the tile table and the request values move out of shared memory."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 150, n).tolist()
    cache = Cache(rng, lens, 16, 1, 64)
    q = to_bf16(values(rng, (n, 4, 64)))
    out, lse, e = decode(B, cache, q, "table")
    assert e == 0
    check(cache, q, out, lse, only=[0, 1, n // 2, n - 2, n - 1] + list(range(0, n, 97)))
    rows = [int(x) for x in np.minimum(lens, rng.integers(0, 3, n))]
    q = to_bf16(values(rng, (sum(rows), 4, 64)))
    out, lse, e = extend(B, cache, q, rows, "csr")
    assert e == 0
    check(cache, q, out, lse, rows, only=[0, 1, n - 1] + list(range(0, n, 97)))


def test_more_keys_than_announced(B):
    """total_kv too small: flagged; the requests that fit are right."""
    rng = np.random.default_rng(63)
    lens, rows = [300, 260, 400], [100, 150, 200]
    cache = Cache(rng, lens, 16, 2, 128)
    q = to_bf16(values(rng, (sum(rows), 8, 128)))
    out, lse, e = extend(B, cache, q, rows, total_kv=600)
    assert e == B.PKV_DEVERR_CAPACITY
    check(cache, q, out, lse, rows, only=[0, 1])


@pytest.mark.parametrize("max_q", [0, 1, 200])
def test_row_bounds_only_choose_the_path(B, max_q):
    """max_q_len below, at and without the real maximum: the same rows within the same bounds."""
    rng = np.random.default_rng(64)
    lens, rows = [500, 40, 300], [200, 1, 33]
    cache = Cache(rng, lens, 32, 2, 128)
    q = to_bf16(values(rng, (sum(rows), 6, 128)))
    out, lse, e = extend(B, cache, q, rows, max_q_len=max_q)
    assert e == 0
    check(cache, q, out, lse, rows)


def test_malformed_row_offsets(B):
    """Offsets that run backwards, overlap or leave the rows: flagged, and nothing else is touched."""
    rng = np.random.default_rng(65)
    lens = [200, 100, 300, 50]
    cache = Cache(rng, lens, 16, 2, 128)
    for n, bad in ((40, [0, 10, 5, 30, 40]), (40, [0, 10, 20, 99, 40]), (40, [-3, 10, 20, 30, 40]), (400, [0, 300, 150, 350, 400])):
        q = to_bf16(values(rng, (n, 8, 128)))
        out, lse, e = extend(B, cache, q, [10, 10, 10, n - 30], qo_indptr=up(np.array(bad, dtype=np.int32)))
        assert e & B.PKV_DEVERR_RANGE


@pytest.mark.parametrize("n,max_q", [(16, 0), (64, 0), (64, 64), (256, 256)])
def test_row_ranges_that_overlap_stay_in_the_workspace(B, n, max_q):
    """Every second request claims all rows (the others run backwards), with the keys split:
    more pieces than the workspace was sized for."""
    rng = np.random.default_rng(67)
    batch = 33
    cache = Cache(rng, [600] * batch, 16, 2, 128)
    q = to_bf16(values(rng, (n, 8, 128)))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = cache.args(B, "table", q, out, lse=lse, kv_chunk=64, max_q_len=max_q,
                   qo_indptr=up(np.array([0, n] * (batch // 2) + [0, n], dtype=np.int32)))
    size = B.pkv_quant_extend_workspace_size(a)
    ws = torch.full((4 * size + (64 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    B.pkv_quant_extend(a, ws[:size], err)
    assert err.item() & B.PKV_DEVERR_RANGE
    assert (ws[size:] == 0xA5).all()


def test_a_bound_without_keys_is_flagged(B):
    """kv_end past the keys of a request that has none."""
    rng = np.random.default_rng(68)
    cache = Cache(rng, [0, 40], 16, 2, 64)
    q = to_bf16(values(rng, (3, 4, 64)))
    out, lse, e = extend(B, cache, q, [1, 2], kv_end=[1, 40, 7])
    assert e == B.PKV_DEVERR_RANGE
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    check(cache, q, out, lse, [1, 2], kv_end=[0, 40, 7])


def test_a_batch_past_the_held_tables(B):
    """Many requests of many rows each: more than the tables of the copied keys hold."""
    rng = np.random.default_rng(69)
    batch = 4100
    lens = (33 + rng.integers(0, 30, batch)).tolist()
    cache = Cache(rng, lens, 16, 1, 64)
    rows = [33] * batch
    q = to_bf16(values(rng, (33 * batch, 4, 64)))
    out, lse, e = extend(B, cache, q, rows, max_q_len=33)
    assert e == 0
    check(cache, q, out, lse, rows, only=[0, 1, 2050, batch - 1])


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("max_q", [0, 1])
@pytest.mark.parametrize("D,ps,H,g,lens,rows", [
    (128, 16, 8, 4, [300, 40, 5, 1000], [4, 1, 3, 8]), (64, 1, 2, 1, [70, 9, 0], [1, 9, 0]), (128, 1, 4, 8, [200], [5]),
    (64, 64, 20, 2, [130, 64, 65], [4, 4, 4]), (128, 32, 2, 7, [33, 900], [2, 2]), (64, 8, 1, 16, [2000], [7]),
    (128, 2, 3, 3, [1, 2, 3, 100], [1, 2, 3, 4]), (64, 4, 8, 5, [17], [3]), (128, 128, 1, 4, [400, 0, 129], [16, 0, 2])])
def test_small_multi_row_calls(B, D, ps, H, g, lens, rows, max_q, given):
    """One launch, a block per request and kv head; max_q = 1 makes it go over the rows 8 or 16 at a time."""
    rng = np.random.default_rng(73 + D + ps + H)
    cache = Cache(rng, lens, ps, H, D)
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    ends = None
    if given:
        ends = np.concatenate([rng.integers(0, n + 1, r) for n, r in zip(lens, rows)]).astype(np.int32)
        ends[::3] = 0
    probe = cache.args(B, "table", q, torch.zeros_like(q), max_q_len=max_q,
                       qo_indptr=up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)))
    if max_q == 1:   # (with more rows announced, the spans may be the better choice)
        assert B.pkv_quant_extend_workspace_size(probe) == 256
    out, lse, e = extend(B, cache, q, rows, "table", ends, max_q_len=max_q)
    assert e == 0
    check(cache, q, out, lse, rows, ends)


@pytest.mark.parametrize("case", [c[:-1] for c in DECODE if c[-1] == 0])
def test_decode_in_spans(B, case):
    D, ps, H, g, lens, layout = case
    rng = np.random.default_rng(74 + D + ps + H)
    cache = Cache(rng, lens, ps, H, D)
    q = to_bf16(values(rng, (len(lens), H * g, D)))
    out, lse, e = decode(B, cache, q, layout, kv_chunk=128)
    assert e == 0
    check(cache, q, out, lse)


@pytest.mark.parametrize("case", [c[:-1] for c in EXTEND if c[-1] == 0 and max(c[5]) * c[3] <= 128])
def test_extend_in_spans(B, case):
    D, ps, H, g, lens, rows, layout = case
    rng = np.random.default_rng(75 + D + ps + H)
    cache = Cache(rng, lens, ps, H, D)
    q = to_bf16(values(rng, (sum(rows), H * g, D)))
    for chunk in (64, 256):
        out, lse, e = extend(B, cache, q, rows, layout, kv_chunk=chunk)
        assert e == 0
        check(cache, q, out, lse, rows)


def test_many_rows_of_a_request_without_keys(B):
    """The copied-keys path where one request has no key at all, and where none has."""
    rng = np.random.default_rng(70)
    for lens in ([0, 300], [0, 0]):
        cache = Cache(rng, lens, 16, 2, 64)
        q = to_bf16(values(rng, (400, 4, 64)))
        ends = np.concatenate([np.zeros(200), rng.integers(0, lens[1] + 1, 200)]).astype(np.int32)
        out, lse, e = extend(B, cache, q, [200, 200], kv_end=ends)
        assert e == 0
        assert (out[:200] == 0).all() and (lse[:200] == -float("inf")).all()
        check(cache, q, out, lse, [200, 200], kv_end=ends)


def test_equal_rows_for_one_slot(B):
    """A slot named twice with the same row holds that row."""
    rng = np.random.default_rng(71)
    ps, H, D = 16, 2, 64
    x = values(rng, (40, H, D))
    slots = rng.permutation(48)[:20].astype(np.int32)
    x[20:] = x[:20]
    pool = torch.zeros((3, H, R.tile_bytes(ps, D)), dtype=torch.uint8, device=DEV)
    want = pool.cpu().numpy()
    g = np.array([0.5, 0.02], dtype=np.float32)
    for part in (0, 1):
        R.write(want, ps, slots, part, *R.quantise(x[:20], g))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.pkv_quant_store(pool, to_bf16(x), to_bf16(x), up(np.concatenate([slots, slots])), err, page_size=ps, k_scale=up(g),
                      v_scale=up(g))
    assert err.item() == 0 and (pool.cpu().numpy() == want).all()


@pytest.mark.parametrize("D,H,n", [(64, 1, 1), (64, 1, 7), (64, 1, 1001), (64, 2, 5), (64, 2, 333), (128, 1, 3), (128, 1, 1001)])
def test_tokens_that_share_a_warp(B, D, H, n):
    """Rows of half a warp or less: padded tokens and slots past the pool among them, then read back
    with a bad page, an empty request and rows past the capacity."""
    rng = np.random.default_rng(76 + D + H + n)
    ps, slots = 4, 4 * (n // 4 + 3)
    x = values(rng, (n, H, D))
    mapping = rng.permutation(slots)[:n].astype(np.int32)
    where = rng.random(n)
    where[0] = 0.5
    mapping[where < 0.1] = -1
    mapping[where > 0.9] += slots
    kept = (where >= 0.1) & (where <= 0.9)
    g = np.array([0.5, 0.125], dtype=np.float32)[:H]   # (products with it are exact)
    before = rng.integers(0, 100, (slots // ps, H, R.tile_bytes(ps, D))).astype(np.uint8)
    want = before.copy()
    for part in (0, 1):
        R.write(want, ps, mapping[kept], part, *R.quantise(x[kept], g))
    pool, err = up(before), torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(page_size=ps, k_scale=up(g), v_scale=up(g))
    B.pkv_quant_store(pool, to_bf16(x), to_bf16(x), up(mapping), err, **kw)
    assert err.item() == (B.PKV_DEVERR_RANGE if (where > 0.9).any() else 0)
    assert (pool.cpu().numpy() == want).all()
    lens = np.array([n // 2, 0, n - n // 2], dtype=np.int32)
    table = np.zeros((3, n + 4), dtype=np.int32)
    for b, m in enumerate(lens):
        table[b, :m] = rng.integers(0, slots, m)
    cap = n - n // 10
    out = [torch.full((cap, H, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    flat = np.concatenate([table[b, :m] for b, m in enumerate(lens)])[:cap].astype(np.int64)
    bad = n // 3
    if n > 100:
        table[0, bad], flat[bad] = slots, 0
    err.zero_()
    B.pkv_quant_gather(pool, up(table), up(np.arange(3, dtype=np.int32)), up(lens), n, out[0], out[1], cu, err, **kw)
    assert err.item() == (B.PKV_DEVERR_RANGE if n > 100 else 0) | (B.PKV_DEVERR_CAPACITY if cap < n else 0)
    assert cu.tolist() == [0] + np.cumsum(lens).tolist()
    for part, o in enumerate(out):
        ref = R.bf16(R.read(want, ps, D, flat, part, g).astype(np.float32))
        if n > 100:
            ref[bad] = 0
        assert (host(o) == ref).all()


def test_two_calls_at_once(B):
    """Two streams, each with its own workspace: decodes beside many-row steps, again and again."""
    rng = np.random.default_rng(72)
    cache = Cache(rng, [900, 30, 400, 2000], 16, 2, 128)
    rows = [200, 3, 100, 64]
    qd, qe = to_bf16(values(rng, (4, 8, 128))), to_bf16(values(rng, (sum(rows), 8, 128)))
    calls = []
    for q, extra, size, call in (
            (qd, {}, B.pkv_quant_decode_workspace_size, B.pkv_quant_decode),
            (qe, dict(qo_indptr=up(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))),
             B.pkv_quant_extend_workspace_size, B.pkv_quant_extend)):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float32, device=DEV)
        a = cache.args(B, "table", q, out, lse=lse, **extra)
        calls.append((call, a, torch.empty(size(a), dtype=torch.uint8, device=DEV),
                      torch.zeros(1, dtype=torch.int32, device=DEV), out, lse, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for call, a, ws, err, _, _, stream in calls:
            call(a, ws, err, stream=stream)
    torch.cuda.synchronize()
    for i, (_, _, _, err, out, lse, _) in enumerate(calls):
        assert err.item() == 0
        check(cache, qe if i else qd, out, lse, rows if i else None)


def test_a_serving_batch_on_its_own_stream(B):
    """Calls on a stream that is not the current one, tensors made on another."""
    rng = np.random.default_rng(66)
    cache = Cache(rng, [700, 20], 16, 2, 128)
    q = to_bf16(values(rng, (2, 8, 128)))
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = cache.args(B, "csr", q, out, lse=lse)
    ws = torch.empty(B.pkv_quant_decode_workspace_size(a), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    B.pkv_quant_decode(a, ws, err, stream=s)
    s.synchronize()
    assert err.item() == 0
    check(cache, q, out, lse)
