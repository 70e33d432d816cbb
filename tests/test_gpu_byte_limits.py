"""The calls over an 8-bit pool at the ends of what they allow: queries, keys and values near the
ends of bf16's range, calls and requests without keys, waits that run out."""
import numpy as np
import pytest
import torch

import _byte_ref as R
from test_gpu_byte import B, Cache, DEV, check, decode, err_word, extend, host, i32, table_of, to_bf16, values  # noqa: F401

pytestmark = pytest.mark.gpu


def weights(B, cache, q, lse, rows, ends=None, **kw):
    """pkv_byte_weights of the rows -> (acc, flags)."""
    acc, err = table_of(cache, None, 0.0), err_word()
    a = cache.args(B, "table", q, None, lse=lse, qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])),
                   kv_end=None if ends is None else i32(ends), acc_out=acc, **kw)
    B.pkv_byte_weights(a, torch.empty(B.pkv_byte_weights_workspace_size(a), dtype=torch.uint8, device=DEV), err)
    return acc, err.item()


def against(rng, big, lens, rows, g, ps=16, D=64, H=2):
    """A cache whose keys are around `big`, and rows that bring the scores back; all of them finite."""
    cache = Cache(rng, lens, ps, H, D, spread=big)
    q = to_bf16(R.bf16(values(rng, (sum(rows), H * g, D)) / np.float32(big)))
    assert torch.isfinite(q).all() and all(np.isfinite(cache.pool.read(s, 0)).all() for s in cache.slots)
    return cache, q


@pytest.mark.parametrize("total", [0, 1 << 22])
@pytest.mark.parametrize("rows,g", [([5, 2], 2), ([40, 33], 2), ([32, 32], 1)])
def test_weights_of_large_queries_over_small_keys(B, rows, g, total):
    """Scores are moderate, though a score times the query's factor alone is past fp32: tiles that all rows see
    and tiles at a bound, in both kernels."""
    rng = np.random.default_rng(50 + sum(rows))
    cache, q = against(rng, 2.0 ** -123, [700, 130], rows, g)
    ends = np.concatenate([rng.integers(l // 2, l + 1, n) for l, n in zip(cache.lens, rows)])
    out, lse, e = extend(B, cache, q, rows, "table", ends)
    assert e == 0
    check(cache, q, out, lse, rows, ends)
    acc, e = weights(B, cache, q, lse, rows, ends, total_kv=total)
    assert e == 0
    check(cache, q, None, None, rows, ends, acc=acc)


@pytest.mark.parametrize("chunk", [0, 64])
@pytest.mark.parametrize("ps,rows", [(64, None), (16, None), (4, None), (1, None), (16, [7, 4]), (64, [64, 20])])
def test_small_queries_over_large_keys(B, ps, rows, chunk):
    """Scores are moderate, though the query's factor alone is below fp32's normal numbers."""
    rng = np.random.default_rng(60 + ps + chunk)
    n = [1, 1] if rows is None else rows
    cache, q = against(rng, 2.0 ** 122, [700, 130], n, 2, ps=ps)
    if rows is None:
        out, lse, e = decode(B, cache, q, kv_chunk=chunk)
        assert e == 0
        check(cache, q, out, lse)
        acc = table_of(cache, None, 0.0)
        out, lse, e = decode(B, cache, q, kv_chunk=chunk, acc_out=acc)
        assert e == 0
        check(cache, q, out, lse, acc=acc)
        return
    out, lse, e = extend(B, cache, q, rows, kv_chunk=chunk)
    assert e == 0
    check(cache, q, out, lse, rows)
    for total in (0, 1 << 22):
        acc, e = weights(B, cache, q, lse, rows, total_kv=total)
        assert e == 0
        check(cache, q, None, None, rows, acc=acc)


def rows_of_one(rng, cache, n, g):
    return to_bf16(values(rng, (n, cache.H * g, cache.D)))


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64)])
def test_held_keys_the_largest_value_that_few_rows_see(B, D, ps):
    """A value that stands for 2^128 in V: rows that do not see its key are as if it were not there."""
    rng = np.random.default_rng(70 + D)
    L, n, g, late = 300, 200, 2, 290
    cache = Cache(rng, [L, 200], ps, 1, D)
    t = R.tile_of(ps)
    slot = cache.slots[0][late]
    cache.pool.E[slot // t, 0, 1] = 247
    cache.pool.codes[slot // t, 0, 1] = 0
    for dim, code in ((5, 0x78), (9, 0xf8)):      # 256 and -256, times 2^120
        cache.pool.codes[slot // t, 0, 1, slot % t, dim] = code
    q = rows_of_one(rng, cache, n + 200, g)
    out, lse, e = extend(B, cache, q, [n, 200])
    assert e == 0
    first = late - (L - n)                        # the first row that sees the key
    qh, k, v = host(q).astype(np.float64), cache.pool.read(cache.slots[0], 0), cache.pool.read(cache.slots[0], 1)
    ref, rl, _, tol, lt, _ = R.attention(qh[:first], k, v, np.arange(L - n + 1, L - n + 1 + first), D ** -0.5, np.ones(1), True)
    R.assert_within(host(out)[:first], ref, tol, "rows that do not see it")
    R.assert_within(host(lse)[:first], rl, lt, "their lse")
    rest = [d for d in range(D) if d not in (5, 9)]
    ref, rl, _, tol, lt, _ = R.attention(qh[first:n], k, v, np.arange(late + 1, L + 1), D ** -0.5, np.ones(1), True)
    R.assert_within(host(out)[first:n][..., rest], ref[..., rest], tol[..., rest], "the other dims of rows that see it")
    check(cache, q, out, lse, [n, 200], only=[1], held=True)


@pytest.mark.parametrize("D,ps,rows", [(64, 16, [200, 20]), (128, 64, [300, 300])])
@pytest.mark.parametrize("big", [2.0 ** 112, 2.0 ** 123, 2.0 ** -100])
def test_held_keys_large_and_small_values(B, D, ps, rows, big):
    """V near the ends of the range: the sums of the rows stay inside fp32."""
    rng = np.random.default_rng(71 + D)
    cache = Cache(rng, [500, 310], ps, 2, D, v_scale=lambda t: np.full(len(t), np.float32(big)))
    q = rows_of_one(rng, cache, sum(rows), 2)
    out, lse, e = extend(B, cache, q, rows)
    assert e == 0
    check(cache, q, out, lse, rows, held=True)


def test_weights_check_a_call_without_keys(B):
    """max_seq_len of 0: what the requests say is looked at as by the other calls."""
    rng = np.random.default_rng(72)
    cache = Cache(rng, [40, 50], 16, 1, 64)
    q = rows_of_one(rng, cache, 4, 2)
    lse = torch.zeros((4, 2), device=DEV)
    none = i32([0, 0])

    def call(**kw):
        kw.setdefault("kv_end", i32([0] * 4))
        out = torch.empty_like(q)
        got = []
        for fn, size, more in ((B.pkv_byte_extend, B.pkv_byte_extend_workspace_size, {}),
                               (B.pkv_byte_weights, B.pkv_byte_weights_workspace_size, dict(acc_out=table_of(cache, rng, 7.0)))):
            fields = dict(lse=lse, qo_indptr=i32([0, 2, 4]), max_seq_len=0)
            fields.update(kw, **more)
            a = cache.args(B, "table", q, out, **fields)
            err = err_word()
            fn(a, torch.empty(size(a), dtype=torch.uint8, device=DEV), err)
            got.append(err.item())
        assert (host(fields["acc_out"]) == 7).all()
        assert got[0] == got[1], got
        return got[1]

    assert call(seq_lens=none) == 0
    assert call() == 4
    assert call(seq_lens=none, req_pool_idx=i32([cache.rpi[0], 55])) == 1
    assert call(seq_lens=none, qo_indptr=i32([0, 2, 9])) == 1
    assert call(seq_lens=i32([0, -1])) == 1


@pytest.mark.parametrize("total", [0, 1 << 22])
@pytest.mark.parametrize("n", [3, 600])
def test_weights_check_the_bounds_of_requests_without_keys(B, total, n):
    """A bound that is not 0 for a row of a request without keys is outside; the other requests get theirs."""
    rng = np.random.default_rng(73 + n)
    rows = [2, n, 5]
    cache = Cache(rng, [300, 0, 70], 16, 2, 64)
    q = rows_of_one(rng, cache, sum(rows), 2)
    ends = np.concatenate([[300, 7], np.zeros(n), [70, 1, 0, 69, 30]]).astype(np.int32)
    out, lse, e = extend(B, cache, q, rows, "table", ends)
    assert e == 0
    want, e = weights(B, cache, q, lse, rows, ends, total_kv=total)
    assert e == 0
    for at, end in ((2, 1), (2 + n - 1, -1), (2 + n // 2, 2 ** 31 - 1)):
        bad = ends.copy()
        bad[at] = end
        acc, e = weights(B, cache, q, lse, rows, bad, total_kv=total)
        assert e == 1 and torch.equal(acc, want), (at, end)


def cold():
    """Whatever lay in L2 is gone."""
    torch.empty(1 << 29, dtype=torch.uint8, device=DEV).zero_()


@pytest.mark.parametrize("call", ["decode", "decode of few", "extend", "held", "weights"])
def test_waits_run_out_when_nothing_is_cached(B, call):
    """With a limit of 1 ns a wait is one look, before copies from memory can have landed: the flag says so, and the
    next call is right."""
    rng = np.random.default_rng(74)
    cache = Cache(rng, [2000] * (3 if call == "decode of few" else 24), 16, 2, 128)
    n = {"extend": 2, "held": 90, "weights": 40}.get(call, 1)
    rows = [n] * len(cache.lens)
    q = rows_of_one(rng, cache, sum(rows), 4)
    out, lse, err = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV), err_word()
    kw = {} if n == 1 else dict(qo_indptr=i32(np.concatenate([[0], np.cumsum(rows)])))
    good = decode(B, cache, q) if n == 1 else extend(B, cache, q, rows)
    assert good[2] == 0
    acc = table_of(cache, None, 0.0)
    if call == "weights":
        kw.update(acc_out=acc)
        lse = good[1]
    a = cache.args(B, "table", q, out, lse=lse, **kw)
    fn, size = {1: (B.pkv_byte_decode, B.pkv_byte_decode_workspace_size)}.get(n, (B.pkv_byte_extend, B.pkv_byte_extend_workspace_size))
    if call == "weights":
        fn, size = B.pkv_byte_weights, B.pkv_byte_weights_workspace_size
    ws = torch.empty(size(a), dtype=torch.uint8, device=DEV)
    cold()
    B.pkv_set_wait_limit(1)
    try:
        fn(a, ws, err)
        assert err.item() == B.PKV_DEVERR_TIMEOUT
    finally:
        B.pkv_set_wait_limit(0)
    err.zero_()
    fn(a, ws, err)
    assert err.item() == 0
    if call == "weights":
        check(cache, q, None, None, rows, acc=acc, only=[0, len(rows) - 1])
    else:
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
