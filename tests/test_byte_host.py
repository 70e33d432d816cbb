"""The 8-bit pool and the eviction on the host: the argument blocks' layouts, refusals before any
launch, and the reference's own pins."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import _byte_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


@pytest.mark.parametrize("name,struct", [("pkv_byte_args", "ByteArgs"), ("pkv_evict_args", "EvictArgs")])
def test_args_layout_matches_c(B, tmp_path, name, struct):
    cls = getattr(B, struct)
    fields = [f[0] for f in cls._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pkv.h"', "int main(void){",
             'printf("%%zu\\n", sizeof(%s));' % name]
    lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f) for f in fields] + ["return 0;}"]
    src, exe = tmp_path / "q.c", tmp_path / "q"
    src.write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    vals = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert vals[0] == ctypes.sizeof(cls)
    for f, off in zip(fields, vals[1:]):
        assert getattr(cls, f).offset == off, f


@pytest.mark.parametrize("ps,d,h,want", [(1, 64, 1, 160), (1, 128, 8, 2080), (8, 64, 20, 20544), (16, 128, 8, 32896),
                                         (64, 128, 1, 16512), (64, 128, 100, 1638656), (1024, 64, 2, 16512), (3, 128, 1, 0),
                                         (2048, 128, 1, 0), (16, 96, 1, 0), (16, 64, 0, 0)])
def test_tile_bytes(B, ps, d, h, want):
    assert B.pkv_byte_tile_bytes(ps, d, h) == want
    if want:
        assert R.tile_bytes(ps, d, h) == want


def test_store_workspace(B):
    assert B.pkv_byte_store_workspace_size(0, 16) == 256 and B.pkv_byte_store_workspace_size(100, 16) == 6400
    assert B.pkv_byte_store_workspace_size(-1, 16) == 0 and B.pkv_byte_store_workspace_size(1 << 40, 16) == 0
    assert B.pkv_byte_store_workspace_size(4, 24) == 0


def test_reference_scales():
    """The least exponent, at its borders, and codes that are exact in every scale."""
    for top, E in ((448.0, 127), (449.0, 128), (450.0, 128), (224.0, 126), (0.0, 1), (1e-38, 1), (1.0, 119), (1.75, 119), (1.76, 120)):
        assert R.scale_byte(np.array([top, -top / 2])) == E
    assert R.scale_byte(np.array([np.inf, np.nan, 2.0])) == 120
    top = np.float32(np.uint32(0x7f7f0000).view(np.float32))     # the largest bf16
    assert R.scale_byte(np.array([top])) == 247
    x = R.decode(np.arange(127).astype(np.uint8))
    assert (R.encode(x) == np.arange(127)).all() and (R.encode(-x) == np.arange(127) + 128).all()
    assert R.encode(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7f] * 3


def test_reference_store_and_read():
    rng = np.random.default_rng(0)
    x = R.bf16(rng.standard_normal((40, 3, 64)) * 5)
    pool = R.Pool(np.zeros((6, R.tile_bytes(16, 64, 3)), dtype=np.uint8), 16, 64, 3)
    slots = np.arange(20, 60)
    for a in (0, 7, 13):                                      # three calls, one tile cut by each border
        e = {0: 7, 7: 13, 13: 40}[a]
        pool.store(x[a:e], x[a:e] * 0.5, slots[a:e])
    y = pool.read(slots, 0)
    assert (np.abs(y - x) <= 2.0 ** -4 * np.abs(x) * (1 + 2.0 ** -3) + 2.0 ** -15 * np.abs(x).max()).all()
    assert (pool.read(slots, 1) == y * 0.5).all()


def test_reference_eviction():
    """Six pages of two: the last stays, the first is protected, of equal ones the later goes."""
    table = np.zeros((2, 16), dtype=np.int32)
    pages = [9, 3, 7, 5, 2, 8]
    table[1, :11] = np.concatenate([[2 * p, 2 * p + 1] for p in pages])[:11]
    acc = np.zeros((2, 16), dtype=np.float32)
    acc[1, :11] = [0, 0, 1, 1, 2, 0, 1, 1, 3, 3, 0]
    t, a, lens, free, state = R.evict(table, acc, [1], [0], [11], [7], [1], [0], 2, np.zeros(9, np.int32), [6, 3])
    assert lens.tolist() == [5] and state == [3, 6] and free[3:6].tolist() == [3, 7, 5]
    assert (t[1, :5] // 2).tolist() == [9, 9, 2, 2, 8] and a[1, :11].tolist() == [0, 0, 3, 3, 0] + [0] * 6


def _args(B, **kw):
    a = B.ByteArgs()
    v = dict(layout=B.PKV_LAYOUT_REQ_TO_TOKEN, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, sm_scale=0.1,
             max_seq_len=64, total_q=2, num_tiles=8, tile_stride=8320, q_row_stride=8 * 128, q=256, pool=256, out=256,
             req_to_token=256, r2t_rows=4, r2t_row_stride=64, r2t_width=64, req_pool_idx=256, seq_lens=256, acc_row_stride=64)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


BAD = [(dict(batch=-1), 1), (dict(num_q_heads=9), 1), (dict(num_q_heads=40), 2), (dict(head_dim=96), 2), (dict(page_size=24), 2),
       (dict(layout=2), 1), (dict(sm_scale=0.0), 1), (dict(sm_scale=float("inf")), 1), (dict(kv_chunk=32), 1),
       (dict(tile_stride=8304), 1), (dict(tile_stride=8328), 1), (dict(q_row_stride=1020), 1), (dict(num_tiles=1 << 40), 2),
       (dict(r2t_row_stride=63), 1), (dict(q=0), 1), (dict(pool=264), 1), (dict(seq_lens=0), 1), (dict(total_q=1 << 27), 2)]


@pytest.mark.parametrize("change,status", BAD)
@pytest.mark.parametrize("call", ["decode", "extend", "weights"])
def test_attention_refusals(B, call, change, status):
    flag = ctypes.c_int32(0)
    kw = dict() if call == "decode" else dict(qo_indptr=256)
    if call == "weights":
        kw.update(lse=256, acc_out=256, out=0)
    a = _args(B, **dict(kw, **change))
    fn = getattr(B._lib, "pkv_byte_" + call)
    assert fn(ctypes.byref(a), 256, 1 << 40, ctypes.byref(flag), None) == status
    assert B._lib.pkv_last_error()
    size = getattr(B._lib, "pkv_byte_%s_workspace_size" % call)
    assert size(ctypes.byref(_args(B, **kw))) >= 256


def test_weights_refusals(B):
    flag = ctypes.c_int32(0)

    def call(name, **kw):
        return getattr(B._lib, "pkv_byte_" + name)(ctypes.byref(_args(B, **kw)), 256, 1 << 40, ctypes.byref(flag), None)

    rows = dict(qo_indptr=256, lse=256, acc_out=256)
    assert call("weights", **dict(rows, lse=0)) == 1 and call("weights", **dict(rows, acc_out=0)) == 1
    assert call("weights", **dict(rows, qo_indptr=0)) == 1 and call("weights", **dict(rows, acc_row_stride=63)) == 1
    csr = dict(layout=B.PKV_LAYOUT_CSR, kv_indptr=256, kv_indices=256, kv_last_page_len=256)
    assert call("weights", **dict(rows, **csr)) == 2 and call("decode", acc_out=256, **csr) == 2
    assert call("extend", **rows) == 1 and call("decode", acc_in=256) == 1
    assert call("decode", qo_indptr=256) == 1 and call("decode", kv_end=256) == 1
    # too little workspace, none, a misaligned one
    a = _args(B, acc_out=256)
    need = B._lib.pkv_byte_decode_workspace_size(ctypes.byref(a))
    assert need > B._lib.pkv_byte_decode_workspace_size(ctypes.byref(_args(B, lse=256, acc_out=256)))
    for ws, n, st in ((256, need - 1, 3), (0, need, 1), (264, need, 1)):
        assert B._lib.pkv_byte_decode(ctypes.byref(a), ws, n, ctypes.byref(flag), None) == st
    assert B._lib.pkv_byte_decode(ctypes.byref(a), 256, need, None, None) == 1
    assert B._lib.pkv_byte_decode(None, 256, need, ctypes.byref(flag), None) == 1
    assert call("decode", batch=0, total_q=0) == 0


def test_store_and_gather_refusals(B):
    flag = ctypes.c_int32(0)
    good = dict(pool=256, tiles=4, ts=8320, H=2, D=128, ps=16, k=256, v=256, kst=256, vst=256, slots=256, n=3, ws=256, wb=256)

    def store(**kw):
        v = dict(good, **kw)
        return B._lib.pkv_byte_store(v["pool"], v["tiles"], v["ts"], v["H"], v["D"], v["ps"], v["k"], v["v"], v["kst"], v["vst"],
                                     v["slots"], v["n"], v["ws"], v["wb"], ctypes.byref(flag), None)

    for kw, st in ((dict(n=-1), 1), (dict(H=0), 1), (dict(D=32), 2), (dict(ps=48), 2), (dict(ts=8319), 1), (dict(ts=8304), 1),
                   (dict(pool=8), 1), (dict(kst=255), 1), (dict(vst=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(slots=0), 1),
                   (dict(wb=255), 3), (dict(ws=0), 1), (dict(ws=128), 1), (dict(pool=0), 1), (dict(tiles=-1), 1),
                   (dict(tiles=1 << 30), 2)):
        assert store(**kw) == st, kw
    assert store(n=0, k=0, v=0, slots=0, ws=0, wb=0) == 0

    def gather(**kw):
        v = dict(good, table=256, rows=4, stride=64, width=64, rpi=256, lens=256, batch=2, most=10, out=256, cap=20, cu=256)
        v.update(kw)
        return B._lib.pkv_byte_gather(v["pool"], v["tiles"], v["ts"], v["H"], v["D"], v["ps"], v["table"], v["rows"], v["stride"],
                                      v["width"], v["rpi"], None, v["lens"], v["batch"], v["most"], v["out"], v["out"], v["cap"],
                                      v["cu"], ctypes.byref(flag), None)

    for kw, st in ((dict(batch=-1), 1), (dict(stride=63), 1), (dict(cap=-1), 1), (dict(cu=0), 1), (dict(table=0), 1),
                   (dict(lens=0), 1), (dict(D=96), 2), (dict(ps=2048), 2), (dict(out=0), 1), (dict(most=-1), 1)):
        assert gather(**kw) == st, kw


def test_evict_refusals(B):
    flag = ctypes.c_int32(0)
    fields = [f[0] for f in B.EvictArgs._fields_]

    def call(ws=256, nbytes=1 << 30, err=True, **kw):
        a = B.EvictArgs()
        v = dict({f: 256 for f in fields}, batch=2, page_size=16, max_seq_len=64, num_pool_pages=8, r2t_rows=4, r2t_row_stride=64,
                 r2t_width=64, acc_row_stride=64, free_pages_len=8)
        v.update(kw)
        for k, x in v.items():
            setattr(a, k, x)
        return B._lib.pkv_evict(ctypes.byref(a), ws, nbytes, ctypes.byref(flag) if err else None, None)

    for kw, st in ((dict(batch=-1), 1), (dict(batch=8193), 2), (dict(page_size=12), 2), (dict(page_size=2048), 2), (dict(max_seq_len=-1), 1),
                   (dict(r2t_row_stride=60), 1), (dict(acc_row_stride=60), 1), (dict(free_pages_len=-1), 1), (dict(free_pages=0), 1),
                   (dict(req_to_token=0), 1), (dict(req_to_token_out=0), 1), (dict(acc=0), 1), (dict(acc_out=0), 1), (dict(seq_lens=0), 1),
                   (dict(seq_lens_out=0), 1), (dict(budget=0), 1), (dict(req_pool_idx=0), 1), (dict(free_state=0), 1),
                   (dict(free_state_out=0), 1), (dict(num_pool_pages=1 << 40), 2), (dict(num_pool_pages=-1), 1),
                   (dict(ws=0), 1), (dict(ws=264), 1), (dict(err=False), 1),
                   (dict(nbytes=B.pkv_evict_workspace_size(2, 64, 16) - 1), 3)):
        assert call(**kw) == st, kw
    assert call(batch=0) == 0        # (the free list's state is its own output: nothing to do)
    assert B.pkv_evict_workspace_size(8193, 64, 16) == 0 and B.pkv_evict_workspace_size(2, -1, 16) == 0
    assert B.pkv_evict_workspace_size(2, 64, 17) == 0 and B.pkv_evict_workspace_size(0, 0, 1) >= 256
