"""The 4-bit pool on the host: the argument block's layout, refusals before any launch, and
the reference's own pins."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import _quant_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


def test_quant_args_layout_matches_c(B, tmp_path):
    fields = [f[0] for f in B.QuantArgs._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pkv.h"', "int main(void){",
             'printf("%zu\\n", sizeof(pkv_quant_args));']
    lines += ['printf("%%zu\\n", offsetof(pkv_quant_args, %s));' % f for f in fields] + ["return 0;}"]
    src, exe = tmp_path / "q.c", tmp_path / "q"
    src.write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    vals = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert vals[0] == ctypes.sizeof(B.QuantArgs)
    for f, off in zip(fields, vals[1:]):
        assert getattr(B.QuantArgs, f).offset == off, f


@pytest.mark.parametrize("ps,d,want", [(1, 64, 80), (1, 128, 144), (2, 64, 144), (16, 128, 2304), (64, 128, 9216),
                                       (64, 64, 4608), (1024, 128, 9216), (3, 128, 0), (2048, 128, 0), (16, 96, 0), (0, 128, 0)])
def test_tile_bytes(B, ps, d, want):
    assert B.pkv_quant_tile_bytes(ps, d) == want
    if want:
        assert R.tile_bytes(ps, d) == want


def test_reference_rounding():
    """Ties go to the even code; the formats saturate; the e4m3 table has its known ends."""
    assert [R.E2M1[R._nearest(R.E2M1, x)] for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.2500001)] == \
        [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 0.5]
    assert R.E4M3[1] == 2.0 ** -9 and R.E4M3[126] == 448.0 and len(R.E4M3) == 127
    x = torch.linspace(0, 460, 100001)
    want = x.clamp(max=448).to(torch.float8_e4m3fn).float().numpy()
    assert (R.E4M3[R._nearest(R.E4M3, x.numpy())] == want).all()


def test_reference_reads_what_it_writes():
    rng = np.random.default_rng(0)
    x = R.bf16(rng.standard_normal((5, 3, 64)))
    g = np.array([1.0, 0.5, 0.01], dtype=np.float32)
    pool = np.zeros((4, 3, R.tile_bytes(4, 64)), dtype=np.uint8)
    slots = [15, 0, 6, 7, 9]
    c, s = R.quantise(x, g)
    for part in (0, 1):
        R.write(pool, 4, slots, part, c, s)
    for part in (0, 1):
        y = R.read(pool, 4, 64, slots, part, g)
        # half a step of e2m1 (2^-2 relative, or 0.25 of the scale below 1) and of e4m3 (2^-4)
        amax = np.repeat(np.abs(x).reshape(5, 3, 4, 16).max(-1), 16, axis=2)
        assert (np.abs(y - x) <= 0.25 * np.abs(x) + amax / 6 * 0.25 * (1 + 2.0 ** -4) + 6 * 2.0 ** -10 * g[None, :, None]).all()


def _args(B, **kw):
    a = B.QuantArgs()
    v = dict(layout=B.PKV_LAYOUT_CSR, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, sm_scale=0.1,
             max_seq_len=64, total_q=2, num_tiles=8, tile_stride=2 * 2304, q_row_stride=8 * 128, kv_indices_len=8,
             q=256, pool=256, out=256, kv_indptr=256, kv_indices=256, kv_last_page_len=256)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


BAD = [
    (dict(batch=-1), "INVALID_ARG"), (dict(num_q_heads=7), "INVALID_ARG"), (dict(num_q_heads=0), "INVALID_ARG"),
    (dict(num_q_heads=34, q_row_stride=34 * 128, total_q=2), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"),
    (dict(page_size=24), "UNSUPPORTED"), (dict(page_size=2048), "UNSUPPORTED"), (dict(page_size=0), "UNSUPPORTED"),
    (dict(layout=2), "INVALID_ARG"), (dict(layout=9), "INVALID_ARG"), (dict(sm_scale=0.0), "INVALID_ARG"),
    (dict(sm_scale=float("nan")), "INVALID_ARG"), (dict(sm_scale=float("inf")), "INVALID_ARG"),
    (dict(sm_scale=-0.1), "INVALID_ARG"), (dict(kv_chunk=32), "INVALID_ARG"), (dict(kv_chunk=-64), "INVALID_ARG"),
    (dict(tile_stride=2304), "INVALID_ARG"), (dict(tile_stride=2 * 2304 + 8), "INVALID_ARG"),
    (dict(q_row_stride=512), "INVALID_ARG"), (dict(q_row_stride=1028), "INVALID_ARG"),
    (dict(num_tiles=1 << 28), "UNSUPPORTED"), (dict(max_seq_len=-1), "INVALID_ARG"), (dict(total_kv=-1), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(pool=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(q=264), "INVALID_ARG"), (dict(pool=264), "INVALID_ARG"), (dict(out=258), "INVALID_ARG"),
    (dict(kv_indices=None), "INVALID_ARG"), (dict(layout=1), "INVALID_ARG"), (dict(layout=3), "INVALID_ARG"),
    (dict(layout=3, r2t_rows=2, r2t_width=64, r2t_row_stride=32), "INVALID_ARG"),
]


@pytest.mark.parametrize("change,status", BAD, ids=[",".join("%s=%s" % x for x in b[0].items()) for b in BAD])
def test_attention_refusals(B, change, status):
    flag = ctypes.c_int32(0)
    for extend in (False, True):
        a = _args(B, **dict(change, qo_indptr=256 if extend else None))
        fn = B._lib.pkv_quant_extend if extend else B._lib.pkv_quant_decode
        assert fn(ctypes.byref(a), 256, 1 << 40, ctypes.byref(flag), None) == getattr(B, "PKV_ERR_" + status)
        assert B._lib.pkv_last_error().startswith(b"pkv_quant_extend" if extend else b"pkv_quant_decode")
    assert flag.value == 0


def test_attention_refusals_of_the_call(B):
    flag, lib = ctypes.c_int32(0), B._lib
    a = _args(B)
    assert lib.pkv_quant_decode(None, None, 0, ctypes.byref(flag), None) == B.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_decode(ctypes.byref(a), 256, 1 << 40, None, None) == B.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_decode(ctypes.byref(a), 256, 0, ctypes.byref(flag), None) == B.PKV_ERR_CAPACITY
    assert lib.pkv_quant_decode(ctypes.byref(a), None, 1 << 40, ctypes.byref(flag), None) == B.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_decode(ctypes.byref(a), 264, 1 << 40, ctypes.byref(flag), None) == B.PKV_ERR_INVALID_ARG
    # decode takes one row per request and no bounds; extend needs its row offsets
    for bad in (dict(total_q=3), dict(qo_indptr=256), dict(kv_end=256)):
        b = _args(B, **bad)
        assert lib.pkv_quant_decode(ctypes.byref(b), 256, 1 << 40, ctypes.byref(flag), None) == B.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_extend(ctypes.byref(a), 256, 1 << 40, ctypes.byref(flag), None) == B.PKV_ERR_INVALID_ARG
    # an empty batch is a no-op; sizes are known without a device
    e = _args(B, batch=0, total_q=0, q=None, pool=None, out=None)
    assert lib.pkv_quant_decode(ctypes.byref(e), None, 0, ctypes.byref(flag), None) == B.PKV_OK
    assert B.pkv_quant_decode_workspace_size(a) >= 256
    assert B.pkv_quant_extend_workspace_size(_args(B, qo_indptr=256)) >= 256
    assert B.pkv_quant_decode_workspace_size(_args(B, head_dim=80)) == 0
    assert flag.value == 0


def test_row_call_refusals(B):
    lib, flag = B._lib, ctypes.c_int32(0)
    err = ctypes.byref(flag)
    p = ctypes.c_void_p(256)

    def store(pool=p, tiles=4, stride=2 * 2304, h=2, d=128, ps=16, kn=p, vn=p, ks=256, vs=256, slots=p, n=3, e=err):
        return lib.pkv_quant_store(pool, tiles, stride, h, d, ps, None, None, kn, vn, ks, vs, slots, n, e, None)

    def gather(pool=p, tiles=4, stride=2 * 2304, h=2, d=128, ps=16, r2t=p, rows=2, rs=64, w=64, rpi=p, lens=p, b=2, m=64,
               k=p, v=p, cap=10, cu=p, e=err):
        return lib.pkv_quant_gather(pool, tiles, stride, h, d, ps, None, None, r2t, rows, rs, w, rpi, None, lens, b, m, k, v,
                                    cap, cu, e, None)

    for f in (store, gather):
        for bad in (dict(e=None), dict(tiles=-1), dict(h=0), dict(stride=2304), dict(stride=2 * 2304 + 8), dict(pool=None),
                    dict(pool=ctypes.c_void_p(264))):
            assert f(**bad) == B.PKV_ERR_INVALID_ARG, (f, bad)
        for bad in (dict(d=96), dict(ps=24), dict(ps=2048), dict(ps=0)):
            assert f(**bad) == B.PKV_ERR_UNSUPPORTED, (f, bad)
    for bad in (dict(n=-1), dict(ks=255), dict(vs=0), dict(kn=None), dict(vn=None), dict(slots=None)):
        assert store(**bad) == B.PKV_ERR_INVALID_ARG, bad
    assert store(n=0, kn=None, vn=None, slots=None) == B.PKV_OK
    for bad in (dict(b=-1), dict(rs=32), dict(cap=-1), dict(m=-1), dict(k=None), dict(v=None), dict(r2t=None),
                dict(rpi=None), dict(lens=None), dict(cu=None)):
        assert gather(**bad) == B.PKV_ERR_INVALID_ARG, bad
    assert flag.value == 0


def test_binding_refuses_wrong_tensors(B):
    """Shapes and types the C call cannot see are refused by the binding (no device needed)."""
    pool = torch.zeros((4, 2, 2304), dtype=torch.uint8)
    kv = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32)
    for bad in (dict(pool=pool.to(torch.int8)), dict(pool=pool[..., :2000]), dict(pool=pool[:, :, None]),
                dict(k=kv.float()), dict(v=kv[:2]), dict(k=kv.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(slots=slots.long()), dict(slots=slots[:2]), dict(ks=torch.ones(3)), dict(vs=torch.ones(2).double())):
        a = dict(pool=pool, k=kv, v=kv, slots=slots, ks=None, vs=None)
        a.update(bad)
        with pytest.raises(ValueError):
            B.pkv_quant_store(a["pool"], a["k"], a["v"], a["slots"], err, page_size=16, k_scale=a["ks"], v_scale=a["vs"])
    with pytest.raises(B.PkvError):
        B.pkv_quant_store(pool, kv, kv, slots, err, page_size=24)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    ok = dict(page_size=16, sm_scale=0.1, max_seq_len=64, seq_lens=torch.zeros(2, dtype=torch.int32),
              block_table=torch.zeros((2, 4), dtype=torch.int32))
    for bad in (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), dict(block_table=torch.zeros((3, 4), dtype=torch.int32)),
                dict(k_scale=torch.ones(8)), dict(lse=torch.zeros((2, 8), dtype=torch.float16)),
                dict(kv_end=torch.zeros(5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.make_quant_args(B.PKV_LAYOUT_BLOCK_TABLE, q, pool, torch.empty_like(q), **dict(ok, **bad))
    for qq, oo in ((q.float(), q), (q, q.float()), (q, q[:1]), (q.transpose(0, 1).contiguous().transpose(0, 1)[..., ::1], q[:, :4])):
        with pytest.raises(ValueError):
            B.make_quant_args(B.PKV_LAYOUT_BLOCK_TABLE, qq, pool, oo, **ok)
    with pytest.raises(ValueError):      # device tensors only
        B.pkv_quant_store(pool, kv, kv, slots, err, page_size=16)


def test_sizes_with_far_hints(B):
    """Upper bounds far above the real sizes plan as the real sizes do, or for the spans; sizes past the limits are refused."""
    big = 2 ** 31 - 1
    size = B.pkv_quant_extend_workspace_size
    base = dict(qo_indptr=256, total_q=40, max_q_len=40)
    assert size(_args(B, **dict(base, max_q_len=big))) == size(_args(B, **base)) > 256
    assert size(_args(B, **dict(base, total_kv=2 ** 62))) > 0            # (keys past the copies' coordinates: spans)
    assert size(_args(B, **dict(base, total_kv=2 ** 62, max_q_len=1))) >= 256
    assert B.pkv_quant_decode_workspace_size(_args(B, total_kv=2 ** 62)) >= 256
    # 2^28 (row, head) pairs, or 2^31 (request, kv head) pairs
    assert size(_args(B, qo_indptr=256, total_q=2 ** 25)) == 0
    assert size(_args(B, qo_indptr=256, batch=2 ** 30, total_q=2)) == 0
