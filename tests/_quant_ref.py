"""Plain numpy reference of the 4-bit K/V pool and of attention over it.

The stored bytes follow the definition in fp32 (IEEE division and products), so they are
compared for equality; attention is computed in fp64 from the stored values, with a bound
on what the kernels' roundings may add to it.  The number formats are tables of all their
values; nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])      # 0x7f is NaN


def _nearest(table, x):
    """Index of the table's value nearest to each x >= 0 (ties to the even index, saturating)."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(x >= table[-1], len(table) - 1, np.where(up, hi, lo))


def quantise(x, g):
    """x fp32 [n, H, D] (bf16 values), g fp32 [H] -> (codes uint8 [n, H, D/2], scales uint8 [n, H, D/16])."""
    n, H, D = x.shape
    b = x.astype(np.float32).reshape(n, H, D // 16, 16)
    g = np.asarray(g, dtype=np.float32).reshape(1, H, 1)
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, np.float32(0))
    with np.errstate(over="ignore", under="ignore"):
        s = _nearest(E4M3, np.abs(b).max(-1) / (np.float32(6) * g))
        den = (E4M3[s].astype(np.float32) * g)[..., None]
        v = np.where(den > 0, b / np.where(den > 0, den, np.float32(1)), np.float32(0)).astype(np.float32)
    code = _nearest(E2M1, np.abs(v)).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)
    code = np.where(finite[..., None] & (den > 0), code, 0).astype(np.uint8).reshape(n, H, D)
    scale = np.where(finite, s, 0x7f).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def tile_of(ps):
    return min(ps, 64)


def tile_bytes(ps, D):
    return -(-tile_of(ps) * D * 9 // 8 // 16) * 16


def _fields(ps, D, part):
    t = tile_of(ps)
    return part * t * D // 2, t * D + part * t * D // 16


def write(pool, ps, slots, part, codes, scales):
    """Writes rows into a pool array uint8 [tiles, H, bytes]; part 0 = K, 1 = V."""
    t, D = tile_of(ps), codes.shape[2] * 2
    c0, s0 = _fields(ps, D, part)
    for i, s in enumerate(slots):
        a = s % t
        pool[s // t, :, c0 + a * D // 2:c0 + (a + 1) * D // 2] = codes[i]
        pool[s // t, :, s0 + a * D // 16:s0 + (a + 1) * D // 16] = scales[i]


def read(pool, ps, D, slots, part, g=None):
    """fp64 values [n, H, D] of the rows at `slots` (code x scale, x g where given)."""
    slots = np.asarray(slots, dtype=np.int64)
    t = tile_of(ps)
    c0, s0 = _fields(ps, D, part)
    tiles, at = pool[slots // t], slots % t
    H = pool.shape[1]
    codes = np.take_along_axis(tiles, np.broadcast_to((c0 + at[:, None] * (D // 2) + np.arange(D // 2))[:, None], (len(slots), H, D // 2)), 2)
    scales = np.take_along_axis(tiles, np.broadcast_to((s0 + at[:, None] * (D // 16) + np.arange(D // 16))[:, None], (len(slots), H, D // 16)), 2)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(len(slots), H, D)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where((scales & 0x7f) == 0x7f, np.nan, np.append(E4M3, 0.0)[scales & 0x7f])
    s = np.where(scales >> 7, -s, s)
    v = v * np.repeat(s, 16, axis=2)
    return v if g is None else v * np.asarray(g, dtype=np.float64).reshape(1, H, 1)


def bf16(x):
    """fp32 -> bf16 (nearest even) -> fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def attention(q, k, v, ends, sm_scale):
    """q [n, Hq, D], k / v [L, H, D] fp64, ends [n] -> (out, lse, out bound, lse bound).

    What the kernels may add to the exact result:
    - a score is a sum of D products accumulated in fp32: D 2^-23 sum |q k| each, so a
      weight is off by ds = sm_scale D 2^-23 max sum |q k| relative, and by 2^-21 for the
      exponential;
    - a weight is rounded to 16 bits (fp16, 2^-11), or by 2^-25 where it is subnormal
      (the largest weight is 1 or more);
    - sums of n terms in fp32: n 2^-23 relative;
    - the output is rounded to bf16 (2^-8).
    """
    n, Hq, D = q.shape
    L, H, _ = k.shape
    g = Hq // H
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol, ltol = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for h in range(Hq):
        kh, vh = k[:, h // g], v[:, h // g]
        s = q[:, h] @ kh.T * sm_scale
        mag = (np.abs(q[:, h]) @ np.abs(kh).T).max(initial=0.0) * sm_scale
        ds = mag * D * 2.0 ** -23
        for i in range(n):
            e = int(ends[i])
            if e == 0:
                continue
            x = s[i, :e]
            m = x.max()
            p = np.exp(x - m)
            den = p.sum()
            out[i, h] = p @ vh[:e] / den
            lse[i, h] = m + np.log(den)
            absv = p @ np.abs(vh[:e]) / den
            rel = 2.0 ** -11 + 2 * (ds + 2.0 ** -21 + e * 2.0 ** -23)
            tol[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + (1 + 2.0 ** -8) * (rel * absv + e * 2.0 ** -25 * np.abs(vh[:e]).max())
            ltol[i, h] = ds + 2.0 ** -21 + e * 2.0 ** -23 + 2.0 ** -22 * (abs(m) + abs(lse[i, h]) + 1)
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what):
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - ref) <= tol)
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError("%s: %d of %d outside the bound; first at %s: got %r, expected %r, bound %.3e" % (
            what, (~ok).sum(), ok.size, at, got[at], ref[at], np.broadcast_to(tol, ok.shape)[at]))
