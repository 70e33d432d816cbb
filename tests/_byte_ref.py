"""Plain numpy reference of the 8-bit K/V pool, of attention over it, of the weights that keys
receive, and of eviction.

Stored bytes and evictions follow the definitions exactly and are compared for equality;
attention is computed in fp64 from the stored values, with a bound on what the kernels'
roundings may add.  Nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

from _quant_ref import E4M3, _nearest, assert_within, bf16  # noqa: F401

NAN = 0x7f


def tile_of(ps):
    return min(ps, 64)


def tile_bytes(ps, D, H):
    pad = 128 if tile_of(ps) >= 16 else 32
    return H * 2 * tile_of(ps) * D + -(-2 * H // pad) * pad


def scale_byte(x):
    """Least E >= 1 with max |finite x| <= 448 2^(E - 127)."""
    x = np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64)
    top = float(x.max(initial=0.0))
    E = max(1, int(np.frexp(max(top, 1e-300) / 448)[1]) + 126)     # (one too few at most)
    return E if top <= 448 * 2.0 ** (E - 127) else E + 1


def encode(x):
    """e4m3 bytes of fp64 values (to nearest, ties to even, at most 448; NaN and infinities are NaN)."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x)
    code = _nearest(E4M3, np.where(bad, 0, np.abs(x))).astype(np.uint8)
    return np.where(bad, NAN, code | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


_VALUES = np.append(E4M3, np.nan)
_VALUES = np.concatenate([_VALUES, -_VALUES])


def decode(code):
    return _VALUES[code]


class Pool:
    """A pool array uint8 [tiles, bytes] and its parts as views."""

    def __init__(self, data, ps, D, H):
        self.data, self.ps, self.D, self.H, self.t = data, ps, D, H, tile_of(ps)
        n = H * 2 * self.t * D
        self.codes = data[:, :n].reshape(len(data), H, 2, self.t, D)
        self.E = data[:, n:n + 2 * H].reshape(len(data), H, 2)
        assert np.shares_memory(self.codes, data) and np.shares_memory(self.E, data)

    def store(self, k, v, slots):
        """One call's rows k, v [n, H, D] at `slots` (negative: padded; each slot at most once)."""
        slots = np.asarray(slots, dtype=np.int64)
        live = np.flatnonzero(slots >= 0)
        live = live[np.argsort(slots[live], kind="stable")]
        tiles, first = np.unique(slots[live] // self.t, return_index=True)
        for tile, rows in zip(tiles, np.split(live, first[1:])):
            at = slots[rows] % self.t
            others = np.setdiff1d(np.arange(self.t), at)
            for h in range(self.H):
                for part, x in ((0, k), (1, v)):
                    y = np.asarray(x)[rows, h].astype(np.float64)
                    E, old = scale_byte(y), int(self.E[tile, h, part])
                    if 0 not in at:
                        E = max(E, min(old, 247))
                        if E > old:
                            self.codes[tile, h, part, others] = encode(decode(self.codes[tile, h, part, others]) * 2.0 ** (old - E))
                    self.codes[tile, h, part, at] = encode(y * 2.0 ** (127 - E))
                    self.E[tile, h, part] = E

    def read(self, slots, part):
        """fp64 values [n, H, D]."""
        slots = np.asarray(slots, dtype=np.int64)
        return decode(self.codes[slots // self.t, :, part, slots % self.t]) * 2.0 ** (self.E[slots // self.t, :, part].astype(np.float64) - 127)[..., None]

    def largest(self, slots):
        """The largest value that V's scales at `slots` allow, [H]."""
        slots = np.asarray(slots, dtype=np.int64)
        return 448 * 2.0 ** (self.E[slots // self.t, :, 1].astype(np.float64).max(0, initial=1) - 127)


def attention(q, k, v, ends, sm_scale, most, held=False):
    """q [n, Hq, D], k / v [L, H, D] fp64, ends [n], most [H] -> (out, lse, weights [n, Hq, L], bounds of the three).

    What the kernels may add to the exact result:
    - a score is a sum of D products accumulated in fp32: D 2^-23 sum |q k| each, and two products
      with factors, 2^-23 of the score; a weight is off by that and by 2^-21 for the exponential,
      relative;
    - a weight (times its scale) is rounded to fp16, 2^-11 relative, or by 2^-36 of the row's largest
      times the largest scale where it is subnormal (the largest weight is held as 2^11 or more);
      over held keys to bf16, 2^-8 relative;
    - sums of n terms in fp32: n 2^-23 relative;
    - the output is rounded to bf16: 2^-8 relative, and half of the subnormals' step of 2^-133 below 2^-126.
    """
    n, Hq, D = q.shape
    L, H, _ = k.shape
    g = Hq // H
    out, lse, w = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, L))
    tol, ltol, wtol = np.zeros((n, Hq, D)), np.zeros((n, Hq)), np.zeros((n, Hq, L))
    for h in range(Hq):
        kh, vh = k[:, h // g], v[:, h // g]
        s = q[:, h] @ kh.T * sm_scale
        mag = np.abs(q[:, h]) @ np.abs(kh).T * sm_scale
        for i in range(n):
            e = int(ends[i])
            if e == 0:
                continue
            x = s[i, :e]
            m = x.max()
            p = np.exp(x - m)
            den = p.sum()
            ds = mag[i, :e].max() * (D * 2.0 ** -23 + 2.0 ** -22)
            out[i, h] = p @ vh[:e] / den
            lse[i, h] = m + np.log(den)
            w[i, h, :e] = p / den
            absv = p @ np.abs(vh[:e]) / den
            rel = (2.0 ** -8 if held else 2.0 ** -11) + 2 * (ds + 2.0 ** -21 + e * 2.0 ** -23)
            low = 0.0 if held else e * 2.0 ** -36 * most[h // g]
            tol[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + (1 + 2.0 ** -8) * (rel * absv + low) + 2.0 ** -134
            ltol[i, h] = ds + 2.0 ** -21 + e * 2.0 ** -23 + 2.0 ** -22 * (abs(m) + abs(lse[i, h]) + 1)
            wtol[i, h, :e] = w[i, h, :e] * (2 * ds + ltol[i, h] + 2.0 ** -20) + 2.0 ** -125
    return out, lse, w, tol, ltol, wtol


def evict(table, acc, rows, starts, lens, budget, first, last, ps, free, state):
    """The definition, request after request -> new (table, acc, lens, free, state)."""
    table, acc, free = table.copy(), acc.copy(), free.copy()
    out, gone_ids = [], []
    for b, (r, s, L) in enumerate(zip(rows, starts, lens)):
        n = -(-L // ps)
        may = [p for p in range(n - 1) if p * ps >= first[b] and (p + 1) * ps <= L - last[b]]
        drop = min(len(may), max(0, n - max(1, budget[b] // ps)))
        score = {p: np.float32(acc[r, s + p * ps:s + (p + 1) * ps].astype(np.float64).sum()) for p in may}
        worst = sorted(may, key=lambda p: (np.inf if np.isnan(score[p]) else score[p], bool(np.isnan(score[p])), -p))[:drop]
        gone = sorted(worst)
        gone_ids += [int(table[r, s + p * ps]) // ps for p in gone]
        cols = np.arange(L)
        keep = cols[~np.isin(cols // ps, gone)]
        t, a = table[r, s + keep], acc[r, s + keep]
        table[r, s:s + len(keep)] = t
        acc[r, s:s + len(keep)], acc[r, s + len(keep):s + L] = a, 0
        out.append(len(keep))
    head, count = state
    if gone_ids:
        free[head - len(gone_ids):head] = gone_ids
    return table, acc, np.array(out, dtype=np.int32), free, [head - len(gone_ids), count + len(gone_ids)]
