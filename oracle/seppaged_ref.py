"""Oracle of the rotary positions and of the paged e4m3 cache (test infrastructure), fp64 numpy.

The separator rule is [AS] "Approach" (initial tokens, separators, n most recent neighbours), here
over a cache that keeps every token ([AS] "Key results": training-free use) or, with n at
least the length, over all of them ([AS] hybrid full-attention layers). The storage format is this
library's own and written out here from its definition:

* an e4m3 number has a sign, 4 exponent bits (bias 7) and 3 mantissa bits; the largest is 448, the
  code 0x7f is NaN, there is no infinity;
* a page (a fixed number of consecutive tokens) has, per KV head, one scale for K and one for V: the
  power of two 2^e with the smallest e >= -100 such that every finite value is at most 448 * 2^e, and
  0 while all values are 0. It starts with the page's slot 0 and then only grows; rows already held are
  then rounded again in the larger scale.
"""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_EXPONENT = -100


def e4m3_values():
    """Value of each of the 256 codes, from the bit fields."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        exp, man = (code >> 3) & 15, code & 7
        if exp == 15 and man == 7:
            out[code] = np.nan
        elif exp == 0:
            out[code] = sign * man * 2.0 ** -9
        else:
            out[code] = sign * (1.0 + man / 8.0) * 2.0 ** (exp - 7)
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # ascending, 0 .. 448


def e4m3_encode(x):
    """Codes of the nearest e4m3 numbers (ties to the even code); anything not finite is NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def e4m3_decode(code):
    return _VALUES[np.asarray(code, dtype=np.uint8)]


def page_scale(values):
    """Scale of a page from all its values (any shape)."""
    v = np.abs(np.asarray(values, dtype=np.float64)).ravel()
    v = v[np.isfinite(v)]
    top = float(v.max()) if v.size else 0.0
    if top == 0.0:
        return 0.0
    e = MIN_EXPONENT
    while E4M3_MAX * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def rope_turn(x, pos, freq, magnitude=1.0, interleaved=False, inverse=False):
    """x [..., d] with the pairs of its first 2 len(freq) elements turned by pos * freq (pos broadcast
    on x's leading axes), as a complex product; inverse: by the negative angle."""
    x = np.array(x, dtype=np.float64)
    h = len(freq)
    one = np.arange(h)
    i1, i2 = (2 * one, 2 * one + 1) if interleaved else (one, one + h)
    ang = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(freq, dtype=np.float64)
    z = (x[..., i1] + 1j * x[..., i2]) * (magnitude * np.exp((-1j if inverse else 1j) * ang))
    x[..., i1], x[..., i2] = z.real, z.imag
    return x


class PagedSim:
    """Pages of one KV head set: codes, scales and flags after a series of appends."""

    def __init__(self, num_pages, Hkv, d, page, freq=None, magnitude=1.0, interleaved=False):
        self.page, self.rope = page, (freq, magnitude, interleaved)
        self.codes = {x: np.zeros((num_pages, Hkv, page, d), dtype=np.uint8) for x in "kv"}
        self.scale = {x: np.zeros((num_pages, Hkv)) for x in "kv"}
        self.flags = np.zeros((num_pages, page), dtype=np.uint8)

    def append(self, table, first, k, v, sep):
        """One call's new tokens of one sequence: k, v [c, Hkv, d], positions first .. first + c - 1."""
        c = k.shape[0]
        pos = np.arange(first, first + c)
        rows = {"k": np.asarray(k, dtype=np.float64), "v": np.asarray(v, dtype=np.float64)}
        if self.rope[0] is not None:
            rows["k"] = rope_turn(rows["k"], pos[:, None], *self.rope)
        for i in range(c):
            if pos[i] >= 0:
                self.flags[table[pos[i] // self.page], pos[i] % self.page] = sep[i]
        for pg in sorted({p // self.page for p in pos if p >= 0}):
            sel = [i for i in range(c) if pos[i] >= 0 and pos[i] // self.page == pg]
            slot0, id_ = pos[sel[0]] % self.page, table[pg]
            for x in "kv":
                for h in range(k.shape[1]):
                    new = page_scale(rows[x][sel, h])
                    if slot0 > 0:
                        old = self.scale[x][id_, h]
                        if new > old > 0.0:
                            held = e4m3_decode(self.codes[x][id_, h, :slot0])
                            self.codes[x][id_, h, :slot0] = e4m3_encode(held * (old / new))
                        new = max(new, old)
                    self.scale[x][id_, h] = new
                    val = rows[x][sel, h]
                    val = val / new if new > 0.0 else np.where(np.isfinite(val), 0.0, np.nan)
                    self.codes[x][id_, h, slot0:slot0 + len(sel)] = e4m3_encode(val)

    def rows(self, x, table, length):
        """Values [length, Hkv, d] of a sequence."""
        ids = [table[j // self.page] for j in range(length)]
        sl = [j % self.page for j in range(length)]
        return e4m3_decode(self.codes[x][ids, :, sl]) * self.scale[x][ids][:, :, None]

    def kept_flags(self, table, length):
        return np.array([self.flags[table[j // self.page], j % self.page] != 0 for j in range(length)],
                        dtype=bool)


def paged_attend(q, k, v, flag, a, n, scale):
    """The newest len(q) tokens' attention: q [c, Hq, d], k, v [len, Hkv, d], flag [len].

    Returns o [c, Hq, d], lse [c, Hq] and, for error bounds, the weighted magnitudes sum_j p_j |v_j|
    [c, Hq, d]. A query that keeps nothing has o = 0, lse = -inf."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    c, Hq, d = q.shape
    length, G = k.shape[0], q.shape[1] // k.shape[1]
    o, mag, lse = np.zeros((c, Hq, d)), np.zeros((c, Hq, d)), np.full((c, Hq), -math.inf)
    j = np.arange(length)
    anchor = (j < a) | np.asarray(flag, dtype=bool)
    for i in range(c):
        p = length - c + i
        keep = np.nonzero((j <= p) & ((p - j < n) | anchor))[0]
        if keep.size == 0:
            continue
        for h in range(k.shape[1]):
            hs = slice(h * G, h * G + G)
            s = scale * (q[i, hs] @ k[keep, h].T)
            top = s.max(1, keepdims=True)
            w = np.exp(s - top)
            total = w.sum(1, keepdims=True)
            o[i, hs] = (w / total) @ v[keep, h]
            mag[i, hs] = (w / total) @ np.abs(v[keep, h])
            lse[i, hs] = (top + np.log(total))[:, 0]
    return o, lse, mag
