"""Per-head norm and rotation, the paged cache's rows, and attention of drafted
tokens (test oracle, float64; the quantisers step by step in binary32).

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""

from __future__ import annotations

import numpy as np

from .formats import QK
from .quant import quantize_q4_0, quantize_q8_0

KV_FMTS = ("bf16", "q8_0", "q4_0")

# 2 pi to the 64 bits of a long double
_TWO_PI = np.longdouble("6.283185307179586476925286766559005768")


def rope_ref(x, pos, inv_freq, interleaved=False, norm=False, g=None, eps=1e-6):
    """float64 [T, H, D] rows of x normalised (norm) and turned by pos[t] * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    T, H, D = y.shape
    if norm:
        y /= np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + np.float64(np.float32(eps)))
        if g is not None:
            y *= np.asarray(g, dtype=np.float64)
    half = len(inv_freq)
    out = y.copy()
    for t in range(T):
        for i in range(half):
            # the exact angle, reduced before cos and sin see it
            th = float(np.fmod(np.longdouble(int(pos[t])) * np.longdouble(np.float32(inv_freq[i])), _TWO_PI))
            c, s = np.cos(th), np.sin(th)
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = y[t, :, ia], y[t, :, ib]
            out[t, :, ia] = a * c - b * s
            out[t, :, ib] = a * s + b * c
    return out


def rope_tolerance(x, ref, interleaved, half, norm=False, g=None, eps=1e-6, bf16=False):
    """Bound on a binary32 evaluation: with u = 2^-24, cos and sin are off by
    2 u, the two products and the sum by 3 u, and a normalised element by the
    4e-6 of the row norm; all relative to |a| + |b| of the element's pair.  A
    result in bf16 adds half a step."""
    y = np.abs(rope_ref(x, np.zeros(len(x), int), np.zeros(0), norm=norm, g=g, eps=eps))
    pair = y.copy()
    if half:
        if interleaved:
            both = y[..., 0:2 * half:2] + y[..., 1:2 * half:2]
            pair[..., 0:2 * half:2] = pair[..., 1:2 * half:2] = both
        else:
            both = y[..., :half] + y[..., half:2 * half]
            pair[..., :half] = pair[..., half:2 * half] = both
    tol = pair * (6 * 2.0**-24 + (4e-6 if norm else 0)) + 1e-30
    return tol + (2.0**-8 * np.abs(ref) if bf16 else 0)


def row_places(D):
    """Place of element 32 b + 2 c + e in a quantised row: 2 NB c + 2 b + e."""
    e = np.arange(D)
    return 2 * (D // QK) * ((e % QK) // 2) + 2 * (e // QK) + e % 2


def bf16_rne(x):
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def kv_encode(fmt, x):
    """float32 [..., D] -> (codes uint8 [..., row bytes], scales uint8 [..., D / 16])."""
    x = np.asarray(x, dtype=np.float32)
    D = x.shape[-1]
    if fmt == "bf16":
        return bf16_rne(x).view(np.uint8).reshape(*x.shape[:-1], 2 * D), np.zeros((*x.shape[:-1], 0), np.uint8)
    flat = x.reshape(-1, D)
    blk = (quantize_q8_0 if fmt == "q8_0" else quantize_q4_0)(flat)
    scales = blk[..., :2].copy()
    d = scales.view("<f2")
    d[np.isinf(d)] = np.copysign(np.float16(65504), d[np.isinf(d)])
    if fmt == "q8_0":
        codes = (blk[..., 2:].view(np.int8).astype(np.int16) + 128).astype(np.uint8).reshape(-1, D)
    else:
        codes = np.concatenate((blk[..., 2:] & 15, blk[..., 2:] >> 4), -1).reshape(-1, D)
    row = np.empty_like(codes)
    row[:, row_places(D)] = codes
    if fmt == "q4_0":
        row = row[:, 0::2] | (row[:, 1::2] << 4)
    return row.reshape(*x.shape[:-1], -1), scales.reshape(*x.shape[:-1], -1)


def kv_decode(fmt, codes, scales):
    """The values of kv_encode's bytes, float64 [..., D]."""
    if fmt == "bf16":
        u = np.ascontiguousarray(codes).view(np.uint16).astype(np.uint32) << 16
        return u.view(np.float32).astype(np.float64)
    D = scales.shape[-1] * 16
    if fmt == "q4_0":
        codes = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], D)
    q = codes[..., row_places(D)].astype(np.float64) - (128 if fmt == "q8_0" else 8)
    return q * np.repeat(np.ascontiguousarray(scales).view(np.float16).astype(np.float64), QK, axis=-1)


class Pages:
    """One buffer of a cache on the host, [pages][heads][chunk] bytes."""

    def __init__(self, fmt, pages, heads, page, D, fill=0xFF):
        self.fmt, self.page, self.D = fmt, page, D
        self.row = {"bf16": 2 * D, "q8_0": D, "q4_0": D // 2}[fmt]
        self.sc = 0 if fmt == "bf16" else D // 16
        self.raw = np.full((pages, heads, page * (self.row + self.sc)), fill, np.uint8)
        self.codes = self.raw[..., :page * self.row].reshape(pages, heads, page, self.row)
        self.scales = self.raw[..., page * self.row:].reshape(pages, heads, page, self.sc)
        assert np.shares_memory(self.codes, self.raw)

    def put(self, slot, x):
        c, s = kv_encode(self.fmt, x)  # [heads, ...]
        self.codes[slot // self.page, :, slot % self.page] = c
        self.scales[slot // self.page, :, slot % self.page] = s

    def get(self, slots):
        """float64 [n, heads, D]."""
        slots = np.asarray(slots)
        p, t = slots // self.page, slots % self.page
        return kv_decode(self.fmt, self.codes[p, :, t], self.scales[p, :, t])


def tree_attn_ref(q, k, v, sees, scale):
    """One sequence: q [n, hq, D], k and v [keys, heads, D], sees bool [n, keys].

    Returns (o float64 [n, hq, D], a = sum p |v| / sum p, e = max_j scale *
    sum_i |q_i k_ij| per row [n, hq, 1]); rows that see nothing are 0.  Values
    that a row does not see do not enter it, whatever they are.
    """
    n, hq, D = q.shape
    o, a, e = np.zeros((n, hq, D)), np.zeros((n, hq, D)), np.zeros((n, hq, 1))
    group = hq // k.shape[1]
    for i in range(n):
        at = np.nonzero(sees[i])[0]
        if not len(at):
            continue
        for h in range(hq):
            kk, vv, x = k[at, h // group], v[at, h // group], np.asarray(q[i, h], np.float64)
            s = scale * (kk @ x)
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h], a[i, h] = p @ vv, p @ np.abs(vv)
            e[i, h] = scale * np.abs(kk * x).sum(-1).max()
    return o, a, e


def tree_attn_tolerance(o, a, e, D, bf16_rows, bf16_cache, keys=0, vmax=0.0):
    """Bound on |o_gpu - o|.

    A score's error d makes p wrong by a factor e^(2 d) at most against the
    others, so o by 2 d * sum p |v|; p, its sum and the sum of p v add their
    own roundings.  float32 rows: q in terms that keep 2^-21, binary32 sums of
    D products (D u each, u = 2^-24, + 8 u for scales and exp's argument); p
    to 2^-17, sums over keys in tiles 2^-17.  bf16 rows: q and p are rounded
    once, to fp16 (half a step 2^-11) or for a bf16 cache to bf16 (2^-8), and
    o once to bf16 (2^-8).

    p times a key's scale is held in fp16, whose smallest step is 2^-24, with
    the largest scale (up to three bits below its bound) and p = 1 at 2^11: a
    term is off by half a step, 2^-25 / 2^(11 - 3) = 2^-33 of the largest value
    vmax, each of `keys` keys once (quantised caches)."""
    u = 2.0**-24
    floor = 0.0 if bf16_cache else keys * 2.0**-33 * vmax
    if not bf16_rows:
        return a * (2 * e * (2.0**-21 + (D + 8) * u) + 2.0**-16) + floor + 1e-30
    r = 2.0**-8 if bf16_cache else 2.0**-11
    return a * (np.expm1(2 * e * (r + (D + 8) * u)) + 2 * r + 2.0**-16) + 2.0**-8 * np.abs(o) + floor + 1e-30
