"""Plain 64-bit and list implementations of the rotary positions, the 8-bit
paged cache, its attention and its page handling, for the tests. They share no
code with the package."""
from __future__ import annotations

import math

import numpy as np


def e4m3_table() -> np.ndarray:
    """The 256 values from the format's definition (NaN at 0x7F and 0xFF)."""
    v = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = math.nan if b & 0x7F == 0x7F else -x if s else x
    return v


TABLE = e4m3_table()
POSITIVE = TABLE[:0x7F]    # ascending


def quantise(x: np.ndarray) -> np.ndarray:
    """fp64 -> e4m3 bytes, nearest, ties to the even byte; |x| <= 448; NaN and
    infinities -> 0x7F (the sign of a NaN is not looked at)."""
    bad = ~np.isfinite(x)
    a = np.where(bad, 0.0, np.abs(x))
    hi = np.searchsorted(POSITIVE, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    up = POSITIVE[hi] - a
    down = a - POSITIVE[lo]
    b = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    b = np.where(a == POSITIVE[hi], hi, b)
    return np.where(bad, 0x7F, b | (np.signbit(x) << 7)).astype(np.uint8)


def scale_exp(amax: float) -> int:
    """Smallest k in [-120, 120] with amax <= 448 * 2^k."""
    k = -120
    while k < 120 and amax > 448.0 * 2.0 ** k:
        k += 1
    return k


def append(cache, scales, table, lens, rows, cu):
    """In place on uint8 cache [P, H, page, D] and scales [P, H, page / block]."""
    P, H, page, D = cache.shape
    block = page // scales.shape[2]
    for s, held in enumerate(lens):
        at, end = int(held), int(held + cu[s + 1] - cu[s])
        while at < end:
            stop = min(end, (at // block + 1) * block)
            pg, a = table[s][at // page], at % page
            b, begin = a + stop - at, a // block * block
            for h in range(H):
                x = rows[cu[s] + at - held: cu[s] + stop - held, h].astype(np.float64)
                fin = np.abs(x[np.isfinite(x)])
                new = 2.0 ** scale_exp(fin.max() if fin.size else 0.0)
                old = float(scales[pg, h, a // block])
                if a > begin:
                    if old >= new:
                        new = old
                    else:
                        cache[pg, h, begin:a] = quantise(TABLE[cache[pg, h, begin:a]] * (old / new))
                scales[pg, h, a // block] = new
                cache[pg, h, a:b] = quantise(x / new)
            at = stop


def attend(q, cache, scales, table, lens, cu, kv_heads, sm_scale, shared, visible=None):
    """fp64 out, lse, and what a tolerance needs: sum p |v| and the largest
    sum of magnitudes of a logit."""
    T, H, D = q.shape
    P, _, page, _ = cache.shape
    block = page // scales.shape[2]
    G = H // kv_heads
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    mass = np.zeros((T, H, D))
    dz = np.zeros((T, H))
    for s in range(len(lens)):
        for t in range(cu[s], cu[s + 1]):
            n = int(lens[s]) if visible is None else min(int(lens[s]), int(visible[t]))
            n = max(n, 0)
            j = [i for i in range(n) if 0 <= table[s][i // page] < P]
            if not j:
                continue
            pg = np.array([table[s][i // page] for i in j])
            slot = np.array([i % page for i in j])
            for h in range(kv_heads):
                vh = h if shared else kv_heads + h
                k = TABLE[cache[pg, h, slot]] * scales[pg, h, slot // block][:, None]
                v = TABLE[cache[pg, vh, slot]] * scales[pg, vh, slot // block][:, None]
                for g in range(h * G, (h + 1) * G):
                    qq = q[t, g].astype(np.float64)
                    with np.errstate(all="ignore"):
                        z = (k @ qq) * sm_scale
                        top = z.max()
                        if np.isnan(z).any():
                            out[t, g], lse[t, g] = np.nan, np.nan
                            continue
                        if top == -np.inf:
                            continue
                        p = np.exp(z - top)
                        w = p / p.sum()
                        out[t, g] = w @ v
                        mass[t, g] = w @ np.abs(v)
                        lse[t, g] = top + np.log(p.sum())
                        dz[t, g] = (np.abs(k) @ np.abs(qq)).max() * abs(sm_scale)
    return out, lse, mass, dz


def attend_tolerance(out, lse, mass, dz, D, rows, eps):
    """Elementwise bounds for (out, lse).

    A logit: D products, exact in fp32 (8 or 11 bits of q times 4 bits of the
    row), summed in fp32 in any order, each addition off by at most one unit in
    the last place (tensor cores may truncate, 2^-23) of the sum of magnitudes
    dz; two scalings and the exponential's argument add 4 roundings: e_z =
    (D + 8) 2^-23 dz.
    A weight: relative 2 e_z (its own and the sum's), the exponential 2^-22, a
    16-bit rounding of at most half a step of fp16, 2^-12.
    The sum over the rows, in fp32 in any order with rescalings: (rows + 64) 2^-23
    of the sum of magnitudes, `mass`. One rounding to the output's type, eps / 2.
    """
    ez = (D + 8) * 2.0 ** -23 * dz
    rel = 2 * np.expm1(np.minimum(ez, 1.0)) + 2.0 ** -22 + 2.0 ** -12 + (rows + 64) * 2.0 ** -23
    bound = mass * rel[..., None]
    tiny = 2.0 ** -25  # half a step of fp16's subnormals (bf16's are far smaller)
    with np.errstate(invalid="ignore"):
        tol_out = bound + eps / 2 * (np.abs(out) + bound) + tiny
        tol_lse = ez + (rows + 64) * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(lse)
    return tol_out, tol_lse


def rope(x, freqs, positions, offset, layout, amplitude, transpose):
    """fp64 turn of [T, H, D], and amplitude (|a| + |b|) of each element's pair."""
    y = x.astype(np.float64).copy()
    mag = np.zeros_like(y)
    n = 2 * len(freqs)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs)[None]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1 if transpose else 1)
    if layout == "half":
        ia = offset + np.arange(n // 2)
        ib = ia + n // 2
    else:
        ia = offset + 2 * np.arange(n // 2)
        ib = ia + 1
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = amplitude * (a * c - b * s)
    y[..., ib] = amplitude * (b * c + a * s)
    mag[..., ia] = mag[..., ib] = abs(amplitude) * (np.abs(a) + np.abs(b))
    return y, mag


# ------------------------------------------------------------- page handling


class Pages:
    """Page tables as lists; the contents of a page are an opaque number."""

    def __init__(self, pages, seqs, width, page):
        self.refs = [0] * pages
        self.table = [[-1] * width for _ in range(seqs)]
        self.lens = [0] * seqs
        self.page = page
        self.width = width
        self.data = list(range(pages))
        self.status = 0

    def fork(self, parents, children):
        n, bits = len(self.lens), 0
        for p, c in zip(parents, children):
            if not (0 <= p < n and 0 <= c < n):
                bits |= 1
                continue
            if self.lens[c] > 0 or self.table[c][0] >= 0:
                bits |= 4
        if len(set(children)) < len(children) or set(children) & set(parents):
            bits |= 2
        if bits:
            self.status |= bits
            return
        for p, c in zip(parents, children):
            held = -(-self.lens[p] // self.page)
            self.table[c] = [self.table[p][e] if e < held else -1 for e in range(self.width)]
            self.lens[c] = self.lens[p]
            for e in range(held):
                self.refs[self.table[c][e]] += 1

    def reserve(self, seqs, rows):
        n, bits = len(self.lens), 0
        for s, r in zip(seqs, rows):
            if not 0 <= s < n:
                bits |= 1
            elif r > 0 and self.lens[s] + r > self.width * self.page:
                bits |= 16
        if len(set(seqs)) < len(seqs):
            bits |= 2
        if bits:
            self.status |= bits
            return
        refs, table, data = list(self.refs), [list(t) for t in self.table], list(self.data)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        for s, r in zip(seqs, rows):
            if r <= 0:
                continue
            for e in range(self.lens[s] // self.page, -(-(self.lens[s] + r) // self.page)):
                old = table[s][e]
                if old >= 0 and refs[old] <= 1:
                    continue
                if not free:
                    self.status |= 8
                    return
                new = free.pop(0)
                table[s][e] = new
                refs[new] = 1
                if old >= 0:
                    refs[old] -= 1
                    if e * self.page < self.lens[s]:
                        data[new] = self.data[old]
        self.refs, self.table, self.data = refs, table, data

    def free(self, seqs):
        for s in dict.fromkeys(seqs):
            if 0 <= s < len(self.lens):
                for p in self.table[s]:
                    if p >= 0:
                        self.refs[p] -= 1
                self.table[s] = [-1] * self.width
                self.lens[s] = 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for m, h in to.items():
            self.refs[h], self.refs[m] = self.refs[m], 0
            self.data[h] = self.data[m]
        self.table = [[to.get(p, p) for p in t] for t in self.table]
        return live
