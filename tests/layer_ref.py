"""Plain 64-bit implementations of the norms with the rotation and of causal
attention over packed sequences, with their gradients, for the tests. They share
no code with the package."""
from __future__ import annotations

import math

import numpy as np

import cache_ref

U = 2.0 ** -24       # a rounding of fp32
TURN = 2.0 ** -20.9  # of amplitude (|a| + |b|): the turn's own error (test_gpu_rope.py)


def norm_rope(x, w, freqs, positions, eps, **kw):
    """(y, tolerance) of x [T, H, D].

    r: a lane sums at most 32 squares and 5 shuffles follow, the mean and eps add two
    roundings: 40 U of the sum, 20 U of its root; the root and the quotient add 2 ulp, 4 U: 24 U.
    Two more products, then the turn. Columns that are not turned have no pair (mag 0): theirs are
    the norm's roundings, 26 U of the value itself, which in a pair is at most mag."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, mag = cache_ref.rope(x * r * w, freqs, positions, kw.get("offset", 0), kw.get("layout", "interleaved"),
                            kw.get("amplitude", 1.0), False)
    return y, TURN * mag + 26 * U * np.maximum(mag, np.abs(y))


def norm_rope_grad(x, w, g, freqs, positions, eps, **kw):
    """(dx, its tolerance, dw, its tolerance)."""
    T, H, D = x.shape
    h, hmag = cache_ref.rope(g, freqs, positions, kw.get("offset", 0), kw.get("layout", "interleaved"),
                             kw.get("amplitude", 1.0), True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = h * w
    back = r * r * (u * x).mean(-1, keepdims=True)
    dx = r * (u - x * back)
    eu = np.abs(w) * TURN * hmag + 2 * U * np.abs(u)
    # the sum as in norm_rope; two factors r, the mean and the products: 52 U
    eb = r * r * ((eu * np.abs(x)).mean(-1, keepdims=True) + 42 * U * np.abs(u * x).mean(-1, keepdims=True)) + 52 * U * np.abs(back)
    tx = r * (eu + np.abs(x) * eb) + 28 * U * r * (np.abs(u) + np.abs(x * back))
    term = h * x * r
    dw = term.sum((0, 1))
    # at most T H sums one after the other, the CTA's groups and the joining
    tw = (TURN * hmag * np.abs(x * r)).sum((0, 1)) + (T * H + 100) * U * np.abs(term).sum((0, 1))
    return dx, tx, dw, tw


def rounded(want, tol, eps, tiny=0.0):
    """The tolerance after one rounding to a type: half a step, and half a step of its subnormals."""
    return tol + eps / 2 * (np.abs(want) + tol) + tiny


def seen(nq, nk, window):
    """[nq, nk] bool: which keys each query of a sequence sees."""
    last = nk - nq + np.arange(nq)[:, None]
    col = np.arange(nk)[None]
    ok = col <= last
    if window:
        ok &= col > last - window
    return ok


def prompt(q, k, v, cu_q, cu_k, scale, window=None):
    """(out, lse, per (sequence, head) list of (z masked, p)); rows of no sequence: 0 and -inf."""
    T, H, D = q.shape
    group = H // k.shape[1]
    out, lse, parts = np.zeros((T, H, v.shape[2])), np.full((T, H), -math.inf), []
    for s in range(len(cu_q) - 1):
        a, b, e, f = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        ok = seen(b - a, f - e, window)
        for h in range(H):
            p = np.zeros(ok.shape)
            if b > a:
                with np.errstate(all="ignore"):
                    z = np.where(ok, q[a:b, h] @ k[e:f, h // group].T * scale, -math.inf)
                top = z.max(-1, keepdims=True) if f > e else np.full((b - a, 1), -math.inf)
                safe = np.where(np.isfinite(top), top, 0.0)
                p = np.exp(z - safe)
                total = p.sum(-1, keepdims=True)
                with np.errstate(all="ignore"):
                    lse[a:b, h] = (np.log(total) + safe)[:, 0]
                p = np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)
                # rows that a query does not see take no part, whatever they hold
                out[a:b, h] = p @ np.where(np.isfinite(v[e:f, h // group]), v[e:f, h // group], 0.0)
            parts.append(p)
    return out, lse, parts


def prompt_grad(q, k, v, cu_q, cu_k, scale, parts, out, g, glse=None):
    """(dq, dk, dv) and the sums of magnitudes that their errors scale with."""
    T, H, D = q.shape
    group = H // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    mq, mk, mv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for s in range(len(cu_q) - 1):
        a, b, e, f = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        for h in range(H):
            p = parts[s * H + h]
            if b == a or f == e:
                continue
            x, y, w, d = q[a:b, h], k[e:f, h // group], v[e:f, h // group], g[a:b, h]
            delta = (d * out[a:b, h]).sum(-1, keepdims=True)
            if glse is not None:
                delta = delta - glse[a:b, h][:, None]
            ds = p * (d @ w.T - delta)
            # what dS's rounding, and that of its parts, scales with
            ms = np.abs(ds)
            dq[a:b, h] += ds @ y * scale
            dk[e:f, h // group] += ds.T @ x * scale
            dv[e:f, h // group] += p.T @ d
            mq[a:b, h] += ms @ np.abs(y) * abs(scale)
            mk[e:f, h // group] += ms.T @ np.abs(x) * abs(scale)
            mv[e:f, h // group] += p.T @ np.abs(d)
    return (dq, dk, dv), (mq, mk, mv)
