"""fp64 CPU oracle of the 8-bit products: rows quantised per 128 elements, and
products of quantised rows with quantised matrices, by group of rows.

TEST INFRASTRUCTURE, as the attention's oracle: only tests may import it, and
it shares no code with the library. Straight from the definitions in the C
header.
"""

from __future__ import annotations

import numpy as np

GROUP = 128


def turn(y, cos, sin, offset, interleaved, inverse):
    """Head rows y [n, heads, dim] fp64 with the elements from `offset` on turned
    by cos / sin [n, rope_dim / 2] (back by them with `inverse`)."""
    y = np.array(y, dtype=np.float64)
    half = cos.shape[1]
    sign = -1.0 if inverse else 1.0
    for i in range(half):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
        c, s = cos[:, None, i], sign * sin[:, None, i]
        ya, yb = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = ya * c - yb * s, yb * c + ya * s
    return y


def silu(g):
    g = np.asarray(g, dtype=np.float64)
    return g / (1.0 + np.exp(-g))


def e4m3(q):
    """The e4m3 values nearest to q, ties to the even code, saturating: 4
    significant bits, none finer than 2^-9, at most 448."""
    q = np.asarray(q, dtype=np.float64)
    m, e = np.frexp(q)
    unit = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.clip(np.round(q / unit) * unit, -448.0, 448.0)


def quantize(y, pow2):
    """Rows y [n, K] fp64 -> (values of the codes [n, K], scales fp64 [n, ceil(K
    / 128)]); NaN for a group with an element that is not finite."""
    n, k = y.shape
    groups = -(-k // GROUP)
    codes, scales = np.empty((n, k)), np.empty((n, groups))
    for g in range(groups):
        part = y[:, GROUP * g:GROUP * (g + 1)]
        bad = ~np.isfinite(part).all(axis=1)
        part = np.where(bad[:, None], 0.0, part)
        top = np.abs(part).max(axis=1)
        if pow2:
            m, e = np.frexp(top / 448.0)
            e = np.where(top > 0, e - (m == 0.5), -100)
            scale = np.ldexp(1.0, np.clip(e, -100, 100))
            q = part / scale[:, None]
        else:
            top = np.maximum(top, 1e-12)
            scale = top / 448.0
            q = part * 448.0 / top[:, None]
        codes[:, GROUP * g:GROUP * (g + 1)] = np.where(bad[:, None], np.nan, e4m3(q))
        scales[:, g] = np.where(bad, np.nan, scale)
    return codes, scales


def product(a, a_scale, w, w_scale):
    """a [m, K], w [n, K] (values of the codes), a_scale [m, B], w_scale [N / 128,
    B] -> (out [m, n], the sum of the terms' magnitudes)."""
    out, mag = np.zeros((a.shape[0], w.shape[0])), np.zeros((a.shape[0], w.shape[0]))
    rows = np.arange(w.shape[0]) // GROUP
    for b in range(a_scale.shape[1]):
        at = slice(GROUP * b, GROUP * (b + 1))
        s = a_scale[:, b:b + 1].astype(np.float64) * w_scale[rows, b][None].astype(np.float64)
        out += s * (a[:, at] @ w[:, at].T)
        mag += np.abs(s) * (np.abs(a[:, at]) @ np.abs(w[:, at]).T)
    return out, mag


def grouped(a, a_scale, w, w_scale, cu, out):
    """product() of each group's rows into a copy of `out`; rows outside all
    groups stay."""
    out, mag = np.array(out, dtype=np.float64), np.zeros(out.shape)
    for g in range(len(w)):
        at = slice(int(cu[g]), int(cu[g + 1]))
        if at.stop > at.start:
            out[at], mag[at] = product(a[at], a_scale[at], w[g], w_scale[g])
    return out, mag
