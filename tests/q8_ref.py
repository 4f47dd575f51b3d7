"""Plain fp64 restatement of the rotary paged appends and the 8-bit cache, for tests.

Written from the formulas in include/loki.h with NumPy, one sequence, head and
block at a time; nothing here comes from the package.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(x):
    """Nearest e4m3 value (ties to even), saturating at 448; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.where(np.isnan(x), np.nan, np.copysign(np.minimum(np.rint(a / step) * step, E4M3_MAX), x))


def pow2_scale(amax):
    if amax <= 0:
        return 2.0 ** -126
    m, x = math.frexp(amax)  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    return 2.0 ** max(-126, x - 9 + (1 if m > 0.875 else 0))


def rope(x, pos, table, interleaved):
    """Rows x [..., n, D] (fp64) at integer positions pos [n]; table [n_pos, r] holds cos | sin."""
    if table is None:
        return np.array(x, dtype=np.float64)
    t = np.asarray(table, dtype=np.float64)[np.asarray(pos)]
    half = t.shape[1] // 2
    c, s = t[:, :half], t[:, half:]
    y = np.array(x, dtype=np.float64)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = np.asarray(x, np.float64)[..., ia], np.asarray(x, np.float64)[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def append_block(codes, scale, rows, first_slot):
    """One scale block: codes [block, D] (values of the codes), its scale, new rows at first_slot.
    Returns (codes, scale, exact values / scale of the new rows)."""
    a = np.abs(rows)
    a = a[np.isfinite(a)]
    grown = pow2_scale(float(a.max()) if a.size else 0.0)
    codes = codes.copy()
    s = grown
    if first_slot > 0:
        s = max(scale, grown)
        if s > scale:
            codes[:first_slot] = e4m3_round(codes[:first_slot] * (scale / s))
    codes[first_slot:first_slot + len(rows)] = e4m3_round(rows / s)
    return codes, s


def attend(q, K, V, scale):
    """Softmax attention of one query over rows K, V (fp64); zeros without rows."""
    if len(K) == 0:
        return np.zeros(V.shape[1])
    a = scale * (K @ q)
    p = np.exp(a - a.max())
    return (p / p.sum()) @ V


def attend_tol(q, K, V, scale, ref, half_step):
    """How far an fp32 computation of attend() may be off.

    Scores: the products' sum of D terms in fp32 is off by at most (D + 8)
    2^-24 sum|q k|, a query carried in 22 bits relative to its largest entry
    adds 2^-22 max|q| sum|k|, and the base-2 exponent rounds once, |a| 2^-22.
    A score off by E changes its weight by a factor e^E, so the output (a
    weighted mean) by at most 2 E max|v|. Weights carried in 21 bits, and the
    sums of n terms: (2^-20 + (n + 16) 2^-24) max|v|. Then one rounding of the
    output: half_step |ref|.
    """
    if len(K) == 0:
        return np.zeros_like(ref)
    D = K.shape[1]
    ab, aq = np.abs(K), np.abs(q)
    E = scale * ((D + 8) * 2.0 ** -24 * (ab @ aq) + 2.0 ** -22 * aq.max() * ab.sum(1)).max()
    E += np.abs(scale * (K @ q)).max() * 2.0 ** -22
    vmax = np.abs(V).max()
    return (2 * E + 2.0 ** -20 + (len(K) + 16) * 2.0 ** -24) * vmax + half_step * np.abs(ref)
