"""The draws' definitions (``include/tn_sampling.h``) with exact comparisons, on the CPU.

Weights are computed in 64 bits and taken as whole numbers of 2^-1074, so sums
and comparisons with u and top_p times a sum are exact; only the exponentials are
rounded (2^-52)."""
import math
from fractions import Fraction

import numpy as np


def _whole(x):
    """A float as a whole number of 2^-1074."""
    n, d = float(x).as_integer_ratio()
    return n * ((1 << 1074) // d)


def _order(row):
    if np.iscomplexobj(row):
        re, im = row.real.astype(np.float32), row.imag.astype(np.float32)
        return re * re + im * im
    return row.astype(np.float32)


def left(row, mask, scale, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Entries left: {index: (weight, log weight)} in ascending order, or a string for a row
    that has none."""
    v = _order(row)
    amplitudes = np.iscomplexobj(row)
    here = np.ones(len(v), bool) if mask is None else np.asarray(mask, bool)
    here = here & (v != (0 if amplitudes else -np.inf))
    if not here.any():
        return "empty"
    if np.isnan(v[here]).any() or np.isposinf(v[here]).any():
        return "undefined"
    at = np.flatnonzero(here)
    at = at[np.lexsort((at, -v[at].astype(np.float64)))]        # largest first, then lowest index
    t = np.float32(temperature)
    if t == 0 or top_k == 1:
        return {int(at[0]): (1, 0.0)}
    beta = float(np.float32(scale) / t)
    m = float(v[at[0]])
    logw = [(beta * (math.log(float(x)) - math.log(m)) if amplitudes else beta * (float(x) - m)) for x in v[at]]
    if amplitudes and beta == 1.0:
        w = [_whole(x) for x in v[at]]
    else:
        w = [_whole(math.exp(x)) for x in logw]
    n = len(at) if top_k <= 0 else min(top_k, len(at))
    if np.float32(top_p) < 1:
        p, s, n2 = Fraction(float(np.float32(top_p))), 0, 0
        need = p.numerator * sum(w[:n])
        while n2 == 0 or s * p.denominator < need:
            s += w[n2]
            n2 += 1
        n = n2
    least = Fraction(float(np.float32(min_p)))
    keep = [i for i in range(n) if w[i] * least.denominator >= least.numerator * w[0]]
    return {int(at[i]): (w[i], logw[i]) for i in sorted(keep, key=lambda i: at[i])}


def draw(entries, u):
    """(id, log p) of a draw."""
    if entries == "empty":
        return -1, -math.inf
    if entries == "undefined":
        return -1, math.nan
    total, f, s = sum(w for w, _ in entries.values()), Fraction(float(u)), 0
    aim = f.numerator * total
    for e, (w, logw) in entries.items():
        s += w
        # an entry whose 64-bit weight is 0 is passed over but where u is 0
        if s * f.denominator > aim or u == 0:
            big = max(l for _, l in entries.values())
            z = math.fsum(math.exp(l - big) for _, l in entries.values())
            return e, logw - big - math.log(z)
    raise AssertionError("u >= 1")
