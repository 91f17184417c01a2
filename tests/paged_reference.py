"""Plain fp64 attention over packed rows, and how far an fp16-operand kernel
may be from it (test helper; shares no code with the library)."""
import math

import numpy as np

from oracle import tq_oracle as o
from tests.layout import unpack_codes, unpack_signs

H = 2.0 ** -11   # fp16 rounding, relative to the value
HS = 2.0 ** -25  # fp16 rounding below 2^-14, absolute
F = 2.0 ** -23   # an fp32 add that may truncate

OUT = {"bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25)}


def unpack(rows, t):
    """Packed rows (codes, signs, norms as numpy arrays) as the oracle's dict."""
    codes, signs, norms = rows
    e = {"codes": unpack_codes(codes, t.d, t.w), "norm": norms[:, 0].astype(np.float64),
         "gamma": norms[:, 1].astype(np.float64)}
    if t.m:
        e["bits"] = unpack_signs(signs, t.m)
    return e


def attend(y, limits, scale, ke, tk, ve, tv, dtype, many=False):
    """y: rows x d; row i sees the first limits[i] keys.  Returns the exact
    output and, per coordinate, the most that fp16 operands (rotated query and
    its projection, centroids, weights; each rounded once) with fp32 sums and
    one rounding of the output can be off.  many: of the kernel of many rows,
    whose keys' and values' operands are centroids times norms, absolute below
    2^-14 of the largest norm (at most twice that), whose residual norms are
    fp16 operands too, whose projections share the query's scale, and some of
    whose exponentials are polynomials (2^-18.4)."""
    d, n = tk.d, len(ke["norm"])
    yt, p = o.prepare_query(y, tk)
    x = scale * o.score(yt, p, ke, tk)
    c = np.abs(tk.centroids[ke["codes"]])
    # a logit's error: each product has two rounded factors; the query's is
    # absolute where it is below 2^-14 of the row's largest (at most twice that)
    top = np.abs(yt).max(1, initial=0.0)[:, None]
    terms = np.abs(yt) @ c.T
    err = terms * (2 * H + H * H) + 2 * top * HS * c.sum(1)[None]
    size = terms
    if tk.m:
        g = ke["gamma"][None] * math.sqrt(math.pi / 2) / tk.m
        ap = np.abs(p)
        # p itself comes from the query as two fp16 terms and fp32 sums
        perr = (np.abs(yt) @ np.abs(tk.S).T) * (H * H + (d / 16 + 2) * F)
        err += g * (ap.sum(1) * H + perr.sum(1) + 2 * ap.max(1, initial=0.0) * HS * d)[:, None]
        if many:
            err += (g * H + HS / 64) * (ap.sum(1) * (1 + H) + perr.sum(1))[:, None] + g * (128 * top * HS * d)
        size = size + g * ap.sum(1)[:, None]
    if many:
        kmost = 2 * ke["norm"].max(initial=0.0) / np.maximum(ke["norm"], 1e-30)[None]
        err += kmost * HS * (np.abs(yt).sum(1) + (ap.sum(1) / 64 if tk.m else 0.0))[:, None]
    # fp32: the rotation's 21 adds, the MMA's sums, the scaling
    err = (err + size * (d / 8 + 24) * F) * abs(scale) * ke["norm"][None] + np.abs(x) * 4 * F + 2.0 ** -21
    see = np.arange(n)[None] < np.asarray(limits)[:, None]
    x = np.where(see, x, -np.inf)
    m = x.max(1, initial=-np.inf, keepdims=True)
    w = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    total = w.sum(1, keepdims=True)
    w = w / np.where(total > 0, total, 1.0)
    eps = np.where(see, np.expm1(err) + (2.0 ** -18.4 if many else 0.0), 0.0)
    mean = (w * eps).sum(1, keepdims=True)
    rel = (1 + eps) / np.maximum(1 - mean, 0.1) - 1 + 2 * H + H * H + (n / 16 + 40) * F
    cv = tv.centroids[ve["codes"]]
    out = ((w * ve["norm"][None]) @ cv) @ tv.R
    vn = ve["norm"][None] * np.ones((len(x), 1))
    vtop = 2 * np.where(see, vn, 0.0).max(1, initial=0.0)[:, None]
    # a weight below 2^-14 of the scale is rounded absolutely; the largest weight is 1 before division by the sum
    small = np.where(see, vtop * HS, 0.0) / np.maximum(total, 1.0)
    e = (w * vn * rel + small) @ np.abs(cv)
    if many:
        e += vtop * HS
    bound = e @ np.abs(tv.R)
    r, a = OUT[dtype]
    return out, bound + (np.abs(out) + bound) * r + a
