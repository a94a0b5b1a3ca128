"""CPU oracle for the norms, gated residuals and 8-bit checkpoints around the attention,
and for the attention's backward from saved tensors.

TEST INFRASTRUCTURE ONLY, like ssta_oracle: plain float64 numpy, every formula written
out, no code shared with the CUDA library.  ``kind`` is "none", "layer" or "rms"; a
modulation [G, C] has one row per ``mod_rows`` rows (0: one row for all).
"""
from __future__ import annotations

import math

import numpy as np

from .ssta_oracle import geometry, valid_token_mask

__all__ = ["norm_stats", "norm_fwd", "norm_bwd", "residual_norm_fwd", "residual_norm_bwd", "checkpoint_encode",
           "checkpoint_decode", "attention_bwd_saved"]

GROUP = 128


def norm_stats(x, kind, eps):
    """(mean or None, 1 / deviation) of each row of x [R, C]."""
    mean = x.mean(axis=1) if kind == "layer" else None
    d = x if mean is None else x - mean[:, None]
    return mean, 1.0 / np.sqrt((d * d).mean(axis=1) + eps)


def _normalise(x, mean, rstd):
    return (x if mean is None else x - mean[:, None]) * rstd[:, None]


def _rows_of(v, rows, mod_rows):
    """A modulation [G, C] spread over the rows (1-row axis kept out of the way: None stays None)."""
    if v is None:
        return None
    m = min(mod_rows or rows, rows)
    return v[np.arange(rows) // m]


def _sum_groups(t, mod_rows):
    rows = t.shape[0]
    m = min(mod_rows or rows, rows)
    return np.stack([t[i:i + m].sum(axis=0) for i in range(0, rows, m)])


def norm_fwd(x, kind, eps, weight=None, scale=None, shift=None, mod_rows=0):
    """(y, mean, rstd): y = norm(x) * weight * (1 + scale) + shift."""
    mean, rstd = norm_stats(x, kind, eps)
    y = _normalise(x, mean, rstd)
    if weight is not None:
        y = y * weight
    if scale is not None:
        y = y * (1.0 + _rows_of(scale, len(x), mod_rows))
    if shift is not None:
        y = y + _rows_of(shift, len(x), mod_rows)
    return y, mean, rstd


def _through_norm(xh, g, rstd, kind):
    out = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        out = out - g.mean(axis=1, keepdims=True)
    return out * rstd[:, None]


def norm_bwd(dy, x, mean, rstd, kind, weight=None, scale=None, dres=None, mod_rows=0):
    """(dx, dweight, dscale, dshift) with the statistics the forward saved; an absent weight counts as 1, an
    absent scale as 0."""
    rows, C = x.shape
    w = np.ones(C) if weight is None else weight
    s = np.zeros((rows, C)) if scale is None else _rows_of(scale, rows, mod_rows)
    xh = _normalise(x, mean, rstd)
    dx = _through_norm(xh, dy * w * (1.0 + s), rstd, kind)
    if dres is not None:
        dx = dx + dres
    dweight = (dy * (1.0 + s) * xh).sum(axis=0)
    return dx, dweight, _sum_groups(dy * xh * w, mod_rows), _sum_groups(dy, mod_rows)


def residual_norm_fwd(x, y, kind, post_kind, eps, res_scale=1.0, post_weight=None, gate=None, weight=None, scale=None,
                      shift=None, mod_rows=0):
    """dict of r = res_scale * x + gate * post_norm(y) * post_weight, n = norm(r) modulated, and the statistics."""
    h, pm, pr = (y, None, None) if post_kind == "none" else norm_fwd(y, post_kind, eps, post_weight)
    r = res_scale * x + (h if gate is None else _rows_of(gate, len(x), mod_rows) * h)
    n = m = rs = None
    if kind != "none":
        n, m, rs = norm_fwd(r, kind, eps, weight, scale, shift, mod_rows)
    return dict(r=r, n=n, post_mean=pm, post_rstd=pr, mean=m, rstd=rs)


def residual_norm_bwd(dr, dn, r, y, mean, rstd, post_mean, post_rstd, kind, post_kind, res_scale=1.0,
                      post_weight=None, gate=None, weight=None, scale=None, mod_rows=0):
    """dict of dx, dy and the vectors' gradients; dr or dn may be None, y may be None without a post norm."""
    some = dr if dr is not None else dn
    rows, C = some.shape
    out = dict(dweight=None, dscale=None, dshift=None, dpost_weight=None, dgate=None)
    dR = np.zeros((rows, C)) if dr is None else dr
    if dn is not None:
        dR, out["dweight"], out["dscale"], out["dshift"] = norm_bwd(dn, r, mean, rstd, kind, weight, scale, dR, mod_rows)
    out["dx"] = res_scale * dR
    pw = np.ones(C) if post_weight is None else post_weight
    g = np.ones((rows, C)) if gate is None else _rows_of(gate, rows, mod_rows)
    dh = dR * g * pw
    if y is not None:
        yh = y if post_kind == "none" else _normalise(y, post_mean, post_rstd)
        out["dgate"] = _sum_groups(dR * yh * pw, mod_rows)
        out["dpost_weight"] = (dR * g * yh).sum(axis=0)
    out["dy"] = dh if post_kind == "none" else _through_norm(yh, dh, post_rstd, post_kind)
    return out


# The magnitudes an e4m3 code can hold: three fraction bits, exponents -6 .. 8, subnormals below, no 480.
_E4M3 = np.array(sorted({m * 2.0 ** -9 for m in range(8)}
                        | {(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)} - {480.0}))


def _nearest_e4m3(u):
    """Nearest magnitude of the table with the sign of u; a tie goes to the even position (the even fraction)."""
    a = np.abs(u)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, len(_E4M3) - 1)
    lo = hi - 1
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(_E4M3[pick], u)


def checkpoint_encode(x, fmt):
    """(codes as the numbers they stand for before scaling [R, C], exponent bytes [R, ceil(C / 128)]) of float64
    x [R, C].  A group's exponent E is the smallest in 1 .. 254 for which its largest magnitude times 2^(127 - E)
    stays below 127.5 (int8) or within 448 (e4m3); 255, and codes 0, for a group with an infinity, a NaN or a
    magnitude whose nearest value would be 2^128."""
    R, C = x.shape
    codes = np.zeros((R, C))
    exps = np.zeros((R, -(-C // GROUP)), dtype=np.uint8)
    for i in range(R):
        for j in range(exps.shape[1]):
            v = x[i, j * GROUP:(j + 1) * GROUP]
            if not np.isfinite(v).all():
                exps[i, j] = 255
                continue
            a = np.abs(v).max()
            E = 1 if a == 0 else max(1, math.frexp(a)[1] + 127 - 10)     # at or below the smallest that fits
            while not (a * 2.0 ** (127 - E) < 127.5 if fmt == "int8" else a * 2.0 ** (127 - E) <= 448.0):
                E += 1
            u = v * 2.0 ** (127 - E)
            u = np.rint(u) if fmt == "int8" else _nearest_e4m3(u)
            if np.abs(u).max() * 2.0 ** (E - 127) >= 2.0 ** 128:
                exps[i, j] = 255
                continue
            exps[i, j] = E
            codes[i, j * GROUP:(j + 1) * GROUP] = u
    return codes, exps


def checkpoint_decode(codes, exps):
    """Values [R, C] of checkpoint_encode's result."""
    scale = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127.0))
    return codes * np.repeat(scale, GROUP, axis=1)[:, :codes.shape[1]]


def attention_bwd_saved(d, qp, kp, vp, op, lse, dOp, kept, scale=None):
    """Gradients of Step 4's attention from what a forward saved: P = exp(q k^T * scale - lse) over the valid keys of
    the kept tiles, D = rowsum(dO * O), dS = P * (dO v^T - D).  Returns (dQ, dK, dV) [B,H,Lq,D]."""
    g = geometry(d)
    scale = 1.0 / math.sqrt(g.D) if not scale else scale
    valid = valid_token_mask(d)
    dQ, dK, dV = (np.zeros(qp.shape) for _ in range(3))
    for b, h, i in np.ndindex(kept.shape[:3]):
        rows = np.arange(i * g.N, min((i + 1) * g.N, g.Lq))
        rows = rows[valid[rows]]
        keys = np.concatenate([np.arange(j * g.N, min((j + 1) * g.N, g.Lq)) for j in np.nonzero(kept[b, h, i])[0]]
                              or [np.zeros(0, dtype=np.int64)])
        keys = keys[valid[keys]]
        if rows.size == 0 or keys.size == 0:
            continue
        q, k, v, do = qp[b, h, rows], kp[b, h, keys], vp[b, h, keys], dOp[b, h, rows]
        p = np.exp(q @ k.T * scale - lse[b, h, rows][:, None])
        ds = p * (do @ v.T - (do * op[b, h, rows]).sum(axis=1, keepdims=True))
        dQ[b, h, rows] = scale * ds @ k
        dK[b, h, keys] += scale * ds.T @ q
        dV[b, h, keys] += p.T @ do
    return dQ, dK, dV
