"""Inputs, bounds and checks shared by the GPU tests of the norms, gated residuals and
8-bit checkpoints.

Bounds.  Every result is compared with the float64 oracle element by element against

    half a step of the stored type times |reference|  +  K * u * A,   u = 2^-24,

where A is the same formula with every term replaced by its magnitude (differences become
sums, so a cancelling row has a large A), K covers the longest chain of fp32 roundings: a
row of 8,192 channels is summed as at most 64 terms per thread, then at most 5 shuffles
and 32 warps, about 100 roundings, and rsqrtf is off by 2 ulp; K = 256 per norm (512 where
two norms follow one another) doubles that.  A sum over R rows adds R further roundings.
Half a step is eps / 2 of the type: 2^-8 for bf16, 2^-24 for fp32.
"""
from __future__ import annotations

import numpy as np
import torch

import block_sparse_video_ssta_b200 as S
import oracle

U = 2.0 ** -24
K = 256.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    """Seeded inputs of one configuration, on the GPU and as float64 arrays of the same values."""

    def __init__(self, rows, C, dtype="bf16", param_dtype="f32", norm="layer", post="none", vectors=True, mod_rows=0,
                 res_scale=1.0, eps=1e-6, stride=6, seed=0, offset=0.5):
        self.rows, self.C, self.dtype, self.norm, self.post = rows, C, dtype, norm, post
        self.mod_rows, self.res_scale, self.eps = mod_rows, res_scale, eps
        gen = torch.Generator().manual_seed(seed * 7919 + rows * 31 + C)
        n = lambda *s: torch.randn(s, generator=gen)
        dt, pt = DT[dtype], DT[param_dtype]
        G = -(-rows // min(mod_rows or rows, rows))
        self.G = G
        act = lambda o=0.0: (n(rows, C) * torch.exp(0.5 * n(C)) + o).to(dt).cuda()
        self.x, self.y, self.dr, self.dn = act(offset), act(), act(), act()
        self.weight = self.post_weight = self.scale = self.shift = self.gate = None
        if vectors:
            if norm != "none":
                self.weight = (1 + 0.3 * n(C)).to(pt).cuda()
                mod = (0.5 * n(G, stride * C)).to(pt).cuda()
                self.scale, self.shift = mod[:, :C], mod[:, (stride - 1) * C:]
            self.gate = (0.5 * n(G, stride * C)).to(pt).cuda()[:, C:2 * C] if stride > 1 else (0.5 * n(G, C)).to(pt).cuda()
            if post != "none":
                self.post_weight = (1 + 0.3 * n(C)).to(pt).cuda()
        self.desc = S.norm_desc(rows, C, dtype, param_dtype, norm, post, eps, res_scale, mod_rows, stride * C)
        self.half = torch.finfo(dt).eps / 2

    def np(self, name):
        return f64(getattr(self, name))


def check(name, got, want, tol):
    a = f64(got).reshape(want.shape)
    assert np.isfinite(a).all(), f"{name}: not finite"
    err = np.abs(a - want)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{name}: off by {err[worst]:.3e} at {worst}, bound {np.broadcast_to(tol, err.shape)[worst]:.3e}"


def _rows(v, case):
    m = min(case.mod_rows or case.rows, case.rows)
    return None if v is None else np.abs(v)[np.arange(case.rows) // m]


def _col(v):
    return v[:, None]


def normal_magnitude(x, mean, rstd):
    """Magnitude of (x - mean) * rstd with its statistics' own errors: each term counted as added, and once more
    times the value for the deviation."""
    m = np.zeros(len(x)) if mean is None else np.abs(mean) + np.abs(x).mean(axis=1)
    X = (np.abs(x) + _col(m)) * _col(rstd)
    xh = np.abs(x if mean is None else x - _col(mean)) * _col(rstd)
    return X + xh * (1 + (X * xh).mean(axis=1, keepdims=True))


def modulated_magnitude(X, case, weight, scale, shift):
    w = 1.0 if weight is None else np.abs(weight)
    s = 0.0 if scale is None else _rows(scale, case)
    return X * w * (1 + s) + (0.0 if shift is None else _rows(shift, case))


def grad_magnitude(g, X, rstd):
    return _col(rstd) * (g + g.mean(axis=1, keepdims=True) + X * (g * X).mean(axis=1, keepdims=True))


def stat_bounds(x, mean, rstd):
    """(bound of mean, bound of rstd)."""
    m = K * U * np.abs(x).mean(axis=1)
    shift = np.abs(x).mean(axis=1) * rstd if mean is not None else 0.0
    return m, K * U * rstd * (1 + shift)
