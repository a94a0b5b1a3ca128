"""Backward of the gated residual in blocks of 512 threads (above 2,048 channels; above 4,096 with
two vectors per thread), with enough rows that every block refills its table of row scalars and
group scales and wraps its stages many times: every element against float64 on the GPU.

Bounds as relative 2-norms.  Rows: half a step of the type for the stored value, and for the
fp32 arithmetic before it 16 u (u = 2^-24) for dx: at most eight roundings in a row (rstd and
mean as they are given; the vectors' product 2, g 1, the normalised value 2, the two
corrections 1, their sums 2), of terms whose 2-norms together are within twice the result's;
32 u for dy, which goes through both norms.  Sums of the vectors' gradients over n rows:
4 u sqrt(n), the square-root growth of rounding in a sum of independent terms."""
import pytest
import torch

import block_sparse_video_ssta_b200 as S
from norm_helpers import U, Case

pytestmark = pytest.mark.gpu

VECTORS = ("post_weight", "gate", "weight", "scale", "shift")
CASES = [("bf16", 8192, None), ("bf16", 8192, "int8"), ("f32", 8192, "e4m3"), ("f32", 6152, None), ("bf16", 4104, "e4m3"),
         ("f32", 4104, "int8"), ("bf16", 4096, "e4m3"), ("f32", 2056, None), ("bf16", 2600, "int8")]


@pytest.mark.parametrize("post", ["rms", "none"])
@pytest.mark.parametrize("dtype,C,saved", CASES)
def test_wide_rows_in_long_runs(cuda_ok, dtype, C, saved, post):
    rows, mod_rows = 15_001, 7_423     # about 150 rows per block, and a last group of 155 in short runs
    c = Case(rows, C, dtype, "f32", "layer", post, True, mod_rows, 0.5, offset=0.1)
    f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift, save_y=saved, save_r=saved)
    r, y = (f.saved_r, f.saved_y) if saved else (f.r, c.y)
    g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, r, y, f.mean, f.rstd, None, f.post_rstd, c.post_weight, c.gate,
                                 c.weight, c.scale)
    value = lambda t: (S.ssta_checkpoint_load(t) if saved else t).double()
    group = torch.arange(rows, device="cuda") // mod_rows
    rows_of = lambda t: t.double().index_select(0, group)
    sums = lambda t: torch.stack([t[i * mod_rows:(i + 1) * mod_rows].sum(0) for i in range(c.G)])
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    w, pw = c.weight.double(), 1.0 if c.post_weight is None else c.post_weight.double()
    rh = (value(r) - f.mean.double()[:, None]) * f.rstd.double()[:, None]
    dn = c.dn.double()
    tol = 4 * U * rows ** 0.5
    want = {"shift": sums(dn), "scale": sums(dn * rh) * w, "weight": (dn * rh * (1 + rows_of(c.scale))).sum(0)}
    gr = dn * w * (1 + rows_of(c.scale))
    dR = c.dr.double() + (gr - gr.mean(1, keepdim=True) - rh * (gr * rh).mean(1, keepdim=True)) * f.rstd.double()[:, None]
    del rh, gr, dn
    assert rel(g.dx, 0.5 * dR) <= c.half + 16 * U
    yh = value(y) if post == "none" else value(y) * f.post_rstd.double()[:, None]
    want["gate"] = sums(dR * yh) * pw
    dh = dR * rows_of(c.gate)
    if post != "none":
        want["post_weight"] = (dh * yh).sum(0)
    dh = dh * pw
    if post != "none":
        dh = (dh - yh * (dh * yh).mean(1, keepdim=True)) * f.post_rstd.double()[:, None]
    assert rel(g.dy, dh) <= c.half + 32 * U
    for n, t in want.items():
        assert rel(getattr(g, "d" + n), t) <= tol, n
