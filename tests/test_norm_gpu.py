"""Norms and gated residuals on the GPU against the float64 oracle (bounds: norm_helpers).
The backward's reference gets the statistics, and the checkpoints' values, that the kernel
is given, so the two compute the same formula on the same numbers."""
import numpy as np
import pytest
import torch

import block_sparse_video_ssta_b200 as S
import oracle
from norm_helpers import (K, U, Case, check, f64, grad_magnitude, modulated_magnitude, normal_magnitude, stat_bounds,
                          _rows)

pytestmark = pytest.mark.gpu

# (rows, C): one row, one vector, every width class of the kernels and its neighbours, partial groups of 128
SIZES = [(1, 8), (1, 2048), (3, 128), (17, 120), (33, 136), (5, 256), (7, 264), (9, 512), (6, 520), (64, 1000), (19, 1024),
         (9, 1032), (70, 2048), (5, 2056), (13, 4096), (3, 4104), (4, 8192), (601, 64)]
# dtype, param_dtype, norm, post, vectors, mod_rows, res_scale
MODES = [("bf16", "f32", "layer", "none", True, 0, 1.0), ("bf16", "bf16", "rms", "rms", True, 2, 0.5),
         ("f32", "f32", "layer", "layer", True, 3, 1.0), ("f32", "bf16", "rms", "none", False, 0, -2.0),
         ("bf16", "f32", "none", "layer", True, 1, 1.0)]
ALL = [s + m for i, s in enumerate(SIZES) for j, m in enumerate(MODES) if i % 3 == j % 3 or i in (1, 9, 12)]


# rows beyond what the kernels for few rows take, in every width class of the others; the widest in fp32
ALL += [s + m for s in [(1300, 512), (650, 520), (650, 768), (650, 776), (650, 1024), (350, 1032), (350, 1536), (350, 2048)]
        for m in MODES[1:4]]
ALL += [s + m for s in [(6, 6144), (5, 4104), (7, 8192)] for m in MODES[2:4]]


def make(rows, C, dtype, param, norm, post, vectors, mod_rows, res_scale, **kw):
    return Case(rows, C, dtype, param, norm, post, vectors, mod_rows, res_scale, **kw)


def check_norm_fwd(c):
    y, mean, rstd, _ = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift)
    x = f64(c.x)
    ry, rm, rr = oracle.norm_fwd(x, c.norm, c.eps, c.np("weight"), c.np("scale"), c.np("shift"), c.mod_rows)
    bm, br = stat_bounds(x, rm, rr)
    if c.norm == "layer":
        check("mean", mean, rm, bm)
    else:
        assert mean is None
    check("rstd", rstd, rr, br)
    A = modulated_magnitude(normal_magnitude(x, rm, rr), c, c.np("weight"), c.np("scale"), c.np("shift"))
    check("y", y, ry, c.half * np.abs(ry) + K * U * A)
    # the same without statistics
    y2, none_m, none_r, _ = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift, stats=False)
    assert none_m is None and none_r is None and torch.equal(y, y2)
    return mean, rstd


def check_norm_bwd(c, mean, rstd, kept, values):
    """kept: what the call is given for x; values: its values."""
    g = S.ssta_norm_bwd(c.desc, c.dn, kept, mean, rstd, c.weight, c.scale, c.dr, want_dshift=True,
                        dweight=torch.empty(c.C, device="cuda"), dscale=torch.empty(c.G, c.C, device="cuda"))
    x, dy, dres = f64(values), f64(c.dn), f64(c.dr)
    m, r, w, s = f64(mean), f64(rstd), c.np("weight"), c.np("scale")
    dx, dw, ds, dt = oracle.norm_bwd(dy, x, m, r, c.norm, w, s, dres, c.mod_rows)
    X = normal_magnitude(x, m, r)
    G = modulated_magnitude(np.abs(dy), c, w, s, None)
    check("dx", g.dx, dx, c.half * np.abs(dx) + K * U * (np.abs(dres) + grad_magnitude(G, X, r)))
    acc = (c.rows + K) * U
    _, aw, as_, at = oracle.norm_bwd(np.abs(dy), X, None, np.ones(c.rows), "rms", None if w is None else np.abs(w),
                                     None if s is None else np.abs(s), None, c.mod_rows)
    check("dweight", g.dweight, dw, acc * aw)
    check("dscale", g.dscale, ds, acc * as_)
    check("dshift", g.dshift, dt, acc * at)
    return g


@pytest.mark.parametrize("cfg", [a for a in ALL if a[4] != "none"], ids=str)
def test_norm_matches_oracle(cuda_ok, cfg):
    c = make(*cfg)
    mean, rstd = check_norm_fwd(c)
    check_norm_bwd(c, mean, rstd, c.x, c.x)
    for fmt in ("int8", "e4m3"):
        ck = S.ssta_checkpoint_save(c.x, fmt)
        check_norm_bwd(c, mean, rstd, ck, S.ssta_checkpoint_load(ck))


def check_residual_fwd(c):
    f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift)
    x, y = f64(c.x), f64(c.y)
    ref = oracle.residual_norm_fwd(x, y, c.norm, c.post, c.eps, c.res_scale, c.np("post_weight"), c.np("gate"),
                                   c.np("weight"), c.np("scale"), c.np("shift"), c.mod_rows)
    H = np.abs(y)
    if c.post != "none":
        bm, br = stat_bounds(y, ref["post_mean"], ref["post_rstd"])
        check("post_rstd", f.post_rstd, ref["post_rstd"], br)
        if c.post == "layer":
            check("post_mean", f.post_mean, ref["post_mean"], bm)
        H = modulated_magnitude(normal_magnitude(y, ref["post_mean"], ref["post_rstd"]), c, c.np("post_weight"), None, None)
    gate = 1.0 if c.gate is None else _rows(c.np("gate"), c)
    R = abs(c.res_scale) * np.abs(x) + gate * H
    check("r", f.r, ref["r"], c.half * np.abs(ref["r"]) + K * U * R)
    if c.norm == "none":
        assert f.n is None and f.mean is None and f.rstd is None
        return f
    # the norm sees r with an error of K u R: X counts R for |r|
    m, r = ref["mean"], ref["rstd"]
    bm, br = stat_bounds(R, m, r)
    check("rstd", f.rstd, r, br * (1 + (R * r[:, None]).max(axis=1)))
    if c.norm == "layer":
        check("mean", f.mean, m, 2 * bm)
    rh = np.abs(ref["r"] - (0 if m is None else m[:, None])) * r[:, None]
    X = normal_magnitude(R, m, r) + (R + R.mean(axis=1, keepdims=True)) * r[:, None] \
        + rh * (R * rh).mean(axis=1, keepdims=True) * r[:, None]
    A = modulated_magnitude(X, c, c.np("weight"), c.np("scale"), c.np("shift"))
    check("n", f.n, ref["n"], c.half * np.abs(ref["n"]) + 2 * K * U * A)
    return f


def check_residual_bwd(c, f, kept_r, kept_y, r_values, y_values, dr=True, dn=True):
    dn = dn and c.norm != "none"
    d_r, d_n = (c.dr if dr else None), (c.dn if dn else None)
    new = lambda *s: torch.empty(s, device="cuda")
    g = S.ssta_residual_norm_bwd(c.desc, d_r, d_n, kept_r if dn else None, kept_y, f.mean if dn else None,
                                 f.rstd if dn else None, f.post_mean, f.post_rstd, c.post_weight, c.gate, c.weight, c.scale,
                                 dgate=new(c.G, c.C), dpost_weight=new(c.C) if c.post != "none" else None,
                                 dweight=new(c.C) if dn else None, dscale=new(c.G, c.C) if dn else None,
                                 want_dshift=dn)
    r, y = f64(r_values), f64(y_values)
    adr, adn = f64(d_r), f64(d_n)
    v = {n: c.np(n) for n in ("post_weight", "gate", "weight", "scale")}
    stats = [f64(t) for t in (f.mean, f.rstd, f.post_mean, f.post_rstd)]
    ref = oracle.residual_norm_bwd(adr, adn, r, y, *stats, c.norm, c.post, c.res_scale, v["post_weight"], v["gate"],
                                   v["weight"], v["scale"], c.mod_rows)
    # magnitudes, formula by formula
    R = np.zeros((c.rows, c.C)) if adr is None else np.abs(adr)
    acc = (c.rows + 2 * K) * U
    if dn:
        X = normal_magnitude(r, stats[0], stats[1])
        R = R + grad_magnitude(modulated_magnitude(np.abs(adn), c, v["weight"], v["scale"], None), X, stats[1])
        mag = lambda z: None if z is None else np.abs(z)
        _, aw, as_, at = oracle.norm_bwd(np.abs(adn), X, None, np.ones(c.rows), "rms", mag(v["weight"]), mag(v["scale"]),
                                         None, c.mod_rows)
        check("dweight", g.dweight, ref["dweight"], acc * aw)
        check("dscale", g.dscale, ref["dscale"], acc * as_)
        check("dshift", g.dshift, ref["dshift"], acc * at)
    else:
        assert g.dweight is None and g.dscale is None and g.dshift is None
    check("dx", g.dx, ref["dx"], c.half * np.abs(ref["dx"]) + abs(c.res_scale) * K * U * R)
    pw = 1.0 if v["post_weight"] is None else np.abs(v["post_weight"])
    gate = np.ones((c.rows, c.C)) if v["gate"] is None else _rows(v["gate"], c)
    Y = np.abs(y) if c.post == "none" else normal_magnitude(y, stats[2], stats[3])
    H = R * gate * pw
    D = H if c.post == "none" else grad_magnitude(H, Y, stats[3])
    check("dy", g.dy, ref["dy"], c.half * np.abs(ref["dy"]) + 2 * K * U * D)
    m = min(c.mod_rows or c.rows, c.rows)
    S3 = np.stack([(R * Y * pw)[i:i + m].sum(axis=0) for i in range(0, c.rows, m)])
    check("dgate", g.dgate, ref["dgate"], acc * S3)
    if c.post != "none":
        check("dpost_weight", g.dpost_weight, ref["dpost_weight"], acc * (R * gate * Y).sum(axis=0))
    return g


@pytest.mark.parametrize("cfg", ALL, ids=str)
def test_residual_norm_matches_oracle(cuda_ok, cfg):
    c = make(*cfg)
    f = check_residual_fwd(c)
    check_residual_bwd(c, f, f.r, c.y, f.r, c.y)
    if c.norm != "none":
        check_residual_bwd(c, f, f.r, c.y, f.r, c.y, dr=False)
        check_residual_bwd(c, f, None, c.y, f.r, c.y, dn=False)
    for fmt in ("int8", "e4m3"):
        s = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift, save_y=fmt,
                                     save_r=fmt)
        assert torch.equal(s.r, f.r) and (f.n is None or torch.equal(s.n, f.n))
        for saved, t in ((s.saved_y, c.y), (s.saved_r, f.r)):    # the fused save is the save of the stored tensor
            alone = S.ssta_checkpoint_save(t, fmt)
            assert torch.equal(saved.codes.view(torch.uint8), alone.codes.view(torch.uint8))
            assert torch.equal(saved.exponents, alone.exponents)
        rv, yv = S.ssta_checkpoint_load(s.saved_r), S.ssta_checkpoint_load(s.saved_y)
        check_residual_bwd(c, s, s.saved_r, s.saved_y, rv, yv)


VECTORS = ("weight", "scale", "shift", "gate", "post_weight")


@pytest.mark.parametrize("given", [(), ("scale",), ("shift",), ("weight",), ("gate",), ("post_weight",), ("weight", "shift"),
                                   ("scale", "gate")], ids=str)
@pytest.mark.parametrize("rows,C", [(9, 264), (1300, 512)])
def test_each_vector_alone(cuda_ok, rows, C, given):
    """Any subset of the vectors; gradients of the absent ones (as 1 or 0) are there for the asking."""
    c = make(rows, C, "bf16", "f32", "layer", "rms", True, rows // 2 + 1, 1.0)
    for v in VECTORS:
        if v not in given:
            setattr(c, v, None)
    mean, rstd = check_norm_fwd(c)
    check_norm_bwd(c, mean, rstd, c.x, c.x)
    f = check_residual_fwd(c)
    check_residual_bwd(c, f, f.r, c.y, f.r, c.y)
    # by default only the given vectors' gradients are computed
    g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.r, c.y, f.mean, f.rstd, f.post_mean, f.post_rstd, c.post_weight, c.gate,
                                 c.weight, c.scale)
    for v in VECTORS:
        assert (getattr(g, "d" + v) is not None) == (getattr(c, "scale" if v == "shift" else v) is not None), v


def test_optional_outputs_do_not_change_the_others(cuda_ok):
    c = make(100, 1000, "bf16", "f32", "rms", "none", True, 30, 1.0)
    _, _, rstd, _ = S.ssta_norm_fwd(c.desc, c.x)
    full = S.ssta_norm_bwd(c.desc, c.dn, c.x, None, rstd, c.weight, c.scale, c.dr)
    none = S.ssta_norm_bwd(c.desc, c.dn, c.x, None, rstd, c.weight, c.scale, c.dr, want_dshift=False)
    assert none.dshift is None and torch.equal(none.dx, full.dx) and torch.equal(none.dscale, full.dscale)
    bare = S.ssta_norm_bwd(c.desc, c.dn, c.x, None, rstd)
    assert bare.dweight is None and bare.dscale is None and bare.dshift is None
    zero = S.ssta_norm_bwd(c.desc, c.dn, c.x, None, rstd, dres=torch.zeros_like(c.dr))
    assert torch.equal(bare.dx, zero.dx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_at_16_byte_offsets(cuda_ok, dtype):
    """16 bytes is all the alignment a tensor needs, also where 32-byte accesses are used otherwise."""
    c = make(300, 520, dtype, dtype, "layer", "rms", True, 77, 1.0)
    item = c.x.element_size()

    def shift(t):
        if t is None:
            return None
        buf = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
        base = 16 if buf.data_ptr() % 32 == 0 else 0
        out = buf[base:base + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        assert out.data_ptr() % 32 == 16
        return out.copy_(t)

    wide = {n: getattr(c, n).contiguous() for n in ("scale", "shift", "gate")}
    d = S.norm_desc(c.rows, c.C, dtype, dtype, "layer", "rms", c.eps, 1.0, c.mod_rows)
    plain = dict(x=c.x, y=c.y, post_weight=c.post_weight, weight=c.weight, **wide)
    back = dict(dr=c.dr, dn=c.dn)

    def go(t, b, out):
        f = S.ssta_residual_norm_fwd(d, t["x"], t["y"], t["post_weight"], t["gate"], t["weight"], t["scale"], t["shift"],
                                     r=out(torch.empty_like(c.x)), n=out(torch.empty_like(c.x)), save_y="int8")
        g = S.ssta_residual_norm_bwd(d, b["dr"], b["dn"], f.r, t["y"], f.mean, f.rstd, f.post_mean, f.post_rstd,
                                     t["post_weight"], t["gate"], t["weight"], t["scale"], dx=out(torch.empty_like(c.x)),
                                     dy=out(torch.empty_like(c.x)))
        ck = S.ssta_checkpoint_save(f.r, "e4m3")
        v = S.ssta_checkpoint_load(ck, out(torch.empty_like(c.x)))
        return [f.r, f.n, f.mean, f.saved_y.codes, g.dx, g.dy, g.dgate, g.dscale, g.dshift, g.dweight, g.dpost_weight, v]

    a = go(plain, back, lambda t: t)
    b = go({n: shift(t) for n, t in plain.items()}, {n: shift(t) for n, t in back.items()}, shift)
    for i, (p, q) in enumerate(zip(a, b)):
        assert torch.equal(p, q), i
    with pytest.raises(S.SstaError) as e:
        S.ssta_norm_fwd(d, torch.empty(c.rows * c.C + 8, dtype=c.x.dtype, device="cuda")[8 // item:][:c.rows * c.C].view(c.rows, c.C))
    assert e.value.code == 3


@pytest.mark.parametrize("dtype,C,saved", [("bf16", 264, None), ("bf16", 128, "int8"), ("f32", 136, "e4m3"), ("f32", 128, None),
                                           ("bf16", 2048, "e4m3")])
def test_long_runs(cuda_ok, dtype, C, saved):
    """Many rows per block (its row table is refilled, its stages wrap, groups end inside tiles), every element
    against float64 autograd on the GPU.  Bounds as relative 2-norms: half a step of the type for the rows, and for the
    vectors' sums over n rows sqrt(n) u * 4, the square-root growth of rounding in a sum of independent terms."""
    rows = 70_001 if C < 1024 else 40_003
    c = make(rows, C, dtype, "f32", "layer", "rms", True, rows // 2 - 77, 0.5, offset=0.1)
    f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift, save_y=saved, save_r=saved)
    r, y = (f.saved_r, f.saved_y) if saved else (f.r, c.y)
    g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, r, y, f.mean, f.rstd, f.post_mean, f.post_rstd, c.post_weight, c.gate,
                                 c.weight, c.scale)
    value = lambda t: (S.ssta_checkpoint_load(t) if saved else t).double()
    group = torch.arange(rows, device="cuda") // (rows // 2 - 77)
    v = {n: getattr(c, n).double().requires_grad_() for n in VECTORS}
    rows_of = lambda n: v[n].index_select(0, group)
    # the norms' gradients at the saved statistics: through(x) = the norm's exact derivative with fixed mean and rstd
    rh = (value(r) - f.mean.double()[:, None]) * f.rstd.double()[:, None]
    yh = value(y) * f.post_rstd.double()[:, None]

    def through(h, grad, rstd, layer):
        out = grad - h * (grad * h).mean(1, keepdim=True) - (grad.mean(1, keepdim=True) if layer else 0)
        return out * rstd.double()[:, None]

    gr = c.dn.double() * v["weight"] * (1 + rows_of("scale"))
    dR = c.dr.double() + through(rh, gr.detach(), f.rstd, True)
    loss = (c.dn.double() * (rh * v["weight"] * (1 + rows_of("scale")) + rows_of("shift"))).sum() + \
        (dR * rows_of("gate") * yh * v["post_weight"]).sum()
    loss.backward()
    dh = dR * rows_of("gate").detach() * v["post_weight"].detach()
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert rel(g.dx, 0.5 * dR) <= c.half and rel(g.dy, through(yh, dh, f.post_rstd, False)) <= c.half + 4 * U
    for n in VECTORS:
        assert rel(getattr(g, "d" + n), v[n].grad) <= 4 * U * rows ** 0.5, n


def test_fused_save_of_the_norm_input(cuda_ok):
    for C in (120, 2048, 2056, 8192):
        c = Case(11, C)
        for fmt in ("int8", "e4m3"):
            y, _, _, saved = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift, save=fmt)
            alone = S.ssta_checkpoint_save(c.x, fmt)
            assert torch.equal(saved.codes.view(torch.uint8), alone.codes.view(torch.uint8))
            assert torch.equal(saved.exponents, alone.exponents)
            assert torch.equal(y, S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift)[0])


@pytest.mark.parametrize("rows,C,mod_rows", [(5, 64, 1), (1000, 2048, 1), (37, 1000, 5), (300, 128, 299), (64, 256, 9999)])
def test_modulation_groups(cuda_ok, rows, C, mod_rows):
    """A modulation row per token, a last group of one row, a group larger than the tensor; dense and strided rows."""
    for stride in (1, 6):
        c = Case(rows, C, mod_rows=mod_rows, stride=stride, norm="rms", post="layer")
        mean, rstd = check_norm_fwd(c)
        check_norm_bwd(c, mean, rstd, c.x, c.x)
        f = check_residual_fwd(c)
        check_residual_bwd(c, f, f.r, c.y, f.r, c.y)


def test_leading_dimensions_and_chunks(cuda_ok):
    """[B, L, C] activations with a [B, 1, C] chunk of one modulation tensor, as a block has them."""
    B, L, C = 3, 10, 256
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(B, L, C, generator=gen).bfloat16().cuda()
    mod = (0.3 * torch.randn(B, 1, 6 * C, generator=gen)).bfloat16().cuda()
    shift, scale, gate = mod.chunk(6, dim=-1)[:3]
    d = S.norm_desc(B * L, C, param_dtype="bf16", mod_rows=L, mod_stride=6 * C)
    y, mean, rstd, ck = S.ssta_norm_fwd(d, x, scale=scale, shift=shift, save="int8")
    assert y.shape == x.shape and mean.shape == (B * L,) and ck.shape == x.shape and ck.exponents.shape == (B, L, 2)
    dense = S.norm_desc(B * L, C, param_dtype="bf16", mod_rows=L)
    y2 = S.ssta_norm_fwd(dense, x, scale=scale.contiguous(), shift=shift.contiguous())[0]
    assert torch.equal(y, y2)
    f = S.ssta_residual_norm_fwd(d, x, y, gate=gate, scale=scale, shift=shift)
    g = S.ssta_residual_norm_bwd(d, x, y, f.r, y, f.mean, f.rstd, gate=gate, scale=scale)
    assert g.dx.shape == x.shape and g.dgate.shape == (B, C)
    # a gap between leading dimensions is refused
    four = torch.zeros(2, 2, 7 * C, dtype=torch.bfloat16, device="cuda")[:, :1, :C]
    with pytest.raises(ValueError, match="row stride"):
        S.ssta_norm_fwd(S.norm_desc(B * L, C, param_dtype="bf16", mod_rows=15, mod_stride=7 * C), x, scale=four)


@pytest.mark.parametrize("C", [128, 1000, 4104])
def test_in_place(cuda_ok, C):
    c = Case(50, C, post="rms", mod_rows=20)
    y = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift)[0]
    x = c.x.clone()
    assert S.ssta_norm_fwd(c.desc, x, c.weight, c.scale, c.shift, y=x)[0] is x and torch.equal(x, y)
    args = (c.post_weight, c.gate, c.weight, c.scale, c.shift)
    f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, *args)
    x, yy = c.x.clone(), c.y.clone()
    S.ssta_residual_norm_fwd(c.desc, x, yy, *args, r=x, n=yy)
    assert torch.equal(x, f.r) and torch.equal(yy, f.n)
    back = lambda dr, dn, **kw: S.ssta_residual_norm_bwd(c.desc, dr, dn, f.r, c.y, f.mean, f.rstd, f.post_mean, f.post_rstd,
                                                         *args[:4], **kw)
    g = back(c.dr, c.dn)
    dr, dn = c.dr.clone(), c.dn.clone()
    back(dr, dn, dx=dr, dy=dn)
    assert torch.equal(dr, g.dx) and torch.equal(dn, g.dy)
    ref = S.ssta_norm_bwd(c.desc, c.dn, c.x, f.mean, f.rstd, c.weight, c.scale, c.dr)
    for out in ("dy", "dres"):
        dy, dres = c.dn.clone(), c.dr.clone()
        got = S.ssta_norm_bwd(c.desc, dy, c.x, f.mean, f.rstd, c.weight, c.scale, dres, dx=dy if out == "dy" else dres)
        assert torch.equal(got.dx, ref.dx) and torch.equal(got.dscale, ref.dscale)


def test_nothing_outside_the_rows_is_written(cuda_ok):
    """Outputs in the middle of larger buffers: what lies before and behind keeps its bytes."""
    rows, C = 21, 1000
    c = Case(rows, C, post="layer", mod_rows=8)

    def framed(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 512,), 77, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)

    bufs, t = {}, {}
    for name, shape, dtype in [("r", (rows, C), torch.bfloat16), ("n", (rows, C), torch.bfloat16),
                               ("dx", (rows, C), torch.bfloat16), ("dy", (rows, C), torch.bfloat16),
                               ("codes", (rows, C), torch.int8), ("exps", (rows, 8), torch.uint8),
                               ("dgate", (c.G, C), torch.float32), ("dscale", (c.G, C), torch.float32),
                               ("dshift", (c.G, C), torch.float32), ("dweight", (C,), torch.float32),
                               ("dpost_weight", (C,), torch.float32)]:
        bufs[name], t[name] = framed(shape, dtype)
    ws_bytes = S.ssta_norm_plan(c.desc).bwd_workspace_bytes
    bufs["ws"], t["ws"] = framed((ws_bytes,), torch.uint8)
    f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift, r=t["r"], n=t["n"],
                                 save_r=S.Checkpoint(t["codes"], t["exps"]))
    S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.r, c.y, f.mean, f.rstd, f.post_mean, f.post_rstd, c.post_weight, c.gate,
                             c.weight, c.scale, workspace=t["ws"],
                             **{n: t[n] for n in ("dx", "dy", "dgate", "dscale", "dshift", "dweight", "dpost_weight")})
    torch.cuda.synchronize()
    for name, buf in bufs.items():
        n = t[name].numel()
        assert (buf[:256] == 77).all() and (buf[256 + n:] == 77).all(), name


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_rows_do_not_touch_one_another(cuda_ok, kind):
    """A row with a NaN or an infinity spoils itself alone; a zero row stays finite."""
    c = Case(40, 2048, norm=kind, post=kind, seed=3)
    ref = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift)
    x, y = c.x.clone(), c.y.clone()
    x[7, 100], y[20, 0], x[30], y[30] = float("nan"), float("inf"), 0, 0
    f = S.ssta_residual_norm_fwd(c.desc, x, y, c.post_weight, c.gate, c.weight, c.scale, c.shift, save_y="int8",
                                 save_r="int8")
    good = [i for i in range(40) if i not in (7, 20, 30)]
    assert torch.equal(f.n[good], ref.n[good]) and torch.equal(f.r[good], ref.r[good])
    assert torch.isfinite(f.n[30].float()).all() and torch.isfinite(f.rstd[30])
    assert torch.isnan(f.n[7].float()).all() and torch.isnan(f.n[20].float()).all()
    e = f.saved_r.exponents
    assert (e[7] == 255).sum() == 1 and e[7, 0] == 255 and (e[good] < 255).all()
    # an infinity in y: the layer norm's mean is infinite and spoils the row; the rms norm's 1 / deviation is 0, which
    # leaves 0 * inf in the one channel and zeros elsewhere
    assert e[20, 0] == 255 and (e[20, 1:] == 255).all().item() == (kind == "layer")
    g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.saved_r, f.saved_y, f.mean, f.rstd, f.post_mean, f.post_rstd,
                                 c.post_weight, c.gate, c.weight, c.scale)
    assert torch.isfinite(g.dx[good].float()).all() and torch.isfinite(g.dy[good].float()).all()
    assert torch.isnan(g.dx[7].float()).any() and torch.isnan(g.dy[20].float()).any()


def test_large_mean_rows(cuda_ok):
    """Rows whose mean is far above their deviation: the mean square of differences does not cancel."""
    for C in (128, 2048, 4096):
        c = Case(16, C, dtype="f32", offset=300.0)
        mean, rstd = check_norm_fwd(c)
        check_norm_bwd(c, mean, rstd, c.x, c.x)


def test_same_bytes_every_time(cuda_ok):
    for rows, C, mod in ((5000, 2048, 0), (3001, 128, 700), (2000, 1544, 1)):
        c = Case(rows, C, post="rms", mod_rows=mod)
        f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift)
        outs = [S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.r, c.y, f.mean, f.rstd, f.post_mean, f.post_rstd,
                                         c.post_weight, c.gate, c.weight, c.scale) for _ in range(3)]
        for name in ("dx", "dy", "dpost_weight", "dgate", "dweight", "dscale", "dshift"):
            assert all(torch.equal(getattr(outs[0], name), getattr(o, name)) for o in outs[1:]), name


def test_gradients_against_differences(cuda_ok):
    """Central differences of the GPU's own fp32 forward along a random direction.  L = sum(dr r + dn n) over
    N = 6 * 1000 elements; with step h the quotient's error is about sqrt(N) K u / h from rounding (each term rounded
    to a few u) and h^2 from the curvature of terms of order one: h = 2^-6 bounds both by 2e-3 sqrt(N)."""
    c = Case(6, 1000, dtype="f32", post="rms", mod_rows=4, eps=1e-2, res_scale=0.7, offset=0.2)
    names = ("x", "y", "post_weight", "gate", "weight", "scale", "shift")

    def loss(**kw):
        a = [kw.get(n, getattr(c, n)) for n in names]
        f = S.ssta_residual_norm_fwd(c.desc, *a, stats=False)
        return ((f.r.double() * c.dr).sum() + (f.n.double() * c.dn).sum()).item()

    f = S.ssta_residual_norm_fwd(c.desc, *[getattr(c, n) for n in names])
    g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.r, c.y, f.mean, f.rstd, f.post_mean, f.post_rstd, c.post_weight,
                                 c.gate, c.weight, c.scale)
    h = 2.0 ** -6
    scale = max(c.dr.double().norm().item(), c.dn.double().norm().item())
    for i, n in enumerate(names):
        t = getattr(c, n)
        v = torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).cuda()
        v /= v.norm()
        wide = torch.empty(c.G, 6 * c.C, device="cuda")[:, :c.C] if n in ("gate", "scale", "shift") else torch.empty_like(t)
        got = []
        for s in (h, -h):
            wide.copy_(t + s * v)
            got.append(loss(**{n: wide}))
        diff = (got[0] - got[1]) / (2 * h)
        want = (getattr(g, "d" + n).double() * v).sum().item()
        assert abs(diff - want) <= 2e-3 * scale, (n, diff, want)


def test_captured_and_replayed(cuda_ok):
    """Forward and backward in one CUDA graph, replayed on inputs changed in place, equal eager calls; a second graph
    with its own workspace replays between them."""
    cases = [Case(333, 1544, post="layer", mod_rows=100, seed=1), Case(64, 128, norm="rms", seed=2)]
    graphs = []
    for c in cases:
        def step(c=c):
            f = S.ssta_residual_norm_fwd(c.desc, c.x, c.y, c.post_weight, c.gate, c.weight, c.scale, c.shift, save_y="int8",
                                         save_r="int8")
            g = S.ssta_residual_norm_bwd(c.desc, c.dr, c.dn, f.saved_r, f.saved_y, f.mean, f.rstd, f.post_mean, f.post_rstd,
                                         c.post_weight, c.gate, c.weight, c.scale)
            return [f.r, f.n, f.saved_r.codes, g.dx, g.dy, g.dgate, g.dscale, g.dshift, g.dweight]
        step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs, step))
    for it in range(3):
        for c in cases:
            c.x.mul_(-1.5)
            c.dn.copy_(c.dn.roll(1, 0))
        for graph, _, _ in graphs:
            graph.replay()
        for graph, outs, step in graphs:
            for a, b in zip(outs, step()):
                assert torch.equal(a, b), it


def test_on_another_stream(cuda_ok):
    c = Case(4000, 2048)
    ref = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift)
    gref = S.ssta_norm_bwd(c.desc, c.dn, c.x, ref[1], ref[2], c.weight, c.scale)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        ext = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)
        for _ in range(20):     # memory of one call may serve the next one of the same stream
            y, mean, rstd, ck = S.ssta_norm_fwd(c.desc, c.x, c.weight, c.scale, c.shift, save="e4m3", stream=stream)
            g = S.ssta_norm_bwd(c.desc, c.dn, c.x, mean, rstd, c.weight, c.scale, stream=stream)
        ext.synchronize()
        assert torch.equal(y, ref[0]) and torch.equal(g.dx, gref.dx) and torch.equal(g.dscale, gref.dscale)


def test_two_streams_at_once(cuda_ok):
    cs = [Case(3000, 2048, seed=i) for i in range(2)]
    refs = [S.ssta_norm_bwd(c.desc, c.dn, c.x, *S.ssta_norm_fwd(c.desc, c.x)[1:3], c.weight, c.scale, c.dr) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            _, m, r, _ = S.ssta_norm_fwd(c.desc, c.x, stream=s)
            outs[i].append(S.ssta_norm_bwd(c.desc, c.dn, c.x, m, r, c.weight, c.scale, c.dr, stream=s))
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        for g in got:
            assert torch.equal(g.dx, ref.dx) and torch.equal(g.dscale, ref.dscale) and torch.equal(g.dweight, ref.dweight)


def test_rows_beyond_32_bit_offsets(cuda_ok):
    """More than 2^31 elements: the last rows equal those of a short tensor with the same rows."""
    rows, C = 1_050_000, 2056
    assert rows * C > 2 ** 31
    small = Case(64, C, norm="rms", stride=1)
    big = torch.zeros((rows, C), dtype=torch.bfloat16, device="cuda")
    big[-64:] = small.x
    d = S.norm_desc(rows, C, norm="rms")
    y, _, rstd, ck = S.ssta_norm_fwd(d, big, small.weight, small.scale, small.shift, save="int8")
    ys, _, rs, cs = S.ssta_norm_fwd(small.desc, small.x, small.weight, small.scale, small.shift, save="int8")
    assert torch.equal(y[-64:], ys) and torch.equal(rstd[-64:], rs)
    assert torch.equal(ck.codes[-64:], cs.codes) and torch.equal(ck.exponents[-64:], cs.exponents)
    assert (ck.codes[:-64] == 0).all()
    del y
    dy = torch.zeros((rows, C), dtype=torch.bfloat16, device="cuda")
    dy[-64:] = small.dn
    for x, xs in ((big, small.x), (ck, cs)):
        g = S.ssta_norm_bwd(d, dy, x, None, rstd, small.weight, small.scale, want_dshift=True)
        gs = S.ssta_norm_bwd(small.desc, small.dn, xs, None, rs, small.weight, small.scale, want_dshift=True)
        assert torch.equal(g.dx[-64:], gs.dx) and (g.dx[:-64] == 0).all()
        # the same 64 terms per channel, added in another order
        for a, b in ((g.dshift, gs.dshift), (g.dscale, gs.dscale), (g.dweight, gs.dweight)):
            assert (a - b).abs().max() <= 64 * U * 64 * b.abs().max()
    assert torch.equal(S.ssta_checkpoint_load(ck)[-64:], S.ssta_checkpoint_load(cs))
    again = S.ssta_checkpoint_save(big, "int8")
    assert torch.equal(again.codes[-64:], cs.codes) and torch.equal(again.exponents[-64:], cs.exponents)


def test_binding_refusals(cuda_ok):
    c = Case(8, 256, mod_rows=4)
    x = c.x
    bad = [
        lambda: S.ssta_norm_fwd(c.desc, x[:4]), lambda: S.ssta_norm_fwd(c.desc, x.float()),
        lambda: S.ssta_norm_fwd(c.desc, torch.empty(8, 512, dtype=x.dtype, device="cuda")[:, ::2]),
        lambda: S.ssta_norm_fwd(c.desc, x, weight=c.weight[:128]), lambda: S.ssta_norm_fwd(c.desc, x, weight=c.weight.bfloat16()),
        lambda: S.ssta_norm_fwd(c.desc, x, scale=c.scale.contiguous()), lambda: S.ssta_norm_fwd(c.desc, x, scale=c.scale[:1]),
        lambda: S.ssta_norm_fwd(c.desc, x, weight=c.weight.cpu()), lambda: S.ssta_norm_fwd(c.desc, x, save="int4"),
        lambda: S.ssta_norm_fwd(c.desc, x, save=S.Checkpoint.empty((4, 256))),
        lambda: S.ssta_norm_fwd(c.desc, x, save=S.Checkpoint.empty((8, 256), dtype=torch.float32)),
        lambda: S.ssta_norm_bwd(c.desc, x, x, None, torch.ones(7, device="cuda")),
        lambda: S.ssta_checkpoint_save(x.half()), lambda: S.ssta_checkpoint_save(x, out=S.Checkpoint.empty((8, 128))),
        lambda: S.ssta_checkpoint_load(x), lambda: S.ssta_checkpoint_load(S.Checkpoint.empty((8, 256)), torch.empty(8, 256)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("case", i, "was accepted")
    for call, code in ((lambda: S.ssta_norm_fwd(S.norm_desc(8, 256, norm="none"), x), 1),
                       (lambda: S.ssta_norm_bwd(c.desc, x, x, None, torch.ones(8, device="cuda")), 1),
                       (lambda: S.ssta_norm_bwd(c.desc, x, x, *torch.ones(2, 8, device="cuda"),
                                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), 4),
                       (lambda: S.ssta_checkpoint_save(torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")), 1)):
        with pytest.raises(S.SstaError) as e:
            call()
        assert e.value.code == code
