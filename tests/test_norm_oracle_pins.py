"""CPU pins of the oracle for the norms, gated residuals and 8-bit checkpoints: gradients
against central differences of the forward in float64, closed forms, and the checkpoint
code's defining properties.

Differences: with step h the truncation error is O(h^2) and the rounding error about
1e-16 / h of the loss; h = 1e-5 leaves both near 1e-10 of the sums involved, so 1e-6 of
the gradient's scale is a wide margin."""
import itertools

import numpy as np
import pytest
import torch

import oracle

KINDS = ("layer", "rms")


def _rng(*seed):
    return np.random.default_rng(list(seed))


def _difference(loss, x, v, h=1e-5):
    """Directional derivative of loss at x along v."""
    return (loss(x + h * v) - loss(x - h * v)) / (2 * h)


@pytest.mark.parametrize("kind,with_vectors,mod_rows", list(itertools.product(KINDS, (False, True), (0, 2, 3))))
def test_norm_bwd_is_the_derivative(kind, with_vectors, mod_rows):
    rng = _rng(1, KINDS.index(kind), with_vectors, mod_rows)
    R, C, eps = 7, 24, 1e-3
    G = 1 if mod_rows == 0 else -(-R // mod_rows)
    x, dy = rng.normal(size=(R, C)) + 0.5, rng.normal(size=(R, C))
    w, s, t = (rng.normal(size=C) + 1, rng.normal(size=(G, C)), rng.normal(size=(G, C))) if with_vectors else (None,) * 3
    y, mean, rstd = oracle.norm_fwd(x, kind, eps, w, s, t, mod_rows)
    dx, dw, ds, dt = oracle.norm_bwd(dy, x, mean, rstd, kind, w, s, None, mod_rows)
    loss = lambda x, w, s, t: (oracle.norm_fwd(x, kind, eps, w, s, t, mod_rows)[0] * dy).sum()
    w1 = np.ones(C) if w is None else w
    s1, t1 = (np.zeros((G, C)) if z is None else z for z in (s, t))
    for arg, grad, f in ((x, dx, lambda z: loss(z, w1, s1, t1)), (w1, dw, lambda z: loss(x, z, s1, t1)),
                         (s1, ds, lambda z: loss(x, w1, z, t1)), (t1, dt, lambda z: loss(x, w1, s1, z))):
        v = rng.normal(size=arg.shape)
        np.testing.assert_allclose(_difference(f, arg, v), (grad * v).sum(), rtol=1e-6, atol=1e-6)
    np.testing.assert_allclose(oracle.norm_bwd(dy, x, mean, rstd, kind, w, s, x, mod_rows)[0], dx + x)


@pytest.mark.parametrize("kind,post,gated,mod_rows",
                         list(itertools.product(("none",) + KINDS, ("none",) + KINDS, (False, True), (0, 3))))
def test_residual_norm_bwd_is_the_derivative(kind, post, gated, mod_rows):
    rng = _rng(2, gated, mod_rows, len(kind), len(post))
    R, C, eps, rs = 5, 16, 1e-3, 0.7
    G = 1 if mod_rows == 0 else -(-R // mod_rows)
    x, y, dr = (rng.normal(size=(R, C)) for _ in range(3))
    dn = rng.normal(size=(R, C)) if kind != "none" else None
    par = dict(post_weight=rng.normal(size=C) + 1 if post != "none" else None,
               gate=rng.normal(size=(G, C)) if gated else None,
               weight=rng.normal(size=C) + 1 if kind != "none" else None,
               scale=rng.normal(size=(G, C)) if kind != "none" else None,
               shift=rng.normal(size=(G, C)) if kind != "none" else None)

    def loss(**kw):
        a = {**dict(x=x, y=y), **par, **kw}
        f = oracle.residual_norm_fwd(a.pop("x"), a.pop("y"), kind, post, eps, rs, mod_rows=mod_rows, **a)
        return (f["r"] * dr).sum() + ((f["n"] * dn).sum() if dn is not None else 0.0)

    f = oracle.residual_norm_fwd(x, y, kind, post, eps, rs, mod_rows=mod_rows, **par)
    b = oracle.residual_norm_bwd(dr, dn, f["r"], y, f["mean"], f["rstd"], f["post_mean"], f["post_rstd"], kind, post, rs,
                                 par["post_weight"], par["gate"], par["weight"], par["scale"], mod_rows)
    base = {**dict(x=x, y=y), **par}
    for name, arg in base.items():
        if arg is None:
            continue
        v = rng.normal(size=arg.shape)
        d = _difference(lambda z: loss(**{name: z}), arg, v)
        np.testing.assert_allclose(d, (b["d" + name] * v).sum(), rtol=1e-6, atol=1e-6, err_msg=name)


def test_layer_norm_closed_form():
    x = np.array([[1.0, 3.0, 1.0, 3.0, 1.0, 3.0, 1.0, 3.0]])
    y, mean, rstd = oracle.norm_fwd(x, "layer", 3.0)         # variance 1, + eps 3 -> 1 / 2
    assert mean[0] == 2.0 and rstd[0] == 0.5
    np.testing.assert_array_equal(y[0], [-0.5, 0.5] * 4)
    y, mean, rstd = oracle.norm_fwd(x, "rms", 4.0)           # mean square 5, + 4 -> 1 / 3
    assert mean is None
    np.testing.assert_allclose(y[0], x[0] / 3)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoint_code_properties(fmt):
    rng = _rng(3, fmt == "int8")
    x = np.concatenate([rng.normal(size=(6, 300)) * s for s in (1.0, 1e-3, 2.0 ** 20, 1e-38, 1e30)])
    x = x.astype(np.float32).astype(np.float64)
    x[3] = 0.0
    codes, exps = oracle.checkpoint_encode(x, fmt)
    v = oracle.checkpoint_decode(codes, exps)
    assert exps.min() >= 1 and exps.max() <= 254
    scale = np.repeat(2.0 ** (exps.astype(np.float64) - 127), 128, axis=1)[:, :300]
    amax = np.stack([np.abs(x[:, j:j + 128]).max(axis=1) for j in range(0, 300, 128)], axis=1)
    top = np.repeat(amax, 128, axis=1)[:, :300]
    if fmt == "int8":
        assert np.abs(codes).max() <= 127 and (codes == np.rint(codes)).all()
        np.testing.assert_array_less(np.abs(v - x), np.maximum(top / 127.5, 2.0 ** -127) + 1e-300)
        assert (np.abs(v - x) <= scale / 2).all()
    else:
        assert np.abs(codes).max() <= 448
        assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)).all()
    # the smallest exponent that fits: one less would not (unless clamped)
    limit = lambda e: amax * 2.0 ** (127.0 - e) < 127.5 if fmt == "int8" else amax * 2.0 ** (127.0 - e) <= 448
    e = exps.astype(np.float64)
    assert limit(e).all() and (~limit(e - 1) | (exps == 1)).all()
    # a second pass changes nothing
    again = oracle.checkpoint_decode(*oracle.checkpoint_encode(v, fmt))
    np.testing.assert_array_equal(again, v)


def test_checkpoint_values_are_exact_in_bf16():
    for fmt in ("int8", "e4m3"):
        x = _rng(4).normal(size=(16, 256)) * np.exp(_rng(5).normal(size=(16, 1)) * 20)
        v = oracle.checkpoint_decode(*oracle.checkpoint_encode(x, fmt))
        t = torch.from_numpy(v)
        assert torch.equal(t.bfloat16().double(), t)


def test_e4m3_table_is_the_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    finite = np.unique(np.abs(codes[np.isfinite(codes)]))
    u = np.concatenate([finite, (finite[1:] + finite[:-1]) / 2, finite[1:] * 0.999, _rng(6).uniform(0, 448, 2000)])
    u = u.astype(np.float32).astype(np.float64)
    # 448 in every group fixes the scale at 1
    x = np.zeros((len(u), 8))
    x[:, 0], x[:, 1] = u, 448.0
    codes, exps = oracle.checkpoint_encode(x, "e4m3")
    assert (exps == 127).all()
    want = torch.from_numpy(u).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(codes[:, 0], want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoint_non_finite_group(fmt):
    x = _rng(7).normal(size=(3, 256))
    x[0, 5], x[1, 200], x[2, 130] = np.inf, np.nan, -np.inf
    codes, exps = oracle.checkpoint_encode(x, fmt)
    assert exps.tolist()[0][0] == 255 and exps[0, 1] < 255 and exps[1, 1] == 255 and exps[2, 1] == 255
    v = oracle.checkpoint_decode(codes, exps)
    assert np.isnan(v[0, :128]).all() and np.isfinite(v[0, 128:]).all() and np.isnan(v[1:, 128:]).all()


def test_attention_bwd_saved_equals_the_recomputing_oracle():
    import ssta_inputs as si
    w = si.with_overrides(si.get_workload("tiny_f32"), T=3, Y=7, X=6, L_text=5)
    x = si.make_inputs(w, 3)
    f = lambda n: None if x[n] is None else x[n].double().numpy()
    qp, kp, vp = (oracle.tile_reorder(w, f(n), f(n + "_text")) for n in "qkv")
    S = oracle.block_scores(w, oracle.tile_pool(w, qp), oracle.tile_pool(w, kp))
    kept = oracle.kept_mask(w, oracle.select_topk(w, S))
    O, lse = oracle.attention(w, qp, kp, vp, kept)
    dO = _rng(8).normal(size=qp.shape)
    for a, b in zip(oracle.attention_bwd_saved(w, qp, kp, vp, O, lse, dO, kept),
                    oracle.attention_bwd(w, qp, kp, vp, dO, kept)):
        np.testing.assert_allclose(a, b, atol=1e-10)
