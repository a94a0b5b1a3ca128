"""ssta_forward with 8-bit checkpoints and ssta_backward at peaked logits: the gradients are
those of the attention over the checkpoints' values, probabilities of a softmax among them.

Bounds.  With u = 2^-24 and h half a step of the stored type (2^-8 for bf16, 2^-24 for fp32),
every rounding is counted at its largest, term by term: a product over 128 channels in fp32 is
off by (K u) times the sum of its terms' magnitudes (K = 136: 128 additions and the handling of
the sum), the exponential and its argument by 2^-20 relative, and the log-sum-exp by the
P-weighted mean of what its logits are off by.  O is stored in the type after P rounded to it met
v; dS and P are rounded to the type before their products, and the gradients once at the end.  A
sum over n rows or keys adds n u of the magnitudes."""
import math

import numpy as np
import pytest
import torch

import block_sparse_video_ssta_b200 as S
import oracle
import ssta_inputs as si
from ssta_inputs import with_overrides
from ssta_parity import gpu_kept, to_np

pytestmark = pytest.mark.gpu

U, K = 2.0 ** -24, 136
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
WORKLOADS = [("tiny_f32", dict(topk=8)), ("tiny_f32", dict(T=5, Y=7, X=6, L_text=45, B=2)),
             ("small_bf16", dict(H=2, T=4, Y=12, X=10, L_text=40)), ("small_bf16", dict(H=1, T=4, Y=8, X=16, tT=2, topk=2))]
IDS = [str(i) for i in range(len(WORKLOADS))]


def backward_bounds(w, q, k, v, dO, kept):
    """Largest errors of (dq, dk, dv), element by element, and the standard deviation of the logits."""
    g, h, scale = oracle.geometry(w), HALF[w.dtype], 1.0 / math.sqrt(w.D)
    valid = oracle.valid_token_mask(w)
    out = [np.zeros(q.shape) for _ in range(3)]
    spread = []
    for b, hd, i in np.ndindex(kept.shape[:3]):
        rows = np.arange(i * g.N, min((i + 1) * g.N, g.Lq))
        rows = rows[valid[rows]]
        keys = np.concatenate([np.arange(j * g.N, min((j + 1) * g.N, g.Lq)) for j in np.nonzero(kept[b, hd, i])[0]])
        keys = keys[valid[keys]]
        Q, Kk, V, G = q[b, hd, rows], k[b, hd, keys], v[b, hd, keys], dO[b, hd, rows]
        s = Q @ Kk.T * scale
        spread.append(s.std())
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        ds_ = K * U * scale * np.abs(Q) @ np.abs(Kk).T
        rel = ds_ + (p * ds_).sum(axis=1, keepdims=True) + 2.0 ** -20 * (1 + np.abs(s - s.max(axis=1, keepdims=True)) * U * 2 ** 20)
        o = p @ V
        o_err = (p * (rel + h)) @ np.abs(V) + h * np.abs(o) + len(keys) * U * p @ np.abs(V)
        d_err = (np.abs(G) * (o_err + K * U * np.abs(o))).sum(axis=1, keepdims=True)
        dp = G @ V.T - (G * o).sum(axis=1, keepdims=True)
        ds = p * dp
        ds_err = np.abs(ds) * (rel + h) + p * (K * U * np.abs(G) @ np.abs(V).T + d_err) * (1 + rel)
        n = U * (len(keys) + len(rows) * kept.shape[2])
        out[0][b, hd, rows] = scale * (ds_err + n * np.abs(ds)) @ np.abs(Kk)
        out[1][b, hd, keys] += scale * (ds_err + n * np.abs(ds)).T @ np.abs(Q)
        out[2][b, hd, keys] += (p * (rel + h + n)).T @ np.abs(G)
    return out, float(np.mean(spread))


def chain(name, ov, fmt, normed, dO=None, edit=None):
    """The chain on logits that a few strong channels make peaked."""
    w = with_overrides(si.get_workload(name), **ov)
    d = S.desc_from(w)
    x = si.make_inputs(w, 5, device="cuda")
    if edit is not None:
        edit(x)
    weights = [None, None]
    strong = torch.ones(w.D, device="cuda")
    strong[[5, 77]] = 6.0
    if normed:
        weights = [strong, strong.clone()]
    else:
        for n in ("q", "k", "q_text", "k_text"):
            if x[n] is not None:
                x[n] = (x[n] * strong).to(x[n].dtype).contiguous()
    r = S.ssta_forward(d, x["q"], x["k"], x["v"], x["q_text"], x["k_text"], x["v_text"], q_weight=weights[0],
                       k_weight=weights[1], checkpoint=fmt)
    if dO is None:
        gen = torch.Generator().manual_seed(3)
        like = lambda t: None if t is None else torch.randn(t.shape, generator=gen).to(t.dtype).cuda()
        dO = lambda w, t, text: (like(t), like(text))
    dOv, dOt = dO(w, r["O"], r["O_text"])
    g = S.ssta_backward(d, r["saved"], dOv, dOt)
    assert S.ssta_read_device_status(g["workspace"]) == 0
    saved = r["saved"]
    values = [to_np(S.ssta_checkpoint_load(c)) for c in (saved.q, saved.k, saved.v)]
    packed = lambda v, t: oracle.tile_reorder(w, to_np(v), to_np(t))
    return w, saved, g, values, packed(dOv, dOt), gpu_kept(w, saved.kv_idx, saved.kv_cnt), packed


def held(name, got, want, bound):
    assert np.isfinite(got).all(), name
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert (err <= bound).all(), f"{name}: off by {err[worst]:.3e} at {worst}, bound {bound[worst]:.3e}; relative {rel:.2e}"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("normed", [False, True], ids=["plain", "normed"])
@pytest.mark.parametrize("name,ov", WORKLOADS, ids=IDS)
def test_gradients_of_the_softmax_over_the_values(cuda_ok, name, ov, normed, fmt):
    w, saved, g, values, dOp, kept, packed = chain(name, ov, fmt, normed)
    ref = oracle.attention_bwd(w, *values, dOp, kept)
    bounds, spread = backward_bounds(w, *values, dOp, kept)
    assert spread >= 3
    h = HALF[w.dtype]
    for i, n in enumerate("qkv"):
        want, bound = ref[i], bounds[i] + h * np.abs(ref[i])
        if i < 2 and normed:
            _, kept_x, rstd, weight = saved.norms[i]
            X = to_np(S.ssta_checkpoint_load(kept_x)).reshape(-1, w.D)
            rstd, weight = to_np(rstd).reshape(-1), to_np(weight)
            grad, bound = want.reshape(-1, w.D), bound.reshape(-1, w.D)
            dx, dweight, _, _ = oracle.norm_bwd(grad, X, None, rstd, "rms", weight)
            xh = np.abs(X) * rstd[:, None]
            through = lambda t: rstd[:, None] * (t + xh * (t * xh).mean(axis=1, keepdims=True))
            bw = (bound * xh).sum(axis=0) + U * (len(X) + K) * (np.abs(grad) * xh).sum(axis=0)
            held(f"d{n}_weight", to_np(g[f"d{n}_weight"]), dweight, bw)
            bound = through(bound * np.abs(weight) + 4 * K * U * np.abs(grad * weight)) + h * np.abs(dx)
            want, bound = dx.reshape(ref[i].shape), bound.reshape(ref[i].shape)
        # pad rows: zero in the oracle's packing of the result and in the reference alike
        held("d" + n, packed(g["d" + n], g[f"d{n}_text"]), want, bound)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name,ov", WORKLOADS, ids=IDS)
def test_probabilities_sum_to_one(cuda_ok, name, ov, fmt):
    """With dO one in channel c of row i and zero elsewhere, channel c of dv summed over the keys is the sum of
    row i of P: 128 rows of every head at once."""
    def one_hot(w, t, text):
        n = w.T * w.Y * w.X
        rows = np.linspace(0, n - 1, w.D).astype(int)
        v = torch.zeros((w.B, w.H, n, w.D), dtype=t.dtype, device=t.device)
        v[:, :, torch.from_numpy(rows).cuda(), torch.arange(w.D, device="cuda")] = 1
        return v.view(t.shape), None if text is None else torch.zeros_like(text)

    w, saved, g, values, dOp, kept, packed = chain(name, ov, fmt, True, one_hot)
    bounds, _ = backward_bounds(w, *values, dOp, kept)
    dv = packed(g["dv"], g["dv_text"])
    bound = (bounds[2] + HALF[w.dtype] * np.abs(dv)).sum(axis=2)
    sums = dv.sum(axis=2)
    assert (np.abs(sums - 1) <= bound).all(), (sums.min(), sums.max(), bound.max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name,ov", WORKLOADS[1:3], ids=IDS[1:3])
def test_an_infinity_stays_visible(cuda_ok, name, ov, fmt):
    """An infinity in v (a group that reads as NaN) leaves NaN in the gradients of every row that keeps it, and the
    other heads as they were (the lists are those of q and k)."""
    want = chain(name, ov, fmt, False)[2]

    def put(x):
        x["v"][0, 0, 1, 2, 3, 4] = float("inf")

    g = chain(name, ov, fmt, False, edit=put)[2]
    assert torch.isnan(g["dq"][0, 0, 1, 2, 3]).any() and torch.isnan(g["dk"][0, 0, 1, 2, 3]).any()
    for n in "qkv":
        assert torch.equal(g["d" + n][:, 1], want["d" + n][:, 1])


def test_status_covers_the_recomputed_attention(cuda_ok, monkeypatch):
    """A device status that only the attention over the values reports reaches the workspace that is returned."""
    forward = S.ssta_attention_fwd

    def late(*args, **kw):
        o, lse, ws = forward(*args, **kw)
        ws[:4].view(torch.int32).fill_(6)
        return o, lse, ws

    w = with_overrides(si.get_workload("tiny_f32"), L_text=5)
    d = S.desc_from(w)
    x = si.make_inputs(w, 0, device="cuda")
    r = S.ssta_forward(d, *(x[n] for n in ("q", "k", "v", "q_text", "k_text", "v_text")), checkpoint="int8")
    assert r["saved"].lse is None and r["LSE"] is not None
    monkeypatch.setattr(S, "ssta_attention_fwd", late)
    assert S.ssta_read_device_status(S.ssta_backward(d, r["saved"], x["q"], x["q_text"])["workspace"]) == 6
    monkeypatch.undo()
    assert S.ssta_read_device_status(S.ssta_backward(d, r["saved"], x["q"], x["q_text"])["workspace"]) == 0
