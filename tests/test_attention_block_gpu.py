"""The operators together, as a transformer's training runs them: ssta_forward with head
norms and 8-bit checkpoints, ssta_backward, and the attention sub-block, against torch's
autograd on the CPU in float64 with the GPU forward's kept lists as constants.

Tolerances (relative L2 of each whole gradient).  fp32: 1e-4, the bound of the attention
backward alone; the norms and projections around it add a few u = 2^-24 each.  bf16: every
tensor between two operators is rounded to 2^-9 relative (root mean square about 2^-10.8),
about 20 of them in a row, forward and backward, with attention's own 1e-2 on top: 5e-2.
Checkpoints: a code is off by at most max|group| / 127.5 (int8; about 1.6 % of the root mean
square of a normal group, uniformly distributed) or 2^-4 (e4m3; 3 %), in up to 9 tensors of
a gradient's formula: 3 times that, 5e-2 and 1e-1, on top of the type's own."""
import numpy as np
import pytest
import torch

import block_sparse_video_ssta_b200 as S
import oracle
import ssta_inputs as si
from block_sparse_video_ssta_b200.attention_block import BlockWeights, ssta_block_backward, ssta_block_forward
from ssta_inputs import with_overrides
from ssta_parity import gpu_kept

pytestmark = pytest.mark.gpu

EPS = 1e-6
TOL = {"f32": 1e-4, "bf16": 5e-2}
SAVED = {None: 0.0, "int8": 5e-2, "e4m3": 1e-1}
WORKLOADS = [("tiny_f32", dict(T=3, Y=7, X=6, L_text=5, B=2)), ("tiny_f32", {}),
             ("small_bf16", dict(H=2, T=4, Y=12, X=10, L_text=40)), ("small_bf16", dict(H=1, T=4, Y=8, X=16, B=2))]


def token_tiles(w):
    """Tile of every token: video in raster order, then text."""
    n = w.T * w.Y * w.X
    g = oracle.geometry(w)
    ids = np.repeat(np.arange(n, dtype=np.float64).reshape(1, 1, w.T, w.Y, w.X, 1), w.D, axis=-1)
    ids = np.broadcast_to(ids, (w.B, w.H) + ids.shape[2:])
    packed = oracle.tile_reorder(w, ids, np.zeros((w.B, w.H, w.L_text, w.D)) if w.L_text else None)[0, 0, :, 0]
    tile = np.zeros(n + w.L_text, dtype=np.int64)
    rows = np.nonzero(oracle.valid_token_mask(w)[:g.NT * g.N])[0]
    tile[packed[rows].astype(np.int64)] = rows // g.N
    tile[n:] = g.NT + np.arange(w.L_text) // g.N
    return torch.from_numpy(tile)


def allowed(w, saved):
    """[B, H, L, L] pairs of tokens that the kept lists connect."""
    kept = torch.from_numpy(gpu_kept(w, saved.kv_idx, saved.kv_cnt))
    t = token_tiles(w)
    return kept[:, :, t][:, :, :, t]


def rms(x, weight):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def attend(q, k, v, mask):
    s = torch.where(mask, q @ k.transpose(-1, -2) / q.shape[-1] ** 0.5, float("-inf"))
    return torch.softmax(s, -1) @ v


def leaf(t):
    return None if t is None else t.detach().double().cpu().requires_grad_()


def close(name, got, want, tol):
    a, b = got.detach().double().cpu().reshape(want.shape), want.detach()
    assert torch.isfinite(a).all(), name
    rel = ((a - b).norm() / b.norm().clamp(min=1e-30)).item()
    assert rel <= tol, f"{name}: relative error {rel:.2e} > {tol:.0e}"


@pytest.mark.parametrize("checkpoint", [None, "int8", "e4m3"])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("name,ov", WORKLOADS, ids=[str(i) for i in range(len(WORKLOADS))])
def test_forward_and_backward_chain(cuda_ok, name, ov, normed, checkpoint):
    w = with_overrides(si.get_workload(name), **ov)
    d = S.desc_from(w)
    x = si.make_inputs(w, 5, device="cuda")
    gen = torch.Generator().manual_seed(3)
    weights = [(1 + 0.2 * torch.randn(w.D, generator=gen)).cuda() if normed else None for _ in range(2)]
    r = S.ssta_forward(d, x["q"], x["k"], x["v"], x["q_text"], x["k_text"], x["v_text"], q_weight=weights[0],
                       k_weight=weights[1], norm_eps=EPS, checkpoint=checkpoint)
    assert (r["qp"] is None) == (checkpoint is not None)
    if not normed:
        plain = S.ssta_forward(d, x["q"], x["k"], x["v"], x["q_text"], x["k_text"], x["v_text"])
        assert torch.equal(plain["O"], r["O"]) and torch.equal(plain["kv_idx"], r["kv_idx"])
    n = w.T * w.Y * w.X
    cat = lambda v, t: v.reshape(w.B, w.H, n, w.D) if t is None else torch.cat([v.reshape(w.B, w.H, n, w.D), t], 2)
    leaves = {m: leaf(cat(x[m], x[m + "_text"])) for m in "qkv"}
    lw = [leaf(t) for t in weights]
    mask = allowed(w, r["saved"])
    O = attend(rms(leaves["q"], lw[0]), rms(leaves["k"], lw[1]), leaves["v"], mask)
    close("O", cat(r["O"], r["O_text"]), O, TOL[w.dtype])
    dO = torch.randn(O.shape, generator=gen).to(r["O"].dtype)
    O.backward(dO.double())
    dOg = dO.cuda()
    g = S.ssta_backward(d, r["saved"], dOg[:, :, :n].reshape(r["O"].shape).contiguous(),
                        dOg[:, :, n:].contiguous() if w.L_text else None)
    assert S.ssta_read_device_status(g["workspace"]) == 0
    tol = TOL[w.dtype] + SAVED[checkpoint]
    for m in "qkv":
        close("d" + m, cat(g["d" + m], g["d" + m + "_text"]), leaves[m].grad, tol)
    for m, t in zip("qk", lw):
        if t is None:
            assert g[f"d{m}_weight"] is None
        else:
            close(f"d{m}_weight", g[f"d{m}_weight"], t.grad, tol)


def test_one_tensor_for_q_k_and_v(cuda_ok):
    """The same tensor passed three times: its head norms and gradients stay apart."""
    w = with_overrides(si.get_workload("tiny_f32"), T=3, Y=7, X=6)
    d = S.desc_from(w)
    x = si.make_inputs(w, 5, device="cuda")["q"]
    weight = torch.linspace(0.5, 1.5, w.D, device="cuda")
    for checkpoint in (None, "int8"):
        a, b = (S.ssta_forward(d, x, y, z, q_weight=weight, checkpoint=checkpoint) for y, z in ((x, x), (x.clone(), x.clone())))
        assert torch.equal(a["O"], b["O"])
        ga, gb = (S.ssta_backward(d, r["saved"], x) for r in (a, b))
        for n in ("dq", "dk", "dv", "dq_weight"):
            assert torch.equal(ga[n], gb[n]), n
        assert ga["dk_weight"] is None


def test_chain_refusals(cuda_ok):
    w = with_overrides(si.get_workload("tiny_f32"), L_text=5)
    d = S.desc_from(w)
    x = si.make_inputs(w, 0, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "q_text", "k_text", "v_text")]
    weight = torch.ones(w.D, device="cuda")
    for kw in (dict(q_weight=weight.half()), dict(q_weight=weight[:64]), dict(k_weight=weight.cpu()), dict(checkpoint="fp8")):
        with pytest.raises(ValueError):
            S.ssta_forward(d, *args, **kw)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.ssta_forward(d, *(t.cpu() for t in args), checkpoint="int8")
    r = S.ssta_forward(d, *args, checkpoint="int8")
    with pytest.raises(ValueError):
        S.ssta_backward(d, r["saved"], x["q"])            # text gradient missing
    with pytest.raises(ValueError):
        S.ssta_backward(d, r["saved"], x["q"].bfloat16(), x["q_text"].bfloat16())


def block_inputs(w, seed=0, normed=True):
    C, L = w.H * w.D, w.T * w.Y * w.X + w.L_text
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    n = lambda *s: torch.randn(s, generator=gen)
    x = n(w.B, L, C).to(dt).cuda()
    mod = (0.3 * n(w.B, 5, C)).cuda()
    weights = BlockWeights((n(3 * C, C) / C ** 0.5).to(dt).cuda(), (n(C, C) / C ** 0.5).to(dt).cuda(),
                           (1 + 0.2 * n(w.D)).cuda() if normed else None, (1 + 0.2 * n(w.D)).cuda() if normed else None)
    return x, mod, weights, n(w.B, L, C).to(dt).cuda(), n(w.B, L, C).to(dt).cuda()


def block_reference(w, x, mod, p, mask):
    ln = lambda t: torch.nn.functional.layer_norm(t, t.shape[-1:], eps=EPS)
    shift, scale, gate, shift2, scale2 = (mod[:, i:i + 1] for i in range(5))
    n1 = ln(x) * (1 + scale) + shift
    heads = lambda t: t.view(w.B, -1, w.H, w.D).transpose(1, 2)
    q, k, v = (heads(t) for t in (n1 @ p.qkv.T).chunk(3, -1))
    o = attend(rms(q, p.q_norm), rms(k, p.k_norm), v, mask)
    r = x + gate * (o.transpose(1, 2).reshape(x.shape) @ p.out.T)
    return r, ln(r) * (1 + scale2) + shift2


@pytest.mark.parametrize("checkpoint", [None, "int8", "e4m3"])
@pytest.mark.parametrize("name,ov", WORKLOADS, ids=[str(i) for i in range(len(WORKLOADS))])
def test_block_forward_and_backward(cuda_ok, name, ov, checkpoint):
    w = with_overrides(si.get_workload(name), **ov)
    d = S.desc_from(w)
    x, mod, p, dr, dn = block_inputs(w)
    r, n2, saved = ssta_block_forward(d, x, mod, p, checkpoint)
    leaves = [leaf(t) for t in (x, mod, p.qkv, p.out, p.q_norm, p.k_norm)]
    R, N = block_reference(w, leaves[0], leaves[1], BlockWeights(*leaves[2:]), allowed(w, saved.attention))
    close("r", r, R, TOL[w.dtype])
    close("n2", n2, N, TOL[w.dtype])
    ((R * dr.double().cpu()).sum() + (N * dn.double().cpu()).sum()).backward()
    g = ssta_block_backward(d, saved, p, dr, dn)
    tol = TOL[w.dtype] + SAVED[checkpoint]
    for name, got, t in zip(("dx", "dmod", "dqkv", "dout", "dq_norm", "dk_norm"),
                            (g.dx, g.dmod, g.dqkv, g.dout, g.dq_norm, g.dk_norm), leaves):
        close(name, got, t.grad, tol)


def test_block_captured_and_on_a_stream(cuda_ok):
    """Forward and backward in one graph, replayed on other inputs, and on a side stream: the bytes of eager calls."""
    w = with_overrides(si.get_workload("small_bf16"), H=2, T=4, Y=12, X=10, L_text=40)
    d = S.desc_from(w)
    x, mod, p, dr, dn = block_inputs(w, 1)

    def step(**kw):
        r, n2, saved = ssta_block_forward(d, x, mod, p, "int8", **kw)
        g = ssta_block_backward(d, saved, p, dr, dn, **kw)
        return [r, n2, g.dx, g.dmod, g.dqkv, g.dout, g.dq_norm, g.dk_norm]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        x.copy_(x.roll(1, 1))
        graph.replay()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_parameters_that_require_gradients(cuda_ok):
    """nn.Parameters and leaves as arguments: the same bytes, and nothing recorded by autograd."""
    w = with_overrides(si.get_workload("small_bf16"), H=1, T=4, Y=8, X=16)
    d = S.desc_from(w)
    x, mod, p, dr, dn = block_inputs(w)
    param = torch.nn.Parameter
    q = BlockWeights(param(p.qkv), param(p.out), param(p.q_norm), param(p.k_norm))
    for checkpoint in (None, "int8"):
        a, b = (ssta_block_forward(d, xx, mod, pp, checkpoint) for xx, pp in ((x, p), (x.clone().requires_grad_(), q)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and not b[0].requires_grad and not b[1].requires_grad
        ga, gb = ssta_block_backward(d, a[2], p, dr, dn), ssta_block_backward(d, b[2], q, dr, dn)
        for n in ("dx", "dmod", "dqkv", "dout", "dq_norm", "dk_norm"):
            assert torch.equal(getattr(ga, n), getattr(gb, n)) and not getattr(gb, n).requires_grad, n


def test_checkpoints_halve_what_is_kept(cuda_ok):
    w = with_overrides(si.get_workload("small_bf16"), H=2, T=8, Y=16, X=24)
    d = S.desc_from(w)
    x, mod, p, _, _ = block_inputs(w)

    def kept(saved):
        a = saved.attention
        parts = [saved.x, saved.y, saved.r, a.q, a.k, a.v, a.o] + [n[1] for n in a.norms]
        return sum(t.nbytes for t in parts)

    dense, small = (kept(ssta_block_forward(d, x, mod, p, c)[2]) for c in (None, "int8"))
    assert small <= 0.505 * dense    # one byte of two, and one exponent per 128


def test_block_refusals(cuda_ok):
    w = with_overrides(si.get_workload("small_bf16"), H=2, T=4, Y=8, X=8)
    d = S.desc_from(w)
    x, mod, p, dr, dn = block_inputs(w)
    bad = [(x[:, 1:], mod, p), (x, mod[:, :4], p), (x, mod, BlockWeights(p.out, p.out)), (x, mod, BlockWeights(p.qkv, p.qkv)),
           (x, mod.half(), p), (x.transpose(0, 1).contiguous().transpose(0, 1)[:, ::1], mod, BlockWeights(p.qkv.float(), p.out))]
    for args in bad:
        with pytest.raises(ValueError):
            ssta_block_forward(d, *args)
    with pytest.raises(ValueError):
        ssta_block_forward(d, x, mod, p, "int4")
    r, n2, saved = ssta_block_forward(d, x, mod, p, "int8")
    with pytest.raises(ValueError):
        ssta_block_backward(d, saved, p, dr[:, 1:], dn)
    for a, b in ((dr, None), (None, dn), (dr, dn[:, 1:])):
        with pytest.raises(ValueError):
            ssta_block_backward(d, saved, p, a, b)
