"""Workloads of the operators around the attention in a transformer block: the norm with modulation before
it, the gated residual with the next norm after it, the 8-bit checkpoints that training keeps, and the
backward passes that read them.

``run`` computes one pass, in plain torch operations (``own`` false) or through the library (``own`` true),
on the state ``prepare`` made; ``exact`` gives the same results from the definitions in float64.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 128          # channels sharing one checkpoint exponent
HEAD_DIM = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases

def _rows_case(op, name, rows, C, **kw):
    """A case on [rows, C]; mod_rows 0 = one modulation row for all rows."""
    case = dict(op=op, name=name, rows=rows, C=C, dtype="bf16", param_dtype="f32", norm="layer", post_norm="none",
                weight=False, mod=True, mod_rows=0, save="none", dres=False, res_scale=1.0)
    case.update(kw)
    return case


def _attn_case(name, H, grid, tile, window, topk, L_text, **kw):
    case = dict(op="attention_bwd", name=name, H=H, T=grid[0], Y=grid[1], X=grid[2], tT=tile[0], tY=tile[1],
                tX=tile[2], wT=window[0], wY=window[1], wX=window[2], topk=topk, L_text=L_text, dtype="bf16",
                save="int8")
    case.update(kw)
    return case


def listed():
    return [
        # the text stream's adaptive LayerNorm: 256 tokens, latency counts
        _rows_case("norm_fwd", "norm_fwd_text", 256, 2048),
        # RMS norm of q (or k) per head before the attention, 16 heads of the 720p 5 s latent
        _rows_case("norm_fwd", "norm_fwd_heads_720p_5s", 16 * 111600, 128, norm="rms", weight=True, mod=False),
        # backward of the text stream's norm
        _rows_case("norm_bwd", "norm_bwd_text", 256, 2048, param_dtype="bf16", dres=True),
        # fp32 training of a narrower model with one modulation row per latent frame (480p: 30 x 53 tokens)
        _rows_case("norm_bwd", "norm_bwd_frames_480p", 49290, 1544, dtype="f32", weight=True, mod_rows=1590, dres=True),
        # a short prompt between two sub-blocks, inference
        _rows_case("residual_fwd", "residual_fwd_prompt", 77, 2048, param_dtype="bf16"),
        # video stream of the 720p 5 s latent between attention and MLP, training: both inputs of the backward kept
        _rows_case("residual_fwd", "residual_fwd_720p_5s", 111600, 2048, save="int8"),
        # sandwich norms, ragged row count and channels that are no multiple of the checkpoint group
        _rows_case("residual_bwd", "residual_bwd_sandwich", 12345, 1000, norm="rms", post_norm="rms", weight=True,
                   mod_rows=4115, save="e4m3", res_scale=0.5, param_dtype="bf16"),
        # video stream of the 720p 10 s latent, backward from 8-bit checkpoints
        _rows_case("residual_bwd", "residual_bwd_720p_10s", 219600, 2048, save="int8"),
        # checkpoint of an odd fp32 activation, there and back
        _rows_case("checkpoint", "checkpoint_odd_f32", 4099, 1000, dtype="f32", save="e4m3"),
        # checkpoint of one activation of the 720p 10 s latent, there and back
        _rows_case("checkpoint", "checkpoint_720p_10s", 219600, 2048, save="int8"),
        # attention backward from checkpoints: a ragged grid with text
        _attn_case("attention_bwd_ragged", 3, (7, 12, 20), (4, 8, 8), (3, 3, 3), 6, 130, save="e4m3"),
        # attention backward from checkpoints: the 480p 5 s latent
        _attn_case("attention_bwd_480p_5s", 16, (31, 30, 53), (4, 8, 8), (3, 3, 3), 34, 0),
    ]


_LARGEST = {}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.5e12 + w["flops"] / 1.4e15


def draw(rng):
    if not _LARGEST:
        for c in listed():
            _LARGEST[c["op"]] = max(_LARGEST.get(c["op"], 0.0), _cost(c))
    op = rng.choice(("norm_fwd", "norm_bwd", "residual_fwd", "residual_bwd", "checkpoint", "attention_bwd"))
    while True:
        case = _draw_attention(rng) if op == "attention_bwd" else _draw_rows(rng, op)
        if _cost(case) <= _LARGEST[op]:
            return case


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rows(rng, op):
    rows = _log_int(rng, 1, 219600)
    C = 8 * _log_int(rng, 8, 512)
    if rng.random() < 0.3:
        C = HEAD_DIM * rng.choice((1, 8, 12, 16, 20, 32))
    case = _rows_case(op, "", rows, C, dtype=rng.choice(("bf16", "bf16", "f32")),
                      param_dtype=rng.choice(("bf16", "f32")), norm=rng.choice(("layer", "rms")),
                      weight=rng.random() < 0.5, mod=rng.random() < 0.75)
    del case["name"]
    if rng.random() < 0.5:
        case["mod_rows"] = -(-rows // rng.choice((1, 2, 3, 5, 8)))
    if op == "norm_bwd":
        case["dres"] = rng.random() < 0.5
    if op.startswith("residual"):
        case["post_norm"] = rng.choice(("none", "none", "layer", "rms"))
        case["res_scale"] = rng.choice((1.0, 1.0, 0.5))
    case["save"] = rng.choice(("int8", "e4m3") if op == "checkpoint" else ("none", "int8", "e4m3"))
    if op == "residual_fwd" and case["save"] != "none":
        # behind a post norm the stream's last bit depends on how a row is summed, and a code next to a border with it
        case["post_norm"] = "none"
    return case


def _draw_attention(rng):
    grid = (rng.randint(2, 31), rng.randint(5, 40), rng.randint(5, 60))
    tile = rng.choice(((4, 8, 8), (4, 8, 8), (2, 8, 8)))
    window = (rng.choice((1, 3)), rng.choice((1, 3)), rng.choice((1, 3, 5)))
    NT = math.prod(-(-n // t) for n, t in zip(grid, tile))
    case = _attn_case("", rng.choice((1, 2, 3, 4, 8, 16)), grid, tile, window,
                      rng.randint(0, max(1, NT // 6)), rng.choice((0, 0, 40, 130, 256)), save=rng.choice(("int8", "e4m3")))
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed, salt=0):
    return torch.Generator(device="cuda").manual_seed(seed * 1009 + salt)


def _normal(shape, gen, std=1.0, mean=0.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std + mean


def _activation(rows, C, gen, dtype):
    """A residual stream: unit normals, a per-channel offset, and a few channels far larger than the rest."""
    chan = torch.ones(C, device="cuda")
    pick = torch.randint(0, C, (max(1, C // 256),), generator=gen, device="cuda")
    chan[pick] = 5.0
    return (_normal((rows, C), gen) * chan + _normal((C,), gen, 0.2)).to(dtype)


def _mod_rows(case):
    return case["mod_rows"] or case["rows"]


def _inputs(case, seed):
    """The tensors of a [rows, C] case, from the seed alone."""
    gen, op = _gen(seed), case["op"]
    rows, C = case["rows"], case["C"]
    dt, pdt = DTYPES[case["dtype"]], DTYPES[case["param_dtype"]]
    G = -(-rows // _mod_rows(case))
    t = {"x": _activation(rows, C, gen, dt)}
    if op == "checkpoint":
        return t
    t["weight"] = _normal((C,), gen, 0.2, 1.0).to(pdt) if case["weight"] else None
    # the modulation comes as one row of several chunks per group, as a linear layer on the conditioning writes it
    mod = _normal((G, 6 * C), gen, 0.3).to(pdt) if case["mod"] else None
    t["shift"], t["scale"], t["gate"] = (mod[:, i * C:(i + 1) * C] if case["mod"] else None for i in range(3))
    if op == "norm_bwd":
        t["dy"] = _normal((rows, C), gen).to(dt)
        t["dres"] = _normal((rows, C), gen).to(dt) if case["dres"] else None
    if op.startswith("residual"):
        t["y"] = _normal((rows, C), gen, 1.5).to(dt)
        t["post_weight"] = _normal((C,), gen, 0.2, 1.0).to(pdt) if case["weight"] and case["post_norm"] != "none" else None
    if op == "residual_bwd":
        t["dr"] = _normal((rows, C), gen).to(dt)
        t["dn"] = _normal((rows, C), gen).to(dt)
    return t


def _stats(x, kind):
    """mean and 1/deviation of each row, as the forward saves them (float32)."""
    x = x.float()
    if kind == "layer":
        mean = x.mean(-1)
        var = ((x - mean[:, None]) ** 2).mean(-1)
        return mean, 1.0 / torch.sqrt(var + EPS)
    return None, 1.0 / torch.sqrt((x * x).mean(-1) + EPS)


def _power_of_two(e):
    """2^e in float32, exactly, from its exponent bits (-126 <= e <= 127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantize(x, fmt):
    """codes [rows, C] (int8 or float8_e4m3fn) and exponents [rows, ceil(C / 128)] (uint8) of a finite tensor."""
    rows, C = x.shape
    n = -(-C // GROUP)
    v = torch.zeros((rows, n * GROUP), device=x.device, dtype=torch.float32)
    v[:, :C] = x.float()
    v = v.view(rows, n, GROUP)
    m, e = torch.frexp(v.abs().amax(-1))                   # amax = m * 2^e, m in [0.5, 1)
    E = e + 127 - 7 + (m * 128 >= 127.5) if fmt == "int8" else e + 127 - 9 + (m * 512 > 448)
    E = torch.where(m > 0, E, 1).clamp(min=1)
    v = v * _power_of_two(127 - E)[..., None]
    codes = torch.round(v).to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)
    return codes.view(rows, n * GROUP)[:, :C].contiguous(), E.to(torch.uint8)


def _dequantize(codes, E):
    scale = _power_of_two(E.int() - 127)
    return codes.float() * scale.repeat_interleave(GROUP, dim=1)[:, :codes.shape[1]]


class _Geometry:
    """Tiles of the grid, the packed rows that hold a token, and the lists of kept tiles."""

    def __init__(self, case, seed):
        self.n = [-(-case[a] // case["t" + a]) for a in "TYX"]
        self.N = math.prod(case["t" + a] for a in "TYX")
        self.NT = math.prod(self.n)
        self.n_text = -(-case["L_text"] // self.N)
        self.NQ = self.NT + self.n_text
        self.L = self.NT * self.N + case["L_text"]
        ax = [torch.arange(n * case["t" + a]).view(n, -1) < case[a] for n, a in zip(self.n, "TYX")]
        v = (ax[0][:, None, None, :, None, None] & ax[1][None, :, None, None, :, None] & ax[2][None, None, :, None, None, :])
        self.valid = torch.cat([v.reshape(-1), torch.ones(case["L_text"], dtype=torch.bool)])
        # each video tile keeps a window around itself, topk tiles drawn by the seed, and the text; text keeps all
        axis = []
        for n, a in zip(self.n, "TYX"):
            w = min(case["w" + a], n)
            start = (torch.arange(n) - case["w" + a] // 2).clamp(0, n - w)
            j = torch.arange(n)
            axis.append((j[None] >= start[:, None]) & (j[None] < start[:, None] + w))
        win = (axis[0][:, None, None, :, None, None] & axis[1][None, :, None, None, :, None]
               & axis[2][None, None, :, None, None, :]).reshape(self.NT, self.NT)
        H = case["H"]
        gen = torch.Generator().manual_seed(seed + 77)
        kept = torch.zeros((H, self.NQ, self.NQ), dtype=torch.bool)
        k = min(case["topk"], self.NT)
        if k:
            order = torch.rand((H, self.NT, self.NT), generator=gen).argsort(-1)[..., :k]
            kept[:, :self.NT, :self.NT].scatter_(2, order, True)
        kept[:, :self.NT, :self.NT] |= win
        kept[:, :, self.NT:] = True
        kept[:, self.NT:, :] = True
        self.kept = kept
        self.cnt = kept.sum(-1).to(torch.int32)                                        # [H, NQ]
        self.max_kept = self.NQ if self.n_text else min(self.NT, k + int(win[0].sum()))
        idx = torch.where(kept, torch.arange(self.NQ), self.NQ).sort(-1).values[..., :self.max_kept]
        self.idx = torch.where(idx < self.NQ, idx, -1).to(torch.int32)


def _tiles(t, geo):
    """[H, L, ...] -> [H, NQ, N, ...], zero where the last text tile ends early."""
    pad = geo.NQ * geo.N - geo.L
    if pad:
        t = torch.cat([t, t.new_zeros((t.shape[0], pad) + tuple(t.shape[2:]))], 1)
    return t.view((t.shape[0], geo.NQ, geo.N) + tuple(t.shape[2:]))


def _attention_inputs(case, seed):
    geo = _Geometry(case, seed)
    gen, H = _gen(seed, 5), case["H"]
    valid = geo.valid.cuda()
    q, k, v = (_normal((H, geo.L, HEAD_DIM), gen) * valid[:, None] for _ in range(3))
    saved = {n: _quantize(t.bfloat16().view(-1, HEAD_DIM), case["save"]) for n, t in (("q", q), ("k", k), ("v", v))}
    qs, ks, vs = (_dequantize(*saved[n]).view(H, geo.L, HEAD_DIM) for n in "qkv")
    # O and LSE as a forward on these values returns them
    qt, kt, vt, ok = _tiles(qs, geo), _tiles(ks, geo), _tiles(vs, geo), _tiles(valid[None], geo)[0]
    head = torch.arange(H, device="cuda")[:, None]
    idx, cnt = geo.idx.cuda(), geo.cnt
    O = torch.empty((H, geo.NQ, geo.N, HEAD_DIM), device="cuda")
    lse = torch.empty((H, geo.NQ, geo.N), device="cuda")
    for i in range(geo.NQ):
        c = int(cnt[:, i].max())
        li = idx[:, i, :c].long()
        alive = (ok[li.clamp(min=0)] & (li >= 0)[..., None]).view(H, 1, -1)
        s = qt[:, i] @ kt[head, li.clamp(min=0)].view(H, -1, HEAD_DIM).transpose(1, 2) / math.sqrt(HEAD_DIM)
        s = torch.where(alive, s, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        O[:, i] = (p / z) @ vt[head, li.clamp(min=0)].view(H, -1, HEAD_DIM)
        lse[:, i] = (m + torch.log(z))[..., 0]
    O = O.view(H, -1, HEAD_DIM)[:, :geo.L].bfloat16()
    saved["o"] = _quantize(O.reshape(-1, HEAD_DIM), case["save"])
    dO = _normal((H, geo.L, HEAD_DIM), gen).bfloat16()
    return geo, saved, lse.view(H, -1)[:, :geo.L].contiguous(), dO


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "attention_bwd":
        geo, saved, lse, dO = _attention_inputs(case, seed)
        st.update(valid=geo.valid.cuda(), geo=geo, saved=saved, lse=lse[None], dO=dO[None],
                  kv_idx=geo.idx.cuda()[None].contiguous(), kv_cnt=geo.cnt.cuda()[None].contiguous())
        del geo.kept
        if own:
            import block_sparse_video_ssta_b200 as S
            st["desc"] = S.desc_from(B=1, D=HEAD_DIM, **{k: case[k] for k in (
                "H", "T", "Y", "X", "tT", "tY", "tX", "wT", "wY", "wX", "topk", "L_text", "dtype")})
            shape = (1, case["H"], geo.L, HEAD_DIM)
            st["ckpt"] = {n: S.Checkpoint(c.view(shape), e.view(shape[:3] + (1,)), torch.bfloat16)
                          for n, (c, e) in saved.items()}
        return st
    t = _inputs(case, seed)
    st.update(t)
    back = case["op"].endswith("_bwd")
    if case["op"] == "norm_bwd":
        st["mean"], st["rstd"] = _stats(t["x"], case["norm"])
        kept = ["x"]
    elif case["op"] == "residual_bwd":
        # x stands for the residual stream r after the block
        st["r"] = st.pop("x")
        st["mean"], st["rstd"] = _stats(st["r"], case["norm"])
        st["post_mean"], st["post_rstd"] = (None, None) if case["post_norm"] == "none" else _stats(t["y"], case["post_norm"])
        kept = ["r", "y"]
    if back and case["save"] != "none":
        for n in kept:
            codes, E = _quantize(st[n], case["save"])
            st[n + "_saved"] = (codes, E)
            if own:
                import block_sparse_video_ssta_b200 as S
                st[n] = S.Checkpoint(codes, E, DTYPES[case["dtype"]])
            else:
                st[n] = None
    if own and case["op"] != "checkpoint":
        import block_sparse_video_ssta_b200 as S
        st["desc"] = S.norm_desc(case["rows"], case["C"], dtype=case["dtype"], param_dtype=case["param_dtype"],
                                 norm=case["norm"], post_norm=case["post_norm"], eps=EPS, res_scale=case["res_scale"],
                                 mod_rows=case["mod_rows"], mod_stride=6 * case["C"])
    return st


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "residual_fwd": _plain_residual_fwd,
            "residual_bwd": _plain_residual_bwd, "checkpoint": _plain_checkpoint,
            "attention_bwd": _plain_attention_bwd}[op](state)


def _run_own(st):
    import block_sparse_video_ssta_b200 as S
    case = st["case"]
    op, save = case["op"], None if case["save"] == "none" else case["save"]
    if op == "norm_fwd":
        y, mean, rstd, saved = S.ssta_norm_fwd(st["desc"], st["x"], st["weight"], st["scale"], st["shift"], save=save)
        return _present(y, mean, rstd, S.ssta_checkpoint_load(saved) if save else None)
    if op == "norm_bwd":
        g = S.ssta_norm_bwd(st["desc"], st["dy"], st["x"], st["mean"], st["rstd"], st["weight"], st["scale"], st["dres"])
        return _present(g.dx, g.dweight, g.dscale, g.dshift)
    if op == "residual_fwd":
        f = S.ssta_residual_norm_fwd(st["desc"], st["x"], st["y"], st["post_weight"], st["gate"], st["weight"],
                                     st["scale"], st["shift"], save_y=save, save_r=save)
        return _present(f.r, f.n, f.post_mean, f.post_rstd, f.mean, f.rstd,
                        S.ssta_checkpoint_load(f.saved_y) if save else None,
                        S.ssta_checkpoint_load(f.saved_r) if save else None)
    if op == "residual_bwd":
        g = S.ssta_residual_norm_bwd(st["desc"], st["dr"], st["dn"], st["r"], st["y"], st["mean"], st["rstd"],
                                     st["post_mean"], st["post_rstd"], st["post_weight"], st["gate"], st["weight"],
                                     st["scale"])
        return _present(g.dx, g.dy, g.dpost_weight, g.dgate, g.dweight, g.dscale, g.dshift)
    if op == "checkpoint":
        return [S.ssta_checkpoint_load(S.ssta_checkpoint_save(st["x"], save))]
    c = st["ckpt"]
    dq, dk, dv, _ = S.ssta_attention_bwd_checkpoint(st["desc"], c["q"], c["k"], c["v"], c["o"], st["lse"], st["dO"],
                                                    st["kv_idx"], st["kv_cnt"])
    return [dq, dk, dv]


def _present(*outs):
    return [o for o in outs if o is not None]


def _per_row(v, st):
    """A modulation [G, C] as float32 rows, or None."""
    if v is None:
        return None
    v = v.float()
    return v if v.shape[0] == 1 else v[torch.arange(st["case"]["rows"], device=v.device) // _mod_rows(st["case"])]


def _group_sum(t, case):
    """Sum [rows, C] over the rows of each modulation group -> [G, C]."""
    m, rows = _mod_rows(case), case["rows"]
    whole = rows // m
    out = t[:whole * m].view(whole, m, -1).sum(1)
    return out if whole * m == rows else torch.cat([out, t[whole * m:].sum(0, keepdim=True)])


def _plain_norm(x, kind):
    """(normalised x, mean, rstd) in float32."""
    mean, rstd = _stats(x, kind)
    return (x if mean is None else x - mean[:, None]) * rstd[:, None], mean, rstd


def _plain_modulate(xh, st):
    if st["weight"] is not None:
        xh = xh * st["weight"].float()
    if st["scale"] is not None:
        xh = xh * (1.0 + _per_row(st["scale"], st)) + _per_row(st["shift"], st)
    return xh


def _plain_saved(x, case):
    return None if case["save"] == "none" else _dequantize(*_quantize(x, case["save"])).to(DTYPES[case["dtype"]])


def _plain_norm_fwd(st):
    case = st["case"]
    xh, mean, rstd = _plain_norm(st["x"].float(), case["norm"])
    y = _plain_modulate(xh, st).to(st["x"].dtype)
    return _present(y, mean, rstd, _plain_saved(st["x"], case))


def _plain_residual_fwd(st):
    case, dt = st["case"], st["x"].dtype
    y = st["y"].float()
    post_mean = post_rstd = None
    h = y
    if case["post_norm"] != "none":
        h, post_mean, post_rstd = _plain_norm(y, case["post_norm"])
        if st["post_weight"] is not None:
            h = h * st["post_weight"].float()
    if st["gate"] is not None:
        h = h * _per_row(st["gate"], st)
    r = case["res_scale"] * st["x"].float() + h
    rh, mean, rstd = _plain_norm(r, case["norm"])
    n = _plain_modulate(rh, st).to(dt)
    r = r.to(dt)
    return _present(r, n, post_mean, post_rstd, mean, rstd, _plain_saved(st["y"], case), _plain_saved(r, case))


def _kept_value(st, name):
    """A tensor the backward reads, as float32: dense, or the values of its checkpoint."""
    return _dequantize(*st[name + "_saved"]) if name + "_saved" in st else st[name].float()


def _plain_norm_grad(xh, g, rstd, kind):
    """Gradient through the normalisation alone."""
    c = g - xh * (g * xh).mean(-1, keepdim=True)
    if kind == "layer":
        c = c - g.mean(-1, keepdim=True)
    return c * rstd[:, None]


def _plain_vector_grads(dy, xh, st):
    """(g = dy through weight and modulation, dweight, dscale, dshift)."""
    case = st["case"]
    g = dy
    dweight = dscale = dshift = None
    s2 = _group_sum(dy * xh, case) if st["weight"] is not None or st["scale"] is not None else None
    if st["scale"] is not None:
        dshift = _group_sum(dy, case)
        dscale = s2 if st["weight"] is None else s2 * st["weight"].float()
        g = g * (1.0 + _per_row(st["scale"], st))
    if st["weight"] is not None:
        dweight = (s2 if st["scale"] is None else s2 * (1.0 + st["scale"].float())).sum(0)
        g = g * st["weight"].float()
    return g, dweight, dscale, dshift


def _plain_norm_bwd(st):
    case = st["case"]
    x = _kept_value(st, "x")
    xh = (x if st["mean"] is None else x - st["mean"][:, None]) * st["rstd"][:, None]
    g, dweight, dscale, dshift = _plain_vector_grads(st["dy"].float(), xh, st)
    dx = _plain_norm_grad(xh, g, st["rstd"], case["norm"])
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return _present(dx.to(st["dy"].dtype), dweight, dscale, dshift)


def _plain_residual_bwd(st):
    case, dt = st["case"], st["dr"].dtype
    r = _kept_value(st, "r")
    rh = (r if st["mean"] is None else r - st["mean"][:, None]) * st["rstd"][:, None]
    g, dweight, dscale, dshift = _plain_vector_grads(st["dn"].float(), rh, st)
    dR = st["dr"].float() + _plain_norm_grad(rh, g, st["rstd"], case["norm"])
    dx = (case["res_scale"] * dR).to(dt)
    y = _kept_value(st, "y")
    yh = y
    if case["post_norm"] != "none":
        yh = (y if st["post_mean"] is None else y - st["post_mean"][:, None]) * st["post_rstd"][:, None]
    pw = None if st["post_weight"] is None else st["post_weight"].float()
    dgate = dpw = None
    dh = dR
    if st["gate"] is not None:
        s3 = _group_sum(dR * yh, case)
        dgate = s3 if pw is None else s3 * pw
        dpw = None if pw is None else (s3 * st["gate"].float()).sum(0)
        dh = dh * _per_row(st["gate"], st)
    elif pw is not None:
        dpw = (dR * yh).sum(0)
    if pw is not None:
        dh = dh * pw
    dy = dh if case["post_norm"] == "none" else _plain_norm_grad(yh, dh, st["post_rstd"], case["post_norm"])
    return _present(dx, dy.to(dt), dpw, dgate, dweight, dscale, dshift)


def _plain_checkpoint(st):
    return [_plain_saved(st["x"], st["case"])]


def _plain_attention_bwd(st):
    geo, H = st["geo"], st["case"]["H"]
    scale = 1.0 / math.sqrt(HEAD_DIM)
    q, k, v, o = (_tiles(_dequantize(*st["saved"][n]).view(H, geo.L, HEAD_DIM), geo) for n in "qkvo")
    dO, lse = _tiles(st["dO"][0].float(), geo), _tiles(st["lse"][0], geo)
    ok = _tiles(st["valid"][None], geo)[0]                                              # [NQ, N]
    D = (dO * o).sum(-1)
    head = torch.arange(H, device="cuda")[:, None]
    dq = torch.zeros_like(q)
    dk, dv = (torch.zeros((H, geo.NQ + 1) + tuple(q.shape[2:]), device="cuda") for _ in range(2))
    for i in range(geo.NQ):
        c = int(geo.cnt[:, i].max())
        li = st["kv_idx"][0, :, i, :c].long()
        src, dst = li.clamp(min=0), torch.where(li >= 0, li, geo.NQ)
        alive = (ok[src] & (li >= 0)[..., None]).view(H, 1, -1) & ok[i][None, :, None]
        ki, vi = k[head, src].view(H, -1, HEAD_DIM), v[head, src].view(H, -1, HEAD_DIM)
        s = (q[:, i] @ ki.transpose(1, 2)) * scale
        p = torch.where(alive, torch.exp(s - lse[:, i, :, None]), 0.0)
        ds = p * (dO[:, i] @ vi.transpose(1, 2) - D[:, i, :, None])
        dq[:, i] = (ds @ ki) * scale
        # a list names a tile once; its entries past the count all go to the spare tile at the end
        dk[head, dst] += ((ds.transpose(1, 2) @ q[:, i]) * scale).view(H, c, geo.N, HEAD_DIM)
        dv[head, dst] += (p.transpose(1, 2) @ dO[:, i]).view(H, c, geo.N, HEAD_DIM)
    out = (t[:, :geo.NQ].reshape(H, -1, HEAD_DIM)[None, :, :geo.L] for t in (dq, dk, dv))
    return [t.bfloat16() for t in out]


# ---------------------------------------------------------------------------------------------- cost

def work(case):
    if case["op"] == "attention_bwd":
        NT = math.prod(-(-case[a] // case["t" + a]) for a in "TYX")
        N = math.prod(case["t" + a] for a in "TYX")
        tokens = case["T"] * case["Y"] * case["X"]
        win = math.prod(min(case["w" + a], -(-case[a] // case["t" + a])) for a in "TYX")
        k = min(case["topk"], NT)
        kept = win + k * (1.0 - win / NT)                     # drawn tiles fall on the window in proportion
        L, Lt, H = NT * N + case["L_text"], case["L_text"], case["H"]
        pairs = tokens * (kept / NT * tokens + Lt) + Lt * (tokens + Lt)
        # read the codes of q, k, v, O, the rows' LSE and dO; write dq, dk, dv
        return {"bytes": H * L * (4 * (HEAD_DIM + 1) + 4 + 2 * HEAD_DIM + 3 * 2 * HEAD_DIM),
                "flops": int(H * pairs * 10 * HEAD_DIM)}
    rows, C, op = case["rows"], case["C"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    n, saved = rows * C, case["save"] != "none"
    code = 1.0 + 1.0 / GROUP
    kept = code if saved else e
    back = {"norm_fwd": 2 * e + saved * (2 * code + e), "residual_fwd": 4 * e + saved * 2 * (2 * code + e),
            "norm_bwd": 2 * e + kept + case["dres"] * e, "residual_bwd": 4 * e + 2 * kept,
            "checkpoint": 2 * e + 2 * code}[op]
    flops = {"norm_fwd": 8, "residual_fwd": 12, "norm_bwd": 14, "residual_bwd": 22, "checkpoint": 4}[op]
    return {"bytes": int(n * back) + rows * 8, "flops": n * flops}


# ---------------------------------------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    return _exact_attention(case, seed) if case["op"] == "attention_bwd" else _exact_rows(case, seed)


def _exact_roundtrip(x, fmt):
    """Nearest representable multiple of a group's power of two, ties to even."""
    limit = 127.5 if fmt == "int8" else 448.0

    def two_to(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c0 in range(0, x.shape[1], GROUP):
        v = x[:, c0:c0 + GROUP].double()
        a = v.abs().amax(1, keepdim=True)
        E = torch.frexp(torch.where(a > 0, a, 2.0 ** -200))[1] - 12
        for _ in range(9):                                   # up to the smallest E that fits
            fits = a * two_to(-E) < limit if fmt == "int8" else a * two_to(-E) <= limit
            E = torch.where(fits, E, E + 1)
        E = E.clamp(min=-126)
        u = v * two_to(-E)
        # the spacing of the codes at u: 1, or eight steps per binade and 2^-9 below the smallest normal
        q = torch.ones_like(u) if fmt == "int8" else two_to((torch.frexp(u)[1] - 4).clamp(min=-9))
        out[:, c0:c0 + GROUP] = torch.round(u / q) * q * two_to(E)
    return out


def _exact_rows(case, seed):
    t = _inputs(case, seed)
    op, save = case["op"], case["save"]
    dtype = DTYPES[case["dtype"]]
    if op == "checkpoint":
        return [_exact_roundtrip(t["x"], save)]
    rows, m = case["rows"], _mod_rows(case)
    group = torch.arange(rows, device="cuda") // m
    G = int(group[-1]) + 1
    vec = {n: None if t.get(n) is None else t[n].double() for n in ("weight", "post_weight", "scale", "shift", "gate")}

    def spread(name):
        return vec[name].index_select(0, group)

    def moments(z, kind):
        mu = z.sum(1) / z.shape[1] if kind == "layer" else None
        c = z if mu is None else z - mu[:, None]
        return mu, ((c * c).sum(1) / z.shape[1] + EPS) ** -0.5

    def standard(z, mu, rs):
        return rs[:, None] * (z if mu is None else z - mu[:, None])

    def modulated(z):
        if vec["weight"] is not None:
            z = vec["weight"] * z
        if vec["scale"] is not None:
            z = z + z * spread("scale") + spread("shift")
        return z

    def by_group(z):
        return torch.zeros((G, z.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, group, z)

    def through(zh, grad, rs, kind):
        n = zh.shape[1]
        out = n * grad - zh * (zh * grad).sum(1, keepdim=True)
        if kind == "layer":
            out = out - grad.sum(1, keepdim=True)
        return out * (rs / n)[:, None]

    x = t["x"].double()
    saved = lambda z: _exact_roundtrip(z, save) if save != "none" else None
    if op == "norm_fwd":
        mu, rs = moments(x, case["norm"])
        return _present(modulated(standard(x, mu, rs)), mu, rs, saved(t["x"]))
    if op == "residual_fwd":
        y = t["y"].double()
        pm = pr = None
        h = y
        if case["post_norm"] != "none":
            pm, pr = moments(y, case["post_norm"])
            h = standard(y, pm, pr)
            if vec["post_weight"] is not None:
                h = h * vec["post_weight"]
        r = case["res_scale"] * x + (h if vec["gate"] is None else spread("gate") * h)
        mu, rs = moments(r, case["norm"])
        outs = [r, modulated(standard(r, mu, rs)), pm, pr, mu, rs]
        # the checkpoint of r holds its stored, rounded values: a value next to a border has no exact answer
        kept = [o for o in outs if o is not None]
        return kept + ([saved(t["y"]), None] if save != "none" else [])

    # the backward's statistics are inputs, float32 as the forward stores them
    def given(z, kind):
        mu, rs = _stats(z, kind)
        return None if mu is None else mu.double(), rs.double()

    def pulled_back(dy, zh):
        grad = dy
        dw = ds = db = None
        prod = by_group(dy * zh)
        if vec["scale"] is not None:
            db, ds = by_group(dy), prod
            if vec["weight"] is not None:
                ds = ds * vec["weight"]
            grad = grad + grad * spread("scale")
        if vec["weight"] is not None:
            dw = (prod * (1 if vec["scale"] is None else 1 + vec["scale"])).sum(0)
            grad = grad * vec["weight"]
        return grad, dw, ds, db

    mu, rs = given(t["x"], case["norm"])
    z = x if save == "none" else _exact_roundtrip(t["x"], save)
    zh = standard(z, mu, rs)
    if op == "norm_bwd":
        grad, dw, ds, db = pulled_back(t["dy"].double(), zh)
        dx = through(zh, grad, rs, case["norm"])
        return _present(dx if t["dres"] is None else dx + t["dres"].double(), dw, ds, db)
    grad, dw, ds, db = pulled_back(t["dn"].double(), zh)
    dR = t["dr"].double() + through(zh, grad, rs, case["norm"])
    del grad, zh, z
    y = t["y"].double() if save == "none" else _exact_roundtrip(t["y"], save)
    yh = y
    if case["post_norm"] != "none":
        pm, pr = given(t["y"], case["post_norm"])
        yh = standard(y, pm, pr)
    prod = by_group(dR * yh)
    dgate = dpw = None
    dh = dR
    if vec["gate"] is not None:
        dgate = prod if vec["post_weight"] is None else prod * vec["post_weight"]
        dh = dh * spread("gate")
    if vec["post_weight"] is not None:
        dpw = (prod if vec["gate"] is None else prod * vec["gate"]).sum(0)
        dh = dh * vec["post_weight"]
    dy = dh if case["post_norm"] == "none" else through(yh, dh, pr, case["post_norm"])
    return _present(case["res_scale"] * dR, dy, dpw, dgate, dw, ds, db)


def _exact_attention(case, seed):
    """Dense rows against all keys with the kept tiles as a mask, a block of query rows at a time."""
    geo, saved, lse, dO = _attention_inputs(case, seed)
    H, L = case["H"], geo.L
    val = {}
    for n, (c, E) in saved.items():
        val[n] = (c.double() * ((E.long() + 896) << 52).view(torch.float64)).view(H, L, HEAD_DIM)
    tile = torch.arange(L, device="cuda") // geo.N
    valid = geo.valid.cuda()
    a = HEAD_DIM ** -0.5
    grads = [torch.zeros((1, H, L, HEAD_DIM), dtype=torch.float64, device="cuda") for _ in range(3)]
    step = max(1, min(L, (1 << 27) // L))
    for h in range(H):
        q, k, v, o = (val[n][h] for n in "qkvo")
        kept = geo.kept[h].cuda()
        for r0 in range(0, L, step):
            rows = slice(r0, min(r0 + step, L))
            g = dO[h, rows].double()
            mask = kept[tile[rows]][:, tile] & valid[None] & valid[rows, None]
            P = torch.exp(a * (q[rows] @ k.T) - lse[h, rows, None].double()) * mask
            grads[2][0, h] += P.T @ g
            P = P * (g @ v.T - (g * o[rows]).sum(1, keepdim=True)) * a
            grads[0][0, h, rows] = P @ k
            grads[1][0, h] += P.T @ q[rows]
    return grads
