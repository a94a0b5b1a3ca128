"""The attention sub-block of a diffusion transformer around SSTA, forward and backward.

The layer the attention runs in ("HunyuanVideo 1.5 Technical Report": a DiT whose
self-attention is SSTA): an adaptive norm of the residual stream, the projections to q, k
and v, RMS norms of q and k per head, the attention, the output projection, the gated
residual, and the adaptive norm before the next sub-block, which is fused with it:

    n1 = norm(x) * (1 + scale) + shift
    q, k, v = heads(n1 Wqkv^T);  O = SSTA(rms(q), rms(k), v);  y = tokens(O) Wo^T
    r = x + gate * y;  n2 = norm(r) * (1 + scale2) + shift2

Tokens are [B, L, C] with C = H * D: the T * Y * X video tokens in raster order, then the
text tokens.  The modulation is [B, 5, C]: shift, scale, gate, shift2, scale2.  The two
projections are library GEMMs; everything else runs in the library's kernels and layout
copies.  With a ``checkpoint`` format everything the backward needs is kept in 8 bits
(9.1 bytes per token and channel, against 18 in bf16): x, the packed q, k, v and O, q
and k before their norms, y and r.  The attention's gradients are then those at the values
of q, k and v (ssta_backward), the output projection's is that of the kept O.
"""
from __future__ import annotations

import weakref
from dataclasses import dataclass, field

import torch

from . import (Desc, SstaSaved, norm_desc, ssta_backward, ssta_checkpoint_load, ssta_forward, ssta_norm_bwd,
               ssta_norm_fwd, ssta_residual_norm_bwd, ssta_residual_norm_fwd, ssta_tile_unorder)
from .norm import _VALUE_DTYPES, Checkpoint, _device, _on

__all__ = ["BlockWeights", "BlockSaved", "BlockGrads", "ssta_block_forward", "ssta_block_backward"]


@dataclass
class BlockWeights:
    """qkv [3 C, C] (rows of q, then k, then v, head-major) and out [C, C] of the activations' dtype; q_norm, k_norm
    [D] (bf16 or f32) or None."""
    qkv: torch.Tensor
    out: torch.Tensor
    q_norm: torch.Tensor | None = None
    k_norm: torch.Tensor | None = None


@dataclass
class BlockSaved:
    """What ssta_block_backward reads; x, y and r are tensors or Checkpoints.  x, mod, the head norms' weights and,
    without checkpoints, r are the caller's own tensors: they stay unchanged until the backward."""
    x: object
    y: object
    r: object
    mean: torch.Tensor
    rstd: torch.Tensor
    mean2: torch.Tensor
    rstd2: torch.Tensor
    mod: torch.Tensor
    attention: SstaSaved
    # r as the forward returned it, and its version (a next residual may be written over it)
    _returned: tuple | None = field(default=None, repr=False, compare=False)

    def __getstate__(self):   # a copy has an r of its own
        return {**self.__dict__, "_returned": None}

    def check_unchanged(self):
        """Raises where the r that the caller was given has been written since the forward."""
        r, version = self._returned or (None, None)
        if r is not None and r() is self.r and self.r._version != version:
            raise ValueError("r was written after ssta_block_forward returned it, and the backward reads it: write the "
                             "next residual elsewhere, or keep a checkpoint")


@dataclass
class BlockGrads:
    """dx [B, L, C]; dmod [B, 5, C] float32; dqkv, dout as the weights; dq_norm, dk_norm [D] float32 or None."""
    dx: torch.Tensor
    dmod: torch.Tensor
    dqkv: torch.Tensor
    dout: torch.Tensor
    dq_norm: torch.Tensor | None
    dk_norm: torch.Tensor | None


def _check(desc, x, mod, w, **more):
    """Shapes, dtypes and strides of the call's tensors (`more`: shaped like x); returns the norms' descriptor."""
    C, L = desc.H * desc.D, desc.T * desc.Y * desc.X + desc.L_text
    rows = [(name, t, (desc.B, L, C)) for name, t in (("x", x), *more.items())]
    for name, t, shape in rows + [("mod", mod, (desc.B, 5, C)), ("qkv", w.qkv, (3 * C, C)), ("out", w.out, (C, C))]:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} is required")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t in (("qkv", w.qkv), ("out", w.out)):
        if t.dtype != x.dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
    if mod.dtype not in _VALUE_DTYPES:
        raise ValueError(f"mod has dtype {mod.dtype}, expected torch.bfloat16 or torch.float32")
    return norm_desc(desc.B * L, C, desc.dtype, _VALUE_DTYPES[mod.dtype], "layer", mod_rows=L, mod_stride=5 * C)


def _split(desc, t):
    """[B, H, L, D] -> (raster, text or None)."""
    n = desc.T * desc.Y * desc.X
    video = t[:, :, :n].reshape(desc.B, desc.H, desc.T, desc.Y, desc.X, desc.D).contiguous()
    return video, t[:, :, n:].contiguous() if desc.L_text else None


def _heads(desc, t):
    """[B, L, H * D] tokens -> (raster, text or None)."""
    return _split(desc, t.view(desc.B, -1, desc.H, desc.D).transpose(1, 2))


def _tokens(desc, video, text, out=None):
    """(raster, text) -> [B, L, H * D], into `out` [B, L, H, D] when given."""
    n = desc.T * desc.Y * desc.X
    if out is None:
        out = torch.empty((desc.B, n + desc.L_text, desc.H, desc.D), dtype=video.dtype, device=video.device)
    out[:, :n] = video.reshape(desc.B, desc.H, n, desc.D).transpose(1, 2)
    if desc.L_text:
        out[:, n:] = text.transpose(1, 2)
    return out.flatten(2)


@torch.no_grad()
def ssta_block_forward(desc: Desc, x, mod, w: BlockWeights, checkpoint=None, stream=None):
    """Returns (r, n2 [B, L, C], saved).  ``checkpoint``: None (keep what the backward reads as it is, x and the
    returned r by reference: ssta_block_backward refuses an r that was written since), "int8" or "e4m3" (mod and the
    head norms' weights are kept by reference all the same).  The gradients are ssta_block_backward's: nothing is recorded for torch's autograd,
    whatever requires a gradient."""
    nd = _check(desc, x, mod, w)
    with _on(stream, _device(x, "x")):
        shift, scale, gate, shift2, scale2 = mod.unbind(1)
        n1, mean, rstd, x_saved = ssta_norm_fwd(nd, x, None, scale, shift, save=checkpoint)
        qkv = torch.matmul(n1, w.qkv.t()).view(desc.B, -1, 3, desc.H * desc.D)
        del n1
        (q, qt), (k, kt), (v, vt) = (_heads(desc, qkv[:, :, i].contiguous()) for i in range(3))
        del qkv
        a = ssta_forward(desc, q, k, v, qt, kt, vt, q_weight=w.q_norm, k_weight=w.k_norm, checkpoint=checkpoint)
        y = torch.matmul(_tokens(desc, a["O"], a["O_text"]), w.out.t())
        f = ssta_residual_norm_fwd(nd, x, y, None, gate, None, scale2, shift2, save_y=checkpoint, save_r=checkpoint)
        saved = BlockSaved(x_saved or x, f.saved_y or y, f.saved_r or f.r, mean, rstd, f.mean, f.rstd, mod, a["saved"])
        if checkpoint is None and not f.r.is_inference():   # inference tensors have no version
            saved._returned = (weakref.ref(f.r), f.r._version)
    return f.r, f.n, saved


@torch.no_grad()
def ssta_block_backward(desc: Desc, saved: BlockSaved, w: BlockWeights, dr, dn2, stream=None) -> BlockGrads:
    """Gradients from those of r and n2 [B, L, C]."""
    mod = saved.mod
    nd = _check(desc, dr, mod, w, dn2=dn2)
    saved.check_unchanged()
    with _on(stream, _device(dr, "dr")):
        shift, scale, gate, _, scale2 = mod.unbind(1)
        g2 = ssta_residual_norm_bwd(nd, dr, dn2, saved.r, saved.y, saved.mean2, saved.rstd2, None, None, None, gate, None,
                                    scale2)
        C = desc.H * desc.D
        dy = g2.dy.view(-1, C)
        o = saved.attention.o
        o = ssta_checkpoint_load(o) if isinstance(o, Checkpoint) else o
        o_tokens = _tokens(desc, *ssta_tile_unorder(desc, o)).view(-1, C)
        dout = torch.matmul(dy.t(), o_tokens)
        dO = torch.matmul(dy, w.out).view(desc.B, -1, C)
        b = ssta_backward(desc, saved.attention, *_heads(desc, dO))
        dqkv = torch.empty((desc.B, dO.shape[1], 3, desc.H, desc.D), dtype=dr.dtype, device=dr.device)
        for i, name in enumerate(("dq", "dk", "dv")):
            _tokens(desc, b[name], b[name + "_text"], dqkv[:, :, i])
        dqkv = dqkv.view(-1, 3 * C)
        # the projection's input again, from what is kept of x
        x = ssta_checkpoint_load(saved.x) if isinstance(saved.x, Checkpoint) else saved.x
        n1 = ssta_norm_fwd(nd, x, None, scale, shift, stats=False)[0].view(-1, C)
        dw = torch.matmul(dqkv.t(), n1)
        dn1 = torch.matmul(dqkv, w.qkv).view(dr.shape)
        g1 = ssta_norm_bwd(nd, dn1, saved.x, saved.mean, saved.rstd, None, scale, g2.dx, dx=g2.dx)
        dmod = torch.stack((g1.dshift, g1.dscale, g2.dgate, g2.dshift, g2.dscale), dim=1)
    return BlockGrads(g1.dx, dmod, dw, dout, b["dq_weight"], b["dk_weight"])
