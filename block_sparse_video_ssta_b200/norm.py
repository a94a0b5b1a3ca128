"""Norms, gated residuals and 8-bit checkpoints around the attention (binding).

What stands before and after the attention in a block of the diffusion transformer
("HunyuanVideo 1.5 Technical Report") and what its training keeps between forward and
backward.  Argument marshalling only, as in the package's other bindings: the functions
carry the C entry points' names (include/ssta.h, which holds the formulas), check their
tensors, and allocate what the caller does not supply.

Activations are dense [..., C] tensors of ``rows`` rows; weights [C]; modulations
[G, C] (any leading dimensions that hold G rows), rows ``mod_stride`` elements apart, so
``mod.chunk(6, dim=-1)`` of a [G, 6 C] tensor can be passed as it is.

A call given a ``stream`` runs and allocates on that stream: order its inputs before it
and its outputs' readers behind it as for any work on that stream.  A tensor that the
caller passes to be written counts as changed in place, as after torch's own operations.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from dataclasses import dataclass

import torch
from torch.autograd.graph import increment_version

from . import SSTA_BF16, SSTA_F32, Desc, _D, _P, _check, _ptr, _torch_dtype, _workspace, lib, ssta_plan

__all__ = [
    "NormDesc", "NormPlan", "norm_desc", "Checkpoint", "NormGrads", "ResidualNorm", "ResidualNormGrads",
    "ssta_norm_plan", "ssta_norm_fwd", "ssta_norm_bwd", "ssta_residual_norm_fwd", "ssta_residual_norm_bwd",
    "ssta_checkpoint_save", "ssta_checkpoint_load", "ssta_attention_bwd_checkpoint",
]

NORMS = {"none": 0, "layer": 1, "rms": 2}
FORMATS = {"int8": 0, "e4m3": 1}
_CODE_DTYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_CODE_NAMES = {v: k for k, v in _CODE_DTYPES.items()}
_VALUE_DTYPES = {torch.bfloat16: SSTA_BF16, torch.float32: SSTA_F32}
GROUP = 128   # channels sharing one exponent


class NormDesc(ctypes.Structure):
    """Mirror of ssta_norm_desc."""
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "mod_rows", "mod_stride")] + [
        (n, ctypes.c_int) for n in ("C", "dtype", "param_dtype", "norm", "post_norm")] + [
        (n, ctypes.c_float) for n in ("eps", "res_scale")]


class _NormPlanInfo(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int64), ("exponents_per_row", ctypes.c_int),
                ("bwd_workspace_bytes", ctypes.c_size_t)]


class _Ckpt(ctypes.Structure):
    """Mirror of ssta_checkpoint."""
    _fields_ = [("codes", _P), ("exponents", _P), ("format", ctypes.c_int)]


_N = ctypes.POINTER(NormDesc)
_C = ctypes.POINTER(_Ckpt)
for _name, _args in {
    "ssta_norm_plan": [_N, ctypes.POINTER(_NormPlanInfo)],
    "ssta_norm_fwd": [_N] + [_P] * 7 + [_C, _P],
    "ssta_norm_bwd": [_N, _P, _P, _C] + [_P] * 10 + [ctypes.c_size_t, _P],
    "ssta_residual_norm_fwd": [_N] + [_P] * 13 + [_C, _C, _P],
    "ssta_residual_norm_bwd": [_N, _P, _P, _P, _C, _P, _C] + [_P] * 16 + [ctypes.c_size_t, _P],
    "ssta_checkpoint_save": [ctypes.c_int64, ctypes.c_int, ctypes.c_int, _P, _C, _P],
    "ssta_checkpoint_load": [ctypes.c_int64, ctypes.c_int, ctypes.c_int, _C, _P, _P],
    "ssta_attention_bwd_checkpoint_workspace": [_D, ctypes.POINTER(ctypes.c_size_t)],
    "ssta_attention_bwd_checkpoint": [_D, _C, _C, _C, _C] + [_P] * 8 + [ctypes.c_size_t, _P],
}.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int


@dataclass
class NormPlan:
    groups: int
    exponents_per_row: int
    bwd_workspace_bytes: int


def norm_desc(rows, C, dtype="bf16", param_dtype="f32", norm="layer", post_norm="none", eps=1e-6, res_scale=1.0,
              mod_rows=0, mod_stride=0) -> NormDesc:
    """Descriptor of rows of C channels.  ``dtype`` and ``param_dtype`` (weights and modulation) may be
    "bf16"/"f32", ``norm`` and ``post_norm`` "none"/"layer"/"rms", or enum values; ``mod_rows`` rows share a
    modulation row (0: all), ``mod_stride`` elements lie between two modulation rows (0: C)."""
    types = {"bf16": SSTA_BF16, "f32": SSTA_F32}
    pick = lambda v, table: table[v] if isinstance(v, str) else int(v)
    return NormDesc(int(rows), int(mod_rows), int(mod_stride), int(C), pick(dtype, types), pick(param_dtype, types),
                    pick(norm, NORMS), pick(post_norm, NORMS), float(eps), float(res_scale))


def ssta_norm_plan(desc: NormDesc) -> NormPlan:
    info = _NormPlanInfo()
    _check(lib.ssta_norm_plan(ctypes.byref(desc), ctypes.byref(info)), "ssta_norm_plan")
    return NormPlan(info.groups, info.exponents_per_row, info.bwd_workspace_bytes)


@functools.lru_cache(maxsize=256)
def _bwd_bytes(rows, C, mod_rows):
    """Workspace of the backwards (no other field of a descriptor changes it)."""
    return ssta_norm_plan(norm_desc(rows, C, mod_rows=mod_rows)).bwd_workspace_bytes


class Checkpoint:
    """An activation kept in 8 bits: ``codes`` [..., C] (torch.int8 or torch.float8_e4m3fn), ``exponents``
    [..., ceil(C / 128)] (torch.uint8), and the ``dtype`` its values are read as.  The value of a code is
    code * 2^(exponent - 127); exponent 255 marks a group that held an infinity or a NaN (its values read as NaN)."""
    __slots__ = ("_codes", "_exponents", "_dtype")

    def __init__(self, codes, exponents, dtype=torch.bfloat16):
        if codes.dtype not in _CODE_NAMES:
            raise ValueError(f"codes have dtype {codes.dtype}, expected torch.int8 or torch.float8_e4m3fn")
        if dtype not in _VALUE_DTYPES:
            raise ValueError(f"values have dtype {dtype}, expected torch.bfloat16 or torch.float32")
        if codes.dim() < 1:
            raise ValueError("codes must have at least one dimension")
        want = tuple(codes.shape[:-1]) + (-(-codes.shape[-1] // GROUP),)
        _ptr(codes, "codes")
        _ptr(exponents, "exponents", torch.uint8, want)
        if exponents.device != codes.device:
            raise ValueError(f"exponents are on {exponents.device}, codes on {codes.device}")
        self._codes, self._exponents, self._dtype = codes, exponents, dtype

    codes = property(lambda self: self._codes)
    exponents = property(lambda self: self._exponents)
    dtype = property(lambda self: self._dtype)

    @property
    def format(self) -> str:
        return _CODE_NAMES[self._codes.dtype]

    @property
    def shape(self):
        return self._codes.shape

    @property
    def device(self):
        return self._codes.device

    @property
    def nbytes(self) -> int:
        return self._codes.numel() + self._exponents.numel()

    @classmethod
    def empty(cls, shape, format="int8", dtype=torch.bfloat16, device="cuda") -> "Checkpoint":
        """An unwritten checkpoint of a tensor of this shape."""
        if format not in _CODE_DTYPES:
            raise ValueError(f"format {format!r}, expected one of {sorted(_CODE_DTYPES)}")
        if dtype not in _VALUE_DTYPES:
            raise ValueError(f"values have dtype {dtype}, expected torch.bfloat16 or torch.float32")
        shape = tuple(shape)
        ckpt = cls.__new__(cls)
        ckpt._codes = torch.empty(shape, dtype=_CODE_DTYPES[format], device=device)
        ckpt._exponents = torch.empty(shape[:-1] + (-(-shape[-1] // GROUP),), dtype=torch.uint8, device=device)
        ckpt._dtype = dtype
        return ckpt

    @classmethod
    def _like(cls, t, format, dtype) -> "Checkpoint":
        """An unwritten checkpoint of a contiguous tensor (or of one shaped like it)."""
        if format not in _CODE_DTYPES:
            raise ValueError(f"format {format!r}, expected one of {sorted(_CODE_DTYPES)}")
        ckpt = cls.__new__(cls)
        ckpt._codes = torch.empty_like(t, dtype=_CODE_DTYPES[format])
        ckpt._exponents = t.new_empty(t.shape[:-1] + (-(-t.shape[-1] // GROUP),), dtype=torch.uint8)
        ckpt._dtype = dtype
        return ckpt

    def _ref(self):
        """The C struct of this moment's addresses, by reference."""
        return ctypes.byref(_Ckpt(self._codes.data_ptr(), self._exponents.data_ptr(), FORMATS[self.format]))


@dataclass
class NormGrads:
    """dx [..., C]; dweight [C], dscale, dshift [G, C] (float32, None where not asked for); the workspace."""
    dx: torch.Tensor
    dweight: torch.Tensor | None
    dscale: torch.Tensor | None
    dshift: torch.Tensor | None
    workspace: torch.Tensor


@dataclass
class ResidualNorm:
    """Outputs of ssta_residual_norm_fwd; n, the statistics and the checkpoints are None where there is none."""
    r: torch.Tensor
    n: torch.Tensor | None
    post_mean: torch.Tensor | None
    post_rstd: torch.Tensor | None
    mean: torch.Tensor | None
    rstd: torch.Tensor | None
    saved_y: Checkpoint | None
    saved_r: Checkpoint | None


@dataclass
class ResidualNormGrads:
    """dx, dy [..., C]; dpost_weight, dweight [C], dgate, dscale, dshift [G, C] (float32, None where not asked
    for); the workspace."""
    dx: torch.Tensor
    dy: torch.Tensor
    dpost_weight: torch.Tensor | None
    dgate: torch.Tensor | None
    dweight: torch.Tensor | None
    dscale: torch.Tensor | None
    dshift: torch.Tensor | None
    workspace: torch.Tensor


_NOTHING = contextlib.nullcontext()


def _on(stream, dev):
    """Context in which `dev` and the call's stream are current."""
    if stream is None:
        return _NOTHING if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream of {stream.device} for tensors on {dev}")
    return torch.cuda.stream(stream)


def _current(dev):
    # the raw handle: torch.cuda.current_stream builds a Stream object, a fifth of a small call
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _device(t, name):
    if not isinstance(t, (torch.Tensor, Checkpoint)) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.device


class _Args:
    """Checks one call's tensors against its descriptor and returns their addresses."""
    __slots__ = ("desc", "dev", "index", "rows", "C", "n", "dtype", "param", "groups", "given")

    def __init__(self, desc: NormDesc, dev):
        self.desc, self.dev, self.index = desc, dev, dev.index
        self.rows, self.C = desc.rows, desc.C
        self.n = self.rows * self.C
        self.given = []   # the caller's tensors that the call writes
        self.dtype = torch.bfloat16 if desc.dtype == SSTA_BF16 else torch.float32
        self.param = torch.bfloat16 if desc.param_dtype == SSTA_BF16 else torch.float32
        m = desc.mod_rows
        self.groups = 1 if m == 0 or m >= self.rows else -(-self.rows // m)

    def _dense(self, t, name, dtype, numel, last):
        try:
            if t.dtype is dtype and t.get_device() == self.index and t.numel() == numel and t.is_contiguous() and (
                    not last or t.shape[-1] == last):
                return t.data_ptr()
        except (AttributeError, IndexError):
            pass
        self._refuse(t, name, dtype, numel, last)

    def _refuse(self, t, name, dtype, numel, last):
        if not isinstance(t, torch.Tensor) or t.device != self.dev:
            raise ValueError(f"{name} must be a tensor on {self.dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {numel // last if last else numel} "
                         + (f"rows of {last}" if last else "elements"))

    def act(self, t, name):
        return None if t is None else self._dense(t, name, self.dtype, self.n, self.C)

    def weight(self, t, name):
        return None if t is None else self._dense(t, name, self.param, self.C, self.C)

    def stat(self, t, name):
        return None if t is None else self._dense(t, name, torch.float32, self.rows, 0)

    def grad(self, t, name, groups):
        return None if t is None else self._dense(t, name, torch.float32, groups * self.C, self.C)

    def mod(self, t, name):
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index:
            raise ValueError(f"{name} must be a tensor on {self.dev}")
        if t.dtype is not self.param:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {self.param}")
        shape, strides = t.shape, t.stride()
        if not shape or shape[-1] != self.C or t.numel() != self.groups * self.C:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {self.groups} rows of {self.C}")
        if strides[-1] != 1:
            raise ValueError(f"{name} must have contiguous channels")
        if self.groups > 1:
            want = self.desc.mod_stride or self.C
            for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
                if size != 1:
                    if stride != want:
                        raise ValueError(f"{name} has row stride {stride}, expected {want} (the descriptor's mod_stride)")
                    want *= size
        return t.data_ptr()

    def kept(self, t, name):
        """(address of a dense tensor or None, checkpoint or None) of something the backward reads."""
        if not isinstance(t, Checkpoint):
            return self.act(t, name), None
        if t.device != self.dev:
            raise ValueError(f"{name} must be a checkpoint on {self.dev}")
        if t.codes.numel() != self.n or t.shape[-1] != self.C:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {self.rows} rows of {self.C}")
        return None, t._ref()

    def save(self, want, like, name):
        """The checkpoint to write: a new one of a named format, or the caller's."""
        if want is None:
            return None
        if isinstance(want, str):
            return Checkpoint._like(like, want, self.dtype)
        if not isinstance(want, Checkpoint):
            raise ValueError(f"{name} must be a format name or a Checkpoint")
        self.kept(want, name)
        if want.dtype != self.dtype:
            raise ValueError(f"{name} holds values of dtype {want.dtype}, expected {self.dtype}")
        return want

    # Outputs: (tensor, address) of the caller's tensor, checked, or of a new one.

    def out_act(self, t, name, like):
        """Shaped like a checked activation."""
        if t is None:
            t = torch.empty_like(like)
            return t, t.data_ptr()
        self.given.append(t)
        return t, self.act(t, name)

    def out_stat(self, t, name, wanted, like=None):
        if t is None:
            if not wanted:
                return None, None
            t = torch.empty_like(like) if like is not None else torch.empty(self.rows, dtype=torch.float32, device=self.dev)
            return t, t.data_ptr()
        self.given.append(t)
        return t, self.stat(t, name)

    def out_grad(self, t, name, wanted, groups=None, like=None):
        """[C], or [groups, C]."""
        if t is None:
            if not wanted:
                return None, None
            shape = (self.C,) if groups is None else (groups, self.C)
            t = torch.empty_like(like) if like is not None else torch.empty(shape, dtype=torch.float32, device=self.dev)
            return t, t.data_ptr()
        self.given.append(t)
        return t, self.grad(t, name, groups or 1)

    def workspace(self, t):
        if t is None:
            t = _workspace(_bwd_bytes(self.rows, self.C, self.desc.mod_rows), self.dev)
            return t, t.data_ptr()
        return t, self._dense(t, "workspace", torch.uint8, t.numel(), 0)


    def check(self, code, where):
        """Raises on a non-zero status; otherwise the caller's tensors count as written, as after torch's own
        in-place operations (an address does not tell torch)."""
        _check(code, where)
        if self.given:
            increment_version(self.given)


def _ref(ckpt):
    return None if ckpt is None else ckpt._ref()


def ssta_norm_fwd(desc: NormDesc, x, weight=None, scale=None, shift=None, y=None, mean=None, rstd=None, save=None,
                  stats=True, stream=None):
    """norm(x) * weight * (1 + scale) + shift: returns (y, mean, rstd, saved).

    ``save``: None, a format ("int8", "e4m3") or a Checkpoint to write x into; ``stats`` False leaves out mean and
    rstd (inference).  mean is None for the RMS norm.  ``y`` may be ``x``."""
    dev = _device(x, "x")
    with _on(stream, dev):
        a = _Args(desc, dev)
        px = a.act(x, "x")
        y, py = a.out_act(y, "y", x)
        mean, pm = a.out_stat(mean, "mean", stats and desc.norm == 1)
        rstd, pr = a.out_stat(rstd, "rstd", stats, mean)
        saved = a.save(save, x, "save")
        a.check(lib.ssta_norm_fwd(
            ctypes.byref(desc), px, a.weight(weight, "weight"), a.mod(scale, "scale"), a.mod(shift, "shift"),
            py, pm, pr, _ref(saved), _current(dev)), "ssta_norm_fwd")
    return y, mean, rstd, saved


def ssta_norm_bwd(desc: NormDesc, dy, x, mean, rstd, weight=None, scale=None, dres=None, dx=None, dweight=None,
                  dscale=None, dshift=None, want_dshift=None, workspace=None, stream=None) -> NormGrads:
    """Gradients of ssta_norm_fwd.  ``x``: the forward's input, or its Checkpoint; ``dres``: a gradient that reaches
    x past the norm, added to dx.  dweight is computed when ``weight`` is given, dscale and dshift when ``scale`` is
    (``want_dshift`` overrides it for dshift), or when their output is given.  ``dx`` may be ``dy`` or ``dres``."""
    dev = _device(dy, "dy")
    with _on(stream, dev):
        a = _Args(desc, dev)
        pdy = a.act(dy, "dy")
        px, cx = a.kept(x, "x")
        dx, pdx = a.out_act(dx, "dx", dy)
        dweight, pdw = a.out_grad(dweight, "dweight", weight is not None)
        dscale, pds = a.out_grad(dscale, "dscale", scale is not None, a.groups)
        dshift, pdt = a.out_grad(dshift, "dshift", scale is not None if want_dshift is None else want_dshift, a.groups, dscale)
        workspace, pw = a.workspace(workspace)
        a.check(lib.ssta_norm_bwd(
            ctypes.byref(desc), pdy, px, cx, a.stat(mean, "mean"), a.stat(rstd, "rstd"), a.weight(weight, "weight"),
            a.mod(scale, "scale"), a.act(dres, "dres"), pdx, pdw, pds, pdt, pw, workspace.numel(), _current(dev)),
            "ssta_norm_bwd")
    return NormGrads(dx, dweight, dscale, dshift, workspace)


def ssta_residual_norm_fwd(desc: NormDesc, x, y, post_weight=None, gate=None, weight=None, scale=None, shift=None,
                           r=None, n=None, save_y=None, save_r=None, stats=True, stream=None) -> ResidualNorm:
    """r = res_scale * x + gate * post_norm(y) * post_weight and n = norm(r) * weight * (1 + scale) + shift.

    ``save_y``, ``save_r``: None, a format or a Checkpoint to write y and the stored r into; ``stats`` False leaves
    out the statistics (inference).  ``r`` may be ``x``, ``n`` may be ``y``."""
    dev = _device(x, "x")
    with _on(stream, dev):
        a = _Args(desc, dev)
        px, py = a.act(x, "x"), a.act(y, "y")
        r, p_r = a.out_act(r, "r", x)
        n, p_n = a.out_act(n, "n", x) if desc.norm != 0 or n is not None else (None, None)
        pr, p_pr = a.out_stat(None, "post_rstd", stats and desc.post_norm != 0)
        pm, p_pm = a.out_stat(None, "post_mean", stats and desc.post_norm == 1, pr)
        rs, p_rs = a.out_stat(None, "rstd", stats and desc.norm != 0, pr)
        m, p_m = a.out_stat(None, "mean", stats and desc.norm == 1, rs)
        cy, cr = a.save(save_y, y, "save_y"), a.save(save_r, x, "save_r")
        a.check(lib.ssta_residual_norm_fwd(
            ctypes.byref(desc), px, py, a.weight(post_weight, "post_weight"), a.mod(gate, "gate"),
            a.weight(weight, "weight"), a.mod(scale, "scale"), a.mod(shift, "shift"), p_r, p_n, p_pm, p_pr, p_m, p_rs,
            _ref(cy), _ref(cr), _current(dev)), "ssta_residual_norm_fwd")
    return ResidualNorm(r, n, pm, pr, m, rs, cy, cr)


def ssta_residual_norm_bwd(desc: NormDesc, dr, dn, r=None, y=None, mean=None, rstd=None, post_mean=None,
                           post_rstd=None, post_weight=None, gate=None, weight=None, scale=None, dx=None, dy=None,
                           dpost_weight=None, dgate=None, dweight=None, dscale=None, dshift=None, want_dshift=None,
                           workspace=None, stream=None) -> ResidualNormGrads:
    """Gradients of ssta_residual_norm_fwd from ``dr`` and ``dn`` (either may be None).  ``r``, ``y``: as the forward
    had them, dense or Checkpoints (both of one kind).  The gradient of each vector is computed when the vector is
    given (dshift with ``scale``, which ``want_dshift`` overrides), or when its output is; those of the norm's vectors
    need ``dn``.  ``dx`` may be ``dr``, ``dy`` may be ``dn``."""
    like = dr if dr is not None else dn
    dev = _device(like, "dr" if dr is not None else "dn")
    with _on(stream, dev):
        a = _Args(desc, dev)
        (pr_, cr), (py, cy) = a.kept(r, "r"), a.kept(y, "y")
        pdr, pdn = a.act(dr, "dr"), a.act(dn, "dn")
        dx, pdx = a.out_act(dx, "dx", like)
        dy, pdy = a.out_act(dy, "dy", like)
        normed = dn is not None
        dpost_weight, pdp = a.out_grad(dpost_weight, "dpost_weight", post_weight is not None)
        dgate, pdg = a.out_grad(dgate, "dgate", gate is not None, a.groups)
        dweight, pdw = a.out_grad(dweight, "dweight", normed and weight is not None)
        dscale, pds = a.out_grad(dscale, "dscale", normed and scale is not None, a.groups, dgate)
        dshift, pdt = a.out_grad(dshift, "dshift", normed and (scale is not None if want_dshift is None else want_dshift),
                                 a.groups, dscale)
        workspace, pw = a.workspace(workspace)
        a.check(lib.ssta_residual_norm_bwd(
            ctypes.byref(desc), pdr, pdn, pr_, cr, py, cy, a.stat(post_mean, "post_mean"), a.stat(post_rstd, "post_rstd"),
            a.stat(mean, "mean"), a.stat(rstd, "rstd"), a.weight(post_weight, "post_weight"), a.mod(gate, "gate"),
            a.weight(weight, "weight"), a.mod(scale, "scale"), pdx, pdy, pdp, pdg, pdw, pds, pdt, pw, workspace.numel(),
            _current(dev)), "ssta_residual_norm_bwd")
    return ResidualNormGrads(dx, dy, dpost_weight, dgate, dweight, dscale, dshift, workspace)


def ssta_checkpoint_save(x, format="int8", out=None, stream=None) -> Checkpoint:
    """The 8-bit checkpoint of x [..., C] (bf16 or f32), in ``out`` or a new one of ``format``."""
    dev = _device(x, "x")
    if x.dtype not in _VALUE_DTYPES:
        raise ValueError(f"x has dtype {x.dtype}, expected torch.bfloat16 or torch.float32")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    with _on(stream, dev):
        px = _ptr(x, "x")
        if out is None:
            out = Checkpoint._like(x, format, x.dtype)
        elif not isinstance(out, Checkpoint) or out.device != dev or out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError(f"out must be a Checkpoint of shape {tuple(x.shape)} and dtype {x.dtype} on {dev}")
        C = x.shape[-1]
        _check(lib.ssta_checkpoint_save(x.numel() // max(C, 1), C, _VALUE_DTYPES[x.dtype], px, out._ref(), _current(dev)),
               "ssta_checkpoint_save")
    return out


def ssta_checkpoint_load(ckpt: Checkpoint, x=None, stream=None):
    """The values of a checkpoint, [..., C] of its dtype."""
    dev = _device(ckpt, "ckpt")
    if not isinstance(ckpt, Checkpoint):
        raise ValueError("ckpt must be a Checkpoint")
    given = x is not None
    with _on(stream, dev):
        if not given:
            x = torch.empty_like(ckpt._codes, dtype=ckpt._dtype)
            px = x.data_ptr()
        else:
            px = _ptr(x, "x", ckpt.dtype, ckpt.shape)
            if x.device != dev:
                raise ValueError(f"x must be a tensor on {dev}")
        C = x.shape[-1]
        _check(lib.ssta_checkpoint_load(x.numel() // max(C, 1), C, _VALUE_DTYPES[ckpt._dtype], ckpt._ref(), px,
                                        _current(dev)), "ssta_checkpoint_load")
        if given:
            increment_version(x)
    return x


def ssta_attention_bwd_checkpoint(desc: Desc, q, k, v, o, lse, do_packed, kv_idx, kv_cnt, dq=None, dk=None, dv=None,
                                  workspace=None, stream=None):
    """Backward of Step 4 from 8-bit checkpoints of the packed q, k, v and O (one format): returns
    (dq, dk, dv [B,H,Lq,D], workspace).  ``lse`` and ``o`` are those of ssta_attention_fwd over the checkpoints' values
    of q, k and v, not over what these were before (ssta_backward computes both anew)."""
    p = ssta_plan(desc)
    dt = _torch_dtype(desc)
    dev = _device(do_packed, "do_packed")
    shp = (desc.B, desc.H, p.packed_len, desc.D)
    for name, c in (("q", q), ("k", k), ("v", v), ("o", o)):
        if not isinstance(c, Checkpoint) or c.device != dev or tuple(c.shape) != shp or c.dtype != dt:
            raise ValueError(f"{name} must be a Checkpoint of shape {shp} and dtype {dt} on {dev}")
    given = (("lse", lse, torch.float32, shp[:3]), ("do_packed", do_packed, dt, shp),
             ("kv_idx", kv_idx, torch.int32, (desc.B, desc.H, p.num_q_tiles, p.max_kept)),
             ("kv_cnt", kv_cnt, torch.int32, (desc.B, desc.H, p.num_q_tiles)))
    with _on(stream, dev):
        dq, dk, dv = (torch.empty(shp, dtype=dt, device=dev) if t is None else t for t in (dq, dk, dv))
        if workspace is None:
            need = ctypes.c_size_t(0)
            _check(lib.ssta_attention_bwd_checkpoint_workspace(ctypes.byref(desc), ctypes.byref(need)),
                   "ssta_attention_bwd_checkpoint_workspace")
            workspace = _workspace(need.value, dev)
        ptrs = []
        for name, t, want, shape in given + (("dq", dq, dt, shp), ("dk", dk, dt, shp), ("dv", dv, dt, shp),
                                             ("workspace", workspace, torch.uint8, None)):
            ptrs.append(_ptr(t, name, want, shape))
            if t.device != dev:
                raise ValueError(f"{name} must be a tensor on {dev}")
        _check(lib.ssta_attention_bwd_checkpoint(ctypes.byref(desc), _ref(q), _ref(k), _ref(v), _ref(o), *ptrs,
                                                 workspace.numel(), _current(dev)), "ssta_attention_bwd_checkpoint")
    return dq, dk, dv, workspace
