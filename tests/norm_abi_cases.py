"""Host-side argument validation of the norm, residual and checkpoint calls of libssta.so,
run in a child process with no visible CUDA device (as abi_validation_cases.py).
Prints one line per case: name, returned status, expected status."""
import ctypes
import os
import sys

assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "run only with CUDA_VISIBLE_DEVICES=''"
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_sparse_video_ssta_b200 as S  # noqa: E402
from block_sparse_video_ssta_b200.norm import _Ckpt, _NormPlanInfo  # noqa: E402

lib = S.lib
A = 0x10000   # fake, 256-byte aligned, never dereferenced
OK, INVALID, UNSUP, ALIGN, WS, LAUNCH = 0, 1, 2, 3, 4, 5
BIG = 1 << 40
cases = []


def norm(**kw):
    return S.norm_desc(kw.pop("rows", 16), kw.pop("C", 256), **kw)


def ck(codes=A, exps=A, fmt=0):
    return ctypes.byref(_Ckpt(codes, exps, fmt))


def add(name, got, want):
    cases.append((name, got, want))


info = _NormPlanInfo()
plan = lambda d: lib.ssta_norm_plan(None if d is None else ctypes.byref(d), ctypes.byref(info))
add("plan_null", plan(None), INVALID)
add("plan_null_info", lib.ssta_norm_plan(ctypes.byref(norm()), None), INVALID)
add("plan_ok", plan(norm()), OK)
add("plan_one_row", plan(norm(rows=1, C=8)), OK)
add("plan_widest", plan(norm(C=8192)), OK)
add("plan_rows_0", plan(norm(rows=0)), INVALID)
add("plan_rows_neg", plan(norm(rows=-3)), INVALID)
add("plan_rows_2_31", plan(norm(rows=1 << 31)), UNSUP)
add("plan_C_0", plan(norm(C=0)), INVALID)
add("plan_C_12", plan(norm(C=12)), UNSUP)
add("plan_C_8200", plan(norm(C=8200)), UNSUP)
add("plan_mod_rows_neg", plan(norm(mod_rows=-1)), INVALID)
add("plan_mod_rows_beyond", plan(norm(mod_rows=1 << 40)), OK)
add("plan_stride_short", plan(norm(mod_stride=128)), INVALID)
add("plan_stride_odd", plan(norm(mod_stride=260)), UNSUP)
add("plan_dtype", plan(norm(dtype=2)), INVALID)
add("plan_param_dtype", plan(norm(param_dtype=-1)), INVALID)
add("plan_norm", plan(norm(norm=3)), INVALID)
add("plan_post_norm", plan(norm(post_norm=-1)), INVALID)
for e in (0.0, -1.0, float("nan"), float("inf")):
    add(f"plan_eps_{e}", plan(norm(eps=e)), INVALID)
add("plan_res_scale_nan", plan(norm(res_scale=float("nan"))), INVALID)


def fwd(d, x=A, weight=None, scale=None, shift=None, y=A, mean=None, rstd=None, save=None):
    return lib.ssta_norm_fwd(ctypes.byref(d), x, weight, scale, shift, y, mean, rstd, save, None)


# a call that passes every check launches, which fails without a device
add("fwd_valid", fwd(norm(), A, A, A, A, A, A, A, ck()), LAUNCH)
add("fwd_null_x", fwd(norm(), x=None), INVALID)
add("fwd_null_y", fwd(norm(), y=None), INVALID)
add("fwd_norm_none", fwd(norm(norm="none")), INVALID)
add("fwd_rms_mean", fwd(norm(norm="rms"), mean=A), INVALID)
add("fwd_misaligned_x", fwd(norm(), x=A + 8), ALIGN)
add("fwd_misaligned_scale", fwd(norm(), scale=A + 4), ALIGN)
add("fwd_save_null_codes", fwd(norm(), save=ck(codes=None)), INVALID)
add("fwd_save_null_exps", fwd(norm(), save=ck(exps=None)), INVALID)
add("fwd_save_format", fwd(norm(), save=ck(fmt=2)), INVALID)
add("fwd_save_misaligned", fwd(norm(), save=ck(codes=A + 8)), ALIGN)


def bwd(d, dy=A, x=A, saved=None, mean=A, rstd=A, dres=None, dx=A, dw=None, ds=None, dt=None, ws=A, nbytes=BIG):
    return lib.ssta_norm_bwd(ctypes.byref(d), dy, x, saved, mean, rstd, None, None, dres, dx, dw, ds, dt, ws, nbytes,
                             None)


add("bwd_valid", bwd(norm(), dw=A, ds=A, dt=A), LAUNCH)
add("bwd_valid_saved", bwd(norm(), x=None, saved=ck()), LAUNCH)
add("bwd_both_x", bwd(norm(), saved=ck()), INVALID)
add("bwd_no_x", bwd(norm(), x=None), INVALID)
add("bwd_layer_no_mean", bwd(norm(), mean=None), INVALID)
add("bwd_rms_with_mean", bwd(norm(norm="rms")), INVALID)
add("bwd_no_rstd", bwd(norm(), rstd=None), INVALID)
add("bwd_no_dy", bwd(norm(), dy=None), INVALID)
add("bwd_no_dx", bwd(norm(), dx=None), INVALID)
add("bwd_no_workspace", bwd(norm(), ws=None), WS)
add("bwd_short_workspace", bwd(norm(), nbytes=64), WS)
add("bwd_ws_misaligned", bwd(norm(), ws=A + 16), ALIGN)
add("bwd_dx_misaligned", bwd(norm(), dx=A + 2), ALIGN)


def rfwd(d, x=A, y=A, pw=None, gate=None, w=None, s=None, t=None, r=A, n=A, pm=None, pr=None, m=None, rs=None,
         cy=None, cr=None):
    return lib.ssta_residual_norm_fwd(ctypes.byref(d), x, y, pw, gate, w, s, t, r, n, pm, pr, m, rs, cy, cr, None)


add("rfwd_valid", rfwd(norm(post_norm="layer"), A, A, A, A, A, A, A, A, A, A, A, A, A, ck(), ck()), LAUNCH)
add("rfwd_no_norm", rfwd(norm(norm="none"), n=None), LAUNCH)
add("rfwd_no_norm_with_n", rfwd(norm(norm="none")), INVALID)
add("rfwd_no_norm_with_scale", rfwd(norm(norm="none"), n=None, s=A), INVALID)
add("rfwd_no_norm_with_rstd", rfwd(norm(norm="none"), n=None, rs=A), INVALID)
add("rfwd_norm_without_n", rfwd(norm(), n=None), INVALID)
add("rfwd_null_x", rfwd(norm(), x=None), INVALID)
add("rfwd_null_y", rfwd(norm(), y=None), INVALID)
add("rfwd_null_r", rfwd(norm(), r=None), INVALID)
add("rfwd_post_weight_without_norm", rfwd(norm(), pw=A), INVALID)
add("rfwd_post_rstd_without_norm", rfwd(norm(), pr=A), INVALID)
add("rfwd_post_mean_rms", rfwd(norm(post_norm="rms"), pm=A), INVALID)
add("rfwd_gate_misaligned", rfwd(norm(), gate=A + 4), ALIGN)


def rbwd(d, dr=A, dn=A, r=A, cr=None, y=A, cy=None, pm=None, pr=None, m=A, rs=A, pw=None, gate=None, w=None, s=None,
         dx=A, dy=A, dpw=None, dg=None, dw=None, ds=None, dt=None, ws=A, nbytes=BIG):
    return lib.ssta_residual_norm_bwd(ctypes.byref(d), dr, dn, r, cr, y, cy, pm, pr, m, rs, pw, gate, w, s, dx, dy,
                                      dpw, dg, dw, ds, dt, ws, nbytes, None)


add("rbwd_valid", rbwd(norm(post_norm="layer"), pm=A, pr=A, dpw=A, dg=A, dw=A, ds=A, dt=A), LAUNCH)
add("rbwd_valid_saved", rbwd(norm(), r=None, cr=ck(), y=None, cy=ck(), gate=A, dg=A), LAUNCH)
add("rbwd_only_dr", rbwd(norm(), dn=None, r=None, m=None, rs=None, y=None), LAUNCH)
add("rbwd_only_dn", rbwd(norm(), dr=None, y=None), LAUNCH)
add("rbwd_no_gradient", rbwd(norm(), dr=None, dn=None), INVALID)
add("rbwd_dn_without_norm", rbwd(norm(norm="none")), INVALID)
add("rbwd_dn_without_r", rbwd(norm(), r=None), INVALID)
add("rbwd_two_r", rbwd(norm(), cr=ck()), INVALID)
add("rbwd_two_y", rbwd(norm(), cy=ck()), INVALID)
add("rbwd_mixed_kinds", rbwd(norm(), r=None, cr=ck(), dg=A), INVALID)
add("rbwd_mixed_formats", rbwd(norm(), r=None, cr=ck(), y=None, cy=ck(fmt=1), dg=A), INVALID)
add("rbwd_unused_y_of_other_kind", rbwd(norm(), r=None, cr=ck()), LAUNCH)
add("rbwd_dweight_without_dn", rbwd(norm(), dn=None, dw=A), INVALID)
add("rbwd_dgate_without_y", rbwd(norm(), y=None, dg=A), INVALID)
add("rbwd_post_without_y", rbwd(norm(post_norm="rms"), y=None, pr=A), INVALID)
add("rbwd_post_without_rstd", rbwd(norm(post_norm="rms")), INVALID)
add("rbwd_dpost_without_norm", rbwd(norm(), dpw=A), INVALID)
add("rbwd_no_dy", rbwd(norm(), dy=None), INVALID)
add("rbwd_short_workspace", rbwd(norm(), nbytes=0), WS)


def cks(rows=4, C=256, dtype=0, x=A, c=None):
    c = c or ck()
    return lib.ssta_checkpoint_save(rows, C, dtype, x, c, None), lib.ssta_checkpoint_load(rows, C, dtype, c, x, None)


for i, which in enumerate(("save", "load")):
    add(f"ckpt_{which}_valid", cks()[i], LAUNCH)
    add(f"ckpt_{which}_rows_0", cks(rows=0)[i], INVALID)
    add(f"ckpt_{which}_C_0", cks(C=0)[i], INVALID)
    add(f"ckpt_{which}_C_4", cks(C=4)[i], UNSUP)
    add(f"ckpt_{which}_too_many", cks(rows=1 << 60)[i], UNSUP)
    add(f"ckpt_{which}_dtype", cks(dtype=9)[i], INVALID)
    add(f"ckpt_{which}_null_x", cks(x=None)[i], INVALID)
    add(f"ckpt_{which}_format", cks(c=ck(fmt=-1))[i], INVALID)
    add(f"ckpt_{which}_misaligned_x", cks(x=A + 8)[i], ALIGN)
    add(f"ckpt_{which}_misaligned_codes", cks(c=ck(codes=A + 8))[i], ALIGN)
add("ckpt_save_null", lib.ssta_checkpoint_save(4, 256, 0, A, None, None), INVALID)
add("ckpt_load_null", lib.ssta_checkpoint_load(4, 256, 0, None, A, None), INVALID)


def desc(**kw):
    base = dict(B=1, H=2, D=128, T=4, Y=8, X=8, tT=2, tY=4, tX=4, wT=1, wY=1, wX=1, topk=2, L_text=0,
                dtype=S.SSTA_F32, scale=0.0)
    base.update(kw)
    return S.Desc(**base)


def abwd(d, q=None, o=None, lse=A, do=A, dk=A, ws=A, nbytes=BIG, null_v=False):
    return lib.ssta_attention_bwd_checkpoint(ctypes.byref(d), q or ck(), ck(), None if null_v else ck(), o or ck(), lse,
                                             do, A, A, A, dk, A, ws, nbytes, None)


need = ctypes.c_size_t(0)
add("abwd_ws_null", lib.ssta_attention_bwd_checkpoint_workspace(ctypes.byref(desc()), None), INVALID)
add("abwd_ws_bad_desc", lib.ssta_attention_bwd_checkpoint_workspace(ctypes.byref(desc(T=0)), ctypes.byref(need)), INVALID)
add("abwd_ws_ok", lib.ssta_attention_bwd_checkpoint_workspace(ctypes.byref(desc()), ctypes.byref(need)), OK)
add("abwd_ws_bytes", OK if need.value == S.ssta_plan(desc()).bwd_workspace_bytes + 3 * 2 * 256 * 128 * 4 else 99, OK)
add("abwd_null_v", abwd(desc(), null_v=True), INVALID)
add("abwd_mixed_formats", abwd(desc(), o=ck(fmt=1)), INVALID)
add("abwd_null_lse", abwd(desc(), lse=None), INVALID)
add("abwd_misaligned_dk", abwd(desc(), dk=A + 8), ALIGN)
add("abwd_misaligned_codes", abwd(desc(), q=ck(codes=A + 8)), ALIGN)
add("abwd_short_workspace", abwd(desc(), nbytes=need.value - 1), WS)
add("abwd_ws_misaligned", abwd(desc(), ws=A + 16), ALIGN)
add("abwd_bf16_tile_not_128", abwd(desc(dtype=S.SSTA_BF16)), UNSUP)
add("abwd_bad_desc", abwd(desc(topk=-1)), INVALID)
add("abwd_valid", abwd(desc()), LAUNCH)

for name, got, want in cases:
    print(name, got, want)
