"""CPU checks of the norm, residual and checkpoint calls: every refusal of the C ABI
with its status, the planned sizes, and the binding's own refusals."""
import os
import subprocess
import sys

import pytest
import torch

import block_sparse_video_ssta_b200 as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_validation_codes():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "norm_abi_cases.py")], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = [line.split() for line in r.stdout.strip().splitlines()]
    assert len(lines) > 100
    wrong = [(n, got, want) for n, got, want in lines if got != want]
    assert not wrong, wrong


@pytest.mark.parametrize("rows,C,mod_rows,groups", [(1, 8, 0, 1), (256, 2048, 0, 1), (49290, 1544, 1590, 31),
                                                    (100, 128, 1, 100), (7, 136, 3, 3), (10, 256, 64, 1),
                                                    (219600, 2048, 0, 1), (5, 8192, 2, 3)])
def test_plan(rows, C, mod_rows, groups):
    p = S.ssta_norm_plan(S.norm_desc(rows, C, mod_rows=mod_rows))
    assert p.groups == groups and p.exponents_per_row == -(-C // 128)
    # room for the three sums of every group at least, and for no more runs than keep the SMs busy
    assert p.bwd_workspace_bytes >= groups * 3 * C * 4
    assert p.bwd_workspace_bytes <= max(groups, 4 * 2 * 148) * 3 * C * 4 + 256


def test_plan_does_not_depend_on_types():
    sizes = {S.ssta_norm_plan(S.norm_desc(5000, 1000, dtype=d, param_dtype=p, norm=n, post_norm=q)).bwd_workspace_bytes
             for d in ("bf16", "f32") for p in ("bf16", "f32") for n in ("layer", "rms") for q in ("none", "rms")}
    assert len(sizes) == 1


def test_binding_refuses_cpu_tensors():
    d = S.norm_desc(4, 128)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    v = torch.zeros(4)
    for call in (lambda: S.ssta_norm_fwd(d, x), lambda: S.ssta_norm_bwd(d, x, x, v, v),
                 lambda: S.ssta_residual_norm_fwd(d, x, x), lambda: S.ssta_residual_norm_bwd(d, x, x, x, x, v, v),
                 lambda: S.ssta_checkpoint_save(x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_checkpoint_refusals_without_a_device():
    with pytest.raises(ValueError, match="format"):
        S.Checkpoint.empty((4, 128), "int4", device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.Checkpoint(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dtype"):
        S.Checkpoint(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
