"""Checkpoints of groups of very small numbers: the bounds that the header states, where the
exponent byte is held at 1, and what a bf16 reader gets."""
import pytest
import torch

import block_sparse_video_ssta_b200 as S

pytestmark = pytest.mark.gpu


def small(dtype):
    """A row per largest magnitude from the smallest subnormal on, normal values below it."""
    gen = torch.Generator().manual_seed(4)
    tops = torch.pow(2.0, torch.arange(-149, -108, dtype=torch.float64))
    rows = torch.randn(len(tops), 128, generator=gen, dtype=torch.float64).clamp(-3, 3) / 3
    rows[:, 7] = 1.0
    return (rows * tops[:, None]).to(dtype).cuda()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stated_bounds(cuda_ok, dtype, fmt):
    x = small(dtype)
    ck = S.ssta_checkpoint_save(x, fmt)
    E, v, got = ck.exponents.double(), x.double(), S.ssta_checkpoint_load(ck).double()
    assert (E >= 1).all() and (E == 1).any() and (E >= 10).any()
    if fmt == "int8":
        bound = torch.exp2(E - 128).expand_as(v)
        top = v.abs().amax(1, keepdim=True)
        free = top >= 63.75 * 2.0 ** -126
        assert (E[~free] == 1).all() and (torch.exp2(E - 128) <= top / 127.5)[free].all()
    else:
        bound = torch.where(v.abs() < torch.exp2(E - 133), torch.exp2(E - 137), v.abs() * 2.0 ** -4)
    assert ((got - v).abs() <= bound).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read_as_bf16(cuda_ok, fmt):
    """The values of a bf16 tensor are bf16 numbers, those of an int8 checkpoint always; the others are rounded."""
    for dtype in (torch.bfloat16, torch.float32):
        ck = S.ssta_checkpoint_save(small(dtype), fmt)
        exact = S.ssta_checkpoint_load(S.Checkpoint(ck.codes, ck.exponents, torch.float32))
        got = S.ssta_checkpoint_load(S.Checkpoint(ck.codes, ck.exponents, torch.bfloat16))
        assert torch.equal(got, exact.bfloat16())
        same = torch.equal(got.float(), exact)
        assert same == (dtype == torch.bfloat16 or fmt == "int8")
