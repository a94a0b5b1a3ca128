"""What the attention sub-block keeps between forward and backward, when the caller writes to the tensors it got."""
import copy

import pytest
import torch

import block_sparse_video_ssta_b200 as S
import ssta_inputs as si
from block_sparse_video_ssta_b200.attention_block import ssta_block_backward, ssta_block_forward
from ssta_inputs import with_overrides
from test_attention_block_gpu import block_inputs

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dmod", "dqkv", "dout", "dq_norm", "dk_norm")


def block():
    w = with_overrides(si.get_workload("small_bf16"), H=1, T=4, Y=8, X=16, L_text=5)
    return S.desc_from(w), block_inputs(w, 2)


def same(a, b):
    return all(torch.equal(getattr(a, n), getattr(b, n)) for n in NAMES)


def next_residual(r, y):
    """The sub-block behind, over r itself."""
    nd = S.norm_desc(r.numel() // r.shape[-1], r.shape[-1])
    assert S.ssta_residual_norm_fwd(nd, r, y, r=r).r is r


WRITES = {"library": next_residual, "view": lambda r, y: next_residual(r.view(-1, r.shape[-1]), y.view(-1, r.shape[-1])),
          "norm": lambda r, y: S.ssta_norm_fwd(S.norm_desc(r.numel() // 128, 128), r, y=r),
          "load": lambda r, y: S.ssta_checkpoint_load(S.ssta_checkpoint_save(y), r),
          "gradient": lambda r, y: S.ssta_residual_norm_bwd(S.norm_desc(r.numel() // 128, 128, norm="none"), y, None, dx=r),
          "torch": lambda r, y: r.add_(y)}


@pytest.mark.parametrize("write", list(WRITES))
def test_a_written_residual_is_refused(cuda_ok, write):
    d, (x, mod, p, dr, dn) = block()
    r, n2, saved = ssta_block_forward(d, x, mod, p)
    want = ssta_block_backward(d, saved, p, dr, dn)
    assert same(ssta_block_backward(d, saved, p, dr, dn), want)     # as often as one likes
    before = r.clone()
    WRITES[write](r, dr)
    with pytest.raises(ValueError, match="r was written"):
        ssta_block_backward(d, saved, p, dr, dn)
    saved.r = before
    assert same(ssta_block_backward(d, saved, p, dr, dn), want)


@pytest.mark.parametrize("checkpoint", ["int8", "e4m3"])
def test_checkpoints_and_copies_are_their_own(cuda_ok, checkpoint):
    d, (x, mod, p, dr, dn) = block()
    for ck in (checkpoint, None):
        r, n2, saved = ssta_block_forward(d, x, mod, p, ck)
        want = ssta_block_backward(d, saved, p, dr, dn)
        if ck is None:
            saved.r = saved.r.clone()
        next_residual(r, dr)
        assert same(ssta_block_backward(d, saved, p, dr, dn), want)


def test_refused_calls_write_nothing(cuda_ok):
    d, (x, mod, p, dr, dn) = block()
    r, n2, saved = ssta_block_forward(d, x, mod, p)
    nd = S.norm_desc(r.numel() // r.shape[-1], r.shape[-1], eps=0.0)
    with pytest.raises(S.SstaError):
        S.ssta_residual_norm_fwd(nd, r, dr, r=r)
    with pytest.raises(ValueError):
        S.ssta_norm_fwd(S.norm_desc(r.numel() // 128, 128), r, y=r.float())
    want = ssta_block_backward(d, saved, p, dr, dn)
    twin = copy.copy(saved)
    assert same(ssta_block_backward(d, twin, p, dr, dn), want)


def test_inference_mode(cuda_ok):
    d, (x, mod, p, dr, dn) = block()
    want = ssta_block_forward(d, x, mod, p)
    with torch.inference_mode():
        got = ssta_block_forward(d, x, mod, p)
        nd = S.norm_desc(got[0].numel() // 128, 128)
        S.ssta_norm_fwd(nd, got[1], y=got[1])
    assert torch.equal(got[0], want[0])
    assert same(ssta_block_backward(d, got[2], p, dr, dn), ssta_block_backward(d, want[2], p, dr, dn))
