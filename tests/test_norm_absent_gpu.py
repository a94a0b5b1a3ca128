"""What no formula reads does not reach a result: with no gradient of n, the norm's vectors."""
import pytest
import torch

import block_sparse_video_ssta_b200 as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows,C", [(9, 264), (300, 128), (40, 4104)])
@pytest.mark.parametrize("post", ["none", "rms"])
def test_without_a_gradient_of_n_the_norms_vectors_do_not_matter(cuda_ok, rows, C, post, bad):
    gen = torch.Generator().manual_seed(rows)
    n = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()
    dr, r, y, gate = n(rows, C), n(rows, C), n(rows, C), n(1, C).float()
    d = S.norm_desc(rows, C, norm="layer", post_norm=post, res_scale=0.5)
    prstd = torch.ones(rows, device="cuda") if post != "none" else None
    call = lambda **kw: S.ssta_residual_norm_bwd(d, dr, None, r, y, gate=gate, post_rstd=prstd, **kw)
    want = call()
    weight, scale = torch.ones(C, device="cuda"), torch.zeros(1, C, device="cuda")
    weight[3], scale[0, C - 1] = bad, bad
    got = call(weight=weight, scale=scale)
    assert torch.equal(want.dx, 0.5 * dr)
    for name in ("dx", "dy", "dgate"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    assert got.dweight is None and got.dscale is None and got.dshift is None
