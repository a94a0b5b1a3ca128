"""8-bit checkpoints on the GPU: codes and exponents equal the oracle's exactly (the code
has no rounding but its own), values are exact, and the attention's backward from
checkpoints matches the oracle at the checkpoints' values."""
import numpy as np
import pytest
import torch

import block_sparse_video_ssta_b200 as S
import oracle
import ssta_inputs as si
from norm_helpers import f64
from ssta_inputs import with_overrides
from ssta_parity import gpu_kept, run_gpu, to_np

pytestmark = pytest.mark.gpu

FORMATS = ("int8", "e4m3")


def _same(ck, x):
    codes, exps = oracle.checkpoint_encode(f64(x).reshape(-1, x.shape[-1]), ck.format)
    got_e = ck.exponents.cpu().numpy().reshape(exps.shape)
    np.testing.assert_array_equal(got_e, exps)
    np.testing.assert_array_equal(f64(ck.codes.float()).reshape(codes.shape), codes)
    v = S.ssta_checkpoint_load(ck)
    assert v.dtype == x.dtype and v.shape == x.shape
    np.testing.assert_array_equal(f64(v).reshape(codes.shape), oracle.checkpoint_decode(codes, exps))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 8), (1, 128), (5, 120), (7, 136), (3, 2, 256), (65, 1000), (129, 128), (2, 16392)])
def test_codes_are_the_definition(cuda_ok, fmt, dtype, shape):
    gen = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=gen)
    rows = x.view(-1, shape[-1])
    rows *= torch.exp(4 * torch.randn(rows.shape[0], 1, generator=gen))
    _same(S.ssta_checkpoint_save(x.to(dtype).cuda(), fmt), x.to(dtype).cuda())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_at_the_edges(cuda_ok, fmt, dtype):
    """Zeros of both signs, the largest and smallest numbers, subnormals, groups whose largest magnitude sits at a
    power of two or next to the limit of a scale, and every tie between two codes."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    rows = [torch.zeros(128), -torch.zeros(128), torch.full((128,), big), torch.full((128,), tiny),
            torch.full((128,), tiny / 64), torch.linspace(-1, 1, 128) * tiny]
    for top in (127.0, 127.5, 128.0, 126.5, 448.0, 449.0, 464.0, 480.0, 1.0, 2.0, 255.0, 254.0):
        for e in (0, -20, 60, -120):
            r = torch.arange(128) * 0.5 + 0.25
            r[:64] = torch.arange(64) + 0.5            # ties of the int8 code at scale 1
            r[64:96] = (torch.arange(32) * 2 + 1) * 2.0 ** -10    # ties of the e4m3 subnormals at scale 1
            r[96:126] = (2 * torch.arange(30) + 17) * 0.5         # ties of e4m3 binades
            r = r.clamp(max=top)
            r[127] = -top
            rows.append(r * 2.0 ** e)
    x = torch.stack(rows).to(dtype).cuda()
    _same(S.ssta_checkpoint_save(x, fmt), x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_16_bit_pattern(cuda_ok, fmt, dtype):
    """All finite bf16 numbers, each in a group with a fixed large neighbour and alone with smaller ones."""
    bits = torch.arange(65536, dtype=torch.int32)
    v = (bits << 16).view(torch.float32)
    v = v[torch.isfinite(v)]
    alone = torch.zeros(v.numel(), 8)
    alone[:, 0], alone[:, 1], alone[:, 5] = v, v * 0.3, -v * 0.01
    with_top = alone.clone()
    with_top[:, 7] = 448.0
    x = torch.cat([alone, with_top]).to(dtype).cuda()
    _same(S.ssta_checkpoint_save(x, fmt), x)


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_groups_read_as_nan(cuda_ok, fmt):
    x = torch.randn(4, 304, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    x[0, 3], x[1, 130], x[2, 299] = float("inf"), float("nan"), float("-inf")
    ck = S.ssta_checkpoint_save(x, fmt)
    e = ck.exponents.cpu()
    assert e[0, 0] == 255 and e[1, 1] == 255 and e[2, 2] == 255 and int((e == 255).sum()) == 3
    v = S.ssta_checkpoint_load(ck).float().cpu()
    nan = torch.isnan(v)
    want = torch.zeros_like(nan)
    want[0, :128] = want[1, 128:256] = want[2, 256:] = True
    assert torch.equal(nan, want)


def test_buffers_are_reused_and_framed(cuda_ok):
    ck = S.Checkpoint.empty((9, 1000), "int8")
    out = torch.full((11, 1000), 5.0, dtype=torch.bfloat16, device="cuda")
    for seed in range(3):
        x = torch.randn(9, 1000, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        assert S.ssta_checkpoint_save(x, out=ck) is ck
        v = S.ssta_checkpoint_load(ck, out[1:10])
        assert torch.equal(v, S.ssta_checkpoint_load(S.ssta_checkpoint_save(x)))
        assert (out[0] == 5).all() and (out[10] == 5).all()


def test_addresses_are_those_of_the_call(cuda_ok):
    """A checkpoint's tensors cannot be swapped for others, and where their storage moves the call follows."""
    x = torch.randn(16, 256, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    ck = S.ssta_checkpoint_save(x)
    want = S.ssta_checkpoint_load(ck)
    with pytest.raises(AttributeError):
        ck.codes = ck.codes.clone()
    old = ck.codes.clone()
    keep = ck.codes.data
    ck.codes.data = old.clone()       # the same values elsewhere
    keep.zero_()
    assert torch.equal(S.ssta_checkpoint_load(ck), want)


# The kernels behind are those of ssta_attention_bwd; the tolerances are those of its test, for the same arithmetic.
TOL = {"f32": dict(rel=1e-4, mx=1e-4, row=1e-4), "bf16": dict(rel=1e-2, mx=2e-2, row=5e-2)}
ATTENTION = [
    ("tiny_f32", {}, "int8"),
    ("tiny_f32", dict(T=5, Y=7, X=6, L_text=45), "e4m3"),
    ("tiny_f32", dict(combine="and", topk=0), "int8"),                       # nothing kept: all zero
    ("small_bf16", dict(H=2, T=8, Y=16, X=24), "int8"),
    ("small_bf16", dict(H=2, T=7, Y=12, X=20, L_text=300), "e4m3"),
    ("small_bf16", dict(H=2, T=4, Y=8, X=16, tT=2, tY=8, tX=8), "int8"),      # N = 128
    ("small_bf16", dict(H=2, T=8, Y=16, X=24, score_mode="importance", combine="and", topk=6), "e4m3"),
    ("small_bf16", dict(B=2, H=3, T=5, Y=12, X=20, L_text=130), "int8"),
]


def _attention(name, ov, fmt):
    w = with_overrides(si.get_workload(name), **ov)
    x = si.make_inputs(w, 3, device="cuda")
    r = run_gpu(w, x)
    d = S.desc_from(w)
    dO = torch.randn(r["O_packed"].shape, generator=torch.Generator().manual_seed(11)).to(r["O_packed"].dtype).cuda()
    ck = [S.ssta_checkpoint_save(r[n], fmt) for n in ("qp", "kp", "vp", "O_packed")]
    return w, d, r, dO, ck


@pytest.mark.parametrize("name,ov,fmt", ATTENTION, ids=[str(i) for i in range(len(ATTENTION))])
def test_attention_backward_from_checkpoints(cuda_ok, name, ov, fmt):
    w, d, r, dO, ck = _attention(name, ov, fmt)
    dq, dk, dv, ws = S.ssta_attention_bwd_checkpoint(d, *ck, r["LSE"], dO, r["kv_idx"], r["kv_cnt"])
    assert S.ssta_read_device_status(ws) == 0
    values = [to_np(S.ssta_checkpoint_load(c)) for c in ck]
    ref = oracle.attention_bwd_saved(w, *values, to_np(r["LSE"]), to_np(dO), gpu_kept(w, r["kv_idx"], r["kv_cnt"]))
    tol = TOL[w.dtype]
    for n, got, want in zip(("dq", "dk", "dv"), (dq, dk, dv), ref):
        a = to_np(got)
        assert np.isfinite(a).all()
        top = max(np.abs(want).max(), 1e-30)
        assert np.abs(a - want).max() / top <= tol["mx"], n
        assert np.linalg.norm(a - want) / max(np.linalg.norm(want), 1e-30) <= tol["rel"], n
        rn = np.linalg.norm(want.reshape(-1, 128), axis=1)
        en = np.linalg.norm((a - want).reshape(-1, 128), axis=1)
        big = rn > 1e-3 * max(rn.max(), 1e-30)
        assert not big.any() or (en[big] / rn[big]).max() <= tol["row"], n


def test_attention_backward_equals_the_dense_one_on_the_same_values(cuda_ok):
    """The same kernels on the checkpoints' values give the same bytes, whatever the reused workspace and outputs
    held before."""
    w, d, r, dO, ck = _attention("small_bf16", dict(H=2, T=7, Y=12, X=20, L_text=300), "int8")
    values = [S.ssta_checkpoint_load(c) for c in ck]
    want = S.ssta_attention_bwd(d, *values, r["LSE"], dO, r["kv_idx"], r["kv_cnt"])[:3]
    ws = None
    outs = [torch.full_like(values[0], float("nan")) for _ in range(3)]
    for _ in range(3):
        *got, ws = S.ssta_attention_bwd_checkpoint(d, *ck, r["LSE"], dO, r["kv_idx"], r["kv_cnt"], *outs, workspace=ws)
        assert S.ssta_read_device_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ws.fill_(0xff)


def test_attention_backward_captured_and_on_a_stream(cuda_ok):
    w, d, r, dO, ck = _attention("small_bf16", dict(H=2, T=8, Y=16, X=24), "int8")
    call = lambda **kw: S.ssta_attention_bwd_checkpoint(d, *ck, r["LSE"], dO, r["kv_idx"], r["kv_cnt"], **kw)
    want = [t.clone() for t in call()[:3]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    dO.mul_(2)          # gradients are linear in dO, and doubling is exact
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, 2 * b) for a, b in zip(outs, want))


def test_attention_backward_refusals(cuda_ok):
    w, d, r, dO, ck = _attention("small_bf16", dict(H=1, T=4, Y=8, X=16), "int8")
    rest = (r["LSE"], dO, r["kv_idx"], r["kv_cnt"])
    other = S.ssta_checkpoint_save(r["O_packed"], "e4m3")
    with pytest.raises(S.SstaError) as e:
        S.ssta_attention_bwd_checkpoint(d, *ck[:3], other, *rest)
    assert e.value.code == 1
    for bad in ([r["qp"]] + ck[1:], ck[:3] + [S.Checkpoint.empty((1, 1, 8, 128))],
                ck[:3] + [S.Checkpoint(ck[3].codes, ck[3].exponents, torch.float32)]):
        with pytest.raises(ValueError):
            S.ssta_attention_bwd_checkpoint(d, *bad, *rest)
    with pytest.raises(S.SstaError) as e:
        S.ssta_attention_bwd_checkpoint(d, *ck, *rest, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
