"""The global gradient norm and clipping by it, against 64-bit sums.

Bounds: squares are summed in fp32 over at most a few hundred elements (each
sum off by at most 2^9 2^-24 relatively, all terms being positive) and in 64
bits from there, so the norm is within 2^-15; the clipped value is one fp32
factor (quotient and product: 2^-22) and one rounding.
"""
import ctypes
import math

import pytest
import torch

import weight_grad_gemm_gb300 as fg

gpu = pytest.mark.gpu
FAKE = ctypes.c_void_p(0x10000)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def tensors(sizes, dtype, seed=0, offset=0, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        buf = torch.zeros(n + offset, dtype=DT[dtype], device="cuda")
        buf[offset:] = (torch.randn(n, generator=g) * std).to(DT[dtype]).cuda()
        out.append(buf[offset:])
    return out


def norm_of(ts):
    return math.sqrt(sum(float((t.cpu().double() ** 2).sum()) for t in ts))


SIZES = {"none": [], "empty": [0, 0], "one": [1], "mixed": [1, 0, 7, 4096, 65537, 3, 300000, 2],
         "many": [17 + 13 * i for i in range(700)], "long": [5_000_003], "thousands": [5] * 2500}


@gpu
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", list(SIZES))
def test_norm(cuda_device, kind, dtype, offset):
    ts = tensors(SIZES[kind], dtype, offset=offset)
    norm = torch.full((1,), 9.0, device="cuda")
    fg.forge_grad_norm(ts, norm)
    want = norm_of(ts)
    assert abs(norm.item() - want) <= 2.0 ** -15 * want
    again = torch.full((1,), 9.0, device="cuda")
    fg.forge_grad_norm(ts, again)
    assert torch.equal(norm, again)


@gpu
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("std", [1e-37, 1e-30, 1e-23, 1e-18, 1e-15, 1e15, 1e18, 1e25, 1e33])
def test_norm_over_the_whole_range(cuda_device, std, dtype, offset):
    """Gradients whose squares fp32 does not hold (below 2^-149, above 2^128) or
    holds with few digits (below 2^-126); the bound is that of ordinary ones."""
    for sizes in ([1], [7, 4096], SIZES["mixed"]):
        ts = tensors(sizes, dtype, offset=offset, std=std)
        norm = torch.full((1,), 9.0, device="cuda")
        fg.forge_grad_norm(ts, norm)
        want = norm_of(ts)
        assert abs(norm.item() - want) <= 2.0 ** -15 * want + 2.0 ** -149
        # beside ordinary ones, zeros of both signs among them
        zeros = torch.zeros(50001, dtype=DT[dtype], device="cuda")
        zeros[::3] = -0.0
        usual = tensors([3000], dtype, std=max(std, 1e-19))
        fg.forge_grad_norm([zeros, *ts, *usual], norm)
        want = norm_of([*ts, *usual])
        assert abs(norm.item() - want) <= 2.0 ** -15 * want
        fg.forge_grad_norm([zeros], norm)
        assert norm.item() == 0.0


@gpu
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6, math.inf])
def test_clip(cuda_device, dtype, out, max_norm, offset):
    sizes = SIZES["mixed"] + [1000] * 600
    ts = tensors(sizes, dtype, offset=offset)
    norm = torch.empty(1, device="cuda")
    fg.forge_grad_norm(ts, norm)
    os_ = [torch.full((n + 2,), 3.0, dtype=DT[out], device="cuda") for n in sizes]
    fg.forge_clip_grads(ts, norm, [o[:n] for o, n in zip(os_, sizes)], max_norm=max_norm)
    c = min(1.0, max_norm / (norm.item() + 1e-6)) if max_norm < math.inf else 1.0
    for t, o, n in zip(ts, os_, sizes):
        want = t.cpu().double() * c
        err = (o[:n].cpu().double() - want).abs()
        assert torch.all(err <= want.abs() * (2.0 ** -22 + (2.0 ** -8 if out == "bf16" else 0)) + 2.0 ** -126)
        assert (o[n:] == 3.0).all()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_norm", [0.25, 1e6])
def test_clip_in_place_equals_clip_into_copies(cuda_device, dtype, max_norm):
    ts = tensors(SIZES["mixed"], dtype)
    norm = torch.empty(1, device="cuda")
    fg.forge_grad_norm(ts, norm)
    copies = [torch.empty_like(t) for t in ts]
    fg.forge_clip_grads(ts, norm, copies, max_norm=max_norm)
    fg.forge_clip_grads(ts, norm, max_norm=max_norm)
    assert all(torch.equal(a, b) for a, b in zip(ts, copies))
    after = torch.empty(1, device="cuda")
    fg.forge_grad_norm(ts, after)
    bound = min(max_norm, norm.item()) * (1 + 2.0 ** -8)
    assert after.item() <= bound


@gpu
def test_zero_nan_and_infinite_gradients(cuda_device):
    norm = torch.empty(1, device="cuda")
    zero = [torch.zeros(1000, device="cuda")]
    fg.forge_grad_norm(zero, norm)
    fg.forge_clip_grads(zero, norm, max_norm=1.0)
    assert norm.item() == 0.0 and not zero[0].any()
    for bad, nan_norm in ((math.nan, True), (math.inf, False)):
        ts = tensors([1000, 77], "f32")
        ts[1][5] = bad
        fg.forge_grad_norm(ts, norm)
        assert math.isnan(norm.item()) if nan_norm else norm.item() == math.inf
        fg.forge_clip_grads(ts, norm, max_norm=1.0)
        if nan_norm:
            assert all(torch.isnan(t).all() for t in ts)
        else:  # the factor is 0: finite entries vanish, inf * 0 is NaN
            assert not ts[0].any() and math.isnan(ts[1][5].item())


@gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_no_limit_clips_nothing_even_by_an_infinite_norm(cuda_device, out):
    ts = tensors([1000, 77], "f32")
    ts[1][5] = -math.inf
    norm = torch.empty(1, device="cuda")
    fg.forge_grad_norm(ts, norm)
    assert norm.item() == math.inf
    os_ = [torch.full_like(t, 3.0, dtype=DT[out]) for t in ts]
    fg.forge_clip_grads(ts, norm, os_, max_norm=math.inf)
    assert all(torch.equal(o, t.to(DT[out])) for o, t in zip(os_, ts))
    kept = [t.clone() for t in ts]
    fg.forge_clip_grads(ts, norm, max_norm=math.inf)
    assert all(torch.equal(t, u) for t, u in zip(ts, kept))
    fg.forge_clip_grads(ts, torch.full((1,), math.nan, device="cuda"), max_norm=math.inf)
    assert all(torch.isnan(t).all() for t in ts)


@gpu
def test_large_tensor_past_32_bit_offsets(cuda_device):
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-1] = 3.0
    t[0] = 4.0
    norm = torch.empty(1, device="cuda")
    fg.forge_grad_norm([t], norm)
    assert norm.item() == 5.0
    fg.forge_clip_grads([t], norm, max_norm=2.5)
    assert t[-1].item() == 1.5 and t[0].item() == 2.0 and not t[1:1000].any()


@gpu
def test_streams_and_graphs(cuda_device):
    ts = tensors(SIZES["mixed"], "f32")
    norm, side_norm = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    outs = [torch.empty_like(t) for t in ts]
    fg.forge_grad_norm(ts, norm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fg.forge_grad_norm(ts, side_norm, stream=side)
    side.synchronize()
    assert torch.equal(norm, side_norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.forge_grad_norm(ts, side_norm)
        fg.forge_clip_grads(ts, side_norm, outs, max_norm=0.5)
    side_norm.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, side_norm)
    want = 0.5 / (norm.item() + 1e-6)
    assert abs(outs[6][0].item() - ts[6][0].item() * want) <= abs(outs[6][0].item()) * 2.0 ** -21


def test_refusals_before_any_launch():
    L = fg.lib()
    ptrs = (ctypes.c_void_p * 2)(0x10000, 0x20000)
    holes = (ctypes.c_void_p * 2)(0x10000, None)
    n, neg = (ctypes.c_int64 * 2)(5, 6), (ctypes.c_int64 * 2)(5, -1)

    def f(g=ptrs, n=n, P=2, dt=fg.FORGE_F32, norm=FAKE):
        return L.forge_grad_norm(g, n, P, dt, norm, None)

    def c(g=ptrs, n=n, P=2, dt=fg.FORGE_F32, norm=FAKE, max_norm=1.0, out=ptrs, odt=fg.FORGE_F32):
        return L.forge_clip_grads(g, n, P, dt, norm, max_norm, out, odt, None)
    for fn in (f, c):
        for kw in (dict(norm=None), dict(P=-1), dict(g=None), dict(n=None), dict(n=neg), dict(g=holes)):
            assert fn(**kw) == fg.FORGE_ERR_INVALID_ARG, kw
        assert fn(dt=fg.FORGE_E4M3) == fg.FORGE_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(out=None), dict(out=holes)):
        assert c(**kw) == fg.FORGE_ERR_INVALID_ARG, kw
    assert c(odt=fg.FORGE_I32) == fg.FORGE_ERR_UNSUPPORTED_DTYPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU what is not refused stops at the device check")
def test_clip_refuses_outputs_that_overlap_their_gradients():
    L = fg.lib()
    es = {fg.FORGE_F32: 4, fg.FORGE_BF16: 2}
    n = 24
    for dt in es:
        for odt in es:
            for d in range(-100, 101, 4):
                for size in (n, 0):
                    g = (ctypes.c_void_p * 2)(0x90000, 0x10000)
                    o = (ctypes.c_void_p * 2)(0x80000, 0x10000 + d)
                    sizes = (ctypes.c_int64 * 2)(5, size)
                    s = L.forge_clip_grads(g, sizes, 2, dt, FAKE, 1.0, o, odt, None)
                    apart = d >= size * es[dt] or -d >= size * es[odt] or size == 0
                    fine = apart or (d == 0 and dt == odt)
                    assert s == (fg.FORGE_ERR_UNSUPPORTED_DEVICE if fine else fg.FORGE_ERR_INVALID_ARG), (dt, odt, d)


@gpu
def test_binding_refuses_what_does_not_fit(cuda_device):
    ts = tensors([4, 5], "f32")
    norm = torch.empty(1, device="cuda")
    with pytest.raises(TypeError):
        fg.forge_grad_norm([ts[0], ts[1].bfloat16()], norm)
    with pytest.raises(ValueError):
        fg.forge_clip_grads(ts, norm, [ts[0]], max_norm=1.0)
    with pytest.raises(ValueError):
        fg.forge_grad_norm([torch.zeros(4, 4, device="cuda")[:, :2]], norm)
    with pytest.raises(ValueError):
        fg.forge_grad_norm(ts, torch.empty(2, device="cuda"))
    with pytest.raises(ValueError):
        fg.forge_grad_norm([t.cpu() for t in ts], norm)
    with pytest.raises(fg.ForgeError):
        fg.forge_clip_grads(ts, norm, max_norm=-1.0)
