"""The router, its balance loss and their gradient against 64-bit forms.

Choices, counts, offsets, slots and rows are whole numbers and have to be equal.
Probabilities: exp's argument z - max is exact to half a step of fp32 and is
multiplied by log2 e (two roundings), so a term is off by |z - max| 2^-23 +
2^-22 relatively; sums and quotients of positive terms add 2^-18 (at most 1024
terms, in a tree of 32 serial ones); with |z - max| <= 40 every weight is
within 2^-16 relatively.  Sums over tokens are positive terms in fp32 (a thread's
at most 256, 32 lanes, then the blocks' in a tree): 2^-14 on the loss.  bf16
outputs add 2^-8.
"""
import ctypes

import pytest
import torch

import weight_grad_gemm_gb300 as fg

gpu = pytest.mark.gpu
FAKE = ctypes.c_void_p(0x10000)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(T, E, dtype="f32", seed=0, pad=0.05, masked=0.1, ties=False, stride=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2
    if ties:
        z = (z * 2).round() / 2
    z[torch.rand(T, E, generator=g) < masked] = -float("inf")
    z[torch.rand(T, generator=g) < pad] = -float("inf")
    buf = torch.full((T, E + stride), 9.0, dtype=DT[dtype], device="cuda")
    buf[:, :E] = z.to(DT[dtype]).cuda()
    return buf[:, :E]


def reference(z, k, normalize):
    """Every output in 64 bits, from the definition, by sorting whole rows."""
    z = z.detach().cpu().double()
    T, E = z.shape
    live = (z > -float("inf")).any(1)
    p = torch.where(live[:, None], z, torch.zeros_like(z)).softmax(1) * live[:, None]
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    experts = torch.where(z.gather(1, order) > -float("inf"), order, torch.full_like(order, -1))
    w = torch.where(experts >= 0, p.gather(1, order), torch.zeros(T, k, dtype=torch.float64))
    if normalize:
        w = w / w.sum(1, keepdim=True).where(live[:, None], torch.ones(T, 1, dtype=torch.float64))
    counts = torch.bincount(experts[experts >= 0], minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    slots = torch.full((T, k), -1, dtype=torch.int64)
    rows = torch.full((T * k,), -1, dtype=torch.int64)
    at = offsets[:-1].tolist()
    for t in range(T):
        for j in range(k):
            e = int(experts[t, j])
            if e >= 0:
                slots[t, j] = at[e]
                rows[at[e]] = t
                at[e] += 1
    n = max(1, int(live.sum()))
    loss = (counts * p.sum(0) / n).sum() * E / (k * n)
    return dict(experts=experts, weights=w, counts=counts, offsets=offsets, slots=slots, rows=rows, live=live.sum()[None], loss=loss[None], p=p)


def outputs(T, E, k):
    i = lambda *s: torch.full(s, 99, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(experts=i(T, k), weights=torch.full((T, k), 9.0, device="cuda"), counts=i(E), offsets=i(E + 1), slots=i(T, k),
                rows=i(T * k), live=i(1), loss=torch.full((1,), 9.0, device="cuda"))


def route(z, k, normalize, **kw):
    o = outputs(*z.shape, k)
    fg.forge_moe_route(z, o["experts"], o["weights"], o["counts"], o["offsets"], slots=o["slots"], rows=o["rows"],
                       live=o["live"], loss=o["loss"], normalize=normalize, **kw)
    return o


def compare(o, want):
    for name in ("experts", "counts", "offsets", "slots", "rows", "live"):
        assert torch.equal(o[name].cpu().long(), want[name]), name
    w = want["weights"]
    assert torch.all((o["weights"].cpu().double() - w).abs() <= 2.0 ** -16 * w + 2.0 ** -100)
    assert abs(float(o["loss"]) - float(want["loss"])) <= 2.0 ** -14 * float(want["loss"])


SIZES = [(1, 1, 1), (1, 8, 2), (3, 2, 2), (16, 8, 2), (33, 5, 3), (255, 16, 4), (256, 9, 2), (257, 64, 8), (300, 100, 7),
         (2000, 8, 2), (513, 256, 8), (1500, 257, 6), (200, 512, 1), (700, 513, 32), (130, 1024, 32), (5000, 17, 17), (4097, 128, 8)]


@gpu
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(cuda_device, T, E, k, dtype, normalize):
    z = make(T, E, dtype, seed=T + E)
    want = reference(z, k, normalize)
    o = route(z, k, normalize)
    compare(o, want)
    again = route(z, k, normalize)
    assert all(torch.equal(o[n], again[n]) for n in o)


@gpu
@pytest.mark.parametrize("T,E,k", [(500, 8, 2), (400, 300, 5), (700, 33, 33 - 1)])
def test_equal_logits_go_to_the_lower_expert(cuda_device, T, E, k):
    z = make(T, E, "f32", ties=True, masked=0.3)
    z[::7] = 0.0
    z[::14, ::2] = -0.0
    compare(route(z, k, True), reference(z, k, True))


@gpu
@pytest.mark.parametrize("E,k", [(8, 2), (70, 4), (400, 3)])
def test_strided_logits_and_left_out_outputs(cuda_device, E, k):
    z = make(3000, E, "bf16", stride=5)
    want = reference(z, k, True)
    o = route(z, k, True)
    compare(o, want)
    q = outputs(3000, E, k)
    fg.forge_moe_route(z, q["experts"], q["weights"], q["counts"], q["offsets"])
    for n in ("experts", "weights", "counts", "offsets"):
        assert torch.equal(q[n], o[n])
    for only in ("slots", "rows"):
        q = outputs(3000, E, k)
        fg.forge_moe_route(z, q["experts"], q["weights"], q["counts"], q["offsets"], **{only: q[only]})
        assert torch.equal(q[only], o[only])


@gpu
@pytest.mark.parametrize("T", [5, 4000])
@pytest.mark.parametrize("E,k", [(8, 2), (96, 5)])
def test_all_padding_none_and_one_expert(cuda_device, T, E, k):
    z = torch.full((T, E), -float("inf"), device="cuda")
    o = route(z, k, True)
    assert (o["experts"] == -1).all() and not o["weights"].any() and not o["counts"].any() and not o["offsets"].any()
    assert (o["slots"] == -1).all() and (o["rows"] == -1).all() and o["live"].item() == 0 and o["loss"].item() == 0
    z[:, 3] = torch.randn(T, device="cuda")  # fewer than k to choose from
    z[::3, 0] = 50.0
    compare(route(z, k, True), reference(z, k, True))
    compare(route(z, k, False), reference(z, k, False))
    none = outputs(0, E, k)
    fg.forge_moe_route(z[:0], none["experts"], none["weights"], none["counts"], none["offsets"], slots=none["slots"],
                       rows=none["rows"], live=none["live"], loss=none["loss"])
    assert not none["counts"].any() and not none["offsets"].any() and none["live"].item() == 0 and none["loss"].item() == 0


@gpu
@pytest.mark.parametrize("E,k", [(8, 3), (40, 3), (300, 3), (1000, 3)])
def test_nan_and_infinite_logits(cuda_device, E, k):
    z = make(600, E, "f32", pad=0, masked=0)
    z[1, 5], z[2, 0], z[4, 7], z[9] = float("nan"), float("inf"), -float("nan"), float("nan")
    z[11, 2] = torch.finfo(torch.float32).min
    o = route(z, k, True)
    keyed = z.clone()
    keyed[torch.isnan(keyed)] = float("inf")
    keyed[1] = torch.where(torch.isnan(z[1]), float("inf"), z[1])
    want = torch.sort(keyed, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(o["experts"].long(), want)
    bad = torch.tensor([1, 2, 4, 9], device="cuda")
    assert torch.isnan(o["weights"][bad]).all() and torch.isnan(o["loss"]).all()
    good = torch.ones(600, dtype=torch.bool)
    good[bad.cpu()] = False
    w = reference(z[good.cuda()], k, True)["weights"]
    assert torch.all((o["weights"].cpu()[good].double() - w).abs() <= 2.0 ** -16 * w + 2.0 ** -100)
    assert int(o["offsets"][-1]) == 600 * k


def reference_grad(z, ref, counts, k, normalize, gw, gl):
    """By automatic differentiation in 64 bits."""
    z = z.detach().cpu().double().requires_grad_()
    T, E = z.shape
    live = (z > -float("inf")).any(1).detach()
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    p = zz.softmax(1) * live[:, None]
    e = ref["experts"]
    w = torch.where(e >= 0, p.gather(1, e.clamp(min=0)), torch.zeros(()).double())
    if normalize:
        w = w / torch.where(live[:, None], w.sum(1, keepdim=True), torch.ones(()).double())
    n = max(1, int(live.sum()))
    total = 0 * z[live].exp().sum()
    if gw is not None:
        total = total + (gw.cpu().double() * w).sum()
    if gl is not None:
        total = total + gl.cpu().double()[0] * (ref["counts"] * p.sum(0) / n).sum() * E / (k * n)
    (g,) = torch.autograd.grad(total, z)
    return torch.nan_to_num(g, nan=0.0)


@gpu
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (16, 8, 2), (257, 5, 3), (300, 64, 8), (400, 200, 6), (333, 256, 8), (150, 500, 4), (90, 1024, 32)])
def test_gradient(cuda_device, T, E, k, dtype, out, normalize):
    """Bound: each p is within 2^-16 relatively (above), so p (q - sum p q) is within
    2^-15 of p (|q| + sum p |q|), q's own parts taken by magnitude."""
    z = make(T, E, dtype, seed=T)
    ref = reference(z, k, normalize)
    g = torch.Generator().manual_seed(3)
    gw, gl = torch.randn(T, k, generator=g).cuda(), (torch.rand(1, generator=g) + 0.5).cuda()
    counts, live = ref["counts"].int().cuda(), ref["live"].int().cuda()
    experts = ref["experts"].int().cuda()
    for a, b in ((gw, gl), (gw, None), (None, gl), (None, None)):
        d = torch.full((T, E + 3), 4.0, dtype=DT[out], device="cuda")
        fg.forge_moe_route_grad(z, experts, counts, live, d[:, :E], grad_weights=a, grad_loss=b, normalize=normalize)
        want = reference_grad(z, ref, counts, k, normalize, a, b)
        p = ref["p"]
        n = max(1, int(ref["live"]))
        q = torch.zeros(T, E, dtype=torch.float64)
        if b is not None:
            q += float(b) * E / (k * n * n) * ref["counts"]
        if a is not None:
            w = a.cpu().double().abs()
            if normalize:
                mass = (p.gather(1, ref["experts"].clamp(min=0)) * (ref["experts"] >= 0)).sum(1, keepdim=True).clamp(min=1e-300)
                w = (w + (w * ref["weights"]).sum(1, keepdim=True)) / mass
            q.scatter_add_(1, ref["experts"].clamp(min=0), torch.where(ref["experts"] >= 0, w, torch.zeros(()).double()))
        bound = 2.0 ** -15 * p * (q + (p * q).sum(1, keepdim=True))
        bound = bound + (2.0 ** -8 if out == "bf16" else 0) * (want.abs() + bound) + 2.0 ** -120
        assert torch.all((d[:, :E].cpu().double() - want).abs() <= bound)
        assert (d[:, E:] == 4.0).all()
        if dtype == out and a is not None:  # over the logits themselves
            y = z.clone()
            fg.forge_moe_route_grad(y, experts, counts, live, y, grad_weights=a, grad_loss=b, normalize=normalize)
            assert torch.equal(y, d[:, :E])


@gpu
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(cuda_device, normalize):
    T, E, k = 40, 12, 3
    z = make(T, E, masked=0.0)
    ref = reference(z, k, normalize)
    gw, gl = torch.randn(T, k, device="cuda"), torch.ones(1, device="cuda")
    d = torch.empty(T, E, device="cuda")
    fg.forge_moe_route_grad(z, ref["experts"].int().cuda(), ref["counts"].int().cuda(), ref["live"].int().cuda(), d,
                            grad_weights=gw, grad_loss=gl, normalize=normalize)

    def f(x):
        r = reference(x, k, normalize)
        assert torch.equal(r["experts"], ref["experts"])
        return float((gw.cpu().double() * r["weights"]).sum() + r["loss"][0])
    g = torch.Generator().manual_seed(1)
    base = z.cpu().double()
    for _ in range(3):
        v = torch.randn(T, E, generator=g, dtype=torch.float64)
        h = 1e-6
        diff = (f(base + h * v) - f(base - h * v)) / (2 * h)
        assert abs(float((d.cpu().double() * v).sum()) - diff) <= 1e-5 * float((d.cpu().double() * v).abs().sum())


@gpu
def test_gradient_of_a_row_with_nan(cuda_device):
    z = make(50, 20, pad=0, masked=0)
    z[3, 4], z[8, 1] = float("nan"), float("inf")
    o = route(z, 2, True)
    d = torch.empty(50, 20, device="cuda")
    fg.forge_moe_route_grad(z, o["experts"], o["counts"], o["live"], d, grad_weights=torch.ones(50, 2, device="cuda"))
    rows = torch.isnan(d).any(1)
    assert rows[3] and rows[8] and int(rows.sum()) == 2 and torch.isnan(d[3]).all()


@gpu
def test_many_tokens(cuda_device):
    T, E, k = 300001, 8, 2
    z = make(T, E, "bf16")
    o = route(z, k, True)
    experts = torch.sort(z.float(), dim=1, descending=True, stable=True)
    want = torch.where(experts.values[:, :k] > -float("inf"), experts.indices[:, :k], -1)
    assert torch.equal(o["experts"].long(), want)
    flat = want.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    packed = int((flat >= 0).sum())
    assert int(o["offsets"][-1]) == packed
    assert torch.equal(o["rows"][:packed].long(), order[:packed] // k) and (o["rows"][packed:] == -1).all()
    slots = torch.full_like(flat, -1)
    slots[order[:packed]] = torch.arange(packed, device="cuda")
    assert torch.equal(o["slots"].reshape(-1).long(), slots)


@gpu
def test_offsets_past_32_bits(cuda_device):
    T, E, far = 9, 20, (1 << 29) + 8
    buf = torch.empty(8 * far + E, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (T, E), (far, 1))
    z.copy_(make(T, E, "bf16"))
    o = route(z, 3, True)
    compare(o, reference(z, 3, True))
    near, wide = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    gw = torch.ones(T, 3, device="cuda") * torch.arange(3, device="cuda")
    fg.forge_moe_route_grad(z, o["experts"], o["counts"], o["live"], near, grad_weights=gw, grad_loss=o["loss"])
    fg.forge_moe_route_grad(z.contiguous(), o["experts"], o["counts"], o["live"], wide, grad_weights=gw, grad_loss=o["loss"])
    assert torch.equal(near, wide)


@gpu
@pytest.mark.parametrize("T,E,k", [(100, 8, 2), (5000, 64, 6)])
def test_streams_and_graphs(cuda_device, T, E, k):
    z = make(T, E)
    want = route(z, k, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = outputs(T, E, k)
    fg.forge_moe_route(z, other["experts"], other["weights"], other["counts"], other["offsets"], slots=other["slots"],
                       rows=other["rows"], live=other["live"], loss=other["loss"], stream=side)
    side.synchronize()
    graphs, held = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        o = outputs(T, E, k)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fg.forge_moe_route(z, o["experts"], o["weights"], o["counts"], o["offsets"], slots=o["slots"], rows=o["rows"],
                               live=o["live"], loss=o["loss"])
        graphs.append(g)
        held.append(o)
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in (other, *held):
        assert all(torch.equal(o[n], want[n]) for n in want)


def test_refusals_before_any_launch():
    L = fg.lib()
    F = fg.FORGE_F32

    def r(z=FAKE, t=F, T=4, E=8, ld=8, k=2, experts=FAKE, w=FAKE, counts=FAKE, offsets=FAKE, slots=FAKE, rows=FAKE,
          live=FAKE, loss=FAKE):
        return L.forge_moe_route(z, t, T, E, ld, k, 1, experts, w, counts, offsets, slots, rows, live, loss, None)

    def g(z=FAKE, t=F, T=4, E=8, ld=8, k=2, experts=FAKE, counts=FAKE, live=FAKE, gw=FAKE, gl=FAKE,
          d=ctypes.c_void_p(0x90000), o=F, ldo=8):
        return L.forge_moe_route_grad(z, t, T, E, ld, k, 1, experts, counts, live, gw, gl, d, o, ldo, None)
    sizes = (dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(ld=7), dict(k=0), dict(k=9), dict(k=33, E=64, ld=64),
             dict(T=1 << 30, k=2))
    for kw in sizes + (dict(z=None), dict(experts=None), dict(w=None), dict(counts=None), dict(offsets=None)):
        assert r(**kw) == fg.FORGE_ERR_INVALID_ARG, kw
    for kw in sizes + (dict(z=None), dict(d=None), dict(experts=None), dict(counts=None), dict(live=None), dict(ldo=7),
                       dict(d=ctypes.c_void_p(0x10010)), dict(d=FAKE, o=fg.FORGE_BF16)):
        assert g(**kw) == fg.FORGE_ERR_INVALID_ARG, kw
    for t in (fg.FORGE_E4M3, fg.FORGE_I64, 7):
        assert r(t=t) == g(t=t) == g(o=t) == fg.FORGE_ERR_UNSUPPORTED_DTYPE
    odd = ctypes.c_void_p(0x10002)
    for n in ("z", "experts", "w", "counts", "offsets", "slots", "rows", "live", "loss"):
        assert r(**{n: odd}) == fg.FORGE_ERR_MISALIGNED, n
    for n in ("z", "experts", "counts", "live", "gw", "gl"):
        assert g(**{n: odd}) == fg.FORGE_ERR_MISALIGNED, n


@gpu
def test_binding_refuses_what_does_not_fit(cuda_device):
    z = torch.zeros(4, 8, device="cuda")
    o = outputs(4, 8, 2)
    with pytest.raises(ValueError):
        fg.forge_moe_route(z, o["experts"], o["weights"][:3], o["counts"], o["offsets"])
    with pytest.raises(ValueError):
        fg.forge_moe_route(z, o["experts"], o["weights"], o["counts"], o["counts"])
    with pytest.raises(ValueError):
        fg.forge_moe_route(z, o["experts"].long(), o["weights"], o["counts"], o["offsets"])
    with pytest.raises(TypeError):
        fg.forge_moe_route(z.half(), o["experts"], o["weights"], o["counts"], o["offsets"])
    with pytest.raises(ValueError):
        fg.forge_moe_route_grad(z, o["experts"], o["counts"], o["live"], z[:, :7])
    with pytest.raises(fg.ForgeError):
        fg.forge_moe_route(z[:, :1], o["experts"], o["weights"], o["counts"][:1], o["offsets"][:2])


def test_logits_that_may_be_written_over_are_read_by_plain_loads():
    """dlogits may be the logits: read-only loads ask for data that nothing writes while the
    kernel lives."""
    import os
    import re
    path = os.path.join(os.path.dirname(fg.__file__), "csrc", "forge_route.cu")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    grad = code[code.index("forge_route_grad_kernel("):]
    assert not re.findall(r"load_packed<X,", code[code.index("load_logits("):code.index("make_masks(")])
    assert "load_packed<X," not in grad and "__restrict__" not in grad


@gpu
def test_choices_laid_out_another_way_are_refused(cuda_device):
    z = make(12, 8)
    o = route(z, 2, True)
    i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        fg.forge_moe_route(z, o["experts"], o["weights"], o["counts"], o["offsets"], slots=i(2, 12))
    d = torch.empty(12, 8, device="cuda")
    with pytest.raises(ValueError):
        fg.forge_moe_route_grad(z, o["experts"], o["counts"], o["live"], d, grad_weights=torch.ones(2, 12, device="cuda"))
    flat = i(24)
    fg.forge_moe_route(z, o["experts"], o["weights"], o["counts"], o["offsets"], slots=flat)
    assert torch.equal(flat, o["slots"].reshape(-1))
