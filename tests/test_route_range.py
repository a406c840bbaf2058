"""The router and its gradient over the whole range of finite logits.

p depends on differences of a row's logits only, so a row's size must not show: rows that
are masked throughout with a large negative number (the type's lowest among them), rows of
equal large logits, and rows whose logits are far apart.  z - max is rounded once (half a
step, relatively 2^-24) and multiplied by log2 e (a rounded constant and a product, 2^-23
relatively), so a term is off by |z - max| 2^-22 + 2^-22 relatively; with |z - max| <= 104
(below that exp is 0 in fp32 as well: 2^-100 absolutely) that is 2^-15, and a quotient of
sums of such terms within 2^-14.
"""
import os
import subprocess
import sys

import pytest
import torch

import weight_grad_gemm_gb300 as fg
from test_route import DT, reference, route

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = [(8, 2), (64, 8), (200, 4), (256, 8), (600, 7)]
SHIFTS = [-1e10, 1e10, -3e10, 2e9, 1e12, -1e30, 1e30, "min", "max"]


def shift_of(name, dtype):
    lim = torch.finfo(DT[dtype])
    return {"min": lim.min, "max": lim.max}.get(name, name)


def rows_of(E, dtype, shift):
    """Rows of one large number throughout, with two masked experts, with steps of the
    number's own size between experts, and with ordinary logits beside it."""
    g = torch.Generator().manual_seed(E)
    at = torch.tensor(shift_of(shift, dtype), dtype=torch.float64)
    z = torch.full((6, E), float(at), dtype=torch.float64)
    z[1, ::3] = -float("inf")
    # multiples of 2^-7 |at|: whole steps of bf16, towards 0
    z[2] = at * (1 - torch.randint(0, 4, (E,), generator=g) * 2.0 ** -7)
    z[3, 1::2] = torch.randn(E // 2, generator=g).double()
    z[4] = 0.0
    z[4, 3] = at
    z[5] = -at
    z[5, 5:] = at
    return z.to(DT[dtype])


def mixed(E, dtype, shift):
    """Such rows among ordinary ones."""
    g = torch.Generator().manual_seed(7)
    z = torch.randn(70, E, generator=g).to(DT[dtype])
    z[[0, 11, 12, 40, 41, 69]] = rows_of(E, dtype, shift)
    return z.cuda()


def reference_grad(z, ref, k, normalize, gw, gl):
    """By automatic differentiation in 64 bits (every row has a finite logit)."""
    z = z.cpu().double().requires_grad_()
    T, E = z.shape
    p, e = z.softmax(1), ref["experts"]
    w = p.gather(1, e.clamp(min=0)) * (e >= 0)
    if normalize:
        w = w / w.sum(1, keepdim=True)
    loss = (ref["counts"] * p.sum(0) / T).sum() * E / (k * T)
    (grad,) = torch.autograd.grad((gw.cpu().double() * w).sum() + gl.item() * loss, z)
    return grad


def near(got, want, slack=2.0 ** -14):
    return torch.all((got.cpu().double() - want).abs() <= slack * want.abs() + 2.0 ** -100)


@gpu
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("E,k", SIZES)
def test_weights_and_loss(cuda_device, E, k, shift, dtype, normalize):
    for z in (rows_of(E, dtype, shift).cuda(), mixed(E, dtype, shift)):
        want = reference(z, k, normalize)
        o = route(z, k, normalize)
        for name in ("experts", "counts", "offsets", "slots", "rows", "live"):
            assert torch.equal(o[name].cpu().long(), want[name]), name
        assert near(o["weights"], want["weights"])
        assert near(o["loss"], want["loss"], 2.0 ** -13)


@gpu
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("E,k", SIZES)
def test_gradient(cuda_device, E, k, shift, dtype, normalize):
    """p (q - sum p q), each p within 2^-14: within 2^-13 of p (|q| + sum p |q|), |q| at
    most its parts' sum: of the loss E max(counts) / (k n^2), of the weights 2 max|gw| over
    the chosen mass where they are normalised."""
    z = mixed(E, dtype, shift)
    T = z.shape[0]
    ref = reference(z, k, normalize)
    g = torch.Generator().manual_seed(3)
    gw, gl = torch.randn(T, k, generator=g).cuda(), torch.ones(1, device="cuda")
    d = torch.empty(T, E, device="cuda")
    ints = [ref[n].int().cuda() for n in ("experts", "counts", "live")]
    fg.forge_moe_route_grad(z, *ints, d, grad_weights=gw, grad_loss=gl, normalize=normalize)
    want = reference_grad(z, ref, k, normalize, gw, gl)
    assert torch.isfinite(want).all()
    p, n = ref["p"], int(ref["live"])
    mass = (p.gather(1, ref["experts"].clamp(min=0)) * (ref["experts"] >= 0)).sum(1, keepdim=True)
    q = E * float(ref["counts"].max()) / (k * n * n)
    q = q + (2 * float(gw.abs().max()) / mass.clamp(min=1e-300) if normalize else float(gw.abs().max()))
    assert torch.all((d.cpu().double() - want).abs() <= 2.0 ** -13 * p * 2 * q + 2.0 ** -100)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding_by_the_lowest_number_leaves_the_others_alone(cuda_device, dtype):
    """The ordinary tokens' choices and weights are bitwise the ones without such rows."""
    E, k = 64, 8
    z = mixed(E, dtype, 0.5)
    z[50:] = torch.finfo(DT[dtype]).min
    o, alone = route(z, k, True), route(z[:50].clone(), k, True)
    assert torch.equal(o["weights"][:50], alone["weights"]) and torch.equal(o["experts"][:50], alone["experts"])
    assert torch.equal(o["weights"][50:], torch.full((20, k), 1 / k, device="cuda"))
    assert torch.isfinite(o["loss"]).all()


@gpu
@pytest.mark.parametrize("E,k,tokens", [(496, 7, 200000), (917, 32, 19457), (1024, 16, 64)])
def test_blocks_whose_shared_memory_is_just_above_the_default(cuda_device, E, k, tokens):
    """Static and dynamic shared memory count together; in a process of its own, where no other
    size has asked for more."""
    code = f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
import torch
from test_route import route
g = torch.Generator(device="cuda").manual_seed(1)
z = torch.randn({tokens}, {E}, device="cuda", generator=g).bfloat16()
o = route(z, {k}, True)
want = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :{k}]
assert torch.equal(o["experts"].long(), want)
assert torch.equal(o["counts"].long(), torch.bincount(want.reshape(-1), minlength={E}))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
