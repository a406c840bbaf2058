"""Layer norm and its gradient against 64-bit forms.

Bounds.  u = 2^-24.  A sum of D fp32 terms in a tree of at most 16 serial terms a
thread (a thread's share of a longer row: D / 1024) and 10 levels is off by at
most (D / 1024 + 26) u times the sum of magnitudes; T(D) below.  The mean is off by
T(D) mean|x|, so xh by T(D) mean|x| rstd, and (squares of deviations, a
reciprocal of a root) relatively by T(D) + 8 u; sums over R rows, a block's serially, are off
by (R + 600) u times the sum of magnitudes at the very worst.  Outputs add one rounding:
bf16 2^-8.
"""
import ctypes

import pytest
import torch

import weight_grad_gemm_gb300 as fg

gpu = pytest.mark.gpu
FAKE = ctypes.c_void_p(0x10000)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-5
HALF = {"f32": U, "bf16": 2.0 ** -8}


def tree(D):
    return (D / 1024 + 26) * U


def make(R, D, dtype, seed=0, std=1.0, mean=0.3, pad=0, offset=0):
    """[R, D] with rows D + pad apart, from `offset` elements into its buffer on."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((R * (D + pad) + offset,), 7.0, dtype=DT[dtype], device="cuda")
    t = buf[offset:].view(R, D + pad)[:, :D]
    t.copy_((torch.randn(R, D, generator=g) * std + mean).to(DT[dtype]))
    return t


def params(D, seed=1, offset=0):
    g = torch.Generator().manual_seed(seed)
    w, b = torch.randn(2, D + offset, generator=g) * 0.3
    return (1 + w).cuda()[offset:], b.cuda()[offset:]


def reference(x, w, b, eps=EPS):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    var = (x - mu).square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = (x - mu) * rstd
    return xh * w.double() + (0 if b is None else b.double()), mu[:, 0], rstd[:, 0], xh


def check_forward(x, w, b, y, mean, rstd):
    D = x.shape[1]
    want, mu, rs, xh = reference(x, w, b)
    size = x.double().abs().mean(1)
    off = tree(D) * size  # of the mean
    if mean is not None:
        assert torch.all((mean.double() - mu).abs() <= off + 2 * U * mu.abs())
    rel = tree(D) + 8 * U + (off * rs) ** 2
    if rstd is not None:
        assert torch.all((rstd.double() / rs - 1).abs() <= rel)
    dxh = (off * rs + rel)[:, None] * (1 + xh.abs()) + 4 * U * (xh.abs() + (size * rs)[:, None])
    bound = dxh * w.double().abs() + 2 * U * want.abs() + (0 if b is None else U * b.double().abs())
    half = HALF["bf16" if y.dtype == torch.bfloat16 else "f32"]
    bound = bound + half * (want.abs() + bound)
    bad = (y.double() - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), float((y.double() - want).abs().max()))


WIDTHS = [1, 2, 7, 64, 129, 256, 257, 512, 520, 1023, 1024, 1025, 2048, 2056, 4096, 4100, 8192, 8200, 16384, 16392, 20001]


@gpu
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(cuda_device, D, x, y):
    for R in (1, 3, 37):
        X = make(R, D, x, seed=D)
        w, b = params(D)
        Y = make(R, D, y)
        mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        fg.forge_layer_norm(X, w, b, Y, mean=mean, rstd=rstd, eps=EPS)
        check_forward(X, w, b, Y, mean, rstd)
        Z = make(R, D, y)
        fg.forge_layer_norm(X, w, None, Z, eps=EPS)
        check_forward(X, w, None, Z, None, None)


@gpu
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("D,pad,offset", [(256, 8, 8), (256, 3, 0), (1000, 24, 1), (4096, 4, 4), (4096, 1, 3), (777, 0, 5)])
def test_strided_and_misaligned_rows(cuda_device, D, pad, offset, x, y):
    R = 19
    X, Y = make(R, D, x, pad=pad, offset=offset), make(R, D, y, seed=9, pad=pad, offset=offset)
    around = Y.new_empty(0).set_(Y.untyped_storage()).clone()
    w, b = params(D, offset=offset % 4)
    fg.forge_layer_norm(X, w, b, Y, eps=EPS)
    check_forward(X, w, b, Y, None, None)
    after = Y.new_empty(0).set_(Y.untyped_storage()).clone()
    mask = torch.ones_like(after, dtype=torch.bool)
    mask[offset:].view(R, D + pad)[:, :D] = False
    assert torch.equal(after[mask], around[mask])  # nothing between or around the rows


@gpu
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("D", [100, 1024, 4096, 20000])
def test_large_mean_and_constant_rows(cuda_device, D, x):
    X = make(6, D, x, mean=300.0)
    X[1] = 5.0
    X[2] = 0.0
    w, b = params(D)
    Y = torch.empty(6, D, device="cuda")
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    fg.forge_layer_norm(X, w, b, Y, mean=mean, rstd=rstd, eps=EPS)
    check_forward(X, w, b, Y, mean, rstd)
    assert torch.equal(Y[2], b) and mean[2] == 0


@gpu
def test_rows_that_are_not_finite_stay_alone(cuda_device):
    X = make(9, 515, "f32")
    X[3, 7], X[5, 1] = float("nan"), float("inf")
    w, b = params(515)
    Y = torch.empty_like(X)
    fg.forge_layer_norm(X, w, b, Y)
    bad = torch.tensor([3, 5], device="cuda")
    assert torch.isnan(Y[bad]).all()
    good = torch.tensor([0, 1, 2, 4, 6, 7, 8], device="cuda")
    check_forward(X[good], w, b, Y[good], None, None)


def grads(dy, x, w, mean, rstd):
    dy, x, w, mean, rstd = (t.double() for t in (dy, x, w, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def check_backward(dy, x, w, mean, rstd, dx, dw, db, dw0=None, db0=None):
    R, D = x.shape
    want, dW, dB, xh, g = grads(dy, x, w, mean, rstd)
    t = tree(D) + 8 * U
    size = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    xh_off = 4 * U * (xh.abs() + (x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None])
    other = xh_off * (g * xh).mean(1, keepdim=True).abs() + xh.abs() * (g.abs() * xh_off).mean(1, keepdim=True)
    bound = rstd.double()[:, None] * (t * size + other)
    half = HALF["bf16" if dx.dtype == torch.bfloat16 else "f32"]
    bound = bound + half * (want.abs() + bound)
    assert torch.all((dx.double() - want).abs() <= bound + 2.0 ** -126)
    rows = (R + 600) * U
    dyd = dy.double().abs()
    first = 0 if dw0 is None else dw0.double()
    bw = rows * (dyd * xh.abs()).sum(0) + (dyd * xh_off).sum(0) + 2 * U * (dW + first).abs()
    assert torch.all((dw.double() - (dW + first)).abs() <= bw)
    if db is not None:
        first = 0 if db0 is None else db0.double()
        assert torch.all((db.double() - (dB + first)).abs() <= rows * dyd.sum(0) + 2 * U * (dB + first).abs())


def stats(x):
    _, mu, rs, _ = reference(x, torch.ones(x.shape[1], device="cuda"), None)
    return mu.float(), rs.float()


@gpu
@pytest.mark.parametrize("dy,x,dx", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                     ("f32", "bf16", "bf16"), ("bf16", "bf16", "f32")])
@pytest.mark.parametrize("D", WIDTHS)
def test_backward(cuda_device, D, dy, x, dx):
    for R in (1, 5, 700):
        X, dY = make(R, D, x, seed=D), make(R, D, dy, seed=D + 1, mean=0.0, std=0.02)
        w, _ = params(D)
        mean, rstd = stats(X)
        dX = make(R, D, dx)
        dW, dB = torch.full((2, D), 3.0, device="cuda")
        fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, dW, dB)
        check_backward(dY, X, w, mean, rstd, dX, dW, dB)
        again, dX2 = torch.empty(2, D, device="cuda"), torch.empty_like(dX)
        fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX2, again[0], again[1])
        assert torch.equal(again[0], dW) and torch.equal(again[1], dB) and torch.equal(dX2, dX)
        dw0, db0 = torch.randn(2, D, device="cuda")
        a, b = dw0.clone(), db0.clone()
        fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, a, b, accumulate=True)
        check_backward(dY, X, w, mean, rstd, dX, a, b, dw0, db0)
        fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, a)
        assert torch.equal(a, dW)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad,offset", [(256, 8, 8), (1000, 3, 1), (4096, 4, 0), (9000, 8, 8), (9001, 0, 1)])
def test_backward_strided_and_in_place(cuda_device, D, pad, offset, dtype):
    R = 33
    X = make(R, D, dtype, pad=pad, offset=offset)
    dY = make(R, D, dtype, seed=5, mean=0.0, pad=pad, offset=offset)
    w, _ = params(D)
    mean, rstd = stats(X)
    dX, dW, dB = make(R, D, dtype, pad=pad, offset=offset), *torch.empty(2, D, device="cuda")
    fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, dW, dB)
    check_backward(dY, X, w, mean, rstd, dX, dW, dB)
    for over in (dY, X):
        a, b = dY.clone(), X.clone()
        target = a if over is dY else b
        dw, db = torch.empty(2, D, device="cuda")
        ref, rw = torch.empty_like(a), torch.empty(2, D, device="cuda")
        fg.forge_layer_norm_grad(a, b, w, mean, rstd, ref, rw[0], rw[1])
        fg.forge_layer_norm_grad(a, b, w, mean, rstd, target, dw, db)
        assert torch.equal(target, ref) and torch.equal(dw, rw[0]) and torch.equal(db, rw[1])
    Y, Z = torch.empty_like(X), X.clone()
    b0 = torch.zeros(D, device="cuda")
    fg.forge_layer_norm(Z, w, b0, Y)
    fg.forge_layer_norm(Z, w, b0, Z)
    assert torch.equal(Y, Z)


@gpu
def test_gradient_against_differences(cuda_device):
    """d/dh of sum(y dy) along random directions of x, weight and bias, from 64-bit
    central differences of the definition; h^2 terms are below 1e-6 of the value."""
    R, D = 23, 130
    X, dY = make(R, D, "f32"), make(R, D, "f32", seed=3, mean=0.0)
    w, b = params(D)
    y, mean, rstd, _ = reference(X, w, b)
    dX, dW, dB = torch.empty_like(X), *torch.empty(2, D, device="cuda")
    fg.forge_layer_norm_grad(dY, X, w, mean.float(), rstd.float(), dX, dW, dB)
    f = lambda x, w, b: float((reference(x, w, b)[0] * dY.double()).sum())  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(4)
    h = 1e-4
    for t, grad in ((0, dX), (1, dW), (2, dB)):
        args = [X.double(), w.double(), b.double()]
        d = torch.randn(args[t].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        up[t], down[t] = args[t] + h * d, args[t] - h * d
        want = (f(*up) - f(*down)) / (2 * h)
        got = float((grad.double() * d).sum())
        scale = float((grad.double() * d).abs().sum())
        assert abs(got - want) <= 1e-5 * scale


@gpu
def test_empty_and_many_rows(cuda_device):
    D = 96
    w, b = params(D)
    none = torch.empty(0, D, device="cuda")
    fg.forge_layer_norm(none, w, b, none)
    dW, dB = torch.full((2, D), 2.0, device="cuda")
    e = torch.empty(0, device="cuda")
    fg.forge_layer_norm_grad(none, none, w, e, e, none, dW, dB, accumulate=True)
    assert (dW == 2).all() and (dB == 2).all()
    fg.forge_layer_norm_grad(none, none, w, e, e, none, dW, dB)
    assert not dW.any() and not dB.any()
    X, dY = make(70001, D, "bf16"), make(70001, D, "bf16", seed=2)
    Y = torch.empty_like(X)
    fg.forge_layer_norm(X, w, b, Y)
    check_forward(X, w, b, Y, None, None)
    mean, rstd = stats(X)
    dX = torch.empty_like(X)
    fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, dW, dB)
    check_backward(dY, X, w, mean, rstd, dX, dW, dB)


@gpu
def test_offsets_past_32_bits(cuda_device):
    R, D = 5, 4096
    far = (1 << 31) // 2 + 4096  # row distance: the last rows begin past 2^32 elements
    buf = torch.empty(4 * far + D, dtype=torch.bfloat16, device="cuda")
    X = torch.as_strided(buf, (R, D), (far, 1))
    X.copy_(make(R, D, "bf16"))
    w, b = params(D)
    Y = torch.empty(R, D, device="cuda")
    fg.forge_layer_norm(X, w, b, Y)
    check_forward(X, w, b, Y, None, None)
    mean, rstd = stats(X)
    ref, dW, dB = torch.empty(R, D, device="cuda"), *torch.empty(2, D, device="cuda")
    fg.forge_layer_norm_grad(Y, X, w, mean, rstd, ref, dW, dB)
    check_backward(Y, X, w, mean, rstd, ref, dW, dB)


@gpu
def test_streams_and_graphs(cuda_device):
    R, D = 300, 1000
    X, dY = make(R, D, "bf16"), make(R, D, "bf16", seed=3)
    w, b = params(D)
    Y, mean, rstd = torch.empty_like(X), *torch.empty(2, R, device="cuda")
    fg.forge_layer_norm(X, w, b, Y, mean=mean, rstd=rstd)
    dX, dW, dB = torch.empty_like(X), *torch.empty(2, D, device="cuda")
    fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dX, dW, dB)
    outs = lambda: [torch.zeros_like(t) for t in (Y, dX, dW, dB)]  # noqa: E731
    side = torch.cuda.Stream()
    y2, dx2, dw2, db2 = outs()
    side.wait_stream(torch.cuda.current_stream())
    fg.forge_layer_norm(X, w, b, y2, stream=side)
    fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dx2, dw2, db2, stream=side)
    side.synchronize()
    graphs, held = [], []
    for _ in range(2):  # two captured graphs, replayed side by side
        y3, dx3, dw3, db3 = outs()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fg.forge_layer_norm(X, w, b, y3)
            fg.forge_layer_norm_grad(dY, X, w, mean, rstd, dx3, dw3, db3)
        graphs.append(g)
        held.append((y3, dx3, dw3, db3))
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for got in ((y2, dx2, dw2, db2), *held):
        for t, want in zip(got, (Y, dX, dW, dB)):
            assert torch.equal(t, want)


def test_refusals_before_any_launch():
    L = fg.lib()
    F, B = fg.FORGE_F32, fg.FORGE_BF16

    def n(x=FAKE, xt=F, ldx=64, w=FAKE, b=FAKE, R=4, D=64, eps=1e-5, y=ctypes.c_void_p(0x90000), yt=F, ldy=64,
          mean=FAKE, rstd=FAKE):
        return L.forge_layer_norm(x, xt, ldx, w, b, R, D, eps, y, yt, ldy, mean, rstd, None)

    def g(dy=FAKE, dyt=F, lddy=64, x=ctypes.c_void_p(0x50000), xt=F, ldx=64, w=FAKE, mean=FAKE, rstd=FAKE, R=4, D=64,
          dx=ctypes.c_void_p(0x90000), dxt=F, lddx=64, dw=FAKE, db=FAKE):
        return L.forge_layer_norm_grad(dy, dyt, lddy, x, xt, ldx, w, mean, rstd, R, D, dx, dxt, lddx, dw, db, 0, None)
    bad = fg.FORGE_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(y=None), dict(w=None), dict(R=-1), dict(D=0), dict(D=(1 << 30) + 1), dict(ldx=63),
               dict(ldy=63), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(y=ctypes.c_void_p(0x10004)), dict(y=FAKE, yt=B), dict(y=FAKE, ldy=65)):
        assert n(**kw) == bad, kw
    for kw in (dict(dy=None), dict(x=None), dict(dx=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dw=None),
               dict(R=-1), dict(D=0), dict(lddy=63), dict(ldx=63), dict(lddx=63), dict(dx=ctypes.c_void_p(0x50100)),
               dict(dx=FAKE, dxt=B)):
        assert g(**kw) == bad, kw
    for t in (fg.FORGE_E4M3, fg.FORGE_I32, 9):
        assert n(xt=t) == n(yt=t) == g(dyt=t) == g(xt=t) == g(dxt=t) == fg.FORGE_ERR_UNSUPPORTED_DTYPE
    odd = ctypes.c_void_p(0x10002)
    for kw in (dict(x=odd), dict(w=odd), dict(b=odd), dict(mean=odd), dict(rstd=odd)):
        assert n(**kw) == fg.FORGE_ERR_MISALIGNED, kw
    for kw in (dict(dy=odd), dict(x=odd), dict(w=odd), dict(dw=odd), dict(db=odd), dict(mean=odd)):
        assert g(**kw) == fg.FORGE_ERR_MISALIGNED, kw
    assert n(x=ctypes.c_void_p(0x10001), xt=B) == fg.FORGE_ERR_MISALIGNED


@gpu
def test_binding_refuses_what_does_not_fit(cuda_device):
    X = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        fg.forge_layer_norm(X, w, None, torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        fg.forge_layer_norm(X, w[:7], None, X)
    with pytest.raises(TypeError):
        fg.forge_layer_norm(X.half(), w, None, X)
    with pytest.raises(ValueError):
        fg.forge_layer_norm(X.t(), w[:4], None, X.t())
    with pytest.raises(ValueError):
        fg.forge_layer_norm(X.cpu(), w, None, X)
    with pytest.raises(fg.ForgeError):
        fg.forge_layer_norm(X, w, None, X, eps=0.0)
    with pytest.raises(ValueError):
        fg.forge_layer_norm_grad(X, X[:3], w, w[:4], w[:4], X, w, None)


def test_rows_that_may_be_written_over_are_read_by_plain_loads():
    """y may be x, and dx may be dy or x: read-only loads (load_packed, and pointers that promise
    no overlap) ask for data that nothing writes while the kernel lives."""
    import os
    import re
    path = os.path.join(os.path.dirname(fg.__file__), "csrc", "forge_layer_norm.cu")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.findall(r"load_packed<[GX],", code)
    assert not re.findall(r"const [GX]\* __restrict__", code)


@gpu
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("D", [2, 65, 256, 500, 1024, 2000, 4096, 8192, 16384, 16400, 20001])
def test_rows_whose_squares_pass_the_largest_number(cuda_device, D, x, y):
    """Finite rows keep their results up to the type's largest numbers: the deviations' squares,
    and the sum of the row itself, may pass fp32's range.  The bound of ordinary rows holds:
    it is relative to the row's size.  (rstd of the largest rows is below 2^-126, where
    fp32's step is 2^-149.)"""
    X = make(9, D, x, seed=D, mean=0.0).float()
    for r, size in ((1, 1e18), (2, 3e19), (3, 1e25), (5, 1e30), (6, 3e37), (7, 1e38)):
        X[r] = X[r].clamp(-3, 3) * size
    X[8] = torch.finfo(DT[x]).max
    X[8, 0] = 0.0
    X = X.to(DT[x])
    w, b = params(D)
    Y = torch.empty(9, D, dtype=DT[y], device="cuda")
    mean, rstd = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    fg.forge_layer_norm(X, w, b, Y, mean=mean, rstd=rstd, eps=EPS)
    check_forward(X, w, b, Y, mean, None)
    _, _, rs, _ = reference(X, w, b)
    off = tree(D) * X.double().abs().mean(1) * rs
    assert torch.all((rstd.double() - rs).abs() <= (tree(D) + 8 * U + off ** 2) * rs + 2.0 ** -149)
    Z = X.clone()
    if x == y:
        fg.forge_layer_norm(Z, w, b, Z, eps=EPS)  # in place
        assert torch.equal(Z, Y)
    bad = X.clone()
    bad[1, 0], bad[3, D - 1], bad[5, 0] = float("inf"), -float("inf"), float("nan")
    fg.forge_layer_norm(bad, w, b, Y, mean=mean, rstd=rstd, eps=EPS)
    assert torch.isnan(Y[[1, 3, 5]]).all()
    good = torch.tensor([0, 2, 4, 6, 7, 8], device="cuda")
    check_forward(X[good], w, b, Y[good], mean[good], None)
    calm = torch.tensor([0, 4], device="cuda")  # bitwise as without such rows beside them
    alone = torch.empty(2, D, dtype=DT[y], device="cuda")
    fg.forge_layer_norm(X[calm], w, b, alone, eps=EPS)
    assert torch.equal(Y[calm], alone)


@gpu
@pytest.mark.parametrize("D,dtype", [(4096, "bfloat16"), (8192, "float32"), (64, "float32")])
def test_scratch_of_the_gradient_is_what_its_blocks_write(cuda_device, D, dtype):
    """The library's pool keeps what it has reserved: a block's parts are 2 D floats, and the
    blocks that run at once have 64 KB an SM of them (10 MB of 152 SMs; the pool
    reserves in steps of 32 MB).  In a process of its own, whose pool is new."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = f"""
import sys
sys.path.insert(0, {root!r})
import torch
import weight_grad_gemm_gb300 as fg
R, D = 16384, {D}
x = torch.randn(R, D, device="cuda").to(torch.{dtype})
w, dw, db = torch.ones(3, D, device="cuda")
mean, rstd = torch.zeros(R, device="cuda"), torch.ones(R, device="cuda")
dx = torch.empty_like(x)
def run(n):
    fg.forge_layer_norm_grad(x[:n], x[:n], w, mean[:n], rstd[:n], dx[:n], dw, db)
    torch.cuda.synchronize()
run(1)
before = torch.cuda.mem_get_info()[0]
run(R)
used = before - torch.cuda.mem_get_info()[0]
assert used <= 40 << 20, used
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
