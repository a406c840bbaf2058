"""The embedding lookup, its gradient by tokens and the gradient fused with
AdamW, against the formulas in 64 bits on the CPU.

Bounds: a product rounds once; a sum of n fp32 terms in any fixed order is off
by at most (n + 2) 2^-24 times the sum of their magnitudes.  AdamW's m and v are
two-term fp32 sums (2^-22 of their terms' magnitudes); W's step divides by
sqrt(v') + eps with hardware approximations of a few 2^-23 (2^-19 of the step).
"""
import ctypes

import numpy as np
import pytest
import torch

import weight_grad_gemm_gb300 as fg

gpu = pytest.mark.gpu
FAKE = ctypes.c_void_p(0x10000)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01, step=3)


def token_ids(T, V, seed, kind="zipf"):
    g = torch.Generator().manual_seed(seed)
    if kind == "zipf":
        ids = (torch.exp(torch.rand(T, generator=g, dtype=torch.float64) * np.log(V + 1)) - 1).long()
    elif kind == "one":
        ids = torch.full((T,), V // 2)
    elif kind == "two":
        ids = torch.where(torch.rand(T, generator=g) < 0.5, 0, V - 1)
    elif kind == "huge":  # rows of several thousand tokens side by side in the order, and a few medium ones
        rows = torch.tensor([5, 133, 261, 389, 7]) % V
        ids = rows[torch.multinomial(torch.tensor([0.4, 0.3, 0.25, 0.03, 0.02]), T, replacement=True, generator=g)]
    elif kind == "pad":
        return torch.full((T,), -1)
    elif kind == "ordered":
        ids = torch.arange(T) * V // max(T, 1)
    else:
        ids = torch.randint(0, V, (T,), generator=g)
    ids = ids.clamp(0, V - 1)
    return torch.where(torch.rand(T, generator=g) < 0.1, -5, ids)


def randn(shape, seed, dtype, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dtype])


def shifted(t, offset):
    """t on the GPU, `offset` elements past an aligned base."""
    buf = torch.empty(t.numel() + offset + 8, dtype=t.dtype, device="cuda")
    view = buf[offset:offset + t.numel()].view(t.shape)
    view.copy_(t.cuda())
    return view


def sums(dY, ids, V, scale):
    """The gradient, the sum of its terms' magnitudes and the terms' number, in 64 bits."""
    D = dY.shape[1]
    live = ids >= 0
    G = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[live], dY[live].double()) * scale
    A = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[live], dY[live].double().abs()) * abs(scale)
    n = torch.bincount(ids[live], minlength=V).double()[:, None]
    return G, A, n


# ---- lookup ------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("weight", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,offset", [(1, 1, 1, 0), (1, 50, 4096, 0), (5, 7, 3, 0), (3, 9, 1023, 0),
                                          (257, 1000, 264, 0), (64, 300, 520, 1), (64, 300, 520, 4),
                                          (1000, 77, 130, 2), (3000, 5000, 1024, 0), (16, 40, 16384, 0)])
def test_lookup(cuda_device, T, V, D, offset, weight, out):
    W = randn((V, D), T + D, weight)
    ids = token_ids(T, V, T)
    Y = shifted(torch.full((T, D), 9.0).to(DT[out]), offset)
    for idt, scale in ((torch.int32, 1.0), (torch.int64, -0.3)):
        fg.forge_embedding(ids.to(idt).cuda(), shifted(W, offset), Y, scale=scale)
        s32 = torch.tensor(scale)
        want = (W.float()[ids.clamp(min=0)] * s32).masked_fill_((ids < 0)[:, None], 0.0).to(DT[out])
        assert torch.equal(Y.cpu() + 0.0, want + 0.0)  # one fp32 product, one rounding
    assert fg.forge_get_device_status() == fg.FORGE_OK


@gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("weight", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,offset", [(20001, 1, 0), (40003, 79, 0), (60000, 128, 1), (10007, 129, 0), (50000, 256, 2),
                                        (20002, 8, 0), (20001, 128, 0), (30005, 136, 0), (9999, 256, 0), (6001, 512, 0)])
def test_lookup_of_many_narrow_rows(cuda_device, T, D, offset, weight, out):
    """Rows narrow enough for a warp to take several, more of them than warps."""
    V = 3001
    W = randn((V, D), T + D, weight)
    ids = token_ids(T, V, T)
    bad = ids.clone()
    bad[7::1000] = V
    Y = shifted(torch.full((T, D), 9.0).to(DT[out]), offset)
    fg.forge_embedding(bad.cuda(), shifted(W, offset), Y, scale=-0.3)
    assert fg.forge_get_device_status() == fg.FORGE_ERR_INVALID_ARG
    live = (bad >= 0) & (bad < V)
    want = (W.float()[ids.clamp(min=0)] * torch.tensor(-0.3)).masked_fill_(~live[:, None], 0.0).to(DT[out])
    assert torch.equal(Y.cpu() + 0.0, want + 0.0)


@gpu
def test_lookup_refuses_nothing_for_no_tokens_and_records_bad_ids(cuda_device):
    W = torch.ones(10, 8, device="cuda")
    Y = torch.full((3, 8), 5.0, device="cuda")
    fg.forge_embedding(torch.empty(0, dtype=torch.int64, device="cuda"), W, Y[:0])
    fg.forge_embedding(torch.tensor([9, 10, 1 << 40], device="cuda"), W, Y)
    assert fg.forge_get_device_status() == fg.FORGE_ERR_INVALID_ARG
    assert Y[0].eq(1).all() and not Y[1:].any()


@gpu
def test_lookup_past_32_bit_offsets(cuda_device):
    V, D = 70000, 32768
    W = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    W[V - 1] = 3.0
    Y = torch.empty(2, D, dtype=torch.bfloat16, device="cuda")
    fg.forge_embedding(torch.tensor([V - 1, 0], device="cuda"), W, Y, scale=2.0)
    assert Y[0].eq(6).all() and not Y[1].any()


# ---- gradient ------------------------------------------------------------------

GRADS = [(0, 5, 3, "zipf"), (1, 1, 1, "zipf"), (1, 1000, 4096, "uniform"), (7, 3, 5, "zipf"),
         (130, 1000, 264, "zipf"), (1000, 50, 1023, "zipf"), (1000, 70000, 8, "uniform"),
         (5000, 300, 520, "zipf"), (4097, 2, 130, "two"), (3000, 100, 256, "one"), (20000, 1, 16, "one"),
         (513, 40, 72, "pad"), (4096, 4096, 96, "ordered"), (300, 20000, 1000, "zipf"),
         (40000, 3000, 33, "zipf"), (2048, 128, 2056, "zipf"), (12000, 500, 300, "huge"),
         (9000, 400, 7, "huge"), (17, 4, 520, "one"), (16, 4, 520, "one"), (2049, 9, 264, "one")]


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,kind", GRADS)
def test_gradient_matches_the_formula(cuda_device, T, V, D, kind, dtype):
    ids = token_ids(T, V, T + V, kind)
    dY = randn((T, D), T + D, dtype)
    scale = 1.5
    G, A, n = sums(dY, ids, V, scale)
    tol = (n + 2) * 2.0 ** -24 * A
    dW = torch.full((V, D), 7.0, device="cuda")
    fg.forge_embedding_grad(dY.cuda(), ids.to(torch.int32).cuda(), dW, scale=scale)
    assert torch.all((dW.cpu().double() - G).abs() <= tol)
    again = torch.full((V, D), 8.0, device="cuda")
    fg.forge_embedding_grad(dY.cuda(), ids.cuda(), again, scale=scale)  # 64-bit ids, bitwise the same
    assert torch.equal(dW, again)
    start = randn((V, D), 5, "f32")
    acc = start.cuda()
    fg.forge_embedding_grad(dY.cuda(), ids.cuda(), acc, scale=scale, accumulate=True)
    want = start.double() + G
    assert torch.all((acc.cpu().double() - want).abs() <= tol + want.abs() * 2.0 ** -23)
    untouched = (n[:, 0] == 0).nonzero()[:, 0]
    assert torch.equal(acc.cpu()[untouched], start[untouched])
    assert fg.forge_get_device_status() == fg.FORGE_OK


@gpu
@pytest.mark.parametrize("D", [37, 264])
@pytest.mark.parametrize("lengths", [
    [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300],
    [511, 512, 513, 3, 1023, 1024, 1025, 0, 575, 576, 577, 18], [2047, 1], [2048], [2048, 1], [2049, 513], [512] * 9, [513] * 9])
def test_rows_of_every_length(cuda_device, lengths, D):
    """Rows whose numbers of tokens lie at the limits between the ways to add
    them, one after another in the order of tokens and spread over it."""
    n = torch.tensor(lengths)
    order = torch.randperm(int(n.sum()), generator=torch.Generator().manual_seed(len(lengths)))
    for rows in (torch.arange(len(n)) * 128, torch.arange(len(n)) * 5 + 1):  # (in one residue class of 128, in many)
        ids = torch.repeat_interleave(rows, n)[order]
        V = int(rows[-1]) + 2
        dY = randn((len(ids), D), D, "bf16")
        G, A, terms = sums(dY, ids, V, 1.0)
        dW = torch.full((V, D), 7.0, device="cuda")
        fg.forge_embedding_grad(dY.cuda(), ids.cuda(), dW)
        assert torch.all((dW.cpu().double() - G).abs() <= (terms + 2) * 2.0 ** -24 * A)


def in_class(n, c, rows, seed):
    """n tokens of the rows c, c + 128, ... (`rows` of them): one residue class of the order."""
    return torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(seed)) * 128 + c


ORDERS = {  # ids, vocabulary: sorts by one, two and three digits, lists in shared and in global memory
    "two digits": lambda: (torch.randint(0, 10000, (30000,), generator=torch.Generator().manual_seed(1)), 10000),
    "three digits": lambda: (torch.randint(0, 200000, (30000,), generator=torch.Generator().manual_seed(2)), 200000),
    "one digit in global memory": lambda: (in_class(5000, 5, 30, 3), 4000),
    "two digits in global memory": lambda: (in_class(5000, 127, 78, 4), 10000),
    "three digits in global memory": lambda: (in_class(9001, 0, 1562, 5), 200000),
    "three digits, every class": lambda: (torch.cat([in_class(150 + c, c, 1200, c) for c in range(128)]), 1200 * 128),
    "limits of the lists": lambda: (torch.cat([in_class(n, c, 70, c) for c, n in enumerate((128, 129, 4096, 4097, 0, 1))]),
                                    9000),
    "global beside shared": lambda: (torch.cat([in_class(4500, 2, 1500, 6), in_class(6000, 1, 1500, 7),
                                                in_class(300, 3, 1500, 8)]), 192001)}


@gpu
@pytest.mark.parametrize("D", [12, 5])
@pytest.mark.parametrize("kind", list(ORDERS))
def test_order_of_many_tokens(cuda_device, kind, D):
    """Integers, whose sums are exact in any order: each token in its row, once."""
    ids, V = ORDERS[kind]()
    g = torch.Generator().manual_seed(9)
    ids = ids[torch.randperm(len(ids), generator=g)]
    ids = torch.where(torch.rand(len(ids), generator=g) < 0.02, -1, ids)
    dY = torch.randint(-64, 65, (len(ids), D), generator=g).float()
    G, _, n = sums(dY, ids, V, 1.0)
    start = torch.randint(-64, 65, (V, D), generator=g).float()
    for idt in (torch.int32, torch.int64):
        for dt in (torch.float32, torch.bfloat16):
            dW, acc = torch.full((V, D), 7.0, device="cuda"), start.cuda()
            fg.forge_embedding_grad(dY.to(dt).cuda(), ids.to(idt).cuda(), dW)
            fg.forge_embedding_grad(dY.to(dt).cuda(), ids.to(idt).cuda(), acc, accumulate=True)
            assert torch.equal(dW.cpu().double(), G)
            assert torch.equal(acc.cpu().double(), G + start)
    # rows of up to 16 tokens: token after token, as the ids lie
    dY = randn((len(ids), D), 8, "f32")
    fg.forge_embedding_grad(dY.cuda(), ids.cuda(), dW)
    want = torch.zeros(V, D)
    few = (n[:, 0] <= 16)
    for t in torch.nonzero((ids >= 0) & few[ids.clamp(min=0)])[:, 0].tolist():
        want[ids[t]] += dY[t]
    assert torch.equal(dW.cpu()[few], want[few])
    assert fg.forge_get_device_status() == fg.FORGE_OK


@gpu
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("D", [1, 130, 264])
def test_gradient_alignment(cuda_device, D, offset):
    T, V = 500, 60
    ids = token_ids(T, V, 3)
    dY = randn((T, D), 4, "bf16")
    G, A, n = sums(dY, ids, V, 1.0)
    dW = shifted(torch.zeros(V, D), offset)
    fg.forge_embedding_grad(shifted(dY, offset), ids.cuda(), dW)
    assert torch.all((dW.cpu().double() - G).abs() <= (n + 2) * 2.0 ** -24 * A)


@gpu
def test_gradient_is_the_adjoint_of_the_lookup(cuda_device):
    """<dW, E> = <dY, lookup(E)> for any E: the difference quotient of a linear
    map.  Both inner products are taken in 64 bits of fp32 results."""
    T, V, D = 700, 90, 200
    ids = token_ids(T, V, 8).cuda()
    dY = randn((T, D), 1, "f32").cuda()
    E = randn((V, D), 2, "f32").cuda()
    Y, dW = torch.empty(T, D, device="cuda"), torch.empty(V, D, device="cuda")
    fg.forge_embedding(ids, E, Y, scale=0.5)
    fg.forge_embedding_grad(dY, ids, dW, scale=0.5)
    left, right = (dW.double() * E.double()).sum(), (dY.double() * Y.double()).sum()
    size = (dY.double().abs() * Y.double().abs()).sum()
    assert (left - right).abs() <= 100 * 2.0 ** -24 * size


@gpu
def test_gradient_bad_ids_streams_and_graphs(cuda_device):
    T, V, D = 600, 100, 264
    ids = token_ids(T, V, 2)
    dY = randn((T, D), 1, "bf16").cuda()
    dW = torch.empty(V, D, device="cuda")
    fg.forge_embedding_grad(dY, ids.cuda(), dW)
    bad = ids.clone()
    bad[ids < 0] = V + 3
    other = torch.empty(V, D, device="cuda")
    fg.forge_embedding_grad(dY, bad.cuda(), other)
    assert fg.forge_get_device_status() == fg.FORGE_ERR_INVALID_ARG
    assert torch.equal(dW, other)
    idg = ids.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other.zero_()
        fg.forge_embedding_grad(dY, idg, other)
    side.synchronize()
    assert torch.equal(dW, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.forge_embedding_grad(dY, idg, other)
    for _ in range(2):
        other.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dW, other)


def test_what_the_order_writes_is_read_by_plain_loads():
    """The kernels behind the order live while it writes its tables, and
    read-only loads (__ldg) ask for data that nothing writes meanwhile."""
    import os
    import re
    path = os.path.join(os.path.dirname(fg.__file__), "csrc", "forge_embedding.cu")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.findall(r"__ld\w+\(\s*(?:o\.|partial)\w*", code)


@gpu
@pytest.mark.parametrize("T,V,D", [(600, 5000, 264), (3000, 9000, 37), (6000, 700, 520)])
def test_calls_one_after_another_see_their_own_order(cuda_device, T, V, D):
    """Calls on one stream without a wait share their scratch: what one reads
    of the order must not be what the call before left there."""
    dY = randn((T, D), 1, "bf16").cuda()
    ids = [token_ids(T, V, s, kind).cuda() for s in range(4) for kind in ("zipf", "uniform", "one", "ordered")]
    alone, together = [], [torch.empty(V, D, device="cuda") for _ in ids]
    for i in ids:
        dW = torch.empty(V, D, device="cuda")
        fg.forge_embedding_grad(dY, i, dW)
        torch.cuda.synchronize()
        alone.append(dW)
    for _ in range(3):
        for i, dW in zip(ids, together):
            fg.forge_embedding_grad(dY, i, dW)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, together))
        for dW in together:
            dW.fill_(9.0)
    for i, dW in zip(ids, alone):
        G, A, n = sums(dY.cpu(), i.cpu(), V, 1.0)
        assert torch.all((dW.cpu().double() - G).abs() <= (n + 2) * 2.0 ** -24 * A)


@gpu
def test_gradient_past_32_bit_offsets(cuda_device):
    T, D = 33000, 65540  # 2.2e9 elements of dY
    dY = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    dY[-1], dY[0] = 2.0, 1.0
    ids = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    ids[-1], ids[0] = 1, 1
    dW = torch.empty(3, D, device="cuda")
    fg.forge_embedding_grad(dY, ids, dW)
    assert dW[1].eq(3).all() and not dW[0].any() and not dW[2].any()
    del dY, dW
    V, D = 70000, 32768  # 2.3e9 elements of dW
    dW = torch.empty(V, D, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    dY = torch.ones(3, D, device="cuda")
    fg.forge_embedding_grad(dY, ids, dW, scale=0.5)
    assert dW[V - 1].eq(1).all() and dW[0].eq(0.5).all() and not dW[1:V - 1].any()
    fg.forge_embedding_grad(dY, ids, dW, scale=0.5, accumulate=True)
    assert dW[V - 1].eq(2).all() and dW[0].eq(1).all() and not dW[V - 2].any()


# ---- gradient + AdamW -----------------------------------------------------------

def adamw_reference(G, A, n, W, m, v, hp):
    hp = {k: float(np.float32(x)) for k, x in hp.items()}
    b1, b2, step = hp["beta1"], hp["beta2"], int(hp["step"])
    m1 = b1 * m + (1 - b1) * G
    v1 = b2 * v + (1 - b2) * G * G
    den = torch.sqrt(v1 / (1 - b2 ** step)) + hp["eps"]
    up = hp["lr"] / (1 - b1 ** step) * m1 / den
    W1 = W * float(np.float32(1 - hp["lr"] * hp["wd"])) - up  # the decay factor is a 32-bit value
    dG = (n + 2) * 2.0 ** -24 * A                        # of the sum
    dm = (1 - b1) * dG + 2.0 ** -22 * (b1 * m.abs() + (1 - b1) * G.abs())
    dv = (1 - b2) * 2 * G.abs() * dG + 2.0 ** -22 * v1 + 2.0 ** -130
    dW = hp["lr"] / (1 - b1 ** step) * dm / den + up.abs() * (2.0 ** -19 + dv / v1.clamp(min=1e-37)) \
        + 2.0 ** -23 * W.abs()
    return (W1, dW), (m1, dm), (v1, dv)


@gpu
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,kind,offset", [(0, 9, 5, "zipf", 0), (1, 1, 1, "zipf", 0), (40, 700, 264, "zipf", 0),
                                               (3000, 90, 130, "zipf", 0), (900, 50, 1023, "zipf", 0),
                                               (5000, 3, 72, "one", 0), (513, 2000, 520, "zipf", 2),
                                               (64, 30, 4096, "uniform", 0)])
def test_fused_step_matches_the_formula(cuda_device, T, V, D, kind, offset, dtype, state):
    ids = token_ids(T, V, T + 1, kind)
    dY = randn((T, D), 3, dtype, 1e-2)
    W, m = randn((V, D), 4, "f32", 0.02), randn((V, D), 5, state, 1e-3)
    v = (randn((V, D), 6, "f32", 1e-3) ** 2 + 1e-9).to(DT[state])
    G, A, n = sums(dY, ids, V, 0.5)
    gpu_state = [shifted(t, offset) for t in (W, m, v)]
    fg.forge_embedding_adamw(shifted(dY, offset), ids.cuda(), *gpu_state, scale=0.5, **HP)
    want = adamw_reference(G, A, n, W.double(), m.double(), v.double(), HP)
    for name, got, (x, tol) in zip("Wmv", gpu_state, want):
        if name != "W" and state == "bf16":
            tol = tol + x.abs() * 2.0 ** -8
        err = (got.cpu().double() - x).abs()
        assert torch.all(err <= tol), (name, float((err / tol.clamp(min=1e-300)).max()))


@gpu
def test_fused_step_equals_gradient_then_owner_step(cuda_device):
    T, V, D = 3000, 400, 264
    ids = token_ids(T, V, 1).cuda()
    dY = randn((T, D), 3, "bf16", 1e-2).cuda()
    W, m = randn((V, D), 4, "f32", 0.02).cuda(), torch.zeros(V, D, device="cuda")
    v = torch.zeros(V, D, device="cuda")
    dW = torch.empty(V, D, device="cuda")
    fg.forge_embedding_grad(dY, ids, dW, scale=2.0)
    a = [t.clone() for t in (W, m, v)]
    fg.forge_owner_adamw(dW, *a, **HP)
    b = [t.clone() for t in (W, m, v)]
    fg.forge_embedding_adamw(dY, ids, *b, scale=2.0, **HP)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,kind,offset", [(12000, 500, 301, "huge", 0), (9000, 400, 7, "huge", 0),
                                               (12000, 500, 301, "huge", 1), (9000, 400, 264, "huge", 3),
                                               (6000, 30, 1023, "zipf", 0), (40000, 3000, 33, "zipf", 0),
                                               (30000, 200000, 6, "uniform", 0)])
def test_fused_step_with_rows_of_many_tokens(cuda_device, T, V, D, kind, offset, dtype, state):
    ids = token_ids(T, V, T + 1, kind)
    dY = randn((T, D), 3, dtype, 1e-2)
    W, m = randn((V, D), 4, "f32", 0.02), randn((V, D), 5, state, 1e-3)
    v = (randn((V, D), 6, "f32", 1e-3) ** 2 + 1e-9).to(DT[state])
    G, A, n = sums(dY, ids, V, 0.5)
    fused = [shifted(t, offset) for t in (W, m, v)]
    fg.forge_embedding_adamw(shifted(dY, offset), ids.cuda(), *fused, scale=0.5, **HP)
    want = adamw_reference(G, A, n, W.double(), m.double(), v.double(), HP)
    for name, got, (x, tol) in zip("Wmv", fused, want):
        if name != "W" and state == "bf16":
            tol = tol + x.abs() * 2.0 ** -8
        err = (got.cpu().double() - x).abs()
        assert torch.all(err <= tol), (name, float((err / tol.clamp(min=1e-300)).max()))
    dW, owner = torch.empty(V, D, device="cuda"), [t.cuda() for t in (W, m, v)]
    fg.forge_embedding_grad(dY.cuda(), ids.cuda(), dW, scale=0.5)
    fg.forge_owner_adamw(dW, *owner, **HP)
    assert all(torch.equal(a, b) for a, b in zip(fused, owner))


@gpu
@pytest.mark.parametrize("D", [32768, 32769])
def test_fused_step_past_32_bit_offsets(cuda_device, D):
    V = 70000  # 2.3e9 elements of W, m, v
    W, m, v = (torch.zeros(V, D, device="cuda", dtype=dt) for dt in (torch.float32, torch.bfloat16, torch.bfloat16))
    rows = torch.tensor([0, V // 2, V - 2, V - 1])
    ids = torch.cat([rows[torch.tensor([3, 0, 3, 1])], rows[2].repeat(40)]).cuda()  # one row of 40 tokens
    dY = randn((len(ids), D), 1, "f32").cuda()
    start = [randn((4, D), 2 + i, "f32").abs().to(t.dtype).cuda() for i, t in enumerate((W, m, v))]
    for t, a in zip((W, m, v), start):
        t[rows] = a
    fg.forge_embedding_adamw(dY, ids, W, m, v, **HP)
    small = [a.clone() for a in start]  # the same four rows alone
    fg.forge_embedding_adamw(dY, torch.searchsorted(rows.cuda(), ids), *small, **HP)
    for t, a in zip((W, m, v), small):
        assert torch.equal(t[rows], a)
        assert not t[1:100].any() and not t[V - 100:V - 2].any()
    del W, m, v
    T, D = 33000, 65541  # 2.2e9 elements of dY
    dY = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    dY[-1], dY[0], dY[-20:-1] = 2.0, 1.0, 0.5
    ids = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    ids[-1] = ids[0] = 1
    ids[-20:-1] = 2
    got = [torch.zeros(3, D, device="cuda") for _ in range(3)]
    fg.forge_embedding_adamw(dY, ids, *got, **HP)
    want = [torch.zeros(3, D, device="cuda") for _ in range(3)]
    G = torch.tensor([0.0, 3.0, 9.5], device="cuda")[:, None].expand(3, D).contiguous()
    fg.forge_owner_adamw(G, *want, **HP)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- refusals --------------------------------------------------------------------

def test_refusals_before_any_launch():
    L = fg.lib()
    hp = (1e-3, 0.9, 0.999, 1e-8, 0.01)

    def e(ids=FAKE, idt=fg.FORGE_I32, T=4, W=FAKE, wdt=fg.FORGE_F32, V=8, D=8, scale=1.0, Y=FAKE, ydt=fg.FORGE_BF16):
        return L.forge_embedding(ids, idt, T, W, wdt, V, D, scale, Y, ydt, None)

    def g(dY=FAKE, dt=fg.FORGE_BF16, ids=FAKE, idt=fg.FORGE_I32, T=4, V=8, D=8, scale=1.0, dW=FAKE):
        return L.forge_embedding_grad(dY, dt, ids, idt, T, V, D, scale, dW, 0, None)

    def a(dY=FAKE, dt=fg.FORGE_BF16, ids=FAKE, idt=fg.FORGE_I32, T=4, V=8, D=8, scale=1.0, W=FAKE, m=FAKE, v=FAKE,
          st=fg.FORGE_F32, hp=hp, step=1):
        return L.forge_embedding_adamw(dY, dt, ids, idt, T, V, D, scale, W, m, v, st, *hp, step, None)
    bad, dtype, mis = fg.FORGE_ERR_INVALID_ARG, fg.FORGE_ERR_UNSUPPORTED_DTYPE, fg.FORGE_ERR_MISALIGNED
    odd = ctypes.c_void_p(0x10001)
    for kw in (dict(ids=None), dict(W=None), dict(Y=None), dict(T=-1), dict(V=0), dict(D=0),
               dict(scale=float("inf")), dict(T=1 << 31), dict(D=1 << 31)):
        assert e(**kw) == bad, kw
    for kw in (dict(idt=fg.FORGE_F32), dict(wdt=fg.FORGE_E4M3), dict(ydt=fg.FORGE_I32)):
        assert e(**kw) == dtype, kw
    for kw in (dict(ids=odd), dict(W=odd), dict(Y=odd)):
        assert e(**kw) == mis, kw
    for fn in (g, a):
        for kw in (dict(dY=None), dict(ids=None), dict(T=-1), dict(V=0), dict(D=-1), dict(scale=float("nan"))):
            assert fn(**kw) == bad, kw
        for kw in (dict(dt=fg.FORGE_E4M3), dict(idt=fg.FORGE_BF16)):
            assert fn(**kw) == dtype, kw
        for kw in (dict(dY=odd), dict(ids=odd)):
            assert fn(**kw) == mis, kw
    assert g(dW=None) == bad and g(dW=odd) == mis
    assert a(W=None) == bad and a(m=None) == bad and a(v=None) == bad and a(step=0) == bad
    assert a(hp=(1e-3, 1.0, 0.999, 1e-8, 0.0)) == bad and a(st=fg.FORGE_E4M3) == dtype
    assert a(m=odd) == mis and a(W=ctypes.c_void_p(0x10002)) == mis


@gpu
def test_scratch_that_cannot_be_had_is_one_calls_error(cuda_device):
    """A call whose scratch exceeds the address space fails before any launch,
    and the calls after it are not told of it."""
    x, ids = torch.zeros(64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    p, L = ctypes.c_void_p(x.data_ptr()), fg.lib()
    W, Y = torch.ones(4, 8, device="cuda"), torch.empty(3, 8, device="cuda")
    tokens, width = 1 << 30, 1 << 24  # 2^24 columns of partial sums for 18 M pieces: 1.3 PB
    for call in (
            lambda: L.forge_embedding_grad(p, fg.FORGE_F32, ctypes.c_void_p(ids.data_ptr()), fg.FORGE_I32, tokens, 4,
                                           width, 1.0, p, 0, None),
            lambda: L.forge_embedding_adamw(p, fg.FORGE_F32, ctypes.c_void_p(ids.data_ptr()), fg.FORGE_I32, tokens, 4,
                                            width, 1.0, p, p, p, fg.FORGE_F32, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, None)):
        assert call() == fg.FORGE_ERR_CUDA
        fg.forge_embedding(ids, W, Y)
        assert Y.eq(1).all()
        assert call() == fg.FORGE_ERR_CUDA
        Y.fill_(3.0)
        assert Y.eq(3).all()


@gpu
def test_binding_refuses_what_does_not_fit(cuda_device):
    W = torch.zeros(6, 8, device="cuda")
    Y = torch.zeros(3, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fg.forge_embedding(ids[:2], W, Y)
    with pytest.raises(ValueError):
        fg.forge_embedding(ids, W[:, :4], Y)
    with pytest.raises(TypeError):
        fg.forge_embedding(ids.float(), W, Y)
    with pytest.raises(TypeError):
        fg.forge_embedding(ids, W.half(), Y)
    with pytest.raises(TypeError):
        fg.forge_embedding_grad(Y, ids, W.bfloat16())
    with pytest.raises(ValueError):
        fg.forge_embedding_adamw(Y, ids, W, W[:5], W, **HP)
    with pytest.raises(ValueError):
        fg.forge_embedding_grad(Y, ids.cpu(), W)
