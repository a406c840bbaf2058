"""Token log-probabilities with entropy and top alternatives, and their
gradient, against the definition in 64 bits on the CPU.

Bounds, derived from the arithmetic: a term exp(z_j - ref) is off by the
rounding of its exponent (z in fp32: |z| 2^-23 with the rounded factor of the
exponential's base, doubled for the reference) and of the exponential (2^-22);
sums are taken over short fp32 runs.  With Z the largest finite |z| of a row,
unit(Z) = (Z + 16) 2^-21 covers lse, logprob and p relatively; the entropy, a
sum of p_j ln p_j with |ln p_j| up to 2 Z + ln V, gets (1 + ln V) times it.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import weight_grad_gemm_gb300 as fg

gpu = pytest.mark.gpu
FAKE = ctypes.c_void_p(0x10000)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def logits_of(R, V, seed, dtype="f32", ld=None, offset=0, std=3.0):
    """[R, V] logits on the CPU and the same on the GPU with rows ld apart,
    `offset` elements past an aligned base."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, V, generator=g) * std).to(DT[dtype])
    return x, to_gpu(x, ld, offset)


def to_gpu(x, ld=None, offset=0):
    R, V = x.shape
    ld = V if ld is None else ld
    buf = torch.full((R * ld + offset + 8,), 77.0, dtype=x.dtype, device="cuda")
    view = buf[offset:offset + R * ld].view(R, ld)[:, :V]
    view.copy_(x.cuda())
    return view


def reference(x, t, scale, k=0):
    """The definition in float64: logprob, lse, entropy, p, ln p, top index and logprob."""
    z = x.double() * float(np.float32(scale))
    lse = torch.logsumexp(z, 1)
    none = lse == -math.inf
    logp = torch.where(none[:, None], -math.inf, z - lse[:, None])
    p = torch.exp(logp)
    H = -torch.where(p > 0, p * logp, 0.0).sum(1)
    H = torch.where(torch.isnan(lse), math.nan, H)
    skip = torch.zeros(x.shape[0], dtype=torch.bool) if t is None else t < 0
    lp = None
    if t is not None:
        lp = logp.gather(1, t.clamp(min=0).long()[:, None])[:, 0].masked_fill(skip, 0.0)
    order = np.lexsort((np.arange(x.shape[1])[None, :].repeat(x.shape[0], 0), -z.numpy()), axis=1)
    top = torch.from_numpy(order[:, :k].copy()).long()
    return {"logprob": lp, "lse": lse.masked_fill(skip, 0.0), "entropy": H.masked_fill(skip, 0.0),
            "p": p, "logp": logp, "skip": skip, "top_index": top.masked_fill(skip[:, None], -1),
            "top_logprob": logp.gather(1, top).masked_fill(skip[:, None], 0.0)}


def unit(x, scale):
    z = x.double().abs() * scale
    z = torch.where((z < 1e30), z, 0.0)
    return (z.amax(1) + 16) * 2.0 ** -21


def forward(x, t, scale=1.0, k=0):
    R = x.shape[0]
    o = {n: torch.full((R,), 99.0, device="cuda") for n in ("lse", "entropy")}
    lp = None if t is None else torch.full((R,), 99.0, device="cuda")
    ti = torch.full((R, k), 9, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((R, k), 99.0, device="cuda") if k else None
    fg.forge_token_logprob(x, t, lp, top_index=ti, top_logprob=tl, scale=scale, **o)
    torch.cuda.synchronize()
    return {**o, "logprob": lp, "top_index": ti, "top_logprob": tl}


def near(got, want, tol):
    got, want = got.cpu().double(), want.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[inf], want[inf])
    fine = torch.isfinite(want)
    err = (got - want).abs()
    tol = tol.expand_as(want) if tol.dim() else tol.expand(want.shape)
    assert torch.all(torch.isfinite(got[fine])) and torch.all(err[fine] <= tol[fine]), \
        float((err[fine] / tol[fine]).max())


def check(x, xg, t, scale=1.0, k=0, ids=torch.int32):
    tg = None if t is None else t.to(ids).cuda()
    got = forward(xg, tg, scale, k)
    want = reference(x, t, scale, k)
    u = unit(x, scale)
    if t is not None:
        near(got["logprob"], want["logprob"], u)
    near(got["lse"], want["lse"], u)
    near(got["entropy"], want["entropy"], u * (1 + math.log(x.shape[1])))
    if k:
        assert torch.equal(got["top_index"].cpu().long(), want["top_index"])
        near(got["top_logprob"], want["top_logprob"], u[:, None])
    assert fg.forge_get_device_status() == fg.FORGE_OK
    return got, want


def targets(R, V, seed, pad=0.2):
    g = torch.Generator().manual_seed(seed + 1000)
    t = torch.randint(0, V, (R,), generator=g)
    return torch.where(torch.rand(R, generator=g) < pad, -1, t)


SHAPES = [(1, 1, 1), (3, 2, 2), (1, 31, 7), (5, 32, 32), (2, 33, 0), (9, 257, 5), (300, 100, 3),
          (4, 1000, 20), (3, 4099, 32), (2, 8192, 1), (7, 32768, 5), (2, 50001, 20),
          (1, 131072, 5), (700, 2049, 4), (2, 200003, 32)]


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V,k", SHAPES)
def test_forward_matches_the_definition(cuda_device, R, V, k, dtype):
    x, xg = logits_of(R, V, 7 * R + V, dtype)
    check(x, xg, targets(R, V, R + V), k=k)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 63, 4097, 40000])
@pytest.mark.parametrize("pad,offset", [(1, 0), (7, 3), (64, 1)])
def test_forward_strides_alignment_scale_and_wide_ids(cuda_device, V, pad, offset, dtype):
    x, xg = logits_of(6, V, V + pad, dtype, ld=V + pad, offset=offset)
    check(x, xg, targets(6, V, V), scale=0.7, k=min(V, 9), ids=torch.int64)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_masks_that_leave_little_or_nothing(cuda_device, V, dtype):
    x, _ = logits_of(8, V, V, dtype)
    low = torch.finfo(DT[dtype]).min
    x[0] = -math.inf                       # nothing left
    x[1] = -math.inf
    x[1, V - 1] = 2.0                      # one entry left
    x[2, : V // 2] = -math.inf             # masked half
    x[3] = low                             # the type's lowest value everywhere
    x[4, 1:] = low                         # and everywhere but once
    x[5] = low
    x[5, 0] = -math.inf
    t = torch.tensor([3, V - 1, 0, 7, 0, 1, -1, 5])
    # z of the lowest value is about -3e38: its absolute bound is useless, its p is exact
    got, want = check(x[[0, 1, 2, 4, 6, 7]], to_gpu(x[[0, 1, 2, 4, 6, 7]]), t[[0, 1, 2, 4, 6, 7]], k=4)
    assert got["logprob"][0].item() == -math.inf and got["entropy"][0].item() == 0.0
    o = forward(to_gpu(x[[3, 5]]), t[[3, 5]].cuda(), k=3)
    n = torch.tensor([V, V - 1.0]).log()
    near(o["entropy"], n, torch.tensor(16 * 2.0 ** -21) * (1 + math.log(V)))
    assert o["top_index"].cpu().tolist() == [[0, 1, 2], [1, 2, 3]]


@gpu
@pytest.mark.parametrize("V", [33, 6000, 90000])
def test_nan_and_infinities(cuda_device, V):
    x, _ = logits_of(5, V, V)
    x[0, V // 2] = math.nan
    x[1, 5] = math.inf
    x[2, 0] = math.nan
    x[2, 1:] = -math.inf
    t = torch.tensor([1, 5, 0, 2, -1])
    o = forward(to_gpu(x), t.cuda(), k=3)
    for n in ("logprob", "lse", "entropy"):
        assert torch.isnan(o[n][:3]).all() and torch.isfinite(o[n][3:]).all()
    assert torch.isnan(o["top_logprob"][:3]).all()
    assert o["top_index"][:, 0].cpu().tolist()[:3] == [V // 2, 5, 0]
    check(x[3:], to_gpu(x[3:]), t[3:], k=3)


@gpu
@pytest.mark.parametrize("V", [64, 3000, 66000])
@pytest.mark.parametrize("kind", ["constant", "ascending", "descending", "steps", "signs"])
def test_top_ties_and_orders(cuda_device, V, kind):
    j = torch.arange(V, dtype=torch.float32)
    row = {"constant": torch.zeros(V), "ascending": j * 1e-3, "descending": -j * 1e-3,
           "steps": (j % 5), "signs": torch.where(j % 2 == 0, 0.0, -0.0)}[kind]
    x = row.repeat(3, 1).contiguous()
    check(x, to_gpu(x), torch.tensor([0, V - 1, 3]), k=32)
    check(x.bfloat16(), to_gpu(x.bfloat16()), torch.tensor([0, V - 1, 3]), k=17)


@gpu
@pytest.mark.parametrize("k", [5, 32])
@pytest.mark.parametrize("R,V", [(1900, 3001), (1900, 33000), (500, 100003), (40, 100003), (3, 3001)])
def test_top_of_masked_and_equal_rows(cuda_device, R, V, k):
    """Constrained decoding: few entries above a mask of -inf or of a finite
    value, in rows by one to eight warps and by clusters.  Indices are exact."""
    g = torch.Generator(device="cuda").manual_seed(R + V)
    y = torch.randn(R, V, generator=g, device="cuda").mul_(3).bfloat16()
    row = torch.arange(R, device="cuda")[:, None]
    keep = torch.tensor([0, 1, 3, 4, 31, 33, 200], device="cuda")[row % 7]
    rank = torch.rand(R, V, generator=g, device="cuda").argsort(1).argsort(1)
    for mask in (-math.inf, torch.finfo(torch.bfloat16).min, -1e4, 0.0):
        x = torch.where(rank < keep, y, mask)
        x[:, V // 2:] = torch.where(row % 5 == 4, mask, x[:, V // 2:])
        x = torch.where(row % 11 == 10, y, x).bfloat16()
        o = forward(x, None, k=k)
        value, index = torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True)
        assert torch.equal(o["top_index"], index[:, :k].int())
        # relative to the largest entry: the lowest finite value takes all digits of a sum
        top = value[:, :1].double().clamp(min=-1e39)
        want = value[:, :k].double() - top - torch.exp(x.double() - top).sum(1, keepdim=True).log()
        want = torch.where(top == -1e39, -math.inf, want)
        fine = torch.isfinite(want)
        assert torch.equal(o["top_logprob"][~fine].double(), want[~fine])
        bound = (value[:, :1].double().abs().clamp(max=1e4) + want.abs().clamp(max=1e30) + 16) * 2.0 ** -21
        ok = (o["top_logprob"].double() - want).abs() <= bound
        assert ok[fine].all()


@gpu
@pytest.mark.parametrize("plateau", [0.0, -1e4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,vectors,offset", [(2000, 1024, 0), (2000, 1400, 1), (600, 5000, 0), (600, 14000, 3),
                                              (40, 3000, 0), (3, 20000, 0), (1, 12500, 1)])
def test_top_ties_between_the_end_of_a_row_and_its_middle(cuda_device, R, vectors, offset, dtype, plateau):
    """Equal allowed tokens over a plateau, some in the unaligned end of the
    row: the lower column comes first.  The entries lie in vectors 8 modulo 256
    and in the first entry of the end, so that few maxima of a row's threads
    exceed the plateau and its warps read their vectors again; rows by one to
    eight warps and by clusters."""
    N = 4 if dtype == "f32" else 8
    head = (N - offset) % N
    reach = vectors // 8 if R < 300 else vectors  # of the first block of a cluster
    for end in (1, 2, N - 1):
        V = head + vectors * N + end
        ld = (V + N - 1) // N * N
        x = torch.full((R, V), plateau)
        g = torch.Generator().manual_seed(V)
        row = torch.arange(R)
        for i in range(3):  # tied entries of the middle: one, two or three
            v = torch.randint(0, max(1, reach // 256), (R,), generator=g) * 256 + 8
            x[row, torch.where(i <= row % 3, head + v * N + (row + i) % N, V - end)] = 1.0
        x[row, V - end] = 1.0
        x[row[row % 4 != 0], head + 8 * N + 1] = 2.0
        if head:
            x[row[row % 5 == 0], 0] = 1.0
        for k in (1, 2, 3, 4, 9):
            xg = to_gpu(x.to(DT[dtype]), ld, offset)
            o = forward(xg, None, k=k)
            want = torch.sort(xg.float(), dim=1, descending=True, stable=True).indices[:, :k]
            wrong = (o["top_index"] != want).any(1)
            assert not wrong.any(), (end, k, int(wrong.sum()), o["top_index"][wrong][0].tolist(), want[wrong][0].tolist())


@gpu
def test_top_ties_of_a_row_end_that_reaches_the_bound_first(cuda_device):
    x = torch.zeros(2000, 4097)  # rows 4100 apart
    x[:, 32], x[:, 2592], x[:, 4096] = 2.0, 1.0, 1.0
    assert forward(to_gpu(x, 4100), None, k=2)["top_index"].unique(dim=0).tolist() == [[32, 2592]]
    x = torch.zeros(1, 50002)
    x[:, 1056], x[:, 50000], x[:, 50001] = 1.0, 1.0, 1.0
    assert forward(to_gpu(x, 50004), None, k=2)["top_index"].tolist() == [[1056, 50000]]


@gpu
@pytest.mark.parametrize("k", [0, 5, 20])
@pytest.mark.parametrize("R,V,dtype", [(4000, 32768, "bf16"), (4000, 16000, "f32"), (4000, 98304, "bf16"),
                                       (2000, 131072, "bf16"), (2000, 400003, "bf16"), (2000, 49152, "f32"),
                                       (20, 400003, "f32")])
def test_long_rows_of_equal_logits(cuda_device, R, V, dtype, k):
    """Equal terms round the same way each time they are added, below an entry
    of any size; the bound is that of all rows (runs of a tile and of tiles)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for kind in ("one above", "some above"):
        x = torch.zeros(R, V, device="cuda", dtype=DT[dtype])
        if kind == "one above":
            x[:, 7] = torch.linspace(0, 16, R, device="cuda").to(DT[dtype])
        else:
            x.scatter_(1, torch.randint(0, V, (R, 200), generator=g, device="cuda"),
                       torch.randn(R, 200, generator=g, device="cuda").mul_(3).to(DT[dtype]))
        t = torch.arange(R, device="cuda") % V
        o = forward(x, t, k=k)
        for i in range(0, R, 250):
            z = x[i:i + 250].double()
            u = (z.abs().amax(1) + 16) * 2.0 ** -21
            lse = torch.logsumexp(z, 1)
            z -= lse[:, None]
            assert torch.all((o["lse"][i:i + 250] - lse).abs() <= u)
            assert torch.all((o["logprob"][i:i + 250] - z.gather(1, t[i:i + 250, None])[:, 0]).abs() <= u)
            if k:
                assert torch.all((o["top_logprob"][i:i + 250] - z.topk(k, 1).values).abs() <= u[:, None])
            entropy = -(z.exp() * z).sum(1)
            assert torch.all((o["entropy"][i:i + 250] - entropy).abs() <= u * (1 + math.log(V)))


@gpu
def test_optional_outputs_and_no_targets(cuda_device):
    x, xg = logits_of(4, 3001, 5)
    check(x, xg, None, k=6)
    lp = torch.empty(4, device="cuda")
    t = targets(4, 3001, 3, pad=0.0)
    fg.forge_token_logprob(xg, t.cuda(), lp)
    near(lp, reference(x, t, 1.0)["logprob"], unit(x, 1.0))
    fg.forge_token_logprob(xg[:0], t[:0].cuda(), lp[:0])


@gpu
def test_target_outside_the_vocabulary_is_padding_and_recorded(cuda_device):
    x, xg = logits_of(3, 500, 5)
    t = torch.tensor([4, 500, -7])
    o = forward(xg, t.cuda(), k=2)
    assert fg.forge_get_device_status() == fg.FORGE_ERR_INVALID_ARG
    assert o["logprob"][1].item() == 0.0 and o["top_index"][1].tolist() == [-1, -1]
    near(o["logprob"], reference(x, torch.tensor([4, -1, -1]), 1.0)["logprob"], unit(x, 1.0))


@gpu
def test_repeats_bitwise_on_another_stream_and_in_a_graph(cuda_device):
    x, xg = logits_of(50, 30011, 9, "bf16")
    t = targets(50, 30011, 1).cuda()
    a = forward(xg, t, k=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = forward(xg, t, k=8)
    lp = torch.zeros(50, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.forge_token_logprob(xg, t, lp)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a) and torch.equal(lp, a["logprob"])


@gpu
def test_rows_past_32_bit_offsets(cuda_device):
    R, V = 33000, 65537
    x = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    row = logits_of(1, V, 3, "bf16")[0]
    x[R - 1] = row[0].cuda()
    t = torch.full((R,), 11, dtype=torch.int32, device="cuda")
    o = forward(x, t, k=3)
    one = forward(row.cuda(), t[:1], k=3)
    assert abs(o["logprob"][-1].item() - one["logprob"][0].item()) <= float(unit(row, 1.0)[0])
    assert torch.equal(o["top_index"][-1], one["top_index"][0])
    a = torch.ones(R, device="cuda")
    fg.forge_token_logprob_grad(x, t, o["lse"], a, x)  # in place
    want = -reference(row, torch.tensor([11]), 1.0)["p"]
    want[0, 11] += 1
    u = float(unit(row, 1.0)[0])
    near(x[-1:], want, want.abs() * (2.0 ** -8 + 4 * u) + 2.0 ** -120)
    near(x[:1, 1:9].float(), torch.full((1, 8), -1 / V, dtype=torch.float64),
         torch.tensor(2.0 ** -8 / V + 2.0 ** -24))


# ---- the gradient ------------------------------------------------------------

def grad(xg, t, lse, a, H=None, b=None, scale=1.0, out="f32", ld=None, dest=None):
    R, V = xg.shape
    if dest is None:
        buf = torch.full((R, V if ld is None else ld), 55.0, dtype=DT[out], device="cuda")
        dest = buf[:, :V]
    fg.forge_token_logprob_grad(xg, t, lse, a, dest, entropy=H, grad_entropy=b, scale=scale)
    torch.cuda.synchronize()
    return dest


def gradient_reference(x, t, a, b, scale):
    r = reference(x, t, scale)
    dead = r["skip"] | (r["lse"] == -math.inf)
    # p (ln p + H), 0 where p is 0
    ent = torch.where(r["p"] > 0, r["p"] * (torch.where(r["p"] > 0, r["logp"], 0.0) + r["entropy"][:, None]), 0.0)
    g = -a[:, None] * r["p"] - b[:, None] * ent
    rows = torch.nonzero(~dead)[:, 0]
    g[rows, t[rows].long()] += a[rows]
    g = torch.where(dead[:, None], 0.0, g * scale)
    # what an element's own terms allow: p by unit, the entropy's bracket by its parts
    u = unit(x, scale)[:, None]
    size = r["p"] * (a.abs()[:, None] + b.abs()[:, None] *
                     (torch.where(r["p"] > 0, r["logp"].abs(), 0.0) + r["entropy"][:, None] + 2 + math.log(x.shape[1])))
    return g, scale * (4 * u * torch.where(dead[:, None], 0.0, size)) + g.abs() * 2.0 ** -22 + 2.0 ** -120


@gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V,ld,offset", [(1, 1, 1, 0), (3, 2, 9, 1), (5, 33, 33, 0), (4, 1000, 1001, 1),
                                           (3, 4099, 4099, 3), (2, 50001, 50008, 0),
                                           (300, 264, 264, 0), (2, 131072, 131072, 0)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_matches_the_formula(cuda_device, R, V, ld, offset, dtype, out, entropy):
    scale = 0.75
    x, xg = logits_of(R, V, R + V, dtype, ld=ld, offset=offset)
    t = targets(R, V, V)
    f = forward(xg, t.cuda(), scale)
    g = torch.Generator().manual_seed(4)
    a = torch.randn(R, generator=g)
    b = torch.randn(R, generator=g) if entropy else torch.zeros(R)
    got = grad(xg, t.cuda(), f["lse"], a.cuda(), f["entropy"] if entropy else None,
               b.cuda() if entropy else None, scale, out, ld=V + 3)
    want, tol = gradient_reference(x, t, a.double(), b.double(), scale)
    if out == "bf16":
        tol = tol + want.abs() * 2.0 ** -8 + 2.0 ** -120
    near(got, want, tol)
    whole = got._base if got._base is not None else got
    assert (whole[:, V:] == 55.0).all()  # nothing past the row


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_in_place_and_masks(cuda_device, dtype):
    V = 5003
    x, _ = logits_of(6, V, 2, dtype)
    x[0] = -math.inf
    x[1, 7:] = -math.inf
    x[2, : V // 2] = torch.finfo(DT[dtype]).min
    t = torch.tensor([1, 3, V - 1, -1, 0, 9], dtype=torch.int64)
    xg = to_gpu(x)
    f = forward(xg, t.cuda())
    a, b = torch.randn(6), torch.randn(6)
    out = grad(xg, t.cuda(), f["lse"], a.cuda(), f["entropy"], b.cuda(), out=dtype)
    same = grad(xg, t.cuda(), f["lse"], a.cuda(), f["entropy"], b.cuda(), dest=xg)
    assert torch.equal(out, same)
    assert not out[0].any() and not out[3].any() and torch.isfinite(out.float()).all()
    want, tol = gradient_reference(x, t, a.double(), b.double(), 1.0)
    near(out, want, tol + want.abs() * (2.0 ** -8 if dtype == "bf16" else 0))


@gpu
def test_gradient_against_differences(cuda_device):
    """Central differences of the definition in 64 bits, step 1e-4: their own
    error is about h^2 (third derivatives below 1 here) plus 1e-16 / h."""
    R, V, scale = 3, 37, 1.25
    x, xg = logits_of(R, V, 77, std=1.0)
    t = torch.tensor([0, 36, 11])
    a, b = torch.tensor([0.5, -1.0, 2.0]), torch.tensor([0.25, 1.0, -0.5])
    f = forward(xg, t.cuda(), scale)
    got = grad(xg, t.cuda(), f["lse"], a.cuda(), f["entropy"], b.cuda(), scale).cpu().double()

    def value(y):
        r = reference(y, t, scale)
        return a.double() * r["logprob"] + b.double() * r["entropy"]

    h = 1e-4
    diff = torch.empty(R, V, dtype=torch.float64)
    for j in range(V):
        e = torch.zeros(R, V, dtype=torch.float64)
        e[:, j] = h
        diff[:, j] = (value(x.double() + e) - value(x.double() - e)) / (2 * h)
    assert (got - diff).abs().max() <= 2e-5


# ---- refusals ------------------------------------------------------------------

def test_refusals_before_any_launch():
    L = fg.lib()

    def f(x=FAKE, dt=fg.FORGE_F32, R=4, V=64, ld=64, t=FAKE, idt=fg.FORGE_I32, scale=1.0, lp=FAKE, lse=FAKE,
          k=2, ti=FAKE, tl=FAKE):
        return L.forge_token_logprob(x, dt, R, V, ld, t, idt, scale, lp, lse, None, k, ti, tl, None)
    bad = fg.FORGE_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(R=-1), dict(V=0), dict(ld=63), dict(t=None), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(k=-1), dict(k=33), dict(V=1, k=2),
               dict(ti=None), dict(tl=None), dict(R=1 << 31), dict(V=1 << 31, ld=1 << 31)):
        assert f(**kw) == bad, kw
    for kw in (dict(dt=fg.FORGE_E4M3), dict(dt=fg.FORGE_I32), dict(idt=fg.FORGE_F32), dict(idt=9)):
        assert f(**kw) == fg.FORGE_ERR_UNSUPPORTED_DTYPE, kw
    for kw in (dict(x=ctypes.c_void_p(0x10002)), dict(t=ctypes.c_void_p(0x10001)),
               dict(idt=fg.FORGE_I64, t=ctypes.c_void_p(0x10004)), dict(lp=ctypes.c_void_p(0x10001)),
               dict(tl=ctypes.c_void_p(0x10002))):
        assert f(**kw) == fg.FORGE_ERR_MISALIGNED, kw

    def g(x=FAKE, dt=fg.FORGE_BF16, R=4, V=64, ld=64, t=FAKE, idt=fg.FORGE_I32, scale=1.0, lse=FAKE, a=FAKE,
          H=None, b=None, dx=FAKE, odt=fg.FORGE_BF16, ldo=64):
        return L.forge_token_logprob_grad(x, dt, R, V, ld, t, idt, scale, lse, a, H, b, dx, odt, ldo, None)
    for kw in (dict(x=None), dict(t=None), dict(lse=None), dict(a=None), dict(dx=None), dict(b=FAKE), dict(ld=1),
               dict(ldo=63), dict(scale=0.0), dict(V=0), dict(R=-2)):
        assert g(**kw) == bad, kw
    for kw in (dict(dt=fg.FORGE_E4M3), dict(odt=fg.FORGE_E4M3), dict(idt=fg.FORGE_BF16)):
        assert g(**kw) == fg.FORGE_ERR_UNSUPPORTED_DTYPE, kw
    assert g(dx=ctypes.c_void_p(0x10001)) == fg.FORGE_ERR_MISALIGNED
    assert g(lse=ctypes.c_void_p(0x10002)) == fg.FORGE_ERR_MISALIGNED


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU what is not refused stops at the device check")
def test_gradient_refuses_rows_that_share_memory():
    """Every kind of overlap by the bytes of all rows; in place is none."""
    L = fg.lib()
    g = np.random.default_rng(5)
    seen = set()
    for _ in range(20000):
        R, V = int(g.integers(1, 6)), int(g.integers(1, 9))
        es, eo = (int(x) for x in g.choice([2, 4], 2))
        ld, ldo = V + int(g.choice([0, 1, 7, 12])), V + int(g.choice([0, 1, 7, 12]))
        if g.random() < 0.5:
            ldo = max(V, ld * es // eo)
        base = 1 << 20
        other = base + 4 * int(g.integers(-60, 60))
        own = {base + (r * ld + j) * es + i for r in range(R) for j in range(V) for i in range(es)}
        theirs = {other + (r * ldo + j) * eo + i for r in range(R) for j in range(V) for i in range(eo)}
        in_place = other == base and es == eo and (ld == ldo or R == 1)
        bad = not in_place and bool(own & theirs)
        code = {2: fg.FORGE_BF16, 4: fg.FORGE_F32}
        s = L.forge_token_logprob_grad(ctypes.c_void_p(base), code[es], R, V, ld, FAKE, fg.FORGE_I32, 1.0, FAKE, FAKE,
                                       None, None, ctypes.c_void_p(other), code[eo], ldo, None)
        assert s == (fg.FORGE_ERR_INVALID_ARG if bad else fg.FORGE_ERR_UNSUPPORTED_DEVICE), \
            (R, V, es, eo, ld, ldo, other - base, bad)
        seen.add((bad, in_place, es == eo, ld * es == ldo * eo))
    assert len(seen) > 8


@gpu
def test_gradient_beside_its_logits_in_one_buffer(cuda_device):
    R, V = 9, 1000
    x, _ = logits_of(R, V, 3)
    t = targets(R, V, 3)
    f = forward(x.cuda(), t.cuda())
    a = torch.ones(R, device="cuda")
    want = grad(x.cuda(), t.cuda(), f["lse"], a)
    buf = torch.zeros(R, 2 * V, device="cuda")
    buf[:, :V] = x.cuda()
    assert torch.equal(grad(buf[:, :V], t.cuda(), f["lse"], a, dest=buf[:, V:]), want)
    assert torch.equal(buf[:, :V].cpu(), x)
    for dest in (buf[:, 1:V + 1], buf[:, V - 1:2 * V - 1], buf.view(-1)[: R * V].view(R, V),
                 buf.view(torch.bfloat16)[:, :V]):
        with pytest.raises(fg.ForgeError):
            fg.forge_token_logprob_grad(buf[:, :V], t.cuda(), f["lse"], a, dest)
    assert torch.equal(buf[:, :V].cpu(), x)


@gpu
def test_binding_refuses_what_does_not_fit(cuda_device):
    x = torch.zeros(4, 8, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    lp = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        fg.forge_token_logprob(x.t(), t, lp)
    with pytest.raises(ValueError):
        fg.forge_token_logprob(x, t[:3], lp)
    with pytest.raises(ValueError):
        fg.forge_token_logprob(x, t, lp[:3])
    with pytest.raises(TypeError):
        fg.forge_token_logprob(x, t.float(), lp)
    with pytest.raises(TypeError):
        fg.forge_token_logprob(x.half(), t, lp)
    with pytest.raises(ValueError):
        fg.forge_token_logprob(x.cpu(), t, lp)
    with pytest.raises(fg.ForgeError):
        fg.forge_token_logprob(x, t, lp, scale=0.0)
    with pytest.raises(fg.ForgeError):  # host memory behind a device call
        s = fg.lib().forge_token_logprob(ctypes.c_void_p(torch.zeros(32).data_ptr()), fg.FORGE_F32, 4, 8, 8, None,
                                         fg.FORGE_I32, 1.0, None, ctypes.c_void_p(lp.data_ptr()), None, 0, None,
                                         None, None)
        fg._check(s, "forge_token_logprob")
