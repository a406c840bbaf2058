"""Steps of expert layers (weight_grad_gemm_gb300/moe.py) on two streams at once, and captured
and replayed: bitwise what the same steps give one after another."""
import pytest
import torch

import weight_grad_gemm_gb300 as fg
from weight_grad_gemm_gb300 import moe

pytestmark = pytest.mark.gpu

# (a router of several blocks and one of one, widths in vectors and without, operands copied
# into padded rows; a width beyond the registers of the layer norm's gradient)
SIZES = [(3000, 264, 16, 2), (2500, 131, 300, 8), (40, 8200, 2, 1)]


def inputs(T, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]


def step(layer, x, dout):
    out = moe.forward(layer, x)
    loss = layer.kept["loss"]
    return [out, loss, moe.backward(layer, dout)]


def state(layer):
    return [layer.W, layer.Wm, layer.Wv, layer.R, layer.Rm, layer.Rv, layer.scale, layer.shift]


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b, strict=True))


@pytest.mark.parametrize("first,second", [(0, 1), (1, 2), (0, 0)])
def test_two_streams(cuda_device, first, second):
    sizes = [SIZES[first], SIZES[second]]
    data = [inputs(T, D, i) for i, (T, D, _, _) in enumerate(sizes)]
    layers = lambda: [moe.Experts(D, E, k, seed=i) for i, (_, D, E, k) in enumerate(sizes)]  # noqa: E731
    alone = layers()
    want = [[step(layer, *d) for _ in range(3)] for layer, d in zip(alone, data)]
    both = layers()
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(both[i], *data[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i], strict=True):
            assert same(a, b)
        assert same(state(both[i]), state(alone[i]))
    assert fg.forge_get_device_status() == 0


@pytest.mark.parametrize("T,D,E,k", SIZES)
def test_captured(cuda_device, T, D, E, k):
    x, dout = inputs(T, D, 5)
    y, dy = inputs(T, D, 6)
    eager, captured = moe.Experts(D, E, k), moe.Experts(D, E, k)
    kept = [t.clone() for t in state(captured)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (libraries' first calls)
        step(captured, x, dout)
    side.synchronize()
    for t, s in zip(state(captured), kept):
        t.copy_(s)
    captured.t = 0
    # what the step moves besides state(): the statistics of the norm's weights
    for t in (captured.Sm, captured.Sv, captured.Bm, captured.Bv):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(captured, x, dout)
    # every replay is a first step of the weights as they are then
    for a, b in ((x, dout), (y, dy)):
        eager.t = 0
        want = step(eager, a.clone(), b.clone())
        x.copy_(a)
        dout.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want) and same(state(captured), state(eager))
    assert fg.forge_get_device_status() == 0
