"""An expert layer's step (weight_grad_gemm_gb300/moe.py): every call in the order and
with the outputs of the others, against the same step in 64 bits.

The reference makes the roundings that the step has by definition (bf16 h, logits,
packed rows and gradients, e4m3 codes) where they are made, from 64-bit values, and
takes the layer's own choices of experts.  A value next to a border may fall on its
other side: an e4m3 step is 2^-3 of the value, and one entry in 2^9 at most lies within
the 2^-8 half step of a bf16 input of a border, so that sums differ by about 2^-3 2^-4.5
2^-3 (few of many terms) in the norm; bf16 outputs by 2^-9 rms.  4e-3 in all, and 1e-2 for
the gradients, which have two such roundings behind each other.
"""
import pytest
import torch

import weight_grad_gemm_gb300 as fg
from weight_grad_gemm_gb300 import lm, moe

pytestmark = pytest.mark.gpu


def b16(x):
    return x.float().to(torch.bfloat16).double()


def e4m3(x, br):
    """Values of the codes of x (fp32 values) by blocks."""
    R, C = x.shape
    x = x.float()
    a = torch.nn.functional.pad(x.abs(), (0, -C % 128, 0, -R % br))
    a = a.unflatten(-1, (-1, 128)).amax(-1).unflatten(0, (-1, br)).amax(1)
    s = torch.where(a > 0, a / torch.tensor(448.0, device=x.device), 1.0)
    s = s.repeat_interleave(br, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return (x / s).to(torch.float8_e4m3fn).double() * s.double()


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def reference(layer, x, dout):
    T, D = x.shape
    E, k = layer.W.shape[0], layer.top
    s = layer.kept
    X, W, R = x.double(), layer.W.double(), b16(layer.R)
    mu = X.mean(1, keepdim=True)
    rstd = (X.var(1, correction=0, keepdim=True) + 1e-5) ** -0.5
    xh = (X - mu) * rstd
    h = b16(xh * layer.scale.double() + layer.shift.double())
    logits = b16(h @ R)
    p = logits.softmax(1)
    experts = s["experts"].long()
    w = p.gather(1, experts)
    w = w / w.sum(1, keepdim=True)
    Wq = torch.stack([e4m3(layer.W[e], 128) for e in range(E)])
    hq = e4m3(h, 1)
    y = torch.stack([b16(hq @ Wq[e]) for e in range(E)], 1)  # [T, E, D]
    mine = y.gather(1, experts[..., None].expand(T, k, D))
    out = b16(X + (w[..., None] * mine).sum(1))
    d = dout.double()
    dw = (d[:, None] * mine).sum(2)
    dy = b16(w[..., None] * d[:, None])  # [T, k, D]
    dW = torch.zeros_like(W)
    dh = torch.zeros_like(X)
    for j in range(k):
        q = e4m3(dy[:, j], 1)
        for e in range(E):
            at = experts[:, j] == e
            dW[e] += h[at].T @ dy[at, j]
            dh[at] += b16(q[at] @ Wq[e].T)
    counts = torch.bincount(experts.reshape(-1), minlength=E).double()
    n = T
    loss = (counts * p.mean(0)).sum() * E / (k * n)
    g = torch.zeros_like(p).scatter_(1, experts, (dw - (dw * w).sum(1, keepdim=True)) / p.gather(1, experts).sum(1, keepdim=True))
    g = g + float(layer.balance) * E * counts / (k * n * n)
    dlogits = b16(p * (g - (p * g).sum(1, keepdim=True)))
    dh = dh + b16(dlogits @ R.T)
    gg = dh * layer.scale.double()
    dx = rstd * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True)) + d
    return dict(out=out, loss=loss, dW=dW, dR=h.T @ dlogits, dscale=(dh * xh).sum(0), dshift=dh.sum(0), dx=dx)


@pytest.mark.parametrize("T,D,E,k", [(300, 256, 4, 2), (777, 136, 8, 2), (64, 512, 16, 4), (1, 128, 3, 1), (1000, 130, 1, 1)])
def test_step_of_the_layer(cuda_device, T, D, E, k):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16).cuda()
    dout = (torch.randn(T, D, generator=g) * 1e-2).to(torch.bfloat16).cuda()
    layer = moe.Experts(D, E, k, seed=1, wd=0.0, balance=0.05)
    out = moe.forward(layer, x)
    want = reference(layer, x, dout)
    assert relative(out, want["out"]) <= 4e-3
    assert abs(float(layer.kept["loss"]) - float(want["loss"])) <= 2e-3 * float(want["loss"])
    o = layer.kept["offsets"]
    assert int(o[-1]) == T * k and torch.equal(layer.kept["counts"].cumsum(0), o[1:])
    dx = moe.backward(layer, dout)
    assert relative(dx, want["dx"]) <= 1e-2
    # from zero state m = (1 - beta1) g
    assert relative(layer.Wm / 0.1, want["dW"]) <= 1e-2
    assert relative(layer.Sm / 0.1, want["dscale"]) <= 1e-2 and relative(layer.Bm / 0.1, want["dshift"]) <= 1e-2
    if E > 1:
        # the router's gradient is a difference of terms larger than itself
        assert relative(layer.Rm / 0.1, want["dR"]) <= 5e-2
    assert fg.forge_get_device_status() == fg.FORGE_OK


def test_a_token_that_is_not_a_number_stays_alone(cuda_device):
    T, D, E = 200, 128, 4
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16).cuda()
    layer = moe.Experts(D, E, 2)
    plain = moe.forward(layer, x)
    x[::5] = float("nan")
    out = moe.forward(layer, x)
    keep = torch.arange(T, device="cuda") % 5 != 0
    assert torch.isnan(out[~keep]).all() and torch.isfinite(out[keep]).all()
    assert torch.equal(out[keep], plain[keep])


def test_lm_step_with_experts_runs(cuda_device):
    g = torch.Generator().manual_seed(1)
    seq = torch.randint(0, 500, (301,), generator=g).cuda()
    ends, layer = lm.Ends(500, 128), moe.Experts(128, 8, 2)
    before = [t.clone() for t in (ends.E, ends.W, layer.W, layer.R, layer.scale, layer.shift)]
    for _ in range(3):
        loss = lm.step(ends, seq[:-1], seq[1:], layer)
    assert torch.isfinite(loss)
    after = (ends.E, ends.W, layer.W, layer.R, layer.scale, layer.shift)
    assert all(torch.isfinite(a).all() and not torch.equal(a, b) for a, b in zip(after, before))
    assert fg.forge_get_device_status() == fg.FORGE_OK
