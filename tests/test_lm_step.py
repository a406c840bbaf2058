"""The two ends of a training step together (weight_grad_gemm_gb300/lm.py): one
step's weights against the same step in 64 bits, and the fused and clipped
forms against each other.

The reference takes the bf16 roundings that the step has by definition (X, the
head's copy, logits, dlogits, dX) where they are made, from 64-bit values; a
value near a rounding boundary may fall on its other side, so state is compared
by its relative norm: bf16's 2^-8 half step on part of the terms, 2e-3 in all.
"""
import pytest
import torch

import weight_grad_gemm_gb300 as fg
from weight_grad_gemm_gb300 import lm

pytestmark = pytest.mark.gpu


def batch(vocab, tokens, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    targets = torch.randint(0, vocab, (tokens,), generator=g)
    ids[::11] = -1
    targets[::7] = -1
    return ids.cuda(), targets.cuda()


def b16(x):
    return x.float().to(torch.bfloat16).double()


def gradients(ends, ids, targets):
    """dW, dE and the loss of one step in 64 bits."""
    E, W = ends.E.double(), ends.W.double()
    live = (ids >= 0)[:, None]
    X = b16(torch.where(live, E[ids.clamp(min=0)] * ends.scale, 0.0))
    Wb = b16(W)
    logits = b16(X @ Wb)
    logp = logits.log_softmax(1)
    counts = targets >= 0
    n = counts.sum()
    t = targets.clamp(min=0)
    loss = -(logp.gather(1, t[:, None])[:, 0] * counts).sum() / n
    d = logp.exp()
    d.scatter_add_(1, t[:, None], torch.full_like(d[:, :1], -1.0))
    d = b16(d * counts[:, None] / n)
    dX = b16(d @ Wb.T)
    dE = torch.zeros_like(E).index_add_(0, ids.clamp(min=0), torch.where(live, dX, 0.0)) * ends.scale
    return X.T @ d, dE, loss


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("vocab,width,tokens", [(1000, 256, 777), (501, 136, 300)])
def test_fused_step(cuda_device, vocab, width, tokens):
    ends = lm.Ends(vocab, width, wd=0.0)
    ids, targets = batch(vocab, tokens, vocab)
    dW, dE, loss = gradients(ends, ids, targets)
    got = lm.step(ends, ids, targets)
    torch.cuda.synchronize()
    assert abs(float(got) - float(loss)) <= 1e-4 * float(loss)
    # from zero state m = (1 - beta1) g
    assert relative(ends.Wm / 0.1, dW) <= 2e-3 and relative(ends.Em / 0.1, dE) <= 2e-3
    assert fg.forge_get_device_status() == fg.FORGE_OK


@pytest.mark.parametrize("max_norm", [1e-2, 1e6])
def test_clipped_step(cuda_device, max_norm):
    vocab, width, tokens = 900, 256, 500
    ids, targets = batch(vocab, tokens, 3)
    ends, fused = lm.Ends(vocab, width), lm.Ends(vocab, width)
    dW, dE, _ = gradients(ends, ids, targets)
    want = float(torch.sqrt(dW.square().sum() + dE.square().sum()))
    _, norm = lm.step_clipped(ends, ids, targets, max_norm)
    assert abs(float(norm) - want) <= 2e-3 * want
    factor = min(1.0, max_norm / (float(norm) + 1e-6))
    lm.step(fused, ids, targets)
    torch.cuda.synchronize()
    if factor == 1.0:  # nothing clipped: the same arithmetic as the fused step
        for n in ("W", "Wm", "Wv", "E", "Em", "Ev"):
            assert torch.equal(getattr(ends, n), getattr(fused, n)), n
    else:
        assert relative(ends.Wm, fused.Wm * factor) <= 1e-6
        assert relative(ends.Em, fused.Em * factor) <= 1e-6


def test_training_lowers_the_loss(cuda_device):
    g = torch.Generator().manual_seed(1)
    seq = torch.randint(0, 800, (100,), generator=g)[torch.arange(2001) % 100].cuda()
    ends = lm.Ends(800, 128, lr=3e-3)
    losses = [float(lm.step(ends, seq[:-1], seq[1:])) for _ in range(25)]
    assert losses[0] > 5.0 and losses[-1] < 0.5 * losses[0]
