"""The two ends of a language model's training step around a linear head.

The model is an embedding and a head: X = scale * E[ids], logits = X W, with
E [V, D] and W [D, V] fp32 masters; the loss is the mean cross-entropy of the
next tokens, and rows whose target is negative are padding.  A full model puts
its layers between the two; their steps are the library's other calls.

step           the fused form: no gradient of a weight reaches memory.
                   X = forge_embedding(ids, E)
                   logits = X W                            (a plain product, cuBLAS)
                   logprob, lse = forge_token_logprob(logits, targets)
                   dlogits = forge_token_logprob_grad(...)     in place of the logits
                   dX, W = forge_backward_adamw(X, dlogits, W)   dX before the update
                   E = forge_embedding_adamw(dX, ids, E)
step_clipped   the form with global-norm clipping, which needs every gradient
               before it may touch a weight ("Math verified, not asserted", P2):
               dX by forge_dgrad, dW by forge_wgrad_only, dE by
               forge_embedding_grad, then forge_grad_norm and forge_clip_grads
               over both and forge_owner_adamw on each weight.

    python -m weight_grad_gemm_gb300.lm       trains on a repeated sequence
"""
from __future__ import annotations


class Ends:
    """The weights, their AdamW state and the hyperparameters of both ends."""

    def __init__(self, vocab: int, width: int, *, device="cuda", seed=0, lr=1e-3, beta1=0.9,
                 beta2=0.999, eps=1e-8, wd=0.01):
        import torch
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device=device).mul_(0.02)
            return w, torch.zeros_like(w), torch.zeros_like(w)

        self.E, self.Em, self.Ev = weight(vocab, width)
        self.W, self.Wm, self.Wv = weight(width, vocab)
        self.scale = float(width) ** 0.5
        self.hp = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, wd=wd)
        self.t = 0


def forward(ends: Ends, ids, targets):
    """X, the bf16 copy of W it met, logits (bf16), and logprob, lse of the targets."""
    import torch

    import weight_grad_gemm_gb300 as fg
    T, D = ids.numel(), ends.E.shape[1]
    X = torch.empty((T, D), dtype=torch.bfloat16, device=ids.device)
    fg.forge_embedding(ids, ends.E, X, scale=ends.scale)
    Wb = ends.W.to(torch.bfloat16)
    logits = X @ Wb
    logprob, lse = (torch.empty(T, device=ids.device) for _ in range(2))
    fg.forge_token_logprob(logits, targets, logprob, lse=lse)
    return X, Wb, logits, logprob, lse


def _loss_and_dlogits(ends, ids, targets):
    import weight_grad_gemm_gb300 as fg
    X, Wb, logits, logprob, lse = forward(ends, ids, targets)
    count = (targets >= 0).sum().clamp(min=1)
    loss = -logprob.sum() / count
    weight = (-1.0 / count).to(logprob.dtype).expand(targets.numel()).contiguous()
    fg.forge_token_logprob_grad(logits, targets, lse, weight, logits)  # in place
    return X, Wb, logits, loss


def step(ends: Ends, ids, targets):
    """One training step; returns the loss before it (a device scalar)."""
    import torch

    import weight_grad_gemm_gb300 as fg
    X, Wb, dlogits, loss = _loss_and_dlogits(ends, ids, targets)
    ends.t += 1
    dX = torch.empty_like(X)
    fg.forge_backward_adamw(X, dlogits, ends.W, ends.Wm, ends.Wv, dX, Wb=Wb, step=ends.t, **ends.hp)
    fg.forge_embedding_adamw(dX, ids, ends.E, ends.Em, ends.Ev, scale=ends.scale, step=ends.t,
                             **ends.hp)
    return loss


def step_clipped(ends: Ends, ids, targets, max_norm: float):
    """One training step with the gradients clipped to max_norm; returns the
    loss before it and the gradients' norm (device scalars)."""
    import torch

    import weight_grad_gemm_gb300 as fg
    X, Wb, dlogits, loss = _loss_and_dlogits(ends, ids, targets)
    ends.t += 1
    dX = torch.empty_like(X)
    dW, dE = torch.empty_like(ends.W), torch.empty_like(ends.E)
    fg.forge_dgrad(dlogits, Wb, dX)
    fg.forge_wgrad_only(X, dlogits, dW)
    fg.forge_embedding_grad(dX, ids, dE, scale=ends.scale)
    norm = torch.empty(1, device=dW.device)
    fg.forge_grad_norm([dW, dE], norm)
    fg.forge_clip_grads([dW, dE], norm, max_norm=max_norm)
    fg.forge_owner_adamw(dW, ends.W, ends.Wm, ends.Wv, step=ends.t, **ends.hp)
    fg.forge_owner_adamw(dE, ends.E, ends.Em, ends.Ev, step=ends.t, **ends.hp)
    return loss, norm


def main(vocab=5000, width=256, tokens=4096, steps=30):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, vocab, (tokens + 1,), generator=g, device="cuda")
    ids = ids[torch.arange(tokens + 1, device="cuda") % 300]  # a sequence that repeats
    for clipped in (False, True):
        ends = Ends(vocab, width)
        losses = []
        for _ in range(steps):
            if clipped:
                loss, norm = step_clipped(ends, ids[:-1], ids[1:], 0.25)
            else:
                loss = step(ends, ids[:-1], ids[1:])
            losses.append(loss)
        print(f"{'clipped' if clipped else 'fused'}: loss {float(losses[0]):.3f} -> "
              f"{float(losses[-1]):.3f} in {steps} steps"
              + (f", last norm {float(norm):.3f}" if clipped else ""))


if __name__ == "__main__":
    main()
