"""An expert layer of a language model, there and back, around the grouped weight gradient.

    out = x + sum over the k chosen experts e of w_e (norm(x) W_e)

with W [E, D, D] fp32 masters, a router Wr [D, E] and the balance loss added to
the model's.  A step of it is the library's calls in the order that they need:

forward    h = forge_layer_norm(x)                              bf16, statistics kept
           logits = h Wr                                        (a plain product, cuBLAS)
           experts, weights, offsets, slots, rows, loss = forge_moe_route(logits)
           packed = forge_embedding(rows, h)                    rows by expert
           codes = forge_quantize_e4m3_blocks(packed; W)        rows; 128 x 128 squares
           y = forge_grouped_linear_e4m3(codes, offsets)
           out = x + sum_j weights[j] y[slots[j]]               (indexing)
backward   dy = weights dout by packed rows, dweights = dout . y
           dpacked = forge_grouped_linear_e4m3(dy's codes, W's, transpose)
           W, m, v = forge_grouped_wgrad_adamw(packed, dy, offsets)   after W's codes are read
           dh = forge_embedding_grad(dpacked, rows)             the rows' sum by token
           dlogits = forge_moe_route_grad(dweights, balance)
           dh += dlogits Wr^T; Wr = forge_wgrad_adamw(h, dlogits)
           dx = dout + forge_layer_norm_grad(dh); its weight and bias by forge_owner_adamw
"""
from __future__ import annotations


class Experts:
    """The layer's weights, their AdamW state, the hyperparameters and what a forward pass
    keeps for the way back."""

    def __init__(self, width: int, experts: int, top: int, *, device="cuda", seed=0, balance=1e-2,
                 lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01):
        import torch
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape, std):
            w = torch.randn(*shape, generator=g, device=device).mul_(std)
            return w, torch.zeros_like(w), torch.zeros_like(w)

        self.W, self.Wm, self.Wv = weight(experts, width, width, std=width ** -0.5)
        self.R, self.Rm, self.Rv = weight(width, experts, std=width ** -0.5)
        self.scale, self.Sm, self.Sv = weight(width, std=0.0)
        self.scale += 1.0
        self.shift, self.Bm, self.Bv = weight(width, std=0.0)
        self.top = top
        self.balance = torch.full((1,), float(balance), device=device)
        self.hp = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, wd=wd)
        self.t = 0
        self.kept = None


def _codes(x, block_rows):
    import torch

    import weight_grad_gemm_gb300 as fg
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((*x.shape[:-2], -(-x.shape[-2] // block_rows), -(-x.shape[-1] // 128)),
                         device=x.device)
    fg.forge_quantize_e4m3_blocks(x, codes, scales, block_rows=block_rows)
    return codes, scales


def forward(layer: Experts, x):
    """out [T, D] (bf16) of x [T, D] (bf16); the balance loss is layer.kept["loss"]."""
    import torch

    import weight_grad_gemm_gb300 as fg
    T, D = x.shape
    E, k = layer.W.shape[0], layer.top
    i32 = dict(dtype=torch.int32, device=x.device)
    h = torch.empty_like(x)
    mean, rstd = torch.empty(T, device=x.device), torch.empty(T, device=x.device)
    fg.forge_layer_norm(x, layer.scale, layer.shift, h, mean=mean, rstd=rstd)
    Rb = layer.R.to(torch.bfloat16)
    logits = h @ Rb
    experts, slots, rows = (torch.empty(s, **i32) for s in ((T, k), (T, k), (T * k,)))
    counts, offsets, live = (torch.empty(n, **i32) for n in (E, E + 1, 1))
    weights, loss = torch.empty(T, k, device=x.device), torch.empty(1, device=x.device)
    fg.forge_moe_route(logits, experts, weights, counts, offsets, slots=slots, rows=rows, live=live,
                       loss=loss)
    packed = torch.empty((T * k, D), dtype=x.dtype, device=x.device)
    fg.forge_embedding(rows, h, packed)
    A, sA = _codes(packed, 1)
    W, sW = _codes(layer.W, 128)
    y = torch.zeros_like(packed)
    fg.forge_grouped_linear_e4m3(A, sA, W, sW, offsets, y)
    at = slots.long()
    mine = y[at.clamp(min=0)].float() * (at >= 0)[..., None]  # [T, k, D]
    layer.kept = dict(x=x, h=h, mean=mean, rstd=rstd, Rb=Rb, logits=logits, experts=experts, counts=counts,
                      live=live, weights=weights, offsets=offsets, rows=rows, at=at, packed=packed, W=W,
                      sW=sW, mine=mine, loss=loss)
    return (x.float() + (weights[..., None] * mine).sum(1)).to(x.dtype)


def backward(layer: Experts, dout):
    """dx [T, D] (bf16) of dout [T, D] (bf16), and one AdamW step on every weight."""
    import torch

    import weight_grad_gemm_gb300 as fg
    s = layer.kept
    T, D = dout.shape
    step = dict(step=layer.t + 1, **layer.hp)
    dweights = (dout.float()[:, None] * s["mine"]).sum(2)
    dy = torch.zeros((T * layer.top + 1, D), dtype=dout.dtype, device=dout.device)
    # (choices without a slot go to a row behind the last)
    dy[torch.where(s["at"] >= 0, s["at"], T * layer.top).reshape(-1)] = \
        (s["weights"][..., None] * dout.float()[:, None]).to(dout.dtype).reshape(-1, D)
    dy = dy[:-1]
    A, sA = _codes(dy, 1)
    dpacked = torch.zeros_like(dy)
    fg.forge_grouped_linear_e4m3(A, sA, s["W"], s["sW"], s["offsets"], dpacked, transpose=True)
    fg.forge_grouped_wgrad_adamw(s["packed"], dy, layer.W, layer.Wm, layer.Wv, s["offsets"], **step)
    dh = torch.empty((T, D), device=dout.device)
    fg.forge_embedding_grad(dpacked, s["rows"], dh)
    dlogits = torch.empty_like(s["logits"])
    fg.forge_moe_route_grad(s["logits"], s["experts"], s["counts"], s["live"], dlogits,
                            grad_weights=dweights, grad_loss=layer.balance)
    dh += (dlogits @ s["Rb"].T).float()
    fg.forge_wgrad_adamw(s["h"], dlogits, layer.R, layer.Rm, layer.Rv, **step)
    dx = torch.empty_like(dout)
    dscale, dshift = torch.empty(D, device=dout.device), torch.empty(D, device=dout.device)
    fg.forge_layer_norm_grad(dh, s["x"], layer.scale, s["mean"], s["rstd"], dx, dscale, dshift)
    fg.forge_owner_adamw(dscale, layer.scale, layer.Sm, layer.Sv, **step)
    fg.forge_owner_adamw(dshift, layer.shift, layer.Bm, layer.Bv, **step)
    layer.t += 1
    layer.kept = None
    return dx + dout
