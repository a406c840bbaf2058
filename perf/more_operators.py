"""The operators of an expert layer around its weight gradients, measured case by case: layer
norm and its gradient, the router with its balance loss and their gradient, e4m3 codes with a
scale for each block of 128, and the products of such codes, dense and by experts.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run``
does one pass (the elementary torch form, or the library's kernels where ``own`` is true),
``work`` gives the bytes and operations a pass cannot do without and ``exact`` the outputs in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5
PAD_SHARE = 1 / 32  # tokens that are padding: all their router logits are -inf
BLOCK = 128


def listed():
    return [
        # the norm in front of a projection in one decode step: 16 tokens, no statistics kept
        {"name": "norm_decode", "op": "norm", "rows": 16, "width": 4096, "x": "bf16", "y": "bf16", "bias": True, "stats": False},
        # a training batch of bf16 activations, statistics kept for the way back
        {"name": "norm_batch", "op": "norm", "rows": 16384, "width": 4096, "x": "bf16", "y": "bf16", "bias": True, "stats": True},
        # a ragged microbatch in fp32 of an odd width, the weight's gradient added to an accumulator
        {"name": "norm_grad_micro", "op": "norm_grad", "rows": 777, "width": 1023, "dy": "f32", "x": "f32", "dx": "f32",
         "bias": True, "accumulate": True},
        # a training batch's gradient in bf16
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 16384, "width": 4096, "dy": "bf16", "x": "bf16", "dx": "bf16",
         "bias": True, "accumulate": False},
        # the routing of one decode step: 16 tokens to 2 of 8 experts
        {"name": "route_decode", "op": "route", "tokens": 16, "experts": 8, "top": 2, "logits": "f32", "normalize": True,
         "grad": False},
        # a training step's routing there and back, 2 of 8 experts, bf16 logits (many of them equal)
        {"name": "route_train_top2", "op": "route", "tokens": 16384, "experts": 8, "top": 2, "logits": "bf16",
         "normalize": True, "grad": True},
        # many small experts: 8 of 256 for every token of a large batch, there and back
        {"name": "route_train_top8", "op": "route", "tokens": 65536, "experts": 256, "top": 8, "logits": "f32",
         "normalize": False, "grad": True},
        # a ragged batch of activations, a scale for each 128 entries of a row, rows that end inside a block
        {"name": "codes_rows", "op": "codes", "rows": 2049, "width": 4100, "x": "bf16", "block_rows": 1},
        # an fp32 master weight, a scale for each 128 x 128 square
        {"name": "codes_weight", "op": "codes", "rows": 14336, "width": 4096, "x": "f32", "block_rows": 128},
        # one decode step's product with a projection of 4096 x 14336: all of it is reading the weight
        {"name": "linear_decode", "op": "linear", "tokens": 16, "inner": 4096, "outer": 14336, "transpose": False, "experts": 0,
         "y": "bf16"},
        # the input gradient of a ragged batch, rows of 4100 codes that no 16-byte copy can address
        {"name": "linear_dx", "op": "linear", "tokens": 4099, "inner": 4096, "outer": 4100, "transpose": True, "experts": 0,
         "y": "f32"},
        # an expert layer's down-projection: 16384 tokens to 2 of 8 experts, packed by expert
        {"name": "linear_experts", "op": "linear", "tokens": 32768, "inner": 14336, "outer": 4096, "transpose": False,
         "experts": 8, "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "codes", "linear", "linear"])
    kind = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op in ("norm", "norm_grad"):
        width = _log(rng, 32, 16384)
        case = {"op": op, "rows": _log(rng, 1, min(65536, (1 << 26) // width)), "width": width, "x": kind(), "bias": rng.random() < 0.7}
        if op == "norm":
            return {**case, "y": kind(), "stats": rng.random() < 0.5}
        return {**case, "dy": kind(), "dx": kind(), "accumulate": rng.random() < 0.3}
    if op == "route":
        experts = _log(rng, 2, 512)
        return {"op": op, "tokens": _log(rng, 1, min(65536, (1 << 24) // experts)), "experts": experts,
                "top": rng.randint(1, min(8, experts)), "logits": kind(), "normalize": rng.random() < 0.5, "grad": rng.random() < 0.5}
    if op == "codes":
        width = _log(rng, 64, 16384)
        return {"op": op, "rows": _log(rng, 1, min(65536, (1 << 26) // width)), "width": width, "x": kind(),
                "block_rows": rng.choice([1, 1, BLOCK])}
    inner, outer = _log(rng, 128, 14336), _log(rng, 128, 14336)
    round_to = rng.choice([1, 4, 16, 128])
    inner, outer = (max(round_to, n // round_to * round_to) for n in (inner, outer))
    experts = rng.choice([0, 0, _log(rng, 2, min(64, max(2, (1 << 29) // (inner * outer))))])
    return {"op": op, "tokens": _log(rng, 1, min(16384, (1 << 39) // (inner * outer))), "inner": inner, "outer": outer,
            "transpose": rng.random() < 0.5, "experts": experts, "y": kind()}


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _blocks(n):
    return -(-n // BLOCK)


def _activations(g, rows, width, dtype=torch.float32):
    """Activations whose features have magnitudes of their own, a few of them large, and a mean."""
    scale = torch.exp(_randn(g, width, std=0.7))
    return _randn(g, rows, width).mul_(scale).add_(0.3).to(dtype)


def _amax_scales(x, block_rows):
    """amax / 448 of each block_rows x 128 block of x [..., R, C], 1 where a block is zero."""
    R, C = x.shape[-2:]
    a = torch.nn.functional.pad(x.float().abs(), (0, -C % BLOCK, 0, -R % block_rows))
    a = a.unflatten(-1, (-1, BLOCK)).amax(-1).unflatten(-2, (-1, block_rows)).amax(-2)
    return torch.where(a > 0, a / a.new_full((), 448.0), 1.0)  # by a tensor: a quotient, not a product with 1 / 448


def _spread(s, rows, cols, block_rows):
    """A block's value at each of its entries."""
    return s.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _codes(x, block_rows):
    s = _amax_scales(x, block_rows)
    return (x.float() / _spread(s, *x.shape[-2:], block_rows)).to(torch.float8_e4m3fn), s


def _routed(g, rows, experts):
    """Offsets of rows packed by expert, popular and unpopular ones, a few rows behind the last."""
    p = torch.exp(_randn(g, experts, std=0.8))
    e = torch.multinomial(p, rows, replacement=True, generator=g) if rows > 1 else torch.zeros(rows, dtype=torch.int64, device="cuda")
    counts = torch.bincount(e[: rows - rows // 64], minlength=experts)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        R, D = case["rows"], case["width"]
        s["x"] = _activations(g, R, D, DTYPES[case["x"]])
        s["weight"] = 1.0 + _randn(g, D, std=0.2)
        s["bias"] = _randn(g, D, std=0.2) if case["bias"] else None
        if op == "norm":
            s["y"] = torch.empty(R, D, device="cuda", dtype=DTYPES[case["y"]])
            s["mean"], s["rstd"] = (torch.empty(R, device="cuda") if case["stats"] else None for _ in range(2))
        else:
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, correction=0) + EPS).float()
            s["dy"] = _randn(g, R, D, std=1e-2, dtype=DTYPES[case["dy"]])
            s["dx"] = torch.empty(R, D, device="cuda", dtype=DTYPES[case["dx"]])
            s["dweight"] = _randn(g, D, std=1e-2) if case["accumulate"] else torch.empty(D, device="cuda")
            s["dbias"] = _randn(g, D, std=1e-2) if case["bias"] else None
    elif op == "route":
        T, E, k = case["tokens"], case["experts"], case["top"]
        z = _randn(g, T, E) + _randn(g, E, std=0.7)
        pad = torch.rand(T, 1, generator=g, device="cuda") < PAD_SHARE
        s["logits"] = z.masked_fill_(pad, -math.inf).to(DTYPES[case["logits"]])
        for name, shape in (("experts", (T, k)), ("slots", (T, k)), ("rows", (T * k,)), ("counts", (E,)), ("offsets", (E + 1,)), ("live", (1,))):
            s[name] = torch.empty(shape, dtype=torch.int32, device="cuda")
        s["weights"], s["loss"] = torch.empty(T, k, device="cuda"), torch.empty(1, device="cuda")
        if case["grad"]:
            s["grad_weights"] = _randn(g, T, k, std=0.1)
            s["grad_loss"] = torch.rand(1, generator=g, device="cuda") + 0.5
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "codes":
        R, C, br = case["rows"], case["width"], case["block_rows"]
        s["x"] = _activations(g, R, C, DTYPES[case["x"]]) if br == 1 else _randn(g, R, C, std=0.02, dtype=DTYPES[case["x"]])
        s["codes"] = torch.empty(R, C, device="cuda", dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(-(-R // br), _blocks(C), device="cuda")
    else:
        T, N, M, E = case["tokens"], case["inner"], case["outer"], case["experts"]
        s["A"], s["sA"] = _codes(_activations(g, T, M if case["transpose"] else N), 1)
        s["W"], s["sW"] = _codes(_randn(g, *([E] if E else []), N, M, std=0.02), BLOCK)
        s["Y"] = torch.zeros(T, N if case["transpose"] else M, device="cuda", dtype=DTYPES[case["y"]])
        s["offsets"] = _routed(g, T, E) if E else None
        s["bounds"] = s["offsets"].tolist() if E else None
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    return _kernels(s) if own else _plain(s)


ROUTE = ("experts", "weights", "slots", "rows", "counts", "offsets", "live", "loss")


def _kernels(s):
    import weight_grad_gemm_gb300 as fg
    case = s["case"]
    op = case["op"]
    if op == "norm":
        fg.forge_layer_norm(s["x"], s["weight"], s["bias"], s["y"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
        return {k: s[k] for k in ("y", "mean", "rstd")}
    if op == "norm_grad":
        fg.forge_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                 accumulate=case["accumulate"])
        return {k: s[k] for k in ("dx", "dweight", "dbias")}
    if op == "route":
        fg.forge_moe_route(s["logits"], s["experts"], s["weights"], s["counts"], s["offsets"], slots=s["slots"], rows=s["rows"],
                           live=s["live"], loss=s["loss"], normalize=case["normalize"])
        out = {k: s[k] for k in ROUTE}
        if case["grad"]:
            fg.forge_moe_route_grad(s["logits"], s["experts"], s["counts"], s["live"], s["dlogits"], grad_weights=s["grad_weights"],
                                    grad_loss=s["grad_loss"], normalize=case["normalize"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "codes":
        fg.forge_quantize_e4m3_blocks(s["x"], s["codes"], s["scales"], block_rows=case["block_rows"])
        return {k: s[k] for k in ("codes", "scales")}
    if s["offsets"] is None:
        fg.forge_linear_e4m3(s["A"], s["sA"], s["W"], s["sW"], s["Y"], transpose=case["transpose"])
    else:
        fg.forge_grouped_linear_e4m3(s["A"], s["sA"], s["W"], s["sW"], s["offsets"], s["Y"], transpose=case["transpose"])
    return s["Y"]


def _plain(s):
    case = s["case"]
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "route": _plain_route, "codes": _plain_codes,
            "linear": _plain_linear}[case["op"]](s, case)


def _plain_norm(s, case):
    x = s["x"].float()
    mean = x.sum(1) / case["width"]
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / case["width"] + EPS)
    y = d * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    stats = case["stats"]
    return {"y": y.to(s["y"].dtype), "mean": mean if stats else None, "rstd": rstd if stats else None}


def _plain_norm_grad(s, case):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True)) / case["width"])
    out = {"dx": dx.to(s["dx"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if s["dbias"] is not None else None}
    if case["accumulate"]:
        out["dweight"] = s["dweight"].add_(out["dweight"])
        out["dbias"] = None if s["dbias"] is None else s["dbias"].add_(out["dbias"])
    return out


def _probabilities(z):
    """Softmax rows of z; a row without a finite entry gives zeros."""
    top = z.max(1, keepdim=True).values
    live = top > -math.inf
    e = torch.exp(z - torch.where(live, top, 0.0))
    return e / torch.where(live, e.sum(1, keepdim=True), 1.0), live[:, 0]


def _plain_route(s, case):
    T, E, k = case["tokens"], case["experts"], case["top"]
    z = s["logits"].float()
    p, live = _probabilities(z)
    top = torch.sort(z, dim=1, descending=True, stable=True)
    experts = top.indices[:, :k].masked_fill(top.values[:, :k] == -math.inf, -1)
    chosen = torch.where(experts >= 0, p.gather(1, experts.clamp(min=0)), 0.0)
    total = chosen.sum(1, keepdim=True) if case["normalize"] else torch.ones_like(chosen[:, :1])
    total = torch.where(live[:, None], total, 1.0)
    weights = chosen / total
    flat = torch.where(experts >= 0, experts, E).reshape(-1)
    counts = (flat[:, None] == torch.arange(E, device=z.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.sort(flat, stable=True).indices
    place = torch.arange(T * k, device=z.device)
    packed = place < offsets[-1]
    slots = torch.empty_like(place)
    slots[order] = torch.where(packed, place, -1)
    count = live.sum()
    n = count.clamp(min=1).float()
    loss = (counts * (p.sum(0) / n)).sum() * E / (k * n)
    i32 = torch.int32
    out = {"experts": experts.to(i32), "weights": weights, "slots": slots.reshape(T, k).to(i32),
           "rows": torch.where(packed, order // k, -1).to(i32), "counts": counts.to(i32), "offsets": offsets.to(i32),
           "live": count.to(i32)[None], "loss": loss[None]}
    if case["grad"]:
        q = (s["grad_loss"] * counts * (E / (k * n * n))).expand(T, E).clone()
        by = s["grad_weights"]
        if case["normalize"]:
            by = by - (by * weights).sum(1, keepdim=True)
        by = torch.where(experts >= 0, by / total, 0.0)
        q.scatter_add_(1, experts.clamp(min=0), by)
        out["dlogits"] = (p * (q - (p * q).sum(1, keepdim=True))).to(s["dlogits"].dtype)
    return out


def _plain_codes(s, case):
    codes, scales = _codes(s["x"], case["block_rows"])
    return {"codes": codes, "scales": scales}


def _values(codes, scales, block_rows, dtype):
    return codes.to(dtype) * _spread(scales.to(dtype), *codes.shape[-2:], block_rows)


def _product(s, case, dtype):
    A = _values(s["A"], s["sA"], 1, dtype)
    weight = lambda W, sW: _values(W, sW, BLOCK, dtype).T if case["transpose"] else _values(W, sW, BLOCK, dtype)  # noqa: E731
    if s["bounds"] is None:
        return A @ weight(s["W"], s["sW"])
    Y = torch.zeros_like(s["Y"], dtype=dtype)
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            Y[lo:hi] = A[lo:hi] @ weight(s["W"][e], s["sW"][e])
    return Y


def _plain_linear(s, case):
    return _product(s, case, torch.float32).to(s["Y"].dtype)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        R, D = case["rows"], case["width"]
        return {"bytes": R * D * (SIZE[case["x"]] + SIZE[case["y"]]) + (8 if case["bias"] else 4) * D + (8 * R if case["stats"] else 0),
                "flops": 8 * R * D}
    if op == "norm_grad":
        R, D = case["rows"], case["width"]
        params = (8 if case["bias"] else 4) * (2 if case["accumulate"] else 1) + 4
        return {"bytes": R * D * (SIZE[case["dy"]] + SIZE[case["x"]] + SIZE[case["dx"]]) + params * D + 8 * R, "flops": 14 * R * D}
    if op == "route":
        T, E, k, size = case["tokens"], case["experts"], case["top"], SIZE[case["logits"]]
        there = T * E * size + 16 * T * k + 8 * E + 12
        back = 2 * T * E * size + 8 * T * k + 4 * E + 8 if case["grad"] else 0
        return {"bytes": there + back, "flops": (12 if case["grad"] else 5) * T * E}
    if op == "codes":
        R, C = case["rows"], case["width"]
        return {"bytes": R * C * (SIZE[case["x"]] + 1) + 4 * -(-R // case["block_rows"]) * _blocks(C), "flops": 3 * R * C}
    T, N, M, E = case["tokens"], case["inner"], case["outer"], max(1, case["experts"])
    K, out = (M, N) if case["transpose"] else (N, M)
    E = min(E, T)
    return {"bytes": T * (K + 4 * _blocks(K)) + E * (N * M + 4 * _blocks(N) * _blocks(M)) + T * out * SIZE[case["y"]],
            "flops": 2 * T * N * M}


# ---- the definition, in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(torch.zeros((), device="cuda", dtype=torch.float64) if s["bias"] is None else s["bias"].double(),
                          (x - mean[:, None]).mul_(rstd[:, None]), s["weight"].double())
        return {"y": y, "mean": mean if case["stats"] else None, "rstd": rstd if case["stats"] else None}
    if op == "norm_grad":
        # dx as the derivative of xhat: (I - 1 1'/D - xhat xhat'/D) rstd, applied to dy * w
        D = case["width"]
        dy, rstd = s["dy"].double(), s["rstd"].double()
        xh = s["x"].double().sub_(s["mean"].double()[:, None]).mul_(rstd[:, None])
        dw = torch.einsum("rd,rd->d", dy, xh)
        db = torch.einsum("rd->d", dy)
        g = dy * s["weight"].double()
        along = torch.einsum("rd,rd->r", g, xh) / D
        dx = (g - g.mean(1, keepdim=True)).sub_(xh.mul_(along[:, None])).mul_(rstd[:, None])
        start = lambda t: t.double() if case["accumulate"] else 0.0  # noqa: E731
        return {"dx": dx, "dweight": dw + start(s["dweight"]), "dbias": None if s["dbias"] is None else db + start(s["dbias"])}
    if op == "route":
        return _exact_route(s, case)
    if op == "codes":
        R, C, br = case["rows"], case["width"], case["block_rows"]
        a = torch.zeros(-(-R // br) * br, _blocks(C) * BLOCK, device="cuda", dtype=torch.float64)
        a[:R, :C] = s["x"].double().abs()
        a = a.reshape(-1, br, _blocks(C), BLOCK).permute(0, 2, 1, 3).flatten(2).max(-1).values / 448
        return {"codes": None, "scales": torch.where(a == 0, 1.0, a)}
    return _product(s, case, torch.float64)


def _exact_route(s, case):
    T, E, k = case["tokens"], case["experts"], case["top"]
    z = s["logits"].double()
    live = torch.isfinite(z).any(1)
    logp = torch.where(live[:, None], z, 0.0).log_softmax(1)
    p = logp.exp() * live[:, None]
    # the k largest, one after another, each the first of its value
    left, one = z.clone(), []
    for _ in range(k):
        best = left.max(1, keepdim=True).values
        at = (left == best).to(torch.int8).argmax(1, keepdim=True)
        one.append(torch.where(best > -math.inf, at, -1))
        left.scatter_(1, at, -math.inf)
    experts = torch.cat(one, 1)
    hit = torch.zeros(T, E + 1, device="cuda", dtype=torch.float64)
    hit.scatter_(1, torch.where(experts >= 0, experts, E), 1.0)
    hit = hit[:, :E]
    counts = hit.sum(0)
    n = max(1, int(live.sum()))
    mass = (p * hit).sum(1, keepdim=True) if case["normalize"] else torch.ones_like(p[:, :1])
    mass = torch.where(live[:, None], mass, 1.0)
    weights = torch.where(experts >= 0, p.gather(1, experts.clamp(min=0)), 0.0) / mass
    ends = counts.cumsum(0)
    # a choice's slot: its expert's beginning and the tokens before it that chose the expert
    before = (hit.cumsum(0) - hit + (ends - counts)).gather(1, experts.clamp(min=0))
    slots = torch.where(experts >= 0, before, -1.0).to(torch.int64)
    rows = torch.full((T * k + 1,), -1, device="cuda", dtype=torch.int64)
    rows[torch.where(slots < 0, T * k, slots).reshape(-1)] = torch.arange(T, device="cuda").repeat_interleave(k)
    rows[T * k] = -1
    out = {"experts": experts, "weights": weights, "slots": slots, "rows": rows[:-1], "counts": counts.to(torch.int64),
           "offsets": torch.cat([ends.new_zeros(1), ends]).to(torch.int64), "live": live.sum()[None],
           "loss": ((p.sum(0) / n * counts).sum() * E / (k * n))[None]}
    if case["grad"]:
        gw = torch.zeros(T, E + 1, device="cuda", dtype=torch.float64)
        gw.scatter_(1, torch.where(experts >= 0, experts, E), s["grad_weights"].double())
        gw = gw[:, :E] * hit
        if case["normalize"]:
            gw = (gw - (gw * p).sum(1, keepdim=True) / mass) / mass * hit
        q = gw + float(s["grad_loss"]) * E / (k * n * n) * counts
        out["dlogits"] = p * q - p * (p * q).sum(1, keepdim=True)
    return out
