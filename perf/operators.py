"""The operators at the two ends of a language model's training step, measured case by case:
token log-probabilities of logits (with entropy and the top alternatives) and their gradient,
the embedding lookup, its gradient by tokens and its gradient fused with AdamW, and the global
gradient norm over many tensors with clipping.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run``
does one pass (the elementary torch form, or the library's kernels where ``own`` is true),
``work`` gives the bytes and operations a pass cannot do without and ``exact`` the outputs in
64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}
SIZE = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
ADAM = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "wd": 0.01}
ADAM = {k: float(np.float32(v)) for k, v in ADAM.items()} | {"step": 4}  # the 32-bit values that the library receives
PAD_SHARE = 1 / 32  # tokens that are padding (a negative id): no logit, row or gradient of theirs counts


def listed():
    return [
        # the answers of one decode step: 16 sequences, the 20 best alternatives of each, an odd vocabulary
        {"name": "logprob_decode", "op": "logprob", "rows": 16, "vocab": 50001, "stride": 50001, "masked": 0,
         "dtype": "f32", "ids": "i64", "top": 20, "scale": 1.25},
        # scoring of rolled-out answers: log-probability and entropy of every token, five alternatives
        {"name": "logprob_rollout", "op": "logprob", "rows": 8192, "vocab": 131072, "stride": 131072, "masked": 64,
         "dtype": "bf16", "ids": "i32", "top": 5, "scale": 1.0},
        # a policy gradient with an entropy term on a short ragged batch, fp32 logits in a padded buffer
        {"name": "logprob_grad_entropy", "op": "logprob_grad", "rows": 513, "vocab": 50001, "stride": 50008, "masked": 0,
         "dtype": "f32", "out": "f32", "ids": "i64", "entropy": True, "scale": 0.8},
        # the cross-entropy gradient of a training batch, bf16 logits to the bf16 dY of the head's weight gradient
        {"name": "logprob_grad_train", "op": "logprob_grad", "rows": 8192, "vocab": 131072, "stride": 131072, "masked": 64,
         "dtype": "bf16", "out": "bf16", "ids": "i32", "entropy": False, "scale": 1.0},
        # the lookup of one decode step
        {"name": "embedding_decode", "op": "embedding", "tokens": 64, "vocab": 131072, "width": 4096,
         "weight": "bf16", "out": "bf16", "ids": "i64", "scale": 1.0},
        # the lookup of a training batch from the fp32 master weight, scaled by the square root of the width
        {"name": "embedding_batch", "op": "embedding", "tokens": 65536, "vocab": 131072, "width": 4096,
         "weight": "f32", "out": "bf16", "ids": "i32", "scale": 64.0},
        # a microbatch's gradient added to an accumulator, odd width
        {"name": "embedding_grad_micro", "op": "embedding_grad", "tokens": 2048, "vocab": 50001, "width": 1023,
         "grad": "f32", "ids": "i64", "scale": 1.0, "accumulate": True},
        # a training batch's gradient, written whole
        {"name": "embedding_grad_batch", "op": "embedding_grad", "tokens": 32768, "vocab": 131072, "width": 4096,
         "grad": "bf16", "ids": "i32", "scale": 64.0, "accumulate": False},
        # a small model's fused step with bf16 state
        {"name": "embedding_adamw_small", "op": "embedding_adamw", "tokens": 4096, "vocab": 32768, "width": 520,
         "grad": "bf16", "state": "bf16", "ids": "i64", "scale": 1.0},
        # a training batch's fused step, fp32 state: the gradient never reaches memory
        {"name": "embedding_adamw_batch", "op": "embedding_adamw", "tokens": 32768, "vocab": 131072, "width": 4096,
         "grad": "bf16", "state": "f32", "ids": "i32", "scale": 64.0},
        # the clipping of a small model's gradients: many short tensors of odd sizes
        {"name": "clip_small", "op": "clip", "layers": 6, "width": 257, "hidden": 1001, "grad": "f32", "out": "f32",
         "max_norm": 1.0},
        # the clipping of a large model's fp32 gradients (wgrad shapes of 4096 and 14336) into bf16 copies
        {"name": "clip_model", "op": "clip", "layers": 4, "width": 4096, "hidden": 14336, "grad": "f32", "out": "bf16",
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "logprob_grad", "embedding", "embedding_grad", "embedding_adamw", "clip"])
    ids = rng.choice(["i32", "i64"])
    scale = rng.choice([1.0, 0.5, 1.25, 64.0])
    if op in ("logprob", "logprob_grad"):
        vocab = _log(rng, 1000, 160000)
        rows = _log(rng, 1, min(16384, (1 << 29) // vocab))
        case = {"op": op, "rows": rows, "vocab": vocab, "stride": vocab + rng.choice([0, 0, 1, 7, 64]),
                "masked": rng.choice([0, 0, vocab // 50]), "dtype": rng.choice(["f32", "bf16"]), "ids": ids,
                "scale": rng.choice([1.0, 0.5, 1.25])}
        if op == "logprob":
            return {**case, "top": rng.choice([0, 1, 5, 20, 32])}
        return {**case, "out": rng.choice(["f32", "bf16"]), "entropy": rng.random() < 0.5}
    if op == "embedding":
        width = _log(rng, 64, 8192)
        return {"op": op, "tokens": _log(rng, 1, min(131072, (1 << 28) // width)), "vocab": _log(rng, 1000, 160000),
                "width": width, "weight": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "ids": ids,
                "scale": scale}
    if op in ("embedding_grad", "embedding_adamw"):
        width = _log(rng, 64, 8192)
        case = {"op": op, "tokens": _log(rng, 1, min(65536, (1 << 27) // width)),
                "vocab": _log(rng, 1000, min(160000, (1 << 28) // width)), "width": width,
                "grad": rng.choice(["f32", "bf16"]), "ids": ids, "scale": scale}
        if op == "embedding_grad":
            return {**case, "accumulate": rng.random() < 0.3}
        return {**case, "state": rng.choice(["f32", "bf16"])}
    width = _log(rng, 64, 4096)
    return {"op": op, "layers": rng.randint(1, 4), "width": width, "hidden": int(width * rng.uniform(2.5, 3.5)),
            "grad": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]),
            "max_norm": rng.choice([0.5, 1.0, 1e6])}


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _pad(g, ids, share=PAD_SHARE):
    return torch.where(torch.rand(ids.shape, generator=g, device="cuda") < share, -1, ids)


def _token_ids(g, tokens, vocab, dtype):
    """Token ids with the frequencies of text: id r has probability about 1 / ((r + 1) ln vocab)."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(vocab + 1)).to(torch.int64).sub_(1).clamp_(0, vocab - 1)
    return _pad(g, ids).to(dtype)


def _distinct(tokens, vocab):
    """The expected number of distinct rows that tokens of _token_ids touch."""
    r = np.arange(vocab, dtype=np.float64)
    p = np.log((r + 2) / (r + 1)) / math.log(vocab + 1)
    return float(np.sum(-np.expm1(tokens * (1 - PAD_SHARE) * np.log1p(-p))))


def _logits(g, case):
    """Logits of a model that is sure of some of its tokens, and the tokens asked for; the last
    ``masked`` columns pad the vocabulary and are masked."""
    R, V, ld = case["rows"], case["vocab"], case["stride"]
    live = V - case["masked"]
    t = torch.randint(0, live, (R,), generator=g, device="cuda")
    buf = torch.randn(R, ld, generator=g, device="cuda").mul_(2.5)
    sure = torch.rand(R, 1, generator=g, device="cuda") * 16
    buf.scatter_add_(1, t[:, None], sure)
    buf[:, live:V] = -math.inf
    return buf.to(DTYPES[case["dtype"]])[:, :V], _pad(g, t).to(DTYPES[case["ids"]])


def _lse_entropy(x, targets, scale):
    """What the forward pass hands the gradient: log-sum-exp and entropy of each row."""
    z = x.float() * scale
    lse = torch.logsumexp(z, 1)
    z -= lse[:, None]
    entropy = -(torch.exp(z) * z.clamp(min=-1e4)).sum(1)
    skip = targets < 0
    return lse.masked_fill(skip, 0.0), entropy.masked_fill(skip, 0.0)


def _clip_sizes(case):
    d, h = case["width"], case["hidden"]
    return ([(d, d)] * 4 + [(h, d)] * 3 + [(d,)] * 2) * case["layers"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "logprob":
        R, k = case["rows"], case["top"]
        s["logits"], s["targets"] = _logits(g, case)
        s["logprob"], s["lse"], s["entropy"] = (torch.empty(R, device="cuda") for _ in range(3))
        s["top_index"] = torch.empty(R, k, device="cuda", dtype=torch.int32) if k else None
        s["top_logprob"] = torch.empty(R, k, device="cuda") if k else None
    elif op == "logprob_grad":
        R, V = case["rows"], case["vocab"]
        s["logits"], s["targets"] = _logits(g, case)
        s["lse"], s["entropy"] = _lse_entropy(s["logits"], s["targets"], case["scale"])
        s["grad_logprob"] = _randn(g, R, std=0.5) - 1.0
        s["grad_entropy"] = _randn(g, R, std=0.05) if case["entropy"] else None
        s["dlogits"] = torch.empty(R, case["stride"], device="cuda", dtype=DTYPES[case["out"]])[:, :V]
    elif op == "embedding":
        T, V, D = case["tokens"], case["vocab"], case["width"]
        s["ids"] = _token_ids(g, T, V, DTYPES[case["ids"]])
        s["W"] = _randn(g, V, D, std=0.02, dtype=DTYPES[case["weight"]])
        s["Y"] = torch.empty(T, D, device="cuda", dtype=DTYPES[case["out"]])
    elif op in ("embedding_grad", "embedding_adamw"):
        T, V, D = case["tokens"], case["vocab"], case["width"]
        s["ids"] = _token_ids(g, T, V, DTYPES[case["ids"]])
        s["dY"] = _randn(g, T, D, std=1e-3, dtype=DTYPES[case["grad"]])
        if op == "embedding_grad":
            s["dW"] = _randn(g, V, D, std=1e-3) if case["accumulate"] else torch.empty(V, D, device="cuda")
        else:
            st = DTYPES[case["state"]]
            s["W"] = _randn(g, V, D, std=0.02)
            s["m"] = _randn(g, V, D, std=1e-3, dtype=st)
            s["v"] = _randn(g, V, D, std=1e-3).square_().to(st)
    else:
        s["grads"] = [_randn(g, *size, std=1e-3, dtype=DTYPES[case["grad"]]) for size in _clip_sizes(case)]
        s["out"] = [torch.empty(*size, device="cuda", dtype=DTYPES[case["out"]]) for size in _clip_sizes(case)]
        s["norm"] = torch.empty(1, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    return _kernels(s) if own else _plain(s)


def _kernels(s):
    import weight_grad_gemm_gb300 as fg
    case = s["case"]
    op = case["op"]
    if op == "logprob":
        fg.forge_token_logprob(s["logits"], s["targets"], s["logprob"], lse=s["lse"], entropy=s["entropy"],
                               top_index=s["top_index"], top_logprob=s["top_logprob"], scale=case["scale"])
        return {k: s[k] for k in ("logprob", "lse", "entropy", "top_index", "top_logprob")}
    if op == "logprob_grad":
        fg.forge_token_logprob_grad(s["logits"], s["targets"], s["lse"], s["grad_logprob"], s["dlogits"],
                                    entropy=s["entropy"], grad_entropy=s["grad_entropy"], scale=case["scale"])
        return s["dlogits"]
    if op == "embedding":
        fg.forge_embedding(s["ids"], s["W"], s["Y"], scale=case["scale"])
        return s["Y"]
    if op == "embedding_grad":
        fg.forge_embedding_grad(s["dY"], s["ids"], s["dW"], scale=case["scale"], accumulate=case["accumulate"])
        return s["dW"]
    if op == "embedding_adamw":
        fg.forge_embedding_adamw(s["dY"], s["ids"], s["W"], s["m"], s["v"], scale=case["scale"], **ADAM)
        return {k: s[k] for k in ("W", "m", "v")}
    fg.forge_grad_norm(s["grads"], s["norm"])
    fg.forge_clip_grads(s["grads"], s["norm"], s["out"], max_norm=case["max_norm"])
    return {"norm": s["norm"], "out": s["out"]}


def _plain(s):
    case = s["case"]
    return {"logprob": _plain_logprob, "logprob_grad": _plain_logprob_grad, "embedding": _plain_embedding,
            "embedding_grad": _plain_embedding_grad, "embedding_adamw": _plain_embedding_adamw,
            "clip": _plain_clip}[case["op"]](s, case)


def _plain_logprob(s, case):
    x, t, k = s["logits"], s["targets"].long(), case["top"]
    skip = t < 0
    z = x.float() * case["scale"]
    top = z.max(1, keepdim=True).values
    ref = torch.where(top == -math.inf, 0.0, top)
    d = z - ref
    e = torch.exp(d)
    total = e.sum(1)
    lse = ref[:, 0] + torch.log(total)
    none = total == 0
    entropy = torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1) / total
    entropy = entropy.masked_fill(none | skip, 0.0)
    of_target = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    logprob = torch.where(none, -math.inf, of_target - lse).masked_fill(skip, 0.0)
    out = {"logprob": logprob, "lse": lse.masked_fill(skip, 0.0), "entropy": entropy, "top_index": None,
           "top_logprob": None}
    if k:
        # one whole number for each logit, ordered by value and then by the lower index
        bits = (x.float() + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
        key += 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
        index = 0xFFFFFFFF - (key.topk(k, dim=1).values & 0xFFFFFFFF)
        lp = torch.where(none[:, None], -math.inf, z.gather(1, index) - lse[:, None])
        out["top_index"] = index.masked_fill(skip[:, None], -1).to(torch.int32)
        out["top_logprob"] = lp.masked_fill(skip[:, None], 0.0)
    return out


def _plain_logprob_grad(s, case):
    x, t = s["logits"], s["targets"].long()
    skip = (t < 0) | (s["lse"] == -math.inf)
    d = x.float() * case["scale"] - s["lse"][:, None]
    p = torch.exp(d)
    by = s["grad_logprob"][:, None]
    if s["grad_entropy"] is not None:
        by = by + s["grad_entropy"][:, None] * (torch.where(p > 0, d, 0.0) + s["entropy"][:, None])
    g = -(p * by)
    g.scatter_add_(1, t.clamp(min=0)[:, None], s["grad_logprob"][:, None])
    g *= case["scale"]
    return g.masked_fill_(skip[:, None], 0.0).to(s["dlogits"].dtype)


def _plain_embedding(s, case):
    ids = s["ids"].long()
    rows = s["W"][ids.clamp(min=0)].float() * case["scale"]
    return rows.masked_fill_((ids < 0)[:, None], 0.0).to(s["Y"].dtype)


def _embedding_sum(s, case):
    ids = s["ids"].long()
    dY = s["dY"].float() * case["scale"]
    dY.masked_fill_((ids < 0)[:, None], 0.0)
    return torch.zeros(case["vocab"], case["width"], device="cuda").index_add_(0, ids.clamp(min=0), dY)


def _plain_embedding_grad(s, case):
    dW = _embedding_sum(s, case)
    return s["dW"].add_(dW) if case["accumulate"] else dW


def _plain_embedding_adamw(s, case):
    G = _embedding_sum(s, case)
    b1, b2, step = ADAM["beta1"], ADAM["beta2"], ADAM["step"]
    m = b1 * s["m"].float() + (1 - b1) * G
    v = b2 * s["v"].float() + (1 - b2) * G * G
    den = torch.sqrt(v / (1 - b2 ** step)) + ADAM["eps"]
    W = s["W"] * (1 - ADAM["lr"] * ADAM["wd"]) - ADAM["lr"] * (m / (1 - b1 ** step)) / den
    s["W"].copy_(W)
    s["m"].copy_(m)
    s["v"].copy_(v)
    return {k: s[k] for k in ("W", "m", "v")}


def _plain_clip(s, case):
    norm = torch.sqrt(torch.stack([g.float().square().sum() for g in s["grads"]]).sum())
    coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm[None], "out": [(g.float() * coef).to(o.dtype) for g, o in zip(s["grads"], s["out"])]}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "logprob":
        R, V, k = case["rows"] * (1 - PAD_SHARE), case["vocab"], case["top"]
        return {"bytes": R * V * SIZE[case["dtype"]] + case["rows"] * (SIZE[case["ids"]] + 12 + 8 * k),
                "flops": 6 * R * V}
    if op == "logprob_grad":
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * (SIZE[case["dtype"]] * (1 - PAD_SHARE) + SIZE[case["out"]])
                + R * (SIZE[case["ids"]] + (16 if case["entropy"] else 8)),
                "flops": 6 * R * V}
    if op == "clip":
        n = sum(math.prod(size) for size in _clip_sizes(case))
        return {"bytes": n * (SIZE[case["grad"]] + SIZE[case["out"]]) + 4, "flops": 3 * n}
    T, V, D = case["tokens"], case["vocab"], case["width"]
    live = T * (1 - PAD_SHARE)
    if op == "embedding":
        return {"bytes": _distinct(T, V) * D * SIZE[case["weight"]] + T * (D * SIZE[case["out"]] + SIZE[case["ids"]]),
                "flops": T * D}
    read = live * D * SIZE[case["grad"]] + T * SIZE[case["ids"]]
    if op == "embedding_grad":
        rows = 2 * _distinct(T, V) if case["accumulate"] else V
        return {"bytes": read + rows * D * 4, "flops": live * D}
    return {"bytes": read + V * D * (8 + 4 * SIZE[case["state"]]), "flops": live * D + 12 * V * D}


# ---- the definition, in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprob":
        z = s["logits"].double().mul_(case["scale"])
        pad = s["targets"].long() < 0
        lse = torch.logsumexp(z, 1)
        logprob = z.gather(1, s["targets"].long().clamp(min=0)[:, None])[:, 0] - lse
        out = {"logprob": logprob, "lse": lse, "entropy": None, "top_index": None, "top_logprob": None}
        if case["top"]:
            out["top_logprob"] = (z.topk(case["top"], dim=1).values - lse[:, None]).masked_fill(pad[:, None], 0.0)
        logp = z.sub_(lse[:, None])
        out["entropy"] = torch.special.entr(logp.exp_()).sum(1)
        for k in ("logprob", "lse", "entropy"):
            out[k] = out[k].masked_fill(pad, 0.0)
        return out
    if op == "logprob_grad":
        t = s["targets"].long()
        p = torch.exp(s["logits"].double().mul_(case["scale"]).sub_(s["lse"].double()[:, None]))
        gl = s["grad_logprob"].double()
        g = p * -gl[:, None]
        if case["entropy"]:
            # d entropy / d z = -p (ln p + H), and -p ln p is entr(p)
            g += s["grad_entropy"].double()[:, None] * (torch.special.entr(p) - p * s["entropy"].double()[:, None])
        rows = torch.nonzero(t >= 0)[:, 0]
        g[rows, t[rows]] += gl[rows]
        return g.mul_(case["scale"]).mul_((t >= 0)[:, None])
    if op == "embedding":
        ids = s["ids"].long()
        return torch.where((ids >= 0)[:, None], s["W"].double()[ids.clamp(min=0)] * case["scale"], 0.0)
    if op in ("embedding_grad", "embedding_adamw"):
        V, D = case["vocab"], case["width"]
        ids = s["ids"].long()
        at = torch.where(ids < 0, V, ids)
        G = torch.zeros(V + 1, D, device="cuda", dtype=torch.float64)
        G = G.index_add_(0, at, s["dY"].double())[:V].mul_(case["scale"])
        if op == "embedding_grad":
            return G.add_(s["dW"].double()) if case["accumulate"] else G
        m = s["m"].double().mul_(ADAM["beta1"]).add_(G, alpha=1 - ADAM["beta1"])
        v = s["v"].double().mul_(ADAM["beta2"]).addcmul_(G, G, value=1 - ADAM["beta2"])
        root = torch.sqrt(v / (1 - ADAM["beta2"] ** ADAM["step"])).add_(ADAM["eps"])
        W = s["W"].double().mul_(1 - ADAM["lr"] * ADAM["wd"]).addcdiv_(m, root, value=-ADAM["lr"] / (1 - ADAM["beta1"] ** ADAM["step"]))
        return {"W": W, "m": m, "v": v}
    total = sum(float(torch.linalg.vector_norm(g.double()) ** 2) for g in s["grads"])
    coef = min(1.0, case["max_norm"] / (math.sqrt(total) + 1e-6))
    return {"norm": np.array([math.sqrt(total)]), "out": [g.double() * coef for g in s["grads"]]}
