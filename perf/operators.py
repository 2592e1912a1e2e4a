"""The operators of a data-parallel training step around the gradient AllReduce: layer norm forward and backward, the
norm of a list of gradients, and clipping by that norm. Cases, inputs, plain forms in torch, and the same in 64 bits."""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-5


def listed():
    return [
        # One decoding step of 8 sequences: no statistics are kept; latency is all that counts.
        {"name": "ln_fwd 8x4096 bf16", "op": "ln_fwd", "rows": 8, "cols": 4096, "dtype": "bfloat16", "wtype": "bfloat16", "stats": False},
        # A training micro-batch of 4 sequences of 4096 tokens, parameters kept in 32 bits.
        {"name": "ln_fwd 16384x4096 bf16", "op": "ln_fwd", "rows": 16384, "cols": 4096, "dtype": "bfloat16", "wtype": "float32", "stats": True},
        # Packed sequences of a narrow model whose width no vector load divides.
        {"name": "ln_fwd 30011x1001 f16", "op": "ln_fwd", "rows": 30011, "cols": 1001, "dtype": "float16", "wtype": "float16", "stats": True},
        # A short fine-tuning batch in 32 bits.
        {"name": "ln_bwd 200x1280 f32", "op": "ln_bwd", "rows": 200, "cols": 1280, "dtype": "float32", "wtype": "float32"},
        # The widest layer's backward pass over a whole micro-batch.
        {"name": "ln_bwd 16384x8192 bf16", "op": "ln_bwd", "rows": 16384, "cols": 8192, "dtype": "bfloat16", "wtype": "float32"},
        # An odd width and an odd number of packed tokens.
        {"name": "ln_bwd 9973x2051 bf16", "op": "ln_bwd", "rows": 9973, "cols": 2051, "dtype": "bfloat16", "wtype": "bfloat16"},
        # The norms of every gradient of a small model, to log them: 288 tensors, half of them vectors.
        {"name": "norm 24x1280 bf16", "op": "norm", "layers": 24, "width": 1280, "dtype": "bfloat16", "mixed": False, "scale": 1.0},
        # Two odd layers with 32-bit vectors: many tensors, few bytes.
        {"name": "norm 2x333 f16+f32", "op": "norm", "layers": 2, "width": 333, "dtype": "float16", "mixed": True, "scale": 0.125},
        # A fine-tuned adapter's few gradients: latency.
        {"name": "clip 1x128 f32", "op": "clip", "layers": 1, "width": 128, "dtype": "float32", "mixed": False, "scale": 1.0, "max_norm": 1.0},
        # A middle-sized model, vectors in 32 bits, the sum over 8 ranks divided on the way.
        {"name": "clip 12x1999 bf16+f32", "op": "clip", "layers": 12, "width": 1999, "dtype": "bfloat16", "mixed": True, "scale": 0.125, "max_norm": 1.0},
        # 0.99 GiB of 32-bit gradients, the size of one rank's buffer in the bandwidth benchmark.
        {"name": "clip 5x2100 f32", "op": "clip", "layers": 5, "width": 2100, "dtype": "float32", "mixed": False, "scale": 1.0, "max_norm": 1.0},
    ]


def spread(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm; about half are multiples of 8."""
    n = round(math.exp(rng.uniform(math.log(low), math.log(high))))
    n = max(low, n // 8 * 8) if rng.random() < 0.5 else n
    return n + 1 if n in (768, 1024, 3072) else n


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "norm", "clip"))
    largest = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        if op.startswith("ln"):
            dtype = rng.choice(tuple(DTYPES))
            case = {"op": op, "rows": spread(rng, 1, 65536), "cols": spread(rng, 64, 16384), "dtype": dtype, "wtype": rng.choice((dtype, "float32"))}
            case |= {"stats": rng.random() < 0.7} if op == "ln_fwd" else {}
        else:
            dtype = rng.choice(tuple(DTYPES))
            case = {"op": op, "layers": spread(rng, 1, 32), "width": spread(rng, 64, 2560), "dtype": dtype,
                    "mixed": dtype != "float32" and rng.random() < 0.5, "scale": rng.choice((1.0, 0.125, 1 / 72))}
            case |= {"max_norm": rng.choice((0.1, 1.0, 1e6))} if op == "clip" else {}
        if work(case)["bytes"] <= largest:
            return case


def sizes(case):
    """The elements of a transformer's gradients, layer by layer: the matrices of the attention and of the feed-forward
    network with their biases, and two layer norms' weights and biases; and whether each is a matrix."""
    w = case["width"]
    layer = [3 * w * w, w * w, 4 * w * w, 4 * w * w, 3 * w, w, 4 * w, w, w, w, w, w]
    return layer * case["layers"], ([True] * 4 + [False] * 8) * case["layers"]


def work(case):
    if case["op"].startswith("ln"):
        n, e = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize
        p = case["cols"] * DTYPES[case["wtype"]].itemsize
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * n * e + 2 * p + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * p + 8 * case["rows"], "flops": 14 * n}
    e = DTYPES[case["dtype"]].itemsize
    each = [n * (4 if case["mixed"] and not m else e) for n, m in zip(*sizes(case))]
    n = sum(sizes(case)[0])
    return {"bytes": sum(each) + 4 * len(each) + 4, "flops": 2 * n} if case["op"] == "norm" else {"bytes": 2 * sum(each) + 4, "flops": 3 * n}


def randn(g, shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"].startswith("ln"):
        dt, wt, shape = DTYPES[case["dtype"]], DTYPES[case["wtype"]], (case["rows"], case["cols"])
        # activations: channels with offsets and scales of their own
        x = (randn(g, shape) * randn(g, shape[1:], 0.2, 1.0) + randn(g, shape[1:], 0.5)).to(dt)
        s = dict(case, x=x, w=randn(g, shape[1:], 0.1, 1.0).to(wt), b=randn(g, shape[1:], 0.1).to(wt))
        if case["op"] == "ln_bwd":  # the statistics that the forward pass left
            var, mean = torch.var_mean(x.float(), 1, correction=0)
            s |= {"dy": randn(g, shape, 0.02).to(dt), "mean": mean, "rstd": torch.rsqrt(var + EPS)}
        return s
    # gradients: views of one flat bucket for each type, as the AllReduce takes them, not padded
    ns, matrix = sizes(case)
    dt = DTYPES[case["dtype"]]
    types = [torch.float32 if case["mixed"] and not m else dt for m in matrix]
    flat = {t: randn(g, sum(n for n, u in zip(ns, types) if u == t), 0.01).to(t) for t in dict.fromkeys(types)}
    out = {t: torch.empty_like(f) for t, f in flat.items()} if case["op"] == "clip" else {}
    views = {t: iter(torch.split(f, [n for n, u in zip(ns, types) if u == t])) for t, f in flat.items()}
    s = dict(case, flat=flat, out=out, grads=[next(views[t]) for t in types])
    if own:  # the lists that a program makes once for the buffers that it keeps
        from ring_allreduce_virtual_gb300 import training
        s["grads"] = training.TensorList(s["grads"])
        views = {t: iter(torch.split(f, [n for n, u in zip(ns, types) if u == t])) for t, f in out.items()}
        s["outs"] = training.TensorList([next(views[t]) for t in types]) if out else None
    return s


def run(s):
    if own:
        from ring_allreduce_virtual_gb300 import training
        if s["op"] == "ln_fwd":
            y, mean, rstd = training.layer_norm_forward(s["x"], s["w"], s["b"], EPS, stats=s["stats"])
            return {"y": y, "mean": mean, "rstd": rstd} if s["stats"] else {"y": y}
        if s["op"] == "ln_bwd":
            dx, dw, db = training.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
            return {"dx": dx, "dw": dw, "db": db}
        if s["op"] == "norm":
            norm, norms = training.grad_norm(s["grads"], scale=s["scale"], per_tensor=True)
            return {"norm": norm, "norms": norms}
        norm = training.clip_grad_norm(s["grads"], s["max_norm"], scale=s["scale"], outs=s["outs"])
        return {"norm": norm, "grads": list(s["out"].values())}
    if s["op"] == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = torch.rsqrt(x.square().mean(1) + EPS)
        y = (x * rstd[:, None] * s["w"].float() + s["b"].float()).to(s["x"].dtype)
        return {"y": y, "mean": mean, "rstd": rstd} if s["stats"] else {"y": y}
    if s["op"] == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        dw, db = (dy * xhat).sum(0), dy.sum(0)
        g = dy * s["w"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dw": dw.to(s["w"].dtype), "db": db.to(s["w"].dtype)}
    if s["op"] == "norm":
        squares = torch.stack([g.float().square().sum() for g in s["grads"]])
        return {"norm": squares.sum().sqrt() * s["scale"], "norms": squares.sqrt() * s["scale"]}
    norm = torch.stack([f.float().square().sum() for f in s["flat"].values()]).sum().sqrt() * s["scale"]
    factor = torch.where((norm > s["max_norm"]) & torch.isfinite(norm), s["max_norm"] / norm, 1.0) * s["scale"]
    return {"norm": norm, "grads": [(f.float() * factor).to(f.dtype) for f in s["flat"].values()]}


def exact(case, seed):
    """The definitions, in 64 bits."""
    global own
    was, own = own, False  # the inputs alone
    s = prepare(case, seed)
    own = was
    if case["op"].startswith("ln"):
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        n = case["cols"]
        if case["op"] == "ln_fwd":
            mu = x.sum(1) / n
            sigma = (((x - mu.unsqueeze(1)) ** 2).sum(1) / n + EPS).sqrt()
            y = w * (x - mu.unsqueeze(1)) / sigma.unsqueeze(1) + b
            return {"y": y, "mean": mu, "rstd": 1 / sigma} if case["stats"] else {"y": y}
        # y = w u + b with u = (x - mu) r: the chain rule through u, r and mu
        mu, r, dy = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1), s["dy"].double()
        u = (x - mu) * r
        du = w * dy
        along = torch.einsum("rc,rc->r", du, u).unsqueeze(1) / n
        dx = (du - u * along - du.sum(1, keepdim=True) / n) * r
        return {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, u), "db": torch.einsum("rc->c", dy)}
    squares = [torch.dot(g.double(), g.double()) for g in s["grads"]]
    norm = torch.stack(squares).sum().sqrt() * case["scale"]
    if case["op"] == "norm":
        return {"norm": norm, "norms": torch.stack(squares).sqrt() * case["scale"]}
    coefficient = min(1.0, case["max_norm"] / float(norm))
    return {"norm": norm, "grads": [f.double() * (case["scale"] * coefficient) for f in s["flat"].values()]}
