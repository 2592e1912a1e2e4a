"""More operators of a data-parallel training step: dropout whose mask is counted out and never stored, the norm of each
query and key head with its rotation, and the losses of policies and preferences with their gradients. Cases, inputs,
plain forms in torch, and the same in 64 bits."""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-6
CLIP = (0.2, 0.28)  # how far a policy's ratio may fall below and rise above 1
KL = 0.04
BETA = 0.1


def listed():
    return [
        # The hidden layer of a fine-tuned adapter over 64 tokens: latency is all that counts.
        {"name": "drop_fwd 64x512 f32", "op": "drop_fwd", "rows": 64, "cols": 512, "dtype": "float32", "residual": False, "p": 0.1, "offset": 0},
        # A layer's output dropped and added to the residual stream, a micro-batch of 16384 tokens, the second of two ranks.
        {"name": "drop_fwd 16384x8192 bf16 add", "op": "drop_fwd", "rows": 16384, "cols": 8192, "dtype": "bfloat16", "residual": True, "p": 0.1, "offset": 16384 * 8192},
        # Packed tokens of an odd width, the part of a batch that starts at an odd element.
        {"name": "drop_bwd 9973x2051 f16", "op": "drop_bwd", "rows": 9973, "cols": 2051, "dtype": "float16", "p": 0.25, "offset": 9973 * 2051 * 3},
        # One decoding step of 8 sequences at far positions.
        {"name": "qk_fwd 8x1 32+8x128 bf16", "op": "qk_fwd", "batch": 8, "tokens": 1, "q": 32, "k": 8, "dim": 128, "rot": 128, "dtype": "bfloat16", "wtype": "bfloat16", "layout": "packed", "inter": False},
        # A micro-batch of 4 sequences of 4096 tokens, heads shared by groups of queries.
        {"name": "qk_fwd 4x4096 64+8x128 bf16", "op": "qk_fwd", "batch": 4, "tokens": 4096, "q": 64, "k": 8, "dim": 128, "rot": 128, "dtype": "bfloat16", "wtype": "float32", "layout": "packed", "inter": False},
        # Heads stored before tokens, odd lengths, a part of each head rotated, neighbours paired.
        {"name": "qk_bwd 3x1371 16+16x80 f16", "op": "qk_bwd", "batch": 3, "tokens": 1371, "q": 16, "k": 16, "dim": 80, "rot": 32, "dtype": "float16", "wtype": "float16", "layout": "heads", "inter": True},
        # The backward pass of the micro-batch.
        {"name": "qk_bwd 4x4096 32+8x128 bf16", "op": "qk_bwd", "batch": 4, "tokens": 4096, "q": 32, "k": 8, "dim": 128, "rot": 128, "dtype": "bfloat16", "wtype": "float32", "layout": "packed", "inter": False},
        # What the policy that sampled 4096 tokens, or the reference policy, gives them: no gradient.
        {"name": "logp 4096x131072 bf16", "op": "logp", "rows": 4096, "vocab": 131072, "dtype": "bfloat16"},
        # A short answer's policy step.
        {"name": "policy 200x32000 bf16", "op": "policy", "rows": 200, "vocab": 32000, "dtype": "bfloat16", "ref": False},
        # A micro-batch of answers, half of the tokens prompts and padding, a vocabulary that no vector load divides.
        {"name": "policy 8192x50001 bf16", "op": "policy", "rows": 8192, "vocab": 50001, "dtype": "bfloat16", "ref": True},
        # Two pairs of short answers in 32 bits, of lengths of their own, packed.
        {"name": "pref 2x100 32000 f32", "op": "pref", "pairs": 2, "length": 100, "packed": True, "vocab": 32000, "dtype": "float32"},
        # Four pairs of padded answers over a large vocabulary.
        {"name": "pref 4x512 131072 bf16", "op": "pref", "pairs": 4, "length": 512, "packed": False, "vocab": 131072, "dtype": "bfloat16"},
    ]


def spread(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm; about half are multiples of 8."""
    n = round(math.exp(rng.uniform(math.log(low), math.log(high))))
    return max(low, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("drop_fwd", "drop_bwd", "qk_fwd", "qk_bwd", "logp", "policy", "pref"))
    largest = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    dtype = rng.choice(tuple(DTYPES))
    while True:
        if op.startswith("drop"):
            case = {"op": op, "rows": spread(rng, 1, 65536), "cols": spread(rng, 64, 16384), "dtype": dtype,
                    "p": rng.choice((0.0, 0.05, 0.1, 0.3, 0.5)), "offset": rng.choice((0, rng.randrange(1 << 20), rng.randrange(1 << 40)))}
            case |= {"residual": rng.random() < 0.5} if op == "drop_fwd" else {}
        elif op.startswith("qk"):
            dim = rng.choice((32, 64, 80, 96, 128, 192, 256))
            k = rng.choice((1, 2, 4, 8, 16))
            case = {"op": op, "batch": spread(rng, 1, 16), "tokens": spread(rng, 1, 8192), "q": k * rng.choice((1, 2, 4, 5, 8)), "k": k, "dim": dim,
                    "rot": rng.choice((dim, dim, dim // 2, dim // 4)) // 2 * 2, "dtype": dtype, "wtype": rng.choice((dtype, "float32")),
                    "layout": rng.choice(("packed", "heads")), "inter": rng.random() < 0.3}
        elif op == "pref":
            case = {"op": op, "pairs": spread(rng, 1, 16), "length": spread(rng, 8, 1024), "packed": rng.random() < 0.5, "vocab": spread(rng, 1000, 160000), "dtype": dtype}
        else:
            case = {"op": op, "rows": spread(rng, 1, 16384), "vocab": spread(rng, 1000, 160000), "dtype": dtype}
            case |= {"ref": rng.random() < 0.5} if op == "policy" else {}
        if work(case)["bytes"] <= largest:
            return case


def lengths(case):
    """The rows of each sequence of a preference batch: chosen answers, then rejected ones. Packed sequences are of odd
    lengths down to a third of the longest."""
    n = 2 * case["pairs"]
    return [case["length"] - (case["length"] * 2 * (i * 7 % n) // (3 * n) if case["packed"] else 0) for i in range(n)]


def work(case):
    op, e = case["op"], DTYPES[case["dtype"]].itemsize
    if op.startswith("drop"):
        n = case["rows"] * case["cols"]
        return {"bytes": (3 if case.get("residual") else 2) * n * e, "flops": 2 * n}
    if op.startswith("qk"):
        tokens = case["batch"] * case["tokens"]
        n = tokens * (case["q"] + case["k"]) * case["dim"]
        w = 2 * case["dim"] * DTYPES[case["wtype"]].itemsize
        table = tokens * (case["rot"] * 4 + 8)  # a row of each table and a position
        if op == "qk_fwd":
            return {"bytes": 2 * n * e + w + table, "flops": 8 * n}
        return {"bytes": 3 * n * e + 2 * w + table, "flops": 16 * n}
    rows = sum(lengths(case)) if op == "pref" else case["rows"]
    n = rows * case["vocab"]
    if op == "logp":
        return {"bytes": n * e + 16 * rows, "flops": 4 * n}
    return {"bytes": 2 * n * e + (28 if op == "policy" else 8) * rows, "flops": 7 * n}


def randn(g, shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op.startswith("drop"):
        shape = (case["rows"], case["cols"])
        s = dict(case, x=randn(g, shape).to(dt), seed=seed * 0x9E3779B97F4A7C15 % (1 << 63), res=None)
        if case.get("residual"):
            s["res"] = randn(g, shape, 2.0).to(dt)
        return s
    if op.startswith("qk"):
        return prepare_qk(case, g)
    rows = sum(lengths(case)) if op == "pref" else case["rows"]
    vocab = case["vocab"]
    logits = torch.empty(rows, vocab, dtype=dt, device="cuda")
    for i in range(0, rows, 1024):
        logits[i: i + 1024] = randn(g, logits[i: i + 1024].shape, 2.5)
    targets = torch.randint(vocab, (rows,), generator=g, device="cuda")
    # what was sampled is among the likely ones
    likely = torch.rand(rows, generator=g, device="cuda") * 12 + 4
    logits[torch.arange(rows, device="cuda"), targets] = likely.to(dt)
    s = dict(case, logits=logits, targets=targets)
    if op == "logp":
        return s
    answer = torch.rand(rows, generator=g, device="cuda") < 0.5  # the others are the prompts'
    logp = log_probs(s)[0]
    if op == "policy":
        # the sampling policy is some updates behind, the reference policy further
        s["old"] = logp + randn(g, (rows,), 0.15)
        s["ref"] = logp + randn(g, (rows,), 0.4) if case["ref"] else None
        s["advantages"] = randn(g, (rows,))
        s["weights"] = answer / answer.sum().clamp(min=1)
        return s
    targets[~answer] = -100
    each = lengths(case)
    s["starts"] = torch.tensor([0] + each, device="cuda").cumsum(0) if case["packed"] else None
    sums = torch.stack([p.sum() for p in torch.split(torch.where(answer, logp, 0), each)])
    s["refs"] = (sums + randn(g, sums.shape, 8.0)).reshape(2, -1)
    if not case["packed"]:
        s["logits"], s["targets"] = logits.view(2 * case["pairs"], -1, vocab), targets.view(2 * case["pairs"], -1)
    return s


def prepare_qk(case, g):
    dt, wt = DTYPES[case["dtype"]], DTYPES[case["wtype"]]
    batch, tokens, nq, nk, dim, rot = (case[n] for n in ("batch", "tokens", "q", "k", "dim", "rot"))
    far = 131072 if tokens == 1 else tokens + 4096
    angles = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    first = torch.randint(far - tokens + 1, (batch, 1), generator=g, device="cuda")
    s = dict(case, cos=angles.cos().float(), sin=angles.sin().float(), pos=first + torch.arange(tokens, device="cuda"),
             wq=randn(g, (dim,), 0.1, 1.0).to(wt), wk=randn(g, (dim,), 0.1, 1.0).to(wt))

    def heads(std, mix):
        if case["layout"] == "heads":  # (batch, heads, tokens, dim) in memory
            q, k = ((randn(g, (batch, n, tokens, dim), std) * mix).to(dt).transpose(1, 2) for n in (nq, nk))
            return q, k
        qkv = randn(g, (batch, tokens, nq + 2 * nk, dim), std).mul_(mix).to(dt)  # the projection's output, values among it
        return qkv[:, :, :nq], qkv[:, :, nq: nq + nk]
    s["qh"], s["kh"] = heads(1.5, randn(g, (dim,), 0.3, 1.0))
    if case["op"] == "qk_bwd":
        s["dq"], s["dk"] = heads(0.02, 1.0)
    return s


# ------------------------------------------------------------ plain forms
LOW = 0xFFFFFFFF


def counter_block(n, stream, seed):
    """Philox4x32-10 (Salmon and others 2011) of the counters (n, stream, 0), n of 64 bits: four words of 32."""
    c = [n & LOW, n >> 32 & LOW, torch.full_like(n, stream), torch.zeros_like(n)]
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64 bits, the sign is one of them
        c = [(b >> 32 & LOW) ^ c[1] ^ k0, b & LOW, (a >> 32 & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return c


def kept(count, p, seed, offset):
    """Which of the elements offset, ..., offset + count - 1 stay: those whose random number of 32 bits is at least p 2^32.
    Its upper and lower half are halfword n mod 8 of block n div 8 of the streams 0 and 1."""
    first = offset // 8
    n = torch.arange(first, (offset + count + 7) // 8, device="cuda")
    halves = []
    for stream in (0, 1):
        words = torch.stack(counter_block(n, stream, seed), 1)
        halves.append(torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[offset - 8 * first:][:count])
    return (halves[0] << 16 | halves[1]) >= round(p * 2.0 ** 32)


def dropped(s):
    x = s["x"]
    keep = kept(x.numel(), s["p"], s["seed"], s["offset"]).view(x.shape)
    y = torch.where(keep, x.float() * (1 / (1 - s["p"])), 0.0)
    return (y if s["res"] is None else y + s["res"].float()).to(x.dtype)


def rotate(x, c, s, inter, back=False):
    """The first elements of each head rotated, pairs of neighbours or of both halves; back: by the opposite angle."""
    n = 2 * c.shape[-1]
    c, s = c[:, :, None], -s[:, :, None] if back else s[:, :, None]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if inter else (x[..., : n // 2], x[..., n // 2: n])
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((y, x[..., n:]), -1)


def qk_forward(x, w, c, s, inter):
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w.float()
    return rotate(y, c, s, inter).to(x.dtype)


def qk_backward(dy, x, w, c, s, inter):
    f, g = x.float(), rotate(dy.float(), c, s, inter, back=True)
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    u, gw = f * r, g * w.float()
    dx = r * (gw - u * (gw * u).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * u).sum((0, 1, 2)).to(w.dtype)


def log_probs(s):
    """(log probability of each target, log of the sum of the row's exponentials, both of 64 bits; the row in 32 bits less
    its largest, the sum of its exponentials), by parts of the rows."""
    logits, targets = s["logits"].flatten(0, -2), s["targets"].flatten()
    lse, at = [], []
    for x, t in zip(logits.split(2048), targets.split(2048)):
        x = x.float()
        m = x.amax(1, keepdim=True)
        lse.append(m[:, 0].double() + (x - m).exp().sum(1).double().log())
        at.append(x.gather(1, t.clamp(min=0)[:, None])[:, 0])
    lse = torch.cat(lse)
    return torch.where(targets < 0, 0.0, torch.cat(at).double() - lse).float(), lse


def logit_gradient(s, lse, coef):
    """coef (one at the target - softmax), rows of coef 0 are 0."""
    logits, targets = s["logits"].flatten(0, -2), s["targets"].flatten()
    d = torch.empty_like(logits)
    for i in range(0, len(logits), 2048):
        x, t, c = logits[i: i + 2048].float(), targets[i: i + 2048], coef[i: i + 2048].float()[:, None]
        g = -c * (x - lse[i: i + 2048, None].float()).exp()
        g.scatter_add_(1, t.clamp(min=0)[:, None], c)
        d[i: i + 2048] = torch.where(c != 0, g, 0.0).to(d.dtype)
    return d.view(s["logits"].shape)


def policy(s):
    logits, targets = s["logits"], s["targets"]
    at = torch.gather(logits, 1, targets[:, None])[:, 0].double()
    lse = log_probs(s)[1]
    lp, w, a = at - lse, s["weights"].double(), s["advantages"].double()  # next to the clipping's border 32 bits may decide otherwise
    ratio = (lp - s["old"].double()).exp()
    inside = ratio.clamp(1 - CLIP[0], 1 + CLIP[1])
    loss = -torch.minimum(ratio * a, inside * a)
    coef = torch.where(ratio * a <= inside * a, -ratio * a, 0.0)
    if s["ref"] is not None:
        r = s["ref"].double() - lp
        loss = loss + KL * (r.exp() - r - 1)
        coef = coef + KL * (1 - r.exp())
    used = w != 0
    loss = torch.where(used, w * loss, 0.0).sum().float()
    return {"loss": loss, "logp": torch.where(used, lp, 0.0).float(), "dlogits": logit_gradient(s, lse, torch.where(used, w * coef, 0.0))}


def preference(s):
    logp, lse = log_probs(s)
    each = lengths(s)
    sums = torch.stack([p.double().sum() for p in torch.split(logp, each)]).view(2, -1)
    h = BETA * ((sums[0] - s["refs"][0].double()) - (sums[1] - s["refs"][1].double()))
    scale = 1 / s["pairs"]
    loss = (torch.exp(-h.abs()).log1p() + torch.clamp(-h, min=0)).sum() * scale
    c = -scale * BETA / (1 + h.exp())
    coef = torch.repeat_interleave(torch.cat((c, -c)), torch.tensor(each, device="cuda"))
    coef = torch.where(s["targets"].flatten() < 0, 0.0, coef)
    return {"loss": loss.float(), "logps": sums.float(), "dlogits": logit_gradient(s, lse, coef)}


def run(s):
    op = s["op"]
    if own:
        from ring_allreduce_virtual_gb300 import training
        if op == "drop_fwd":
            return training.dropout_forward(s["x"], s["p"], s["seed"], s["offset"], s["res"])
        if op == "drop_bwd":
            return training.dropout_backward(s["x"], s["p"], s["seed"], s["offset"])
        if op == "qk_fwd":
            q, k = training.qk_norm_rope_forward(s["qh"], s["kh"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS, s["inter"])
            return {"q": q, "k": k}
        if op == "qk_bwd":
            dq, dk, dwq, dwk = training.qk_norm_rope_backward(s["dq"], s["dk"], s["qh"], s["kh"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS, s["inter"])
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if op == "logp":
            logp, lse = training.token_logprobs_forward(s["logits"], s["targets"])
            return {"logp": logp, "lse": lse}
        if op == "policy":
            loss, logp, dlogits = training.policy_loss_gradient(s["logits"], s["targets"], s["old"], s["advantages"], s["weights"], s["ref"], *CLIP, KL)
            return {"loss": loss, "logp": logp, "dlogits": dlogits}
        loss, logps, dlogits = training.preference_loss_gradient(s["logits"], s["targets"], s["refs"], s["starts"], BETA, scale=1 / s["pairs"])
        return {"loss": loss, "logps": logps, "dlogits": dlogits}
    if op.startswith("drop"):
        return dropped(s)
    if op.startswith("qk"):
        c, sn = s["cos"][s["pos"]], s["sin"][s["pos"]]
        if op == "qk_fwd":
            return {n: qk_forward(s[n + "h"], s["w" + n], c, sn, s["inter"]) for n in ("q", "k")}
        (dq, dwq), (dk, dwk) = (qk_backward(s["d" + n], s[n + "h"], s["w" + n], c, sn, s["inter"]) for n in ("q", "k"))
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "logp":
        logp, lse = log_probs(s)
        return {"logp": logp, "lse": lse.float()}
    return policy(s) if op == "policy" else preference(s)


# ------------------------------------------------------------- in 64 bits
def exact_keep(s, count):
    """The rule of `kept` with the products taken apart into halves of 16 bits, part by part of the elements."""
    def multiply(m, v):  # upper and lower 32 bits
        m1, m0, v1, v0 = m >> 16, m & 65535, v >> 16, v & 65535
        low, mid1, mid2 = m0 * v0, m1 * v0, m0 * v1
        mid = (low >> 16) + (mid1 & 65535) + (mid2 & 65535)
        return m1 * v1 + (mid1 >> 16) + (mid2 >> 16) + (mid >> 16), (mid & 65535) << 16 | low & 65535

    threshold = round(s["p"] * 4294967296)
    keep = torch.empty(count, dtype=torch.bool, device="cuda")
    for i in range(0, count, 1 << 24):
        n = s["offset"] + i + torch.arange(min(1 << 24, count - i), device="cuda")
        block, place = n // 8, n % 8
        number = torch.zeros_like(n)
        for stream in (0, 1):
            x = (block % 4294967296, block // 4294967296, torch.full_like(n, stream), torch.zeros_like(n))
            for turn in range(10):
                ka, kb = ((s["seed"] >> b) % 4294967296 + turn * c & 4294967295 for b, c in ((0, 0x9E3779B9), (32, 0xBB67AE85)))
                (h0, l0), (h1, l1) = multiply(0xD2511F53, x[0]), multiply(0xCD9E8D57, x[2])
                x = (h1 ^ x[1] ^ ka, l1, h0 ^ x[3] ^ kb, l0)
            word = torch.where(place < 2, x[0], torch.where(place < 4, x[1], torch.where(place < 6, x[2], x[3])))
            number = number * 65536 + torch.where(place % 2 == 0, word % 65536, word // 65536)
        keep[i: i + len(n)] = number >= threshold
    return keep


def exact(case, seed):
    """The definitions, in 64 bits."""
    global own
    was, own = own, False  # the inputs alone
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op.startswith("drop"):
        y = s["x"].double() / (1 - case["p"]) * exact_keep(s, s["x"].numel()).view(s["x"].shape)
        return y if s["res"] is None else y + s["res"].double()
    if op.startswith("qk"):
        return exact_qk(s)
    logits, targets = s["logits"].flatten(0, -2), s["targets"].flatten()
    rows = torch.arange(len(logits), device="cuda")
    logp = torch.cat([torch.log_softmax(x.double(), 1)[rows[: len(x)], t.clamp(min=0)] for x, t in zip(logits.split(1024), targets.split(1024))])
    if op == "logp":
        return {"logp": logp, "lse": torch.cat([torch.logsumexp(x.double(), 1) for x in logits.split(1024)])}
    lp = logp.clone().requires_grad_()
    if op == "policy":
        mask = s["weights"] > 0
        change = (lp - s["old"].double()).exp()
        a = s["advantages"].double()
        gain = torch.where(a >= 0, a * change.clamp(max=1 + CLIP[1]), a * change.clamp(min=1 - CLIP[0]))
        each = -gain
        if s["ref"] is not None:
            apart = lp - s["ref"].double()
            each = each + KL * (torch.expm1(-apart) + apart)
        loss = (each[mask] * s["weights"].double()[mask]).sum()
        out = {"loss": loss.detach(), "logp": logp * mask}
    else:
        mask = targets >= 0
        owner = torch.repeat_interleave(torch.arange(2 * case["pairs"], device="cuda"), torch.tensor(lengths(case), device="cuda"))
        sums = torch.zeros(2 * case["pairs"], dtype=torch.float64, device="cuda").index_add(0, owner, lp * mask)
        margin = (sums - s["refs"].double().flatten()).view(2, -1)
        loss = -torch.nn.functional.logsigmoid(BETA * (margin[0] - margin[1])).sum() / case["pairs"]
        out = {"loss": loss.detach(), "logps": sums.detach().view(2, -1)}
    loss.backward()
    coef = torch.where(mask, lp.grad, 0.0)
    d = torch.empty(logits.shape, dtype=torch.float64, device="cuda")
    for i in range(0, len(logits), 1024):
        c = coef[i: i + 1024, None]
        d[i: i + 1024] = -c * torch.softmax(logits[i: i + 1024].double(), 1)
    d[rows, targets.clamp(min=0)] += coef
    return out | {"dlogits": d.view(s["logits"].shape)}


def exact_qk(s):
    """Each pair of elements as a complex number, turned by its angle; the gradients by automatic differentiation."""
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"]].unsqueeze(2)
    half = turn.shape[-1]
    out = {}
    for n in ("q", "k"):
        x, w = s[n + "h"].double().requires_grad_(), s["w" + n].double().requires_grad_()
        u = w * x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        pairs = u[..., : 2 * half].unflatten(-1, (half, 2) if s["inter"] else (2, half))
        if not s["inter"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y = torch.cat(((z if s["inter"] else z.transpose(-1, -2)).flatten(-2), u[..., 2 * half:]), -1)
        if s["op"] == "qk_fwd":
            out[n] = y.detach()
        else:
            out["d" + n], out["dw" + n] = torch.autograd.grad(y, (x, w), s["d" + n].double())
    return out if s["op"] == "qk_fwd" else {n: out[n] for n in ("dq", "dk", "dwq", "dwk")}
