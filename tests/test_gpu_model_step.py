"""The operators of a training step together: a block of a transformer with layer norm, norm and rotation of
heads, dropout and a policy's or a preference's loss, on virtual ranks whose gradients the ring adds up, against
the same step in 64 bits by torch."""
import math

import pytest
import torch

import ring_allreduce_virtual_gb300 as vr
from ring_allreduce_virtual_gb300 import training
from test_gpu_dropout import numbers

pytestmark = pytest.mark.gpu

B, S, HQ, HK, D, V = 2, 16, 4, 2, 16, 97
W = HQ * D
DROP, SEED = 0.2, 1234


def parameters():
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    return {"g": 1 + r(W, std=0.1), "b": r(W, std=0.1), "qkv": r(W, (HQ + 2 * HK) * D, std=W ** -0.5),
            "nq": 1 + r(D, std=0.1), "nk": 1 + r(D, std=0.1), "o": r(W, W, std=W ** -0.5), "head": r(W, V, std=2 * W ** -0.5)}


def attention(q, k, v):
    k, v = (t.repeat_interleave(HQ // HK, 2) for t in (k, v))
    a = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    a = a.masked_fill(torch.ones(S, S, device="cuda", dtype=torch.bool).triu(1), -math.inf).softmax(-1)
    return torch.einsum("bhij,bjhd->bihd", a, v).flatten(2)


def tables():
    angle = torch.arange(S, device="cuda")[:, None] * 100.0 ** (-torch.arange(D // 2, device="cuda") / (D / 2))
    return angle.cos(), angle.sin()


def logits(p, x, offset):
    """This library's operators."""
    h = training.layer_norm(x, p["g"], p["b"])
    qkv = (h @ p["qkv"]).view(B, S, HQ + 2 * HK, D)
    q, k = training.qk_norm_rope(qkv[:, :, :HQ], qkv[:, :, HQ: HQ + HK], p["nq"], p["nk"], *tables(),
                                 torch.arange(S, device="cuda"))
    a = attention(q, k, qkv[:, :, HQ + HK:])
    return training.dropout(a @ p["o"], DROP, SEED, offset, residual=x) @ p["head"]


def logits64(p, x):
    """The same in plain torch over the whole batch."""
    c = x - x.mean(-1, keepdim=True)
    h = c * (c.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * p["g"] + p["b"]
    qkv = (h @ p["qkv"]).view(-1, S, HQ + 2 * HK, D)
    cos, sin = (t.double()[:, None] for t in tables())

    def turned(t, w):
        t = t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = t[..., : D // 2], t[..., D // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    a = attention(turned(qkv[:, :, :HQ], p["nq"]), turned(qkv[:, :, HQ: HQ + HK], p["nk"]), qkv[:, :, HQ + HK:])
    keep = numbers(x.numel(), SEED, 0, "cuda").view(x.shape) >= round(DROP * 2 ** 32)
    return (x + (a @ p["o"]) * keep / (1 - DROP)) @ p["head"]


def batch(ranks):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(ranks * B, S, W, generator=g, device="cuda")
    t = torch.randint(V, (ranks * B, S), generator=g, device="cuda")
    t[:, :3] = -100
    return x, t, g


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_ranks_step_like_one_in_64_bits(kind):
    ranks = 3
    x, t, g = batch(ranks)
    start = parameters()
    p64 = {n: v.double().requires_grad_() for n, v in start.items()}
    z = logits64(p64, x.double())
    lp = torch.log_softmax(z, -1).gather(-1, t.clamp(min=0)[..., None])[..., 0]
    used = t >= 0
    count = int(used.sum())
    if kind == "policy":
        old = (lp + 0.1 * torch.randn(t.shape, generator=g, device="cuda")).detach().float()
        adv = torch.randn(t.shape, generator=g, device="cuda")
        ratio = (lp - old.double()).exp()
        want = (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) * used).sum() / count
    else:
        refs = torch.randn(ranks, 2, B // 2, generator=g, device="cuda") * 3 - 60
        sums = (lp * used).sum(1).view(ranks, 2, -1) - refs.double()
        want = torch.nn.functional.softplus(-0.1 * (sums[:, 0] - sums[:, 1])).sum() / ranks
    want.backward()
    buckets, losses = [], []
    for r in range(ranks):
        part = slice(r * B, (r + 1) * B)
        p = {n: v.clone().requires_grad_() for n, v in start.items()}
        z = logits(p, x[part], r * B * S * W)
        if kind == "policy":
            loss, _, dz = training.policy_loss_gradient(z.detach(), t[part], old[part], adv[part], used[part].float(),
                                                        scale=1 / count)
        else:
            loss, _, dz = training.preference_loss_gradient(z.detach(), t[part], refs[r], scale=1 / ranks)
        z.backward(dz)
        losses.append(loss)
        buckets.append(torch.cat([v.grad.flatten() for v in p.values()]))
    with vr.Communicator(ranks, 2, "simple", 64 << 10) as comm:
        comm.all_reduce(buckets, buckets, "sum")
    norm = training.clip_grad_norm([buckets[0]], 0.5)
    grad = torch.cat([v.grad.flatten() for v in p64.values()])
    # products of up to 100 terms in 32 bits, five of them in a row: 1e-4 of the norm is ample
    assert abs(float(torch.stack(losses).double().sum() - want.detach())) <= 1e-4 * max(1.0, abs(float(want.detach())))
    assert abs(float(norm) - float(grad.norm())) <= 1e-4 * float(grad.norm())
    expect = grad * min(1.0, 0.5 / float(grad.norm()))
    assert (buckets[0].double() - expect).norm() <= 1e-4 * expect.norm()
    for b in buckets[1:]:
        assert torch.equal(b, buckets[1])


def test_differentiable_losses_give_the_same_step():
    x, t, g = batch(1)
    for kind in ("policy", "preference"):
        grads = []
        for direct in (False, True):
            p = {n: v.clone().requires_grad_() for n, v in parameters().items()}
            z = logits(p, x, 0)
            old, adv = torch.full(t.shape, -4.0, device="cuda"), torch.ones(t.shape, device="cuda")
            if direct:
                d = training.policy_loss_gradient(z.detach(), t, old, adv)[2] if kind == "policy" else \
                    training.preference_loss_gradient(z.detach(), t)[2]
                z.backward(d)
            else:
                loss = training.policy_loss(z, t, old, adv)[0] if kind == "policy" else training.preference_loss(z, t)[0]
                loss.backward()
            grads.append(torch.cat([v.grad.flatten() for v in p.values()]))
        assert (grads[0] - grads[1]).norm() <= 1e-5 * grads[0].norm()


def test_captured_step_draws_anew():
    # a forward and backward pass captured into a CUDA graph, drawing anew at each replay
    x, t, _ = batch(1)
    seed = torch.tensor([5], device="cuda")
    w = parameters()["head"].requires_grad_()
    old, adv = torch.full(t.shape, -4.0, device="cuda"), torch.ones(t.shape, device="cuda")

    def step(w, seed):
        y = training.dropout(x, DROP, seed) @ w
        loss, _, d = training.policy_loss_gradient(y.detach(), t, old, adv)
        return loss, torch.autograd.grad(y, w, d)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(w, seed)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, dw = step(w, seed)
        seed += 1
    seed.fill_(20)
    for i in range(3):
        graph.replay()
        want = step(w, 20 + i)
        assert torch.equal(loss, want[0]) and (dw - want[1]).norm() <= 1e-6 * want[1].norm()
