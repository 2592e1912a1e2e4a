"""The data-parallel example: layer norm, AllReduce, norm and clipping as a
training loop uses them together."""
import importlib.util
import os

import pytest
import torch

from ring_allreduce_virtual_gb300 import training

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "data_parallel_step", os.path.join(ROOT, "examples", "data_parallel_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_tensors_that_are_written_count_as_changed():
    x = torch.randn(4, 64, device="cuda")
    y, dx, bucket = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(128, device="cuda")

    def changes(t, f, *args, **kw):
        v = t._version
        r = f(*args, **kw)
        assert t._version > v
        return r

    _, mean, rstd = changes(y, training.layer_norm_forward, x, out=y)
    changes(dx, training.layer_norm_backward, x, x, mean, rstd, None, dx, False, False)
    changes(bucket, training.layer_norm_backward, x, x, mean, rstd, None, False, bucket[:64], bucket[64:])
    for parts in (torch.split(bucket, 50), [x]):
        for grads in (parts, training.TensorList(parts)):
            changes(parts[0], training.clip_grad_norm, grads, 1.0)
            changes(parts[0], training.clip_grad_norm, [t.clone() for t in parts], 1.0, outs=grads)
            kept = [t.clone() for t in parts]
            outs = training.TensorList(kept)
            for _ in range(2):
                changes(kept[-1], training.clip_grad_norm, grads, 1.0, outs=outs)
    v = x._version
    training.grad_norm([x])
    training.layer_norm_backward(x, x, mean, rstd)
    assert x._version == v


@pytest.mark.parametrize("write", [
    lambda h: training.layer_norm_forward(h.detach(), out=h.detach()),
    lambda h: training.clip_grad_norm([h.detach()], 0.1),
])
def test_autograd_refuses_saved_tensors_that_were_written(write):
    w = torch.rand(8, 8, device="cuda", requires_grad=True)
    h = torch.rand(4, 8, device="cuda")
    y = (h @ w).sum()  # saves h
    write(h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_ranks_stay_equal_and_learn():
    losses, norms, replicas = example().train(4, 12)
    assert losses[-1] < 0.7 * losses[0]
    for r in replicas[1:]:
        for name, p in r.params.items():
            assert torch.equal(p, replicas[0].params[name]), name


def test_first_step_is_the_whole_batch_gradient():
    # One step on 3 ranks against torch autograd in 64 bits on the joined batch
    m = example()
    ranks, width, rows, lr, most = 3, 40, 16, 0.25, 0.3
    _, norms, replicas = m.train(ranks, 1, width, rows, lr, most)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.cat([torch.randn(rows, width, generator=gen, device="cuda") for _ in range(ranks)]).double()
    teacher = (torch.randn(width, width, generator=gen, device="cuda") * width ** -0.5).double()
    start = m.Replica(width)
    p = {n: t.detach().double().requires_grad_() for n, t in start.params.items()}

    def norm(h, g, b):
        c = h - h.mean(1, keepdim=True)
        return c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g + b

    h = torch.relu(norm(x, p["g1"], p["b1"]) @ p["w1"])
    (norm(h, p["g2"], p["b2"]) @ p["w2"] - x @ teacher).square().mean().backward()
    want = torch.cat([t.grad.reshape(-1) for t in p.values()])
    total = want.norm()
    # 32-bit products of up to 80 terms in two layers: 1e-4 of the norm is ample
    assert abs(norms[0] - total.item()) <= 1e-4 * total.item()
    moved = torch.cat([(start.params[n] - replicas[0].params[n]).double().reshape(-1) for n in p])
    step = want * lr * min(1.0, most / total.item())
    assert (moved - step.reshape(-1)).norm() <= 1e-4 * step.norm() + 1e-6
