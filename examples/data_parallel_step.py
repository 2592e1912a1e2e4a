"""A data-parallel training loop on virtual ranks, with this library's layer
norm, AllReduce and gradient clipping: every rank has a replica of a small
model and its own part of the batch, its gradients are views of one flat bucket,
the buckets are summed by the ring, and the sum is averaged and clipped on the
way into the update.

    python examples/data_parallel_step.py [--ranks 4] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_virtual_gb300 as vr  # noqa: E402
from ring_allreduce_virtual_gb300 import training  # noqa: E402


class Replica:
    """y = LN(x) W1 -> relu -> LN -> W2, parameters and gradients in flat buckets."""

    def __init__(self, width, seed=0):
        shapes = {"g1": (width,), "b1": (width,), "w1": (width, 2 * width), "g2": (2 * width,),
                  "b2": (2 * width,), "w2": (2 * width, width)}
        n = sum(torch.Size(s).numel() for s in shapes.values())
        self.bucket = torch.zeros(n, device="cuda")
        self.params, at = {}, 0
        gen = torch.Generator("cuda").manual_seed(seed)
        for name, shape in shapes.items():
            p = torch.ones(shape, device="cuda") if name[0] == "g" else torch.zeros(shape, device="cuda")
            if name[0] == "w":
                p = torch.randn(shape, generator=gen, device="cuda") * shape[0] ** -0.5
            p.requires_grad_()
            p.grad = self.bucket[at: at + p.numel()].view(shape)
            at += p.numel()
            self.params[name] = p
        self.grads = training.TensorList([p.grad for p in self.params.values()])

    def loss(self, x, target):
        p = self.params
        h = torch.relu(training.layer_norm(x, p["g1"], p["b1"]) @ p["w1"])
        return (training.layer_norm(h, p["g2"], p["b2"]) @ p["w2"] - target).square().mean()


def train(ranks, steps, width=96, rows=32, lr=0.5, max_norm=0.5):
    """The ranks' mean losses and the gradient norms, step by step, and the replicas."""
    gen = torch.Generator("cuda").manual_seed(1)
    xs = [torch.randn(rows, width, generator=gen, device="cuda") for _ in range(ranks)]
    teacher = torch.randn(width, width, generator=gen, device="cuda") * width ** -0.5
    replicas = [Replica(width) for _ in range(ranks)]
    losses, norms = [], []
    with vr.Communicator(ranks, 4, "simple", 64 << 10) as comm:
        for _ in range(steps):
            for r in replicas:
                r.bucket.zero_()
            step = [r.loss(x, x @ teacher) for r, x in zip(replicas, xs)]
            for loss in step:
                loss.backward()  # into the bucket
            buckets = [r.bucket for r in replicas]
            comm.all_reduce(buckets, buckets, "sum")
            for r in replicas:  # every rank averages, clips and updates its replica
                norm = training.clip_grad_norm(r.grads, max_norm, scale=1 / ranks)
                with torch.no_grad():
                    for p in r.params.values():
                        p.sub_(p.grad, alpha=lr)
            losses.append(torch.stack(step).detach().mean())
            norms.append(norm)
    return [x.item() for x in losses], [x.item() for x in norms], replicas


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    for i, (loss, norm) in enumerate(zip(*train(args.ranks, args.steps)[:2])):
        print(f"step {i:3d}  loss {loss:.5f}  gradient norm {norm:.5f}")
