"""One data-parallel training step with the operators and the AllReduce together.

N logical ranks train the same small student on their own micro-batches:

    h  = layer_norm(x)                       tokens of a micro-batch
    r  = expert_dispatch(h)                  sorted by expert, top-k of a router
    e  = relu(r @ W_expert)                  each expert's own rows
    y  = x + expert_combine(e, weights)      back in token order
    z  = y @ W_out                           logits over the vocabulary
    loss = distill_step(z, teacher's top logits)

and back again; every rank's gradients lie in one flat bucket, the buckets are
averaged with ``allreduce(..., op="avg")`` and every rank takes the same step.

    python examples/moe_distill.py [--ranks 4] [--steps 20]

prints the mean loss of each step and checks that the ranks' weights stay bit
for bit the same.  The matrix products are torch's; everything else on the way
is this package's.  (The router's scores are fixed inputs here, so the
gradient of the choices' weights is computed but goes no further.)
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ring_allreduce_rs_amd as ar  # noqa: E402


class Student:
    """Weights and gradients of one rank, each in one flat fp32 bucket."""

    def __init__(self, hidden, experts, vocab, seed, device="cuda"):
        self.shapes = {"norm_w": (hidden,), "norm_b": (hidden,),
                       "expert": (experts, hidden, hidden), "out": (hidden, vocab)}
        sizes = {k: torch.Size(s).numel() for k, s in self.shapes.items()}
        self.weights = torch.empty(sum(sizes.values()), device=device)
        self.grads = torch.zeros_like(self.weights)
        self.w, self.g, at = {}, {}, 0
        for k, s in self.shapes.items():
            self.w[k] = self.weights[at:at + sizes[k]].view(s)
            self.g[k] = self.grads[at:at + sizes[k]].view(s)
            at += sizes[k]
        gen = torch.Generator(device).manual_seed(seed)
        self.weights.normal_(0.0, hidden ** -0.5, generator=gen)
        self.w["norm_w"].fill_(1.0)
        self.w["norm_b"].zero_()

    def step(self, batch):
        """Forward and backward of one micro-batch into the gradient bucket; the
        loss of each token and the gradient of the choices' weights."""
        x, ids, weights, places, teacher = batch
        experts = self.shapes["expert"][0]
        h, mean, rstd = ar.layer_norm(x, self.w["norm_w"], self.w["norm_b"])
        rows, plan = ar.expert_dispatch(h, ids, experts)
        ends = plan.offsets.tolist()
        acts = torch.zeros_like(rows)
        for e in range(experts):
            s = slice(ends[e], ends[e + 1])
            acts[s] = torch.relu(rows[s] @ self.w["expert"][e].to(x.dtype))
        y = x + ar.expert_combine(acts, weights, plan)
        z = y @ self.w["out"].to(x.dtype)
        share = torch.full((x.shape[0],), 1.0 / x.shape[0], device=x.device)
        loss, dz = ar.distill_step(share, z, places, teacher, temperature=2.0)

        self.g["out"].copy_(y.t().contiguous() @ dz)
        dy = dz @ self.w["out"].to(x.dtype).t().contiguous()
        dacts, dweights = ar.expert_combine_backward(dy, acts, weights, plan)
        dacts *= acts > 0
        drows = torch.zeros_like(rows)
        for e in range(experts):
            s = slice(ends[e], ends[e + 1])
            self.g["expert"][e].copy_(rows[s].t().contiguous() @ dacts[s])
            drows[s] = dacts[s] @ self.w["expert"][e].to(x.dtype).t().contiguous()
        dh = ar.expert_dispatch_backward(drows, plan)
        _, self.g["norm_w"][:], self.g["norm_b"][:] = ar.layer_norm_backward(
            dh, x, mean, rstd, self.w["norm_w"])
        return loss, dweights


def make_batch(tokens, hidden, experts, vocab, topk, top, seed, dtype=torch.bfloat16):
    """Tokens, a router's choices, and the top logits of a fixed random teacher."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").to(dtype)
    scores, ids = torch.randn((tokens, experts), generator=gen, device="cuda").topk(topk, dim=1)
    wt = torch.Generator("cuda").manual_seed(7)
    head = torch.randn((hidden, vocab), generator=wt, device="cuda").to(dtype) * 0.2
    teacher, places = (x @ head).topk(top, dim=1)
    return x, ids, scores.softmax(1), places, teacher.contiguous()


def train(ranks=4, steps=20, tokens=256, hidden=128, experts=8, vocab=1000, topk=2, top=16, lr=10.0):
    """Losses of the steps; raises if the ranks' weights ever differ."""
    students = [Student(hidden, experts, vocab, seed=1) for _ in range(ranks)]
    batches = [make_batch(tokens, hidden, experts, vocab, topk, top, seed=100 + r)
               for r in range(ranks)]
    losses = []
    for _ in range(steps):
        losses.append(sum(float(s.step(b)[0].mean()) for s, b in zip(students, batches)) / ranks)
        ar.allreduce([s.grads for s in students], op="avg", algo="ring_fused")
        for s in students:
            s.weights.sub_(s.grads, alpha=lr)
    if ar.check([s.weights for s in students])["mismatched"]:
        raise AssertionError("the ranks' weights differ")
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=20)
    args = p.parse_args()
    for i, loss in enumerate(train(args.ranks, args.steps)):
        print(f"step {i:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
