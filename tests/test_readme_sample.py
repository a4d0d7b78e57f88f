"""The operators' sample in README.md computes the gradients of what it runs
forward: executed as it stands, with the definitions in 64 bits in place of the
GPU's operators, against autograd."""

import os
import re
import types

import pytest
import torch

from tests import operator_refs as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
README = os.path.join(ROOT, "README.md")


def stand_in(topk):
    """The package's operators by their definitions."""
    def dispatch(x, ids, experts):
        dest, slot, offsets = ref.plan(ids, experts)
        return x[slot.long() // topk], (dest, offsets)

    def dispatch_backward(drows, plan):
        return ref.combine(drows, torch.ones(plan[0].shape), plan[0], plan[1][-1])[0]

    def step(dloss, logits, indices, teacher, temperature=1.0):
        loss, _, d = ref.distill(logits, indices, teacher, temperature, dloss)[0]
        return loss, d
    return types.SimpleNamespace(
        layer_norm=lambda x, w, b: ref.norm(x, w, b, 1e-5)[0],
        layer_norm_backward=lambda dy, x, m, r, w: ref.norm_backward(dy, x, m, r, w)[0],
        expert_dispatch=dispatch, expert_dispatch_backward=dispatch_backward,
        expert_combine=lambda rows, w, plan: ref.combine(rows, w, plan[0], plan[1][-1])[0],
        expert_combine_backward=lambda dy, rows, w, plan: ref.combine_backward(
            dy, rows, w, plan[0], plan[1][-1])[0],
        distill_step=step)


@pytest.mark.skipif(not os.path.exists(README), reason="needs README.md")
def test_gradients_of_the_sample():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    code, = (b for b in blocks if "layer_norm_backward" in b)
    tokens, hidden, vocab, topk, top = 6, 10, 12, 2, 3
    g = torch.Generator().manual_seed(5)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)
    ids = torch.randint(0, 64, (tokens, topk), generator=g)
    places = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(tokens)])
    w_out, share = n(hidden, vocab), torch.rand(tokens, generator=g, dtype=torch.float64)
    leaves = {"x": n(tokens, hidden), "weight": n(hidden), "bias": n(hidden),
              "gates": torch.rand((tokens, topk), generator=g, dtype=torch.float64)}
    teacher = n(tokens, top)
    names = {**leaves, "ar": stand_in(topk), "ids": ids, "places": places, "share": share,
             "teacher": teacher,
             # an expert squares its rows, the head is a product
             "experts_of": lambda rows: rows.square(),
             "experts_backward": lambda dacts, rows: dacts * 2 * rows,
             "head": lambda out: out @ w_out, "head_backward": lambda dlogits: dlogits @ w_out.t()}
    exec(code, names)

    leaf = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    x = leaf["x"]
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
    y = y * leaf["weight"] + leaf["bias"]
    out = leaf["gates"].sum(1, keepdim=True) * y.square()
    T = 2.0
    logp = torch.log_softmax(teacher / T, 1)
    logq = torch.log_softmax(out @ w_out / T, 1).gather(1, places)
    loss = T * T * (logp.exp() * (logp - logq)).sum(1)
    (loss * share).sum().backward()
    # 64 bits all the way: a few hundred roundings of values below 2^12
    tol = 512 * 4096 * 2.0 ** -53
    assert float((names["loss"] - loss.detach()).abs().max()) <= tol
    for k in leaf:
        err = (names["d" + k] - leaf[k].grad).abs().max()
        assert float(err) <= tol, (k, float(err))
