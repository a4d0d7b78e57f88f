"""The operators and the AllReduce together (examples/moe_distill.py): the
gradients of a step against autograd in 64 bits over plain torch operations,
and a few steps of training."""

import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def example():
    spec = importlib.util.spec_from_file_location(
        "moe_distill", os.path.join(ROOT, "examples", "moe_distill.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd():
    ex = example()
    tokens, hidden, experts, vocab, topk, top = 48, 32, 5, 77, 2, 6
    s = ex.Student(hidden, experts, vocab, seed=3)
    batch = ex.make_batch(tokens, hidden, experts, vocab, topk, top, seed=4, dtype=torch.float32)
    x, ids, weights, places, teacher = batch
    loss, dweights = s.step(batch)

    w = {k: v.double().cpu().requires_grad_() for k, v in s.w.items()}
    x, teacher = x.double().cpu(), teacher.double().cpu()
    ids, places = ids.cpu(), places.cpu()
    gates = weights.double().cpu().requires_grad_()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    h = (x - mean) / (var + 1e-5).sqrt() * w["norm_w"] + w["norm_b"]
    each = torch.stack([torch.relu(h @ w["expert"][e]) for e in range(experts)], 1)
    y = x + sum(gates[:, k:k + 1] * each[torch.arange(tokens), ids[:, k]] for k in range(topk))
    z = y @ w["out"]
    logp = torch.log_softmax(teacher / 2.0, 1)
    logq = torch.log_softmax(z / 2.0, 1).gather(1, places)
    want = 4.0 * (logp.exp() * (logp - logq)).sum(1)
    want.mean().backward()
    # fp32 all the way: products of at most 77 terms and a handful of roundings
    # after each other stay below 200 steps of 2^-24 of the largest magnitude
    # on the way, which is below 64
    tol = 200 * 64 * 2.0 ** -24
    assert float((loss.double().cpu() - want.detach()).abs().max()) <= tol
    for k in w:
        err = (s.g[k].double().cpu() - w[k].grad).abs().max()
        assert float(err) <= tol, (k, float(err))
    assert float((dweights.double().cpu() - gates.grad).abs().max()) <= tol


def test_training_with_the_allreduce():
    losses = example().train(ranks=3, steps=12)
    assert losses[-1] < 0.8 * losses[0]
    assert all(b == b for b in losses)
