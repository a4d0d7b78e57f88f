"""The layer's sample in README.md computes the gradients of what it runs
forward: executed as it stands, with the definitions in 64 bits in place of the
GPU's operators, against autograd."""

import os
import re
import types

import pytest
import torch

from tests import model_refs, operator_refs as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
README = os.path.join(ROOT, "README.md")


def gate(h):
    a, u = h.chunk(2, -1)
    return a * torch.sigmoid(a) * u


def stand_in(topk):
    """The package's operators by their definitions; a checkpoint keeps its values as
    they are."""
    def dispatch(x, ids, experts):
        dest, slot, offsets = ref.plan(ids, experts)
        return x[slot.long() // topk], (dest, offsets)

    def gate_backward(dacts, h):
        a, u = h.chunk(2, -1)
        s = torch.sigmoid(a)
        return torch.cat([dacts * u * s * (1 + a * (1 - s)), dacts * a * s], -1), gate(h)

    def product(kind):
        return lambda a, b, plan: model_refs.product(kind, plan[1], a, b)[0]
    return types.SimpleNamespace(
        embedding=lambda table, ids: model_refs.embedding(table, ids, 1.0)[0],
        embedding_backward=lambda dy, ids, vocab: model_refs.embedding_backward(dy, ids, vocab, 1.0)[0],
        expert_dispatch=dispatch,
        expert_dispatch_backward=lambda drows, plan: ref.combine(
            drows, torch.ones(plan[0].shape), plan[0], plan[1][-1])[0],
        expert_combine=lambda rows, w, plan: ref.combine(rows, w, plan[0], plan[1][-1])[0],
        expert_combine_backward=lambda dy, rows, w, plan: ref.combine_backward(
            dy, rows, w, plan[0], plan[1][-1])[0],
        expert_matmul=product("out"), expert_matmul_drows=product("drows"),
        expert_matmul_dweights=product("dweights"),
        silu_gate=lambda h: (gate(h), h), silu_gate_backward=gate_backward)


@pytest.mark.skipif(not os.path.exists(README), reason="needs README.md")
def test_gradients_of_the_sample():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    code, = (b for b in blocks if "silu_gate_backward" in b)
    n_tokens, vocab, hidden, inner, topk = 7, 11, 6, 5, 2
    g = torch.Generator().manual_seed(6)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)
    tokens = torch.randint(0, vocab, (n_tokens,), generator=g)
    ids = torch.randint(0, 64, (n_tokens, topk), generator=g)
    leaves = {"table": n(vocab, hidden), "w1": n(64, 2 * inner, hidden), "w2": n(64, hidden, inner),
              "gates": torch.rand((n_tokens, topk), generator=g, dtype=torch.float64)}
    dy = n(n_tokens, hidden)
    names = {**leaves, "ar": stand_in(topk), "tokens": tokens, "ids": ids, "dy": dy}
    exec(code, names)

    leaf = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    x = leaf["table"][tokens]
    y = torch.zeros_like(x)
    for k in range(topk):
        h = (leaf["w1"][ids[:, k]] * x[:, None]).sum(-1)
        y = y + leaf["gates"][:, k:k + 1] * (leaf["w2"][ids[:, k]] * gate(h)[:, None]).sum(-1)
    y.backward(dy)
    # 64 bits all the way: a few hundred roundings of values below 2^12
    tol = 512 * 4096 * 2.0 ** -53
    assert float((names["y"] - y.detach()).abs().max()) <= tol
    for k in leaf:
        err = (names["d" + k] - leaf[k].grad).abs().max()
        assert float(err) <= tol, (k, float(err))
