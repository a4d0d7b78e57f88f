"""A layer as the operators are used together: embedding, layer norm, dispatch,
the experts' two products with the gated activation between them, combination,
and back through all of them, against autograd in 64 bits over plain torch
operations; and the table's gradient summed over ranks with the AllReduce."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref
from tests.test_gpu_model_forms import F32, Layer, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def gate(h):
    a, u = h.chunk(2, -1)
    return a * torch.sigmoid(a) * u


@pytest.mark.parametrize("tokens,vocab,hidden,inner,experts,topk", [
    (48, 77, 32, 40, 5, 2), (1, 3, 64, 33, 4, 1), (301, 20, 24, 65, 70, 3)])
def test_gradients_against_autograd(tokens, vocab, hidden, inner, experts, topk):
    layer = Layer(tokens, vocab, hidden, inner, experts, topk, F32)
    layer.draw(5)
    y, dgates, dw1, dw2, dtable, codes, scales = layer.run()
    plan = ar.expert_dispatch(ar.embedding(layer.table, layer.tokens), layer.ids, experts)[1]
    values = ref.values(codes, scales).reshape(-1, 2 * inner)

    leaf = {k: getattr(layer, k).double().cpu().requires_grad_() for k in ("table", "w1", "w2", "gates")}
    ids, dest = layer.ids.cpu(), plan.dest.cpu().long()
    x = 2.0 * leaf["table"][layer.tokens.cpu()]
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
    want, most = torch.zeros_like(h), 1.0
    for k in range(topk):
        w1, w2 = leaf["w1"][ids[:, k].long()], leaf["w2"][ids[:, k].long()]
        a = (w1 * h[:, None]).sum(-1)
        # forward at the exact values; back at the checkpoint's, which lie within half a step
        # of them (and within the product's own error)
        v = values[dest[:, k]]
        step = 2.0 ** (scales.reshape(-1, 2, scales.shape[-1]).double().cpu()[dest[:, k]] - 127)
        step = step.repeat_interleave(ref.GROUP, -1)[..., :inner].reshape(tokens, -1)
        assert bool(((v - a).abs() <= 0.5 * step + 2e-5).all())
        held = gate(a + (v - a).detach())
        out = (w2 * held[:, None]).sum(-1)
        out = out + ((w2 * gate(a)[:, None]).sum(-1) - out).detach()
        want = want + leaf["gates"][:, k:k + 1] * out
        most = max(most, *(float(s.detach().abs().sum(-1).max()) for s in (w1 * h[:, None],
                                                                          w2 * held[:, None])))
    want.backward(layer.dy.double().cpu())
    # fp32 all the way.  A stage adds at most 130 terms, or a token's occurrences, and is off
    # by less than 300 steps of 2^-24 of the sum of its terms' magnitudes; a value passes at
    # most eight stages; `most` bounds the sums of the products, and the gradients' largest
    # value stands for those of the way back, whose rows' sums are at most 8 times it
    for name, got, exact in (("y", y, want.detach()), ("gates", dgates, leaf["gates"].grad),
                             ("w1", dw1, leaf["w1"].grad), ("w2", dw2, leaf["w2"].grad),
                             ("table", dtable, leaf["table"].grad)):
        tol = 8 * 300 * 2.0 ** -24 * max(most, 8 * float(exact.abs().max()))
        err = float((got.double().cpu() - exact).abs().max())
        assert err <= tol, (name, err, tol)


def test_summed_over_ranks():
    """Three ranks' gradients of the table, summed in place."""
    layers = []
    for r in range(3):
        layer = Layer(200, 90, 64, 40, 4, 2, F32)
        layer.draw(r)
        layers.append(layer.run()[4])
    want = sum(g.double() for g in layers)
    size = sum(g.double().abs() for g in layers)
    bufs = [g.view(-1) for g in layers]
    torch.cuda.synchronize()
    ar.allreduce(bufs)
    torch.cuda.synchronize()
    for g in layers:
        assert bool(((g.double() - want).abs() <= 2 * 2.0 ** -24 * size).all())


def test_gradients_by_differences():
    """The embedding and the products are linear: the difference along a direction v
    is f(v), whatever the point, and <dy, f(v)> is <gradient, v>."""
    ids = torch.randint(0, 50, (200,), device="cuda")
    v, dy = randn(50, 40), randn(200, 40, seed=1)
    off = torch.tensor([0, 90, 90, 200], dtype=torch.int32, device="cuda")
    at = torch.arange(200, dtype=torch.int32, device="cuda")
    plan = ar.ExpertPlan(at.view(-1, 1), at, off)
    vr, vw, dout = randn(200, 72, seed=2), randn(3, 56, 72, seed=3), randn(200, 56, seed=4)

    def same_slope(a, b, what):
        """Each side a direction, a result and the result's bound."""
        sides = [float((d.double().cpu() * r.double().cpu()).sum()) for d, r, _ in (a, b)]
        tol = sum(float((d.double().cpu().abs() * t.cpu()).sum()) for d, _, t in (a, b))
        assert abs(sides[0] - sides[1]) <= tol, (what, sides, tol)

    same_slope((dy, ar.embedding(v, ids, 3.0), ref.embedding(v, ids, 3.0)[1]),
               (v, ar.embedding_backward(dy, ids, 50, 3.0), ref.embedding_backward(dy, ids, 50, 3.0)[1]),
               "embedding")
    out = (dout, ar.expert_matmul(vr, vw, plan), ref.product("out", off, vr, vw)[1])
    same_slope(out, (vr, ar.expert_matmul_drows(dout, vw, plan),
                     ref.product("drows", off, dout, vw)[1]), "rows")
    same_slope(out, (vw, ar.expert_matmul_dweights(dout, vr, plan),
                     ref.product("dweights", off, dout, vr)[1]), "weights")
