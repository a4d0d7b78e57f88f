"""The training operators record nothing for autograd: a tensor whose gradient
would be lost is refused (before anything that needs a GPU)."""

import pytest
import torch
import torch.autograd.forward_ad as fw

import ring_allreduce_rs_amd as ar

X = torch.randn(4, 32)
STAT = torch.zeros(4)
IDS = torch.zeros((4, 2), dtype=torch.int64)
PLAN = ar.ExpertPlan(IDS.int(), IDS.int().view(-1), torch.zeros(4, dtype=torch.int32))
# every operator, by the tensor that it looks at first
CALLS = {
    "layer_norm": (lambda x: ar.layer_norm(x), X),
    "layer_norm_backward": (lambda dy: ar.layer_norm_backward(dy, X, STAT, STAT), X),
    "expert_dispatch": (lambda x: ar.expert_dispatch(x, IDS, 3), X),
    "expert_dispatch_backward": (lambda d: ar.expert_dispatch_backward(d, PLAN), X.repeat(2, 1)),
    "expert_combine": (lambda r: ar.expert_combine(r, torch.zeros(4, 2), PLAN), X.repeat(2, 1)),
    "expert_combine_backward": (
        lambda dy: ar.expert_combine_backward(dy, X.repeat(2, 1), torch.zeros(4, 2), PLAN), X),
    "distill_loss": (lambda z: ar.distill_loss(z, IDS, torch.zeros(4, 2)), X),
    "distill_backward": (
        lambda z: ar.distill_backward(STAT, z, IDS, torch.zeros(4, 2), STAT), X),
    "distill_step": (lambda z: ar.distill_step(STAT, z, IDS, torch.zeros(4, 2)), X),
}


@pytest.mark.parametrize("name", CALLS)
def test_gradients_are_not_lost(name):
    call, arg = CALLS[name]
    leaf = arg.clone().requires_grad_()
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="requires grad"):
            call(t)
        with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):
            call(t)      # taken as it is
        with pytest.raises(ValueError, match="not on a GPU"):
            call(t.detach())


@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_not_lost(name):
    call, arg = CALLS[name]
    with fw.dual_level():
        dual = fw.make_dual(arg, torch.ones_like(arg))
        with pytest.raises(ValueError, match="tangent"):
            call(dual)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_gradients_of_later_arguments_are_not_lost():
    x, ids = torch.randn(4, 32, device="cuda"), torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    w = torch.nn.Parameter(torch.ones(32, device="cuda"))
    pair = torch.zeros((4, 2), device="cuda")
    row = torch.zeros(4, device="cuda")
    with torch.no_grad():
        _, mean, rstd = ar.layer_norm(x, w, w)
        rows, plan = ar.expert_dispatch(x, ids, 3)

    def leaf(t):
        return t.clone().requires_grad_()
    for call in (lambda: ar.layer_norm(x, w), lambda: ar.layer_norm(x, None, w),
                 lambda: ar.layer_norm_backward(x, leaf(x), mean, rstd),
                 lambda: ar.layer_norm_backward(x, x, leaf(mean), rstd),
                 lambda: ar.layer_norm_backward(x, x, mean, leaf(rstd)),
                 lambda: ar.layer_norm_backward(x, x, mean, rstd, w),
                 lambda: ar.expert_combine(rows, leaf(pair), plan),
                 lambda: ar.expert_combine_backward(x, leaf(rows), pair, plan),
                 lambda: ar.expert_combine_backward(x, rows, leaf(pair), plan),
                 lambda: ar.distill_loss(x, ids, leaf(pair)),
                 lambda: ar.distill_backward(leaf(row), x, ids, pair, row),
                 lambda: ar.distill_backward(row, x, ids, leaf(pair), row),
                 lambda: ar.distill_backward(row, x, ids, pair, leaf(row)),
                 lambda: ar.distill_step(leaf(row), x, ids, pair),
                 lambda: ar.distill_step(row, x, ids, leaf(pair))):
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad():
            call()
