"""The training operators at their limits and beside non-finite values, against
the definitions in 64 bits (tests/operator_refs.py derives the bounds)."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import operator_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def test_norm_gradient_of_rows_past_a_grid():
    """2 x cols / 64 groups of columns are more than the fold's blocks."""
    cols = 2 ** 27 + 33
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((1, cols), generator=g, device="cuda")
    dy = torch.randn((1, cols), generator=g, device="cuda")
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 1.5, device="cuda")
    got = ar.layer_norm_backward(dy, x, mean, rstd)
    want, tol = ref.norm_backward(dy, x, mean, rstd, None)
    for name, v, w, t in zip(("dx", "dweight", "dbias"), got, want, tol):
        assert bool(((v.double() - w.view_as(v)).abs() <= t.view_as(v)).all()), name


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("hidden", [9, 13, 771, 2055])
def test_infinite_rows_beside_a_ragged_end(hidden, t):
    """Infinities in the elements that a row's last 16 bytes share with the ones
    before: the weight's gradient is infinite, not NaN."""
    tokens, topk, experts = 6, 3, 4
    g = torch.Generator("cuda").manual_seed(hidden)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda")
    dy = (torch.rand((tokens, hidden), generator=g, device="cuda") + 0.5).to(t)
    rows, plan = ar.expert_dispatch(dy, ids, experts)
    w = torch.rand((tokens, topk), generator=g, device="cuda")
    inf = float("inf")
    for back in range(1, 10):      # from the row's end
        if back > hidden:
            break
        rows = torch.randn(rows.shape, generator=g, device="cuda").to(t)
        rows[1, -back] = inf
        rows[5, -back] = -inf
        (drows, dw), (tdrows, tdw) = ref.combine_backward(dy, rows, w, plan.dest,
                                                          int(plan.offsets[-1]))
        got = ar.expert_combine_backward(dy, rows, w, plan)
        assert int(torch.isinf(dw).sum()) == 2
        ref.close(got[0], drows, tdrows, "drows")
        ref.close(got[1], dw, torch.where(torch.isinf(dw), 0.0, tdw), "dweights")


# (rows, vocab): rows in registers, more of them than blocks, chunks of one row, a row's
# parts, chunks of a block's row
FORMS = [(6, 300), (6, 32000), (700, 4099), (7000, 1003), (3, 140001), (600, 140001), (3, 5)]


def distill_case(rows, vocab, top, t, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    logits = (torch.randn((rows, vocab), generator=g, device="cuda") * 2.5).to(t)
    at = torch.randint(0, vocab, (rows, top), generator=g, device="cuda")
    teacher = (torch.randn((rows, top), generator=g, device="cuda") * 2 + 4).to(t)
    return logits, at, teacher, torch.rand(rows, generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_infinite_teacher_logits(rows, vocab, t):
    """A kept +inf has no softmax: the row's loss and its gradient at the entries'
    places are NaN, in every form; left out, it is not looked at."""
    logits, at, teacher, dloss = distill_case(rows, vocab, 4, t, 11)
    bad = torch.tensor([1, rows - 1], device="cuda")
    clean, lse = ar.distill_loss(logits, at, teacher)
    clean_step = ar.distill_step(dloss, logits, at, teacher)
    clean_back = ar.distill_backward(dloss, logits, at, teacher, lse)
    teacher[bad, 2] = float("inf")
    at[0, 1] = -1
    teacher[0, 1] = float("inf")
    loss, got = ar.distill_loss(logits, at, teacher)
    step = ar.distill_step(dloss, logits, at, teacher)
    back = ar.distill_backward(dloss, logits, at, teacher, lse)
    assert torch.equal(got, lse)
    named = torch.zeros((rows, vocab), dtype=torch.bool, device="cuda")
    named.scatter_(1, at.clamp(min=0), True)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for v, c in ((loss, clean), (step[0], clean_step[0])):
        assert torch.isnan(v[bad]).all() and torch.isfinite(v[0])
        assert torch.equal(v[1:][keep[1:]], c[1:][keep[1:]])
    for v, c in ((step[1], clean_step[1]), (back, clean_back)):
        assert torch.isnan(v[bad][named[bad]]).all()
        assert torch.equal(v[bad][~named[bad]], c[bad][~named[bad]])
        assert torch.equal(v[1:][keep[1:]], c[1:][keep[1:]]) and torch.isfinite(v[0]).all()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_large_logits_beside_an_infinite_one(rows, vocab, t):
    """A +inf makes the row's sum infinite: q is 0 at every finite logit, however
    large, and NaN at the infinite one, by the step as by loss and backward."""
    logits, at, teacher, dloss = distill_case(rows, vocab, 2, t, 12)
    bad = torch.tensor([1, rows - 1], device="cuda")
    logits[bad, vocab // 2] = float("inf")
    logits[bad, 0] = 200.0        # exp(200) is past fp32
    logits[bad, vocab - 1] = torch.finfo(t).max
    at[bad] = torch.tensor([0, 1], device="cuda")
    loss, lse = ar.distill_loss(logits, at, teacher)
    step = ar.distill_step(dloss, logits, at, teacher)
    back = ar.distill_backward(dloss, logits, at, teacher, lse)
    assert (loss[bad] == float("inf")).all() and (lse[bad] == float("inf")).all()
    assert (step[0][bad] == float("inf")).all()
    p = teacher.double().softmax(1)[bad] * dloss.double()[bad, None]
    # two exponentials, their sum, a quotient and a product, then the last rounding
    tol = p * (2 * ref.EXP + 8 * ref.U + ref.half_step(t))
    for d in (step[1][bad], back[bad]):
        assert torch.isnan(d[:, vocab // 2]).all()
        ref.close(d[:, :2], -p, tol)
        rest = torch.cat([d[:, 2:vocab // 2], d[:, vocab // 2 + 1:]], 1)
        assert not rest.any()


def test_temperatures_whose_inverse_overflows():
    logits, at, teacher, dloss = distill_case(3, 50, 2, F32, 1)
    lse = torch.zeros(3, device="cuda")
    for T in (1e-40, 1e-45):
        for call in (lambda: ar.distill_loss(logits, at, teacher, T),
                     lambda: ar.distill_backward(dloss, logits, at, teacher, lse, T),
                     lambda: ar.distill_step(dloss, logits, at, teacher, T)):
            with pytest.raises(ValueError, match="temperature"):
                call()
