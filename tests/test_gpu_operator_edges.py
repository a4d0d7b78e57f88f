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
