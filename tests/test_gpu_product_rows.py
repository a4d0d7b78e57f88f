"""The experts' products take the rows of their plan's dispatch: another number
of rows is refused, as ``expert_combine`` refuses it."""

import pytest
import torch

import ring_allreduce_rs_amd as ar

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_rows_of_another_dispatch(t):
    x = torch.randn((6, 64), device="cuda").to(t)
    ids = torch.randint(0, 3, (6, 2), device="cuda")
    rows, plan = ar.expert_dispatch(x, ids, 3)
    w = torch.randn((3, 32, 64), device="cuda").to(t)
    dout = ar.expert_matmul(rows, w, plan)
    assert dout.shape == (12, 32) and ar.expert_matmul_drows(dout, w, plan).shape == (12, 64)
    assert ar.expert_matmul_dweights(dout, rows, plan).shape == (3, 32, 64)
    for n in (0, 1, 11, 13):
        r, d = x.new_zeros((n, 64)), x.new_zeros((n, 32))
        for call in (lambda: ar.expert_matmul(r, w, plan),
                     lambda: ar.expert_matmul_drows(d, w, plan),
                     lambda: ar.expert_matmul_dweights(d, r, plan)):
            with pytest.raises(ValueError, match="needs the plan's 12 rows"):
                call()
    other = ar.expert_dispatch(x, ids[:, :1].contiguous(), 3)[1]
    with pytest.raises(ValueError, match="needs the plan's 6 rows"):
        ar.expert_matmul(rows, w, other)
    for bad in (plan.dest.long(), plan.dest.cpu(), plan.dest.view(-1), plan.dest[:, :0],
                plan.dest[:, ::2]):
        with pytest.raises(ValueError, match="plan.dest"):
            ar.expert_matmul(rows, w, plan._replace(dest=bad))
