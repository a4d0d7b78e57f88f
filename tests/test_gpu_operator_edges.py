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
