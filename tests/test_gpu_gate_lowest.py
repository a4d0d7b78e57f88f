"""The gate's gradient where u is the type's lowest value, as a masked place has
it: the gradient is finite although the product dacts u is not."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_gradient_at_the_lowest_value(t):
    low = torch.finfo(t).min
    a = torch.tensor([low, -1e30, -1e4, -200.0, -60.0, -50.0, -20.0, 0.0, 1.0, 2.0, 5.0, 1e4])
    d = torch.tensor([0.01, 0.8, 2.0, -4.0, 100.0, -1e4])
    # a row, with groups of its own, for each a; u lowest, as large upwards, and half as large
    for top in (low, -low, 1.6e38):
        h = torch.cat([a[:, None].expand(-1, 64), torch.full((12, 64), top)], 1).to(t).cuda()
        _, saved = ar.silu_gate(h)
        dacts = d.repeat(11)[:64].to(t).expand(12, 64).contiguous()
        dh, acts = ar.silu_gate_backward(dacts.cuda(), saved)

        v, g = ref.values(saved.codes, saved.scales), dacts.double()
        x, u = v[:, 0], v[:, 1]
        s = torch.sigmoid(x)
        f = 1 + x * (1 - s)
        # the bounds of model_refs.gate_backward; a sigmoid below 2^-126 may be 0, which is e^-200
        # at the most here, and 1e4 * 2^128 * 200 times that is below every type's numbers
        for got, want, rel in ((dh[:, :64], g * u * s * f, (
                ref.RS * s + 2 * ref.U) * x.abs() / f.abs().clamp(min=2.0 ** -4)
                + 3 * ref.U * (1 + (x * (1 - s)).abs()) / f.abs().clamp(min=2.0 ** -4)
                + ref.RS + 4 * ref.U),
                (dh[:, 64:], g * (x * s), ref.RS + 3 * ref.U), (acts, x * s * u, ref.RS + 2 * ref.U)):
            fits = want.abs() < 0.99 * torch.finfo(t).max
            tol = 1.01 * (rel + ref.half_step(t)) * want.abs() + ref.floor_of(t)
            got = got.double().cpu()
            assert bool(torch.isfinite(got[fits]).all())
            assert bool(((got - want).abs() <= tol)[fits].all())
            assert bool((got == want.sign() * torch.inf)[want.abs() > 1.01 * torch.finfo(t).max].all())
