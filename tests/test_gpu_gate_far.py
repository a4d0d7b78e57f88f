"""The gate where the sigmoid is below binary32's normal numbers and what it
multiplies is large: the activation and its gradient are ordinary numbers."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

# sigmoids from e^-64 down to e^-165; the products below are 2^128 times that and more
A = [-64.0, -79.5, -80.0, -80.5, -87.0, -88.0, -90.0, -96.0, -100.0, -110.0, -120.0, -150.0, -165.0,
     64.0, 88.0, 100.0]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("u", [1.0, -1e20, 3e38])
def test_small_sigmoids(u, t):
    # a row, with groups of its own, for each a
    h = torch.cat([torch.tensor(A)[:, None].expand(-1, 64), torch.full((len(A), 64), u)], 1).to(t)
    acts, saved = ar.silu_gate(h.cuda())
    a, w = h[:, :64].double(), h[:, 64:].double()
    checks = [(acts, a * torch.sigmoid(a) * w, ref.RS + 2 * ref.U)]
    v = ref.values(saved.codes, saved.scales)
    x, w = v[:, 0], v[:, 1]
    s = torch.sigmoid(x)
    f = 1 + x * (1 - s)
    for size in (1.0, -1e-3, 3e38):
        d = torch.full((len(A), 64), size).to(t)
        dh, again = ar.silu_gate_backward(d.cuda(), saved)
        # f = 1 + a (1 - s) is off by at most 4 u of 1 + |a| (a <= -64), or of 1 + |a| s (a > 0)
        checks += [(dh[:, :64], d * w * s * f, ref.RS + 8 * ref.U + (x > 0) * (x * ref.RS)),
                   (dh[:, 64:], d * (x * s), ref.RS + 3 * ref.U), (again, x * s * w, ref.RS + 2 * ref.U)]
    seen = 0
    for got, want, rel in checks:
        got = got.double().cpu()
        fits = want.abs() < 0.99 * torch.finfo(t).max
        tol = 1.01 * (rel + ref.half_step(t)) * want.abs() + ref.floor_of(t)
        assert bool(((got - want).abs() <= tol)[fits].all())
        seen += int(((want.abs() > 1e-30) & fits & (a < -88)).sum())
    assert seen > 0 or u == 1.0
