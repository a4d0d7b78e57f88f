"""The experts' products in every kernel that they can take (tests/product_cases.py;
tests/test_product_kernels.py checks on the CPU that these are all), bit for
bit: with small whole numbers every sum is exact in binary32, in whatever order,
so the result is the exact one rounded once."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import product_cases as pc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def placed(v, shift, extra):
    """v's values `shift` elements from an aligned address, `extra` more from row to row."""
    n, width = v.numel() // v.shape[-1], v.shape[-1]
    base = torch.full((shift + n * (width + extra) + 64,), torch.nan, dtype=v.dtype, device=v.device)
    at = base[shift:shift + n * (width + extra)].view(*v.shape[:-1], width + extra)[..., :width]
    at.copy_(v)
    return at


def exact(kind, counts, n, a, b):
    """The product in 64 bits, rounded once; a and b whole numbers."""
    t, a, b = a.dtype, a.double(), b.double()
    shape = {"out": (n, b.shape[1]), "drows": (n, b.shape[-1]),
             "dweights": (len(counts), a.shape[1], b.shape[-1])}[kind]
    y = torch.zeros(shape, dtype=torch.float64, device=a.device)
    lo = 0
    for e, c in enumerate(counts):
        at = slice(lo, lo + c)
        lo += c
        if kind == "dweights":
            y[e] = a[at].t().contiguous() @ b[at]
        else:
            y[at] = a[at] @ (b[e].t().contiguous() if kind == "out" else b[e])
    assert float(y.abs().max()) < 2 ** 24
    return y.to(t)


@pytest.mark.parametrize("sizes,lines", pc.cases())
def test_every_kernel(sizes, lines):
    kind, eb, n, experts, hidden, out = sizes
    t = torch.bfloat16 if eb == 2 else torch.float32
    counts = pc.groups(n, experts)
    g = torch.Generator("cuda").manual_seed(n + hidden)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(t)
    wa, wb = pc.widths(kind, hidden, out)
    a = whole(n, wa)
    b = whole(n, wb) if wb else whole(experts, out, hidden)
    want = exact(kind, counts, n, a, b)
    # what the rows behind the last expert hold does not matter
    a[n - 3:] = torch.nan
    if wb:
        b[n - 3:] = torch.inf
    a = placed(a, lines[0], lines[1])
    b = placed(b, lines[2], lines[3] if wb else 0)
    off = torch.tensor([0, *counts]).cumsum(0).int().cuda()
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    plan = ar.ExpertPlan(at.view(-1, 1), at, off)
    call = {"out": ar.expert_matmul, "drows": ar.expert_matmul_drows,
            "dweights": ar.expert_matmul_dweights}[kind]
    for _ in range(2):
        got = call(a, b, plan)
        assert got.shape == want.shape and torch.equal(got, want)
