"""The experts' products and their gradients against 64 bits
(tests/model_refs.py derives the bounds)."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def plan_of(counts, behind=0):
    """A plan whose experts have `counts` rows, with `behind` rows behind them."""
    off = torch.tensor([0, *counts]).cumsum(0).int().cuda()
    n = int(off[-1]) + behind
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    return ar.ExpertPlan(at.view(-1, 1), at, off), n


def check(counts, hidden, out, t, behind=0, seed=0, kinds=("out", "drows", "dweights")):
    plan, n = plan_of(counts, behind)
    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn((n, hidden), generator=g, device="cuda").to(t)
    dout = torch.randn((n, out), generator=g, device="cuda").to(t)
    w = torch.randn((len(counts), out, hidden), generator=g, device="cuda").to(t)
    # what the rows behind the last expert hold does not matter
    rows[n - behind:], dout[n - behind:] = torch.nan, torch.inf
    got = {"out": lambda: ar.expert_matmul(rows, w, plan),
           "drows": lambda: ar.expert_matmul_drows(dout, w, plan),
           "dweights": lambda: ar.expert_matmul_dweights(dout, rows, plan)}
    a = {"out": (rows, w), "drows": (dout, w), "dweights": (dout, rows)}
    for kind in kinds:
        y, tol = ref.product(kind, plan.offsets, *a[kind])
        first = got[kind]()
        ref.close(first, y, tol, kind)
        assert torch.equal(first, got[kind]())       # to the bit


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("counts,hidden,out,behind", [
    ((1,), 1, 1, 0), ((1, 0, 2), 3, 5, 1), ((0, 0), 8, 8, 4), ((5,), 64, 64, 0),
    ((16, 17, 15, 0, 1), 128, 72, 3), ((128, 127, 129), 64, 128, 0), ((300,), 257, 129, 7),
    ((33, 0, 0, 250, 4), 1000, 771, 5), ((2,) * 70, 40, 24, 0), ((1, 0, 3) * 100, 33, 16, 9),
    ((700, 60), 200, 512, 0), ((256, 512), 256, 256, 0), ((1023, 1, 520), 520, 264, 11)])
def test_products(counts, hidden, out, behind, t):
    check(counts, hidden, out, t, behind, hidden)


@pytest.mark.parametrize("t", [BF, F32])
def test_one_token_through_many_experts(t):
    """A token's choices among experts that have a row at most."""
    counts = [1 if e % 9 == 2 else 0 for e in range(64)]
    check(counts, 2048, 520, t)
    check([0] * 1023 + [1], 72, 40, t)
    check([3] + [0] * 1023, 72, 40, t, 2)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("hidden,out", [(64, 2056), (2056, 64), (1, 300), (300, 1), (4104, 40),
                                        (63, 65), (1001, 255)])
def test_widths(hidden, out, t):
    check((40, 150, 9), hidden, out, t, 2)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("hidden,out", [(1, 200), (2, 1), (3, 70), (4, 9), (5, 5), (6, 31), (7, 2),
                                        (8, 7), (9, 3), (70, 3), (200, 7)])
def test_narrow(hidden, out, t):
    """Lines closer together than 16 bytes, over several steps of the depth."""
    check((200, 0, 131, 1), hidden, out, t, 2)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("counts,hidden,out", [((3, 0, 40), 8192, 200), ((130, 7), 1024, 600),
                                               ((1, 1, 1, 0, 2), 2048, 1400), ((5,), 16384, 70)])
def test_lines_a_power_of_two_apart(counts, hidden, out, t):
    """Tiles that begin inside their depth, with the depth in parts and not."""
    check(counts, hidden, out, t, 1)


def test_large():
    """Tiles of every kind among many rows."""
    check((3000, 100, 0, 2500, 260, 1), 1024, 1280, BF, 30)
    check((900, 100, 0, 600), 512, 640, F32, 3)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("offset,extra", [(1, 0), (3, 6), (8, 8)])
def test_rows_anywhere(offset, extra, t):
    plan, n = plan_of((20, 0, 41), 3)
    w = torch.randn((3, 96, 72), device="cuda").to(t)
    def strided(width):
        base = torch.randn(n * (width + extra) + 64, device="cuda").to(t)
        return base[offset:offset + n * (width + extra)].view(n, -1)[:, :width]
    rows, dout = strided(72), strided(96)
    for kind, got, a, b in (("out", ar.expert_matmul(rows, w, plan), rows, w),
                            ("drows", ar.expert_matmul_drows(dout, w, plan), dout, w),
                            ("dweights", ar.expert_matmul_dweights(dout, rows, plan), dout, rows)):
        y, tol = ref.product(kind, plan.offsets, a, b)
        ref.close(got, y, tol, kind)


@pytest.mark.parametrize("t", [BF, F32])
def test_infinities_stay_in_their_rows(t):
    plan, n = plan_of((30, 40))
    rows, w = torch.ones((n, 80), device="cuda").to(t), torch.ones((2, 50, 80), device="cuda").to(t)
    rows[3, 7], rows[35, 79], rows[36, 0] = torch.inf, torch.nan, -torch.inf
    y, tol = ref.product("out", plan.offsets, rows, w)
    ref.close(ar.expert_matmul(rows, w, plan), y, tol)
    dout = torch.ones((n, 50), device="cuda").to(t)
    y, tol = ref.product("dweights", plan.offsets, dout, rows)
    ref.close(ar.expert_matmul_dweights(dout, rows, plan), y, tol)


def test_offsets_outside_the_rows():
    """Offsets past the rows, or an end before its beginning, count as the rows' end
    and as no rows."""
    rows, w = torch.randn((50, 24), device="cuda"), torch.randn((4, 16, 24), device="cuda")
    dout = torch.randn((50, 16), device="cuda")
    at = torch.arange(50, dtype=torch.int32, device="cuda")
    for off in ([0, 20, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 7, 7, 30, 40],
                [50, 50, 50, 50, 50], [0, 30, 20, 50, 50]):
        plan = ar.ExpertPlan(at.view(-1, 1), at, torch.tensor(off, dtype=torch.int32, device="cuda"))
        y, tol = ref.product("dweights", plan.offsets, dout, rows)
        ref.close(ar.expert_matmul_dweights(dout, rows, plan), y, tol)
        if off[1] > off[2]:
            ar.expert_matmul(rows, w, plan)       # (rows that two experts claim: either's)
            continue
        y, tol = ref.product("out", plan.offsets, rows, w)
        ref.close(ar.expert_matmul(rows, w, plan), y, tol)


def test_no_rows():
    plan, _ = plan_of((0, 0, 0))
    rows, dout = torch.empty((0, 40), device="cuda"), torch.empty((0, 24), device="cuda")
    w = torch.randn((3, 24, 40), device="cuda")
    assert ar.expert_matmul(rows, w, plan).shape == (0, 24)
    assert ar.expert_matmul_drows(dout, w, plan).shape == (0, 40)
    d = ar.expert_matmul_dweights(dout, rows, plan)
    assert d.shape == (3, 24, 40) and not d.any()
