"""Checkpoints in 8 bits bit for bit, and the gated activation with its
gradient against 64 bits (tests/model_refs.py derives the bounds)."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 32), (4, 33), (63, 64), (64, 100), (33, 771),
         (1000, 264), (129, 2048), (7, 8200), (4099, 65), (2, 70001)]


def check_save(x):
    saved = ar.save_8bit(x)
    codes, scales, values = ref.save(x)
    assert torch.equal(saved.scales.cpu(), scales)
    assert torch.equal(saved.codes.cpu(), codes)
    for t in (BF, F32):
        ref.close(ar.restore_8bit(saved, t), values, 0.0)
    return saved


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_save(rows, cols, t):
    g = torch.Generator("cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    check_save((x * torch.randn((rows, cols), generator=g, device="cuda").mul(3).exp()).to(t))


@pytest.mark.parametrize("t", [BF, F32])
def test_borders(t):
    """Magnitudes around 127 scales, ties, the largest and smallest numbers, zeros."""
    f = torch.finfo(t)
    tops = [127.0, 127.5, 128.0, 1.984375, 1.9921875, 2.0, 0.5, f.max, f.tiny, f.tiny / 4, 2.0 ** -120,
            254.0 * 2 ** -130, 0.0, -127.0, -f.max, 3e-39, 1e38]
    x = torch.zeros((len(tops), 32))
    for i, top in enumerate(tops):
        x[i] = torch.linspace(-1, 1, 32) * top
        x[i, 3] = top
        x[i, 4:12] = torch.arange(8) * 0.5 * (top / 127)
    check_save(x.to(t).cuda())


@pytest.mark.parametrize("t", [BF, F32])
def test_groups_that_are_not_finite(t):
    x = torch.randn((6, 100), device="cuda").to(t)
    x[0, 0], x[1, 40], x[2, 99], x[3, 31], x[3, 32] = torch.inf, torch.nan, -torch.inf, 1e30, torch.nan
    saved = check_save(x)
    assert saved.scales[0].tolist()[0] == 255 and torch.isnan(ar.restore_8bit(saved)[2, 96:]).all()


def test_shapes_and_strides():
    check_save(torch.randn((2, 3, 4, 70), device="cuda"))
    check_save(torch.randn(45, device="cuda"))
    base = torch.randn(40 * 50 + 64, device="cuda")
    for t in (BF, F32):
        for off, width in ((0, 32), (1, 33), (3, 49)):
            check_save(base.to(t)[off:off + 40 * 50].view(40, 50)[:, :width])
    assert ar.save_8bit(torch.empty((0, 40), device="cuda")).scales.shape == (0, 2)


def check_gate(h, seed=0):
    n = h.shape[-1] // 2
    acts, saved = ar.silu_gate(h)
    y, tol = ref.gate(h)
    ref.close(acts, y, tol, "acts")
    codes, scales, _ = ref.save(h.reshape(*h.shape[:-1], 2, n))
    assert torch.equal(saved.codes.cpu(), codes) and torch.equal(saved.scales.cpu(), scales)
    g = torch.Generator("cuda").manual_seed(seed)
    d = torch.randn((*h.shape[:-1], n), generator=g, device="cuda").to(h.dtype)
    want, tol = ref.gate_backward(d, saved.codes, saved.scales)
    for got, v, b, what in zip(ar.silu_gate_backward(d, saved), want, tol, ("dh", "acts")):
        ref.close(got, v, b, what)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_gate(rows, cols, t):
    g = torch.Generator("cuda").manual_seed(cols)
    check_gate((torch.randn((rows, 2 * cols), generator=g, device="cuda") * 3).to(t), rows)


@pytest.mark.parametrize("t", [BF, F32])
def test_gate_far_out(t):
    """Large and tiny a and u: the sigmoid at 0 and 1."""
    a = torch.tensor([0.0, 1e-30, -1e-30, 20.0, -20.0, 87.0, -87.0, 100.0, -100.0, 1e4, -1e4, 1e30,
                      -1e30, 5e-39])
    u = torch.tensor([0.0, 1.0, -1e-20, 1e5, 3.0])
    h = torch.cat([a.repeat_interleave(5)[None], u.repeat(14)[None]], 1).to(t).cuda()
    check_gate(h)
    h = torch.cat([a[:, None].expand(14, 64), u.repeat(14)[:14, None].expand(14, 64)], 1).to(t).cuda()
    check_gate(h)     # a group of its own for each


def test_gate_infinite():
    h = torch.zeros((2, 2 * 64), device="cuda")
    h[0, 0], h[0, 64:], h[1, 5], h[1, 70] = torch.inf, 2.0, torch.nan, torch.inf
    acts, saved = ar.silu_gate(h)
    assert acts[0, 0] == torch.inf and not acts[0, 1:].any() and torch.isnan(acts[1, 5])
    dh, again = ar.silu_gate_backward(torch.ones((2, 64), device="cuda"), saved)
    # a group that was not finite is NaN in the gradient, the others are not touched
    assert torch.isnan(dh[0, :32]).all() and torch.isfinite(dh[0, 32:64]).all()
    assert torch.isfinite(dh[1, 32:64]).all() and torch.isnan(again[1, :32]).all()


def test_gate_shapes_and_strides():
    check_gate(torch.randn((2, 3, 140), device="cuda"))
    base = torch.randn(40 * 90 + 64, device="cuda")
    for t in (BF, F32):
        for off, width in ((0, 64), (1, 66), (3, 82)):
            check_gate(base.to(t)[off:off + 40 * 90].view(40, 90)[:, :width])


def test_gradient_by_differences():
    """At the checkpoint's values, (f(h + d) - f(h - d)) / 2 in 64 bits."""
    g = torch.Generator().manual_seed(3)
    h = (torch.randn((4, 80), generator=g)).cuda()
    _, saved = ar.silu_gate(h)
    v = ref.values(saved.codes, saved.scales).view(4, 80)
    d = torch.randn((4, 40), generator=g)
    dh, _ = ar.silu_gate_backward(d.cuda(), saved)
    f = lambda z: (z[:, :40] * torch.sigmoid(z[:, :40]) * z[:, 40:] * d.double()).sum()  # noqa: E731
    for i, j in ((0, 0), (1, 39), (2, 40), (3, 79), (0, 17), (2, 66)):
        step = torch.zeros_like(v)
        step[i, j] = 1e-4
        want = (f(v + step) - f(v - step)) / 2e-4
        # the third derivative is below 1, so differences are good to d^2 |u d| and 64 bits' noise
        size = float(d[i, j % 40].abs() * (1 + v[i, (j + 40) % 80].abs() + v[i, j].abs()))
        assert abs(float(dh[i, j]) - float(want)) <= size * (1e-8 + 2.0 ** -18) + 1e-10
