"""Layer norm forward and backward against the definitions in 64 bits
(tests/operator_refs.py derives the bounds), over widths that meet every
kernel form, odd widths and offsets, strided rows, both parameter types, rows
of one value, far means, non-finite rows, empty batches, other streams and
captured graphs."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import operator_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [1, 2, 7, 8, 63, 64, 130, 511, 512, 771, 1000, 2048, 2049, 4096, 4104, 5001, 8192, 12288,
          16384, 16391, 33000, 70001]


def make(rows, cols, t, p, seed, shift=0.5):
    g = torch.Generator("cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(s, generator=g, device="cuda")
    x = (n(rows, cols) * n(rows, 1).mul(0.3).exp() + shift * n(rows, 1)).to(t)
    return x, (n(cols) * 0.2 + 1).to(p), (n(cols) * 0.1).to(p), (n(rows, cols) * 1e-2).to(t)


def check_forward(x, w, b, eps=1e-5):
    got = ar.layer_norm(x, w, b, eps=eps)
    want, tol = ref.norm(x, w, b, eps)
    assert got[0].dtype == x.dtype and got[0].is_contiguous()
    assert got[1].dtype == got[2].dtype == F32
    for name, g, v, t in zip(("y", "mean", "rstd"), got, want, tol):
        ref.close(g, v, t, name)
    return got


def check_backward(dy, x, mean, rstd, w):
    got = ar.layer_norm_backward(dy, x, mean, rstd, w)
    want, tol = ref.norm_backward(dy, x, mean, rstd, w)
    p = w.dtype if w is not None else x.dtype
    assert got[0].dtype == x.dtype and got[1].dtype == got[2].dtype == p
    ref.close(got[0].reshape(want[0].shape), want[0], tol[0], "dx")
    ref.close(got[1], want[1], tol[1], "dweight")
    ref.close(got[2], want[2], tol[2], "dbias")
    return got


@pytest.mark.parametrize("t,p", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)],
                         ids=["bf16", "bf16-f32", "f32", "f32-bf16"])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 133])
def test_both_directions(rows, cols, t, p):
    x, w, b, dy = make(rows, cols, t, p, rows * 100003 + cols)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(dy, x, mean, rstd, w)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1021, 771), (2500, 96), (700, 4096), (520, 8200),
                                       (4000, 1), (1500, 1024)])
def test_many_rows(rows, cols, t):
    x, w, b, dy = make(rows, cols, t, F32, cols)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(dy, x, mean, rstd, w)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("cols", [64, 1003, 4096, 16391])
@pytest.mark.parametrize("offset,extra", [(1, 0), (3, 5), (8, 8)])
def test_rows_anywhere(cols, offset, extra, t):
    """Rows that start off every 16-byte boundary, at a stride."""
    rows = 37
    base = torch.randn(rows * (cols + extra) + 64, device="cuda").to(t)
    x = base[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    gbase = torch.randn(rows * (cols + extra + 2) + 64, device="cuda").to(t)
    dy = gbase[1:1 + rows * (cols + extra + 2)].view(rows, -1)[:, :cols]
    _, w, b, _ = make(1, cols, t, F32, cols)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(dy, x, mean, rstd, w)
    keep = base.clone()
    ar.layer_norm(x, w, b)
    assert torch.equal(keep, base)


def test_leading_dimensions_and_no_parameters():
    x = torch.randn(3, 4, 5, 96, device="cuda")
    y, mean, rstd = check_forward(x, None, None)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4, 5)
    check_backward(torch.randn_like(x), x, mean, rstd, None)
    w = torch.randn(96, device="cuda")
    check_forward(x, w, None)
    check_forward(x.to(BF), None, w)
    one = torch.randn(4096, device="cuda", dtype=BF)
    y, mean, rstd = check_forward(one, None, None)
    assert mean.shape == ()
    check_backward(torch.randn_like(one), one, mean, rstd, None)


@pytest.mark.parametrize("cols", [64, 771, 4096, 70001])
def test_far_mean_and_flat_rows(cols):
    """A mean thousands of times the spread costs the mean's digits alone; a row
    of one value has rstd 1/sqrt(eps)."""
    x, w, b, dy = make(9, cols, F32, F32, cols)
    x = x * 0.1 + 4096.0
    x[3] = 7.0
    x[4] = 0.0
    y, mean, rstd = check_forward(x, w, b)
    assert torch.equal(y[3], b) and torch.equal(y[4], b)
    check_backward(dy, x, mean, rstd, w)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("cols", [100, 4096, 40000])
def test_non_finite_rows_stay_alone(cols, t):
    x, w, b, dy = make(12, cols, t, t, cols)
    clean = [v.clone() for v in ar.layer_norm(x, w, b)]
    x[2, cols // 2] = float("nan")
    x[5, 0] = float("inf")
    x[7, cols - 1] = -float("inf")
    got = ar.layer_norm(x, w, b)
    bad = torch.tensor([2, 5, 7], device="cuda")
    good = torch.tensor([i for i in range(12) if i not in (2, 5, 7)], device="cuda")
    assert torch.isnan(got[0][bad]).all()
    for g, c in zip(got, clean):
        assert torch.equal(g[good], c[good])
    dx = ar.layer_norm_backward(dy, x, got[1], got[2], w)[0]
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[good]).all()


def test_no_rows():
    x = torch.empty(0, 96, device="cuda", dtype=BF)
    y, mean, rstd = ar.layer_norm(x, torch.ones(96, device="cuda"))
    assert y.shape == (0, 96) and mean.shape == (0,)
    dx, dw, db = ar.layer_norm_backward(x, x, mean, rstd, torch.ones(96, device="cuda"))
    assert dx.shape == (0, 96) and dw.dtype == F32
    assert not dw.any() and not db.any()


def test_gradient_against_differences():
    """dx, dweight and dbias against central differences of sum(y dy) in 64 bits."""
    rows, cols, h = 3, 10, 1e-5
    x, w, b, dy = make(rows, cols, F32, F32, 4)

    def loss(x, w, b):
        return float((ref.norm(x, w, b, 1e-5)[0][0] * dy.double()).sum())
    _, mean, rstd = ar.layer_norm(x, w, b)
    grads = ar.layer_norm_backward(dy, x, mean, rstd, w)
    for which, got in zip(range(3), grads):
        args = [x.double(), w.double(), b.double()]
        want = torch.zeros_like(args[which])
        flat, wf = args[which].view(-1), want.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(*args)
            flat[i] = keep - h
            down = loss(*args)
            flat[i] = keep
            wf[i] = (up - down) / (2 * h)
        # differences: h^2 times the third derivative and rounding / h, both
        # below 1e-8 here; the kernel's own: 40 roundings of values below 1
        ref.close(got, want, 40 * ref.U + 1e-8, f"gradient {which}")


def test_repeats_to_the_bit_on_any_stream():
    x, w, b, dy = make(777, 1000, BF, F32, 5)
    _, mean, rstd = ar.layer_norm(x, w, b)
    first = ar.layer_norm_backward(dy, x, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ar.layer_norm(x, w, b) + ar.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.current_stream().wait_stream(side)
    for a, g in zip(ar.layer_norm(x, w, b) + first, again):
        assert torch.equal(a, g)


def test_captured_graph():
    x, w, b, dy = make(300, 1536, BF, F32, 6)

    def step():
        y, mean, rstd = ar.layer_norm(x, w, b)
        return (y, mean, rstd) + ar.layer_norm_backward(dy, x, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        nx, _, _, ndy = make(300, 1536, BF, F32, 60 + seed)
        x.copy_(nx)
        dy.copy_(ndy)
        graph.replay()
        for g, e in zip(out, step()):
            assert torch.equal(g, e)
        torch.cuda.synchronize()


def test_views_with_even_rows():
    """Leading dimensions that one stride walks, and those that none does."""
    x = torch.randn(6, 40, device="cuda")
    check_forward(x[:, :7], None, None)
    check_forward(x[::2], None, None)
    check_forward(x[1], None, None)
    check_forward(x.view(2, 3, 40)[:, :, 3:9], None, None)
    check_forward(x.view(2, 3, 40)[1:, :, 1:], None, None)
    check_forward(x.view(6, 1, 40)[:, :, :5], None, None)
    check_forward(x[:, :1].t().contiguous().t(), None, None)
    for bad in (x.t(), x[:, ::2], x[:1].expand(6, 40), x.view(2, 3, 40).transpose(0, 1),
                x.as_strided((3, 8), (4, 1)), x.view(2, 3, 40)[:, :2], x[0, 0]):
        with pytest.raises(ValueError):
            ar.layer_norm(bad)


def test_refusals():
    x = torch.randn(4, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    _, mean, rstd = ar.layer_norm(x, w)
    for bad in (lambda: ar.layer_norm(x.half()), lambda: ar.layer_norm(x.cpu()),
                lambda: ar.layer_norm(x.t()), lambda: ar.layer_norm(x[:, ::2]),
                lambda: ar.layer_norm(x, w[:31]), lambda: ar.layer_norm(x, w.cpu()),
                lambda: ar.layer_norm(x, w, w.to(BF)), lambda: ar.layer_norm(x, w.half()),
                lambda: ar.layer_norm(x, eps=-1.0), lambda: ar.layer_norm(x, eps=float("nan")),
                lambda: ar.layer_norm(x[:, :0]), lambda: ar.layer_norm(x[0, 0]),
                lambda: ar.layer_norm(x[:1].expand(4, 32)),
                lambda: ar.layer_norm_backward(x[:3], x, mean, rstd, w),
                lambda: ar.layer_norm_backward(x.to(BF), x, mean, rstd, w),
                lambda: ar.layer_norm_backward(x, x, mean[:3], rstd, w),
                lambda: ar.layer_norm_backward(x, x, mean, rstd.double(), w),
                lambda: ar.layer_norm_backward(x, x, mean, rstd, w[:5])):
        with pytest.raises(ValueError):
            bad()
