"""The training operators in each of their kernels' forms, with more rows than
blocks, against the definitions in 64 bits (tests/operator_refs.py derives the
bounds), and through the C entry points with guard regions around every output
and the scratch."""

import ctypes

import pytest
import torch

import ring_allreduce_rs_amd as ar
from ring_allreduce_rs_amd import _lib
from tests import operator_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def near(got, want, tol, what):
    """ref.close on the GPU: want and its bound may be large."""
    g = got.double()
    odd = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(g), g == want)
    ok = torch.where(odd, same, (g - want).abs() <= tol)
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} off"


# ------------------------------------------------------------------------ layer norm

def norm_case(rows, cols, t, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x = (x * torch.randn((rows, 1), generator=g, device="cuda").mul_(0.3).exp_()
         + 0.5 * torch.randn((rows, 1), generator=g, device="cuda")).to(t)
    w = torch.randn(cols, generator=g, device="cuda") * 0.2 + 1
    b = torch.randn(cols, generator=g, device="cuda") * 0.1
    return x, w, b, (torch.randn((rows, cols), generator=g, device="cuda") * 1e-2).to(t)


# units of 16 bytes in a row: the row kernels' widths (64, 128, 256, 512, 640 and 1024
# threads of one unit, two units, four), each past the rows that get a block of their own
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("ragged", [0, 3])
@pytest.mark.parametrize("units,rows", [(5, 2000), (13, 2000), (30, 2000), (64, 1301), (110, 1301),
                                        (256, 1301), (400, 1301), (512, 1301), (640, 1301),
                                        (900, 1301), (1024, 1301), (1500, 401), (2048, 401),
                                        (4096, 401)])
def test_norm_rows_of_every_width(units, rows, ragged, t):
    cols = units * (8 if t == BF else 4) - ragged
    x, w, b, dy = norm_case(rows, cols, t, units)
    got = ar.layer_norm(x, w, b)
    want, tol = ref.norm(x, w, b, 1e-5)
    for name, v, e, d in zip(("y", "mean", "rstd"), got, want, tol):
        near(v, e, d, name)
    grads = ar.layer_norm_backward(dy, x, got[1], got[2], w)
    want, tol = ref.norm_backward(dy, x, got[1], got[2], w)
    for name, v, e, d in zip(("dx", "dweight", "dbias"), grads, want, tol):
        near(v, e, d, name)


@pytest.mark.parametrize("t,rows,cols", [
    (F32, 2 ** 21 + 77, 3),       # a block a row
    (BF, 2 ** 23 + 301, 264),     # four rows a block
    (BF, 2 ** 28 + 77, 8)])       # 128 rows a block
def test_norm_of_more_rows_than_a_grid(t, rows, cols):
    """The blocks come round to the rows past a grid's."""
    base = torch.randn(4099, cols, device="cuda").to(t)
    x = torch.empty((rows, cols), dtype=t, device="cuda")
    x[:4099], x[-4099:] = base, base
    x[4099:-4099] = 1.0
    w, b = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
    y, mean, rstd = ar.layer_norm(x, w, b)
    want, tol = ref.norm(base, w, b, 1e-5)
    flat = ar.layer_norm(x[5000:5001], w, b)[0]
    for s in (slice(None, 4099), slice(rows - 4099, None)):
        for v, e, d in zip((y[s], mean[s], rstd[s]), want, tol):
            near(v, e, d, "rows")
    assert bool((y[4099:-4099] == flat).all()) and bool((mean[4099:-4099] == 1).all())


# ---------------------------------------------------------------------- distillation

def distill_case(rows, vocab, top, t, seed):
    """Entries left out, rows without any, places named twice."""
    g = torch.Generator("cuda").manual_seed(seed)
    logits = (torch.randn((rows, vocab), generator=g, device="cuda") * 2.5).to(t)
    at = torch.randint(0, vocab, (rows, top), generator=g, device="cuda")
    at[1::3, top // 2:] = at[1::3, :top - top // 2]
    teacher = (logits.gather(1, at).float() * 0.5
               + torch.randn((rows, top), generator=g, device="cuda") * 2 + 4).to(t)
    gone = torch.rand((rows, top), generator=g, device="cuda")
    at = at.masked_fill(gone < 0.05, -1).masked_fill(gone > 0.95, vocab)
    at[torch.rand(rows, generator=g, device="cuda") < 0.1] = -1
    return logits, at, teacher, torch.rand(rows, generator=g, device="cuda") - 0.3


# (rows, row length in units): a block of the row kernel takes two rows and more, the last
# round uneven; 4 units a thread with 64 and 256 threads, 8 with 128, 16 with 256, 512 and
# 1024, these with every place filled and not
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("ragged", [0, 3])
@pytest.mark.parametrize("rows,units", [(7000, 126), (13000, 60), (2047, 1001), (2100, 1001),
                                        (1100, 4000), (1100, 4096), (700, 6253), (300, 16384),
                                        (2600, 4090), (280, 15000)])
def test_distill_rows_one_after_another(rows, units, ragged, t):
    vocab = units * (8 if t == BF else 4) - ragged
    for top, T in ((24, 1.0), (1, 2.0)):
        logits, at, teacher, dloss = distill_case(rows, vocab, top, t, units + top)
        (want, wlse, wd), (tol, tlse, td) = ref.distill(logits, at, teacher, T, dloss)
        loss, d = ar.distill_step(dloss, logits, at, teacher, T)
        near(loss, want, tol, "loss of the step")
        near(d, wd, td, "dlogits of the step")
        loss, lse = ar.distill_loss(logits, at.int(), teacher, T)
        near(loss, want, tol, "loss")
        near(lse, wlse, tlse, "lse")
        (_, _, wd), (_, _, td) = ref.distill(logits, at, teacher, T, dloss, lse)
        near(ar.distill_backward(dloss, logits, at, teacher, lse, T), wd, td, "dlogits")
        del wd, td, d


# ---------------------------------------------------- the C entry points, with guards

class Guards:
    """Arrays between bytes that nothing may write."""
    EDGE, MARK = 4096, 0xA5

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, shift=0):
        size = torch.empty((), dtype=dtype).element_size()
        n = torch.Size(shape).numel() * size
        lo = self.EDGE + shift * size
        buf = torch.full((lo + n + self.EDGE,), self.MARK, dtype=torch.uint8, device="cuda")
        self.all.append((buf, lo, lo + n))
        return buf[lo:lo + n].view(dtype).view(shape)

    def copy(self, t, shift=0):
        v = self(t.shape, t.dtype, shift)
        v.copy_(t)
        return v

    def check(self):
        for buf, lo, hi in self.all:
            assert bool((buf[:lo] == self.MARK).all()) and bool((buf[hi:] == self.MARK).all())


@pytest.fixture()
def ctx():
    c = ar.Context(0, torch.cuda.current_stream().cuda_stream)
    yield c
    c.close()


def ok(ctx, status):
    assert status == _lib.AR_OK, _lib.lib.ar_last_error(ctx.handle)


def p(t):
    return t.data_ptr() if t is not None and t.numel() else None


def scratch(guards, fn, *args):
    n = ctypes.c_size_t()
    assert fn(*args, ctypes.byref(n)) == _lib.AR_OK
    return guards((n.value,), torch.uint8), n.value


def same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.contiguous().view(torch.uint8))


DT = {BF: _lib.DTYPES["bfloat16"], F32: _lib.DTYPES["float32"]}


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (5, 3), (300, 61), (700, 250), (1301, 771),
                                       (1301, 5001), (280, 16384), (130, 16391), (37, 70001)])
def test_norm_between_guards(ctx, rows, cols, t):
    lib = _lib.lib
    x, w, b, dy = norm_case(rows, cols, t, 7)
    want = ar.layer_norm(x, w, b)
    grads = ar.layer_norm_backward(dy, x, want[1], want[2], w)
    for shift in (0, 1):
        g = Guards()
        gx, gdy, gw, gb = (g.copy(v, shift) for v in (x, dy, w, b))
        y, mean, rstd = g(x.shape, t, shift), g((rows,), F32, shift), g((rows,), F32)
        ok(ctx, lib.ar_layer_norm(ctx.handle, p(gx), cols, p(gw), p(gb), DT[F32], p(y), p(mean),
                                  p(rstd), rows, cols, DT[t], 1e-5))
        same((y, mean, rstd), want)
        ws, n = scratch(g, lib.ar_layer_norm_backward_workspace, rows, cols, DT[t])
        for wanted in ((True, True), (True, False), (False, True), (False, False)):
            dx = g(x.shape, t, shift)
            dw, db = (g((cols,), F32, shift) if v else None for v in wanted)
            some = any(wanted)
            ok(ctx, lib.ar_layer_norm_backward(
                ctx.handle, p(gdy), cols, p(gx), cols, p(mean), p(rstd), p(gw), DT[F32], p(dx),
                p(dw), p(db), rows, cols, DT[t], p(ws) if some else None, n if some else 0))
            same([dx] + [v for v in (dw, db) if v is not None],
                 [grads[0]] + [v for v, k in zip(grads[1:], wanted) if k])
        g.check()
        same((gx, gdy, gw, gb), (x, dy, w, b))


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (1, 1, 1, 1), (5, 3, 4, 6), (64, 9, 33, 771), (300, 8, 60, 2048), (2000, 4, 128, 520),
    (1500, 5, 1024, 4100), (3000, 8, 64, 129)])
def test_experts_between_guards(ctx, tokens, topk, experts, hidden, t):
    lib = _lib.lib
    gen = torch.Generator("cuda").manual_seed(hidden)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").to(t)
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=gen, device="cuda")
    w = torch.rand((tokens, topk), generator=gen, device="cuda")
    rows, plan = ar.expert_dispatch(x, ids, experts)
    dy = torch.randn((tokens, hidden), generator=gen, device="cuda").to(t)
    y = ar.expert_combine(rows, w, plan)
    back = ar.expert_combine_backward(dy, rows, w, plan)
    dx = ar.expert_dispatch_backward(back[0], plan)
    for shift in (0, 1):
        g = Guards()
        ws, n = scratch(g, lib.ar_expert_dispatch_workspace, tokens, topk, experts)
        gx, gids, gw, gdy = (g.copy(v, shift) for v in (x, ids, w, dy))
        out = g(rows.shape, t, shift)
        dest, slot, offsets = (g(v.shape, torch.int32, shift) for v in plan)
        ok(ctx, lib.ar_expert_dispatch(ctx.handle, p(gx), hidden, p(gids), 8, tokens, topk, experts,
                                       hidden, DT[t], p(out), p(dest), p(slot), p(offsets), p(ws), n))
        same((out, dest, slot, offsets), (rows, *plan))
        gy, drows, gdx = (g(v.shape, t, shift) for v in (y, back[0], dx))
        dw = g(w.shape, F32, shift)
        sizes = (tokens, topk, experts, hidden, DT[t])
        ok(ctx, lib.ar_expert_combine(ctx.handle, p(out), p(gw), p(dest), p(offsets), *sizes, p(gy)))
        ok(ctx, lib.ar_expert_combine_backward(ctx.handle, p(gdy), hidden, p(out), p(gw), p(dest),
                                               p(offsets), *sizes, p(drows), p(dw)))
        ok(ctx, lib.ar_expert_dispatch_backward(ctx.handle, p(drows), p(dest), p(offsets), *sizes,
                                                p(gdx)))
        same((gy, drows, dw, gdx), (y, *back, dx))
        g.check()
        same((gx, gids, gw, gdy), (x, ids, w, dy))


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab,top", [(3, 5, 2), (700, 1003, 9), (2, 32000, 1024), (7000, 500, 3),
                                            (1100, 9000, 30), (5, 140001, 64), (520, 70001, 5)])
def test_distillation_between_guards(ctx, rows, vocab, top, t):
    lib = _lib.lib
    logits, at, teacher, dloss = distill_case(rows, vocab, top, t, vocab)
    T = 2.0
    first = ar.distill_loss(logits, at, teacher, T)
    back = ar.distill_backward(dloss, logits, at, teacher, first[1], T)
    step = ar.distill_step(dloss, logits, at, teacher, T)
    for shift in (0, 1):
        g = Guards()
        gl, gat, gt, gd = (g.copy(v, shift) for v in (logits, at, teacher, dloss))
        heads = (p(gl), vocab, p(gat), 8, p(gt))
        sizes = (rows, vocab, top, DT[t], T)
        ws, n = scratch(g, lib.ar_distill_workspace, rows, vocab, top, DT[t], 0)
        loss, lse = g((rows,), F32, shift), g((rows,), F32, shift)
        ok(ctx, lib.ar_distill_loss(ctx.handle, *heads, *sizes, p(loss), p(lse), p(ws), n))
        same((loss, lse), first)
        d = g(logits.shape, t, shift)
        ok(ctx, lib.ar_distill_backward(ctx.handle, p(gd), *heads, p(lse), *sizes, p(d)))
        same((d,), (back,))
        ws, n = scratch(g, lib.ar_distill_workspace, rows, vocab, top, DT[t], 1)
        loss, d = g((rows,), F32, shift), g(logits.shape, t, shift)
        ok(ctx, lib.ar_distill_step(ctx.handle, p(gd), *heads, *sizes, p(loss), p(d), p(ws), n))
        same((loss, d), step)
        g.check()
        same((gl, gat, gt, gd), (logits, at, teacher, dloss))
