"""Distillation from a teacher's top logits: loss, lse and gradient against
the definitions in 64 bits (tests/operator_refs.py derives the bounds), over
vocabularies that meet every kernel form, entries left out, places named
twice, masked vocabularies, rows without a teacher and non-finite logits."""

import math

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import operator_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def make(rows, vocab, top, t, seed, index=torch.int64, pad=0.1):
    g = torch.Generator("cuda").manual_seed(seed)
    logits = (torch.randn((rows, vocab), generator=g, device="cuda") * 2.5).to(t)
    at = torch.randint(0, vocab, (rows, top), generator=g, device="cuda")
    teacher = (logits.gather(1, at).float() * 0.5
               + torch.randn((rows, top), generator=g, device="cuda") * 2 + 4).to(t)
    gone = torch.rand((rows, top), generator=g, device="cuda")
    at = at.masked_fill(gone < pad / 2, -1).masked_fill(gone > 1 - pad / 2, vocab)
    at[torch.rand(rows, generator=g, device="cuda") < pad] = -1
    dloss = torch.rand(rows, generator=g, device="cuda") - 0.3
    return logits, at.to(index), teacher, dloss


def check(logits, at, teacher, dloss, temperature):
    loss, lse = ar.distill_loss(logits, at, teacher, temperature)
    (want, wlse, _), (tol, tlse, _) = ref.distill(logits, at, teacher, temperature, dloss)
    ref.close(loss, want, tol, "loss")
    ref.close(lse, wlse, tlse, "lse")
    d = ar.distill_backward(dloss, logits, at, teacher, lse, temperature)
    (_, _, wd), (_, _, td) = ref.distill(logits, at, teacher, temperature, dloss, lse)
    assert d.dtype == logits.dtype and d.is_contiguous()
    ref.close(d, wd, td, "dlogits")
    loss2, d2 = ar.distill_step(dloss, logits, at, teacher, temperature)
    (_, _, wd), (_, _, td) = ref.distill(logits, at, teacher, temperature, dloss)
    ref.close(loss2, want, tol, "loss of the step")
    ref.close(d2, wd, td, "dlogits of the step")
    return loss, lse, d


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 100, 1), (4, 1000, 64), (1, 2049, 1024), (9, 4096, 16),
    (2, 8191, 33), (33, 20001, 100), (1, 32000, 16), (8, 32000, 16), (700, 1003, 8),
    (3, 50021, 100), (1, 131072, 64), (5, 131072, 256), (2, 131073, 64), (3, 65544, 64),
    (2, 200000, 32), (300, 40000, 5)])
def test_loss_and_gradient(rows, vocab, top, t):
    for index, temperature in ((torch.int64, 1.0), (torch.int32, 2.0)):
        check(*make(rows, vocab, top, t, rows + vocab + top, index), temperature)


@pytest.mark.parametrize("temperature", [0.37, 0.7, 3.0, 20.0])
@pytest.mark.parametrize("t", [BF, F32])
def test_temperatures(t, temperature):
    check(*make(6, 9001, 40, t, 3), temperature)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("vocab,offset,extra", [(1001, 1, 6), (32000, 3, 0), (50021, 7, 11)])
def test_rows_anywhere(vocab, offset, extra, t):
    rows = 13
    logits, at, teacher, dloss = make(rows, vocab, 20, t, vocab)
    base = torch.zeros(rows * (vocab + extra) + 64, device="cuda", dtype=t)
    view = base[offset:offset + rows * (vocab + extra)].view(rows, -1)[:, :vocab]
    view.copy_(logits)
    check(view, at, teacher, dloss, 1.0)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("vocab", [100, 32000, 140001])
def test_places_named_twice(vocab, t):
    logits, at, teacher, dloss = make(6, vocab, 48, t, 12, pad=0.0)
    at[:, 24:] = at[:, :24]
    at[1] = 5
    at[2, 10:] = vocab - 1
    check(logits, at, teacher, dloss, 2.0)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(4, 501), (7, 32000), (300, 9000), (2, 140001)])
def test_masked_logits_and_rows_without_a_teacher(rows, vocab, t):
    logits, at, teacher, dloss = make(rows, vocab, 24, t, 7)
    # half of the vocabulary is masked, by -inf and by the type's lowest value
    picked = torch.zeros((rows, vocab + 1), dtype=torch.bool, device="cuda")
    picked.scatter_(1, torch.where((at < 0) | (at > vocab), torch.full_like(at, vocab), at), True)
    mask = (torch.arange(vocab, device="cuda") % 2 == 0) & ~picked[:, :vocab]
    logits.masked_fill_(mask, -math.inf)
    logits[:, -1] = torch.finfo(t).min
    at[0] = -1
    teacher[0] = math.nan          # left out: never looked at
    teacher[1, 3:] = -math.inf     # entries without weight
    teacher[1, 0] = torch.finfo(t).min
    at[1, 0] = 1
    loss, _, d = check(logits, at, teacher, dloss, 1.0)
    assert loss[0] == 0 and not d[0].any()
    teacher[:] = -math.inf
    loss, lse = ar.distill_loss(logits, at, teacher)
    assert not loss.any()
    assert not ar.distill_backward(dloss, logits, at, teacher, lse).any()
    loss, d = ar.distill_step(dloss, logits, at, teacher)
    assert not loss.any() and not d.any()
    # a row without a teacher has gradient 0 whatever its logits hold
    at[:] = -1
    logits[:, 2] = math.nan
    logits[:, 3] = math.inf
    loss, lse = ar.distill_loss(logits, at, teacher)
    assert not loss.any() and torch.isnan(lse).all()
    assert not ar.distill_backward(dloss, logits, at, teacher, lse).any()
    loss, d = ar.distill_step(dloss, logits, at, teacher)
    assert not loss.any() and not d.any()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("vocab", [300, 32000, 131072, 150001])
def test_non_finite_rows_stay_alone(vocab, t):
    logits, at, teacher, dloss = make(7, vocab, 12, t, 8, pad=0.0)
    clean_loss, clean_d = ar.distill_step(dloss, logits, at, teacher)
    clean_b = ar.distill_backward(dloss, logits, at, teacher,
                                  ar.distill_loss(logits, at, teacher)[1])
    logits[1, vocab // 3] = math.nan
    logits[4, vocab - 1] = math.inf
    good = torch.tensor([0, 2, 3, 5, 6], device="cuda")
    loss, d = ar.distill_step(dloss, logits, at, teacher)
    assert not torch.isfinite(loss[[1, 4]]).any() and torch.isnan(d[1]).all()
    assert torch.equal(loss[good], clean_loss[good]) and torch.equal(d[good], clean_d[good])
    loss, lse = ar.distill_loss(logits, at, teacher)
    assert torch.isnan(lse[1]) and lse[4] == math.inf
    b = ar.distill_backward(dloss, logits, at, teacher, lse)
    assert torch.equal(b[good], clean_b[good]) and torch.isnan(b[1]).all()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(3, 5), (3, 700), (2, 32000), (600, 4099), (2, 140001)])
def test_rows_of_the_lowest_value(rows, vocab, t):
    """Every logit of a row masked by the type's lowest value: all are equal, so
    both softmaxes are uniform."""
    logits, at, teacher, dloss = make(rows, vocab, 4, t, 3, pad=0.0)
    at = torch.arange(4, device="cuda").expand(rows, 4).contiguous()
    logits[1] = torch.finfo(t).min
    teacher[1] = torch.finfo(t).min
    check(logits, at, teacher, dloss, 1.0)
    loss, d = ar.distill_step(dloss, logits, at, teacher, 2.0)
    # log(vocab / 4): four logarithms and exponentials of 0, the sum's additions
    bound = (ref.depth(vocab) + 16) * 4 * ref.U * (1 + math.log(vocab))
    assert abs(float(loss[1]) - 4 * math.log(vocab / 4)) <= 4 * bound
    q = torch.full((vocab,), 1 / vocab, dtype=torch.float64, device="cuda")
    q[:4] -= 0.25
    want = q * dloss[1].double() * 2
    ref.close(d[1], want, want.abs() * (bound + ref.half_step(t)) + bound / vocab * want.abs().max())


def test_a_row_of_minus_infinity():
    logits, at, teacher, dloss = make(3, 5000, 8, F32, 9, pad=0.0)
    logits[1] = -math.inf
    loss, lse = ar.distill_loss(logits, at, teacher)
    assert lse[1] == -math.inf and torch.isfinite(loss[[0, 2]]).all()


def test_no_rows():
    for t in (BF, F32):
        logits, at, teacher, dloss = (v[:0] for v in make(2, 99, 4, t, 1))
        loss, lse = ar.distill_loss(logits, at, teacher)
        assert loss.shape == lse.shape == (0,)
        assert ar.distill_backward(dloss, logits, at, teacher, lse).shape == (0, 99)
        assert ar.distill_step(dloss, logits, at, teacher)[1].shape == (0, 99)


def test_past_four_gigabytes():
    rows, vocab, top = 34000, 65536, 4
    logits = torch.zeros((rows, vocab), dtype=BF, device="cuda")
    part, at, teacher, dloss = make(8, vocab, top, BF, 2, pad=0.0)
    logits[-8:] = part
    at_all = torch.full((rows, top), -1, dtype=torch.int64, device="cuda")
    at_all[-8:] = at
    teacher_all = torch.zeros((rows, top), dtype=BF, device="cuda")
    teacher_all[-8:] = teacher
    g = torch.zeros(rows, device="cuda")
    g[-8:] = dloss
    (want, wlse, wd), (tol, tlse, td) = ref.distill(part, at, teacher, 1.0, dloss)
    loss, d = ar.distill_step(g, logits, at_all, teacher_all)
    ref.close(loss[-8:], want, tol)
    ref.close(d[-8:], wd, td)
    assert not loss[:-8].any() and not bool(d[rows // 2].any())
    loss, lse = ar.distill_loss(logits, at_all, teacher_all)
    ref.close(lse[-8:], wlse, tlse)
    d.fill_(7.0)
    d = ar.distill_backward(g, logits, at_all, teacher_all, lse)
    (_, _, wd), (_, _, td) = ref.distill(part, at, teacher, 1.0, dloss, lse[-8:])
    ref.close(d[-8:], wd, td)


def test_gradient_against_differences():
    rows, vocab, top, T, h = 2, 9, 4, 2.0, 1e-5
    logits, at, teacher, dloss = make(rows, vocab, top, F32, 5, pad=0.0)
    at[1, 2] = -1
    at[1, 3] = at[1, 0]
    z = logits.double()

    def loss():
        return float((ref.distill(z, at, teacher, T)[0][0] * dloss.double()).sum())
    want = torch.zeros_like(z)
    for i in range(z.numel()):
        keep = z.view(-1)[i].item()
        z.view(-1)[i] = keep + h
        up = loss()
        z.view(-1)[i] = keep - h
        down = loss()
        z.view(-1)[i] = keep
        want.view(-1)[i] = (up - down) / (2 * h)
    lse = ar.distill_loss(logits, at, teacher, T)[1]
    # the differences are good to 1e-8; q - p takes fewer than 64 roundings of
    # values below 2 (the exponent's argument below 16 included)
    for got in (ar.distill_backward(dloss, logits, at, teacher, lse, T),
                ar.distill_step(dloss, logits, at, teacher, T)[1]):
        ref.close(got, want, 64 * 2 * ref.U + 1e-8)


@pytest.mark.parametrize("rows,vocab", [(5, 40000), (400, 9000), (2, 140001)])
def test_captured_graph_and_other_stream(rows, vocab):
    logits, at, teacher, dloss = make(rows, vocab, 30, BF, 4)

    def step():
        loss, lse = ar.distill_loss(logits, at, teacher, 2.0)
        return (loss, lse, ar.distill_backward(dloss, logits, at, teacher, lse, 2.0),
                *ar.distill_step(dloss, logits, at, teacher, 2.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(other, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        for old, new in zip((logits, at, teacher, dloss), make(rows, vocab, 30, BF, 40 + seed)):
            old.copy_(new)
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_refusals():
    logits, at, teacher, dloss = make(4, 100, 5, F32, 1)
    lse = torch.zeros(4, device="cuda")
    big = torch.zeros((4, 1025), dtype=torch.int64, device="cuda")
    for bad in (lambda: ar.distill_loss(logits.half(), at, teacher),
                lambda: ar.distill_loss(logits.cpu(), at, teacher),
                lambda: ar.distill_loss(logits[0], at, teacher),
                lambda: ar.distill_loss(logits, at[:3], teacher),
                lambda: ar.distill_loss(logits, at.float(), teacher),
                lambda: ar.distill_loss(logits, at, teacher[:, :4]),
                lambda: ar.distill_loss(logits, at, teacher.to(BF)),
                lambda: ar.distill_loss(logits, at.cpu(), teacher),
                lambda: ar.distill_loss(logits, at, teacher, 0.0),
                lambda: ar.distill_loss(logits, at, teacher, -1.0),
                lambda: ar.distill_loss(logits, at, teacher, math.nan),
                lambda: ar.distill_loss(logits, at, teacher, math.inf),
                lambda: ar.distill_loss(logits[:, :0], at, teacher),
                lambda: ar.distill_loss(logits, at[:, :0], teacher[:, :0]),
                lambda: ar.distill_loss(logits, big, big.float()),
                lambda: ar.distill_loss(logits.t().contiguous().t(), at, teacher),
                lambda: ar.distill_backward(dloss[:3], logits, at, teacher, lse),
                lambda: ar.distill_backward(dloss, logits, at, teacher, lse.double()),
                lambda: ar.distill_step(dloss.to(BF), logits, at, teacher)):
        with pytest.raises(ValueError):
            bad()
