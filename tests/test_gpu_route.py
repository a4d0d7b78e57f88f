"""Tokens sorted by expert and back: the sort and the rows bit for bit against
a stable sort on the host, the sums and gradients against 64 bits
(tests/operator_refs.py derives the bounds)."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import operator_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


def choices(tokens, topk, experts, seed, pad=0.1, dtype=I64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, topk), generator=g)
    gone = torch.rand((tokens, topk), generator=g)
    ids[gone < pad / 2] = -1
    ids[gone > 1 - pad / 2] = experts            # past the last expert: none either
    return ids.to(dtype).cuda()


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def check_dispatch(x, ids, experts):
    rows, plan = ar.expert_dispatch(x, ids, experts)
    dest, slot, offsets = ref.plan(ids, experts)
    assert torch.equal(plan.dest.cpu(), dest)
    assert torch.equal(plan.slot.cpu(), slot)
    assert torch.equal(plan.offsets.cpu(), offsets)
    live = int(offsets[-1])
    want = x[slot.long().cuda() // ids.shape[1]]
    want[live:] = 0
    assert rows.is_contiguous() and torch.equal(bits(rows), bits(want.contiguous()))
    return rows, plan


def check_back(plan, hidden, t, seed):
    tokens, topk = plan.dest.shape
    live = int(plan.offsets[-1])
    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn((tokens * topk, hidden), generator=g, device="cuda").to(t)
    weights = torch.rand((tokens, topk), generator=g, device="cuda")
    dy = torch.randn((tokens, hidden), generator=g, device="cuda").to(t)
    # what the rows and weights without an expert hold does not matter
    rows[live:] = float("nan")
    weights[plan.dest >= live] = float("nan")
    y, ty = ref.combine(rows, weights, plan.dest, live)
    ref.close(ar.expert_combine(rows, weights, plan), y, ty, "y")
    ones = torch.ones_like(weights)
    dx, tdx = ref.combine(rows, ones, plan.dest, live)
    ref.close(ar.expert_dispatch_backward(rows, plan), dx, tdx, "dx")
    (drows, dw), (tdrows, tdw) = ref.combine_backward(dy, rows, weights, plan.dest, live)
    got = ar.expert_combine_backward(dy, rows, weights, plan)
    ref.close(got[0], drows, tdrows, "drows")
    ref.close(got[1], dw, tdw, "dweights")


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (1, 1, 1, 1), (1, 8, 64, 2048), (2, 3, 5, 7), (4, 8, 64, 2048), (5, 2, 4, 8), (63, 1, 2, 64),
    (64, 9, 33, 100), (129, 6, 60, 1000), (257, 8, 255, 511), (1000, 2, 256, 520),
    (1500, 5, 1024, 136), (2049, 4, 7, 96), (700, 17, 300, 2056), (3000, 8, 128, 264)])
def test_there_and_back(tokens, topk, experts, hidden, t):
    seed = tokens * 31 + topk
    x = torch.randn((tokens, hidden), device="cuda").to(t)
    for dtype in (I64, I32):
        ids = choices(tokens, topk, experts, seed, dtype=dtype)
        _, plan = check_dispatch(x, ids, experts)
    check_back(plan, hidden, t, seed)


@pytest.mark.parametrize("tokens,topk", [(1, 1), (300, 4), (5000, 8)])
def test_one_expert_takes_all_or_none(tokens, topk):
    x = torch.randn((tokens, 24), device="cuda", dtype=F32)
    for value, experts in ((0, 1), (6, 7), (3, 7), (-1, 7), (7, 7), (2 ** 40 + 3, 7), (-2 ** 62, 7)):
        ids = torch.full((tokens, topk), value, dtype=I64, device="cuda")
        _, plan = check_dispatch(x, ids, experts)
        check_back(plan, 24, F32, 1)


@pytest.mark.parametrize("slots", [4096, 1448 * 8, 20000, 40000 * 8, 70001 * 5])
def test_many_slots(slots):
    """More slots than one round of the sort's blocks takes."""
    topk = 8 if slots % 8 == 0 else 5
    ids = choices(slots // topk, topk, 130, 3, dtype=I32)
    x = torch.randn((slots // topk, 12), device="cuda").to(BF)
    check_dispatch(x, ids, 130)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("hidden,offset,extra", [(64, 1, 0), (1001, 3, 6), (2048, 5, 8)])
def test_rows_anywhere(hidden, offset, extra, t):
    tokens = 45
    base = torch.randn(tokens * (hidden + extra) + 64, device="cuda").to(t)
    x = base[offset:offset + tokens * (hidden + extra)].view(tokens, -1)[:, :hidden]
    ids = choices(tokens, 3, 9, 11)
    rows, plan = check_dispatch(x, ids, 9)
    w = torch.rand((tokens, 3), device="cuda")
    live = int(plan.offsets[-1])
    want, tol = ref.combine_backward(x, rows, w, plan.dest, live)
    for got, v, b in zip(ar.expert_combine_backward(x, rows, w, plan), want, tol):
        ref.close(got, v, b)


def test_values_pass_through_untouched():
    """The way there copies bits: NaN payloads, infinities, -0."""
    pat = torch.tensor([0x7fc1, 0x7f81, 0xffc0 - 65536, 0x7f80, 0xff80 - 65536, 0x8000 - 65536, 1],
                       dtype=torch.int16, device="cuda")
    x = pat.repeat(20)[:21 * 6].view(-1, 6).contiguous().view(BF)
    ids = choices(x.shape[0], 2, 4, 2)
    check_dispatch(x, ids, 4)


def test_no_tokens():
    x = torch.empty((0, 16), device="cuda", dtype=BF)
    rows, plan = ar.expert_dispatch(x, torch.empty((0, 2), dtype=I64, device="cuda"), 5)
    assert rows.shape == (0, 16) and not plan.offsets.any()
    w = torch.empty((0, 2), device="cuda")
    assert ar.expert_combine(rows, w, plan).shape == (0, 16)
    assert ar.expert_dispatch_backward(rows, plan).shape == (0, 16)
    drows, dw = ar.expert_combine_backward(x, rows, w, plan)
    assert drows.shape == (0, 16) and dw.shape == (0, 2)


def test_plans_that_point_elsewhere_count_for_nothing():
    """A dest outside the rows, or an end past them, is never an address."""
    tokens, topk, hidden = 40, 4, 72
    ids = choices(tokens, topk, 6, 5)
    _, plan = ar.expert_dispatch(torch.randn((tokens, hidden), device="cuda"), ids, 6)
    dest, offsets = plan.dest.clone(), plan.offsets.clone()
    dest[3, 1], dest[7, 0], dest[9, 2], dest[11, 3] = -1, tokens * topk, 2 ** 31 - 1, -2 ** 31
    live = int(offsets[-1])
    rows = torch.randn((tokens * topk, hidden), device="cuda")
    w = torch.rand((tokens, topk), device="cuda")
    bad = ar.ExpertPlan(dest, plan.slot, offsets)
    y, tol = ref.combine(rows, w, dest, live)
    ref.close(ar.expert_combine(rows, w, bad), y, tol)
    got = ar.expert_combine_backward(torch.randn((tokens, hidden), device="cuda"), rows, w, bad)
    assert got[1][3, 1] == got[1][7, 0] == got[1][9, 2] == got[1][11, 3] == 0
    offsets[-1] = 2 ** 31 - 1
    y, tol = ref.combine(rows, w, dest, tokens * topk)
    ref.close(ar.expert_combine(rows, w, bad), y, tol)


def test_rows_past_four_gigabytes():
    tokens, topk, hidden = 2100, 8, 131072
    x = torch.randn((tokens, 1), device="cuda").to(BF).expand(tokens, hidden).contiguous()
    ids = choices(tokens, topk, 16, 8, pad=0.0)
    rows, plan = ar.expert_dispatch(x, ids, 16)
    want = x[:, 0][plan.slot.long() // topk]
    for at in (0, 1, 65536, hidden - 1):
        assert torch.equal(rows[:, at], want)
    w = torch.rand((tokens, topk), device="cuda")
    y, tol = ref.combine(rows[:, -1:], w, plan.dest, tokens * topk)
    ref.close(ar.expert_combine(rows, w, plan)[:, -1:], y, tol)


def test_gradients_against_differences():
    """Through there, an elementwise square and back, in 64 bits."""
    tokens, topk, hidden, experts, h = 5, 3, 4, 4, 1e-5
    ids = choices(tokens, topk, experts, 9, pad=0.4)
    x = torch.randn((tokens, hidden), device="cuda")
    w = torch.rand((tokens, topk), device="cuda")
    dy = torch.randn((tokens, hidden), device="cuda")
    rows, plan = ar.expert_dispatch(x, ids, experts)
    drows, dw = ar.expert_combine_backward(dy, rows.square(), w, plan)
    dx = ar.expert_dispatch_backward(drows * 2 * rows, plan)
    dest, slot, offsets = (v.cuda() for v in ref.plan(ids, experts))

    def loss(x, w):
        r = x[slot.long() // topk].square()
        ok = dest < offsets[-1]
        return float((torch.where(ok, w, 0.0)[:, :, None] * r[dest.long()]).sum(1)
                     .mul(dy.double()).sum())
    for which, got in ((0, dx), (1, dw)):
        args = [x.double(), w.double()]
        flat = args[which].view(-1)
        want = torch.zeros_like(args[which])
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(*args)
            flat[i] = keep - h
            down = loss(*args)
            flat[i] = keep
            want.view(-1)[i] = (up - down) / (2 * h)
        # the loss is of second degree: no truncation, rounding / h below 1e-8;
        # the kernels: fewer than 16 roundings of values below 64
        ref.close(got, want, 16 * 64 * ref.U + 1e-8)


def test_captured_graph_and_other_stream():
    tokens, topk, hidden, experts = 900, 4, 320, 24
    x = torch.randn((tokens, hidden), device="cuda").to(BF)
    ids = choices(tokens, topk, experts, 1)
    w = torch.rand((tokens, topk), device="cuda")

    def step():
        rows, plan = ar.expert_dispatch(x, ids, experts)
        y = ar.expert_combine(rows, w, plan)
        drows, dw = ar.expert_combine_backward(y, rows, w, plan)
        return (rows, *plan, y, drows, dw, ar.expert_dispatch_backward(drows, plan))
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
        ids.copy_(choices(tokens, topk, experts, 70 + seed))
        x.copy_(torch.randn((tokens, hidden), device="cuda"))
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_refusals():
    x = torch.randn(6, 16, device="cuda")
    ids = torch.zeros((6, 2), dtype=I64, device="cuda")
    rows, plan = ar.expert_dispatch(x, ids, 3)
    w = torch.rand(6, 2, device="cuda")
    for bad in (lambda: ar.expert_dispatch(x.half(), ids, 3),
                lambda: ar.expert_dispatch(x.cpu(), ids, 3),
                lambda: ar.expert_dispatch(x[0], ids, 3),
                lambda: ar.expert_dispatch(x, ids[:5], 3),
                lambda: ar.expert_dispatch(x, ids.to(torch.int16), 3),
                lambda: ar.expert_dispatch(x, ids.cpu(), 3),
                lambda: ar.expert_dispatch(x, ids.t().contiguous().t(), 3),
                lambda: ar.expert_dispatch(x, ids, 0),
                lambda: ar.expert_dispatch(x, ids, 1025),
                lambda: ar.expert_dispatch(x, ids[:, :0], 3),
                lambda: ar.expert_combine(rows[:11], w, plan),
                lambda: ar.expert_combine(rows, w.to(BF), plan),
                lambda: ar.expert_combine(rows, w[:, :1], plan),
                lambda: ar.expert_combine(rows, w, plan._replace(dest=plan.dest.long())),
                lambda: ar.expert_combine(rows, w, plan._replace(offsets=plan.offsets.cpu())),
                lambda: ar.expert_combine(rows.t().contiguous().t(), w, plan),
                lambda: ar.expert_dispatch_backward(rows.cpu(), plan),
                lambda: ar.expert_combine_backward(x[:5], rows, w, plan),
                lambda: ar.expert_combine_backward(x.to(BF), rows, w, plan)):
        with pytest.raises(ValueError):
            bad()
