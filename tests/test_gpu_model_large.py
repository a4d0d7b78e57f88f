"""The embedding, the experts' products and the gated activation past the sizes
where a 32-bit offset or one grid of blocks ends.  What is far apart is
compared bit for bit: rows are copied or repeated, and sums are of small whole
numbers, exact in binary32 in whatever order."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def poison(shape, t):
    """Leaves the allocator a block of this size without zeros for the next output."""
    torch.cuda.empty_cache()
    torch.full(shape, torch.nan, dtype=t, device="cuda")


def whole(*shape, t=BF, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(t)


# ------------------------------------------------------------------------- embedding

# a table past 2^32 bytes, one past 2^32 elements and past the 2^35 bytes that a grid clears
@pytest.mark.parametrize("t,vocab,hidden", [(BF, 600011, 4096), (F32, 600011, 2049),
                                            (BF, 2 ** 22 + 5, 4096)])
def test_far_rows_of_a_table(t, vocab, hidden):
    at = torch.tensor([0, 1, 7, vocab // 2, vocab // 2 + 1, vocab - 300, vocab - 2, vocab - 1])
    for dtype in (torch.int32, torch.int64):
        ids = torch.cat([at, torch.tensor([-1, vocab])]).to(dtype).cuda()
        rows = torch.randn((8, hidden), device="cuda").to(t)
        table = torch.zeros((vocab, hidden), dtype=t, device="cuda")
        table[at.cuda()] = rows
        y = ar.embedding(table, ids)
        assert torch.equal(y[:8], rows) and not y[8:].any()
        del table
        poison((vocab, hidden), t)
        dtable = ar.embedding_backward(torch.cat([rows, rows[:2]]), ids, vocab)
        assert torch.equal(dtable[at.cuda()], rows)
        dtable[at.cuda()] = 0.0
        for part in dtable.split(1 << 17):
            assert not part.any()
        del dtable, part


@pytest.mark.parametrize("t,tokens,hidden", [(BF, 2 ** 21 + 77, 2048), (BF, 2 ** 27 + 1001, 3),
                                             (F32, 2 ** 27 + 1001, 4)])
def test_more_tokens_than_a_grid(t, tokens, hidden):
    table = torch.randn((4099, hidden), device="cuda").to(t)
    ids = torch.arange(tokens, dtype=torch.int32, device="cuda").remainder_(4100)    # (4099: none)
    y = ar.embedding(table, ids)
    table = torch.cat([table, table.new_zeros((1, hidden))])
    for part, at in zip(y.split(1 << 22), ids.split(1 << 22)):
        assert torch.equal(part, table[at.long()])


def test_gradient_of_more_tokens_than_a_grid():
    """2^21 pieces and more, one id with a sixteenth of the tokens."""
    tokens, vocab = 2 ** 27 + 1001, 70001
    g = torch.Generator("cuda").manual_seed(2)
    ids = torch.randint(-1, vocab + 1, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    ids[5::16] = 40000
    dy = whole(tokens, 4, t=F32, seed=3)
    got = ar.embedding_backward(dy, ids, vocab)
    want = torch.zeros((vocab, 4), device="cuda")
    for i, d in zip(ids.split(1 << 24), dy.split(1 << 24)):
        often = i == 40000
        want[40000] += d[often].sum(0)
        rest = (i >= 0) & (i < vocab) & ~often
        want.index_add_(0, i[rest].long(), d[rest])
    assert float(want.abs().max()) < 2 ** 23
    assert torch.equal(got, want)


# --------------------------------------------------------------- the experts' products

def plan_of(counts, behind=0):
    off = torch.tensor([0, *counts]).cumsum(0).int().cuda()
    at = torch.arange(int(off[-1]) + behind, dtype=torch.int32, device="cuda")
    return ar.ExpertPlan(at.view(-1, 1), at, off)


@pytest.mark.parametrize("t", [BF, F32])
def test_far_experts(t):
    """Weights past 2^32 bytes; rows in the first and the last expert."""
    experts, hidden, out = 1024, 2048, 1100
    plan = plan_of([3, *[0] * (experts - 2), 40], 2)
    w = whole(experts, out, hidden, t=t)
    rows, dout = whole(45, hidden, t=t, seed=1), whole(45, out, t=t, seed=2)
    first, last, none = slice(0, 3), slice(3, 43), slice(43, 45)
    got = ar.expert_matmul(rows, w, plan)
    for at, e in ((first, 0), (last, -1)):
        assert torch.equal(got[at], (rows[at].double() @ w[e].double().t().contiguous()).to(t))
    assert not got[none].any()
    got = ar.expert_matmul_drows(dout, w, plan)
    for at, e in ((first, 0), (last, -1)):
        assert torch.equal(got[at], (dout[at].double() @ w[e].double()).to(t))
    assert not got[none].any()
    del w, got
    poison((experts, out, hidden), t)
    got = ar.expert_matmul_dweights(dout, rows, plan)
    for at, e in ((first, 0), (last, -1)):
        assert torch.equal(got[e], (dout[at].double().t().contiguous() @ rows[at].double()).to(t))
    for part in got[1:-1].split(64):
        assert not part.any()


@pytest.mark.parametrize("t,out", [(BF, 2056), (F32, 1032)])
def test_far_rows(t, out):
    """Rows past 2^32 bytes, most of them the second expert's."""
    hidden, counts = 64, (1000, 2 ** 21 - 333, 777)
    plan = plan_of(counts, 2)
    n = plan.slot.numel()
    off = plan.offsets.tolist()
    w = whole(3, out, hidden, t=t)
    rows, dout = whole(n, hidden, t=t, seed=1), whole(n, out, t=t, seed=2)
    y, dx = ar.expert_matmul(rows, w, plan), ar.expert_matmul_drows(dout, w, plan)
    dw = ar.expert_matmul_dweights(dout, rows, plan)
    for e in range(3):
        we, total = w[e].double(), torch.zeros((out, hidden), dtype=torch.float64, device="cuda")
        wt = we.t().contiguous()
        for lo in range(off[e], off[e + 1], 1 << 17):
            at = slice(lo, min(lo + (1 << 17), off[e + 1]))
            assert torch.equal(y[at], (rows[at].double() @ wt).to(t))
            assert torch.equal(dx[at], (dout[at].double() @ we).to(t))
            total += dout[at].double().t().contiguous() @ rows[at].double()
        assert float(total.abs().max()) < 2 ** 23
        assert torch.equal(dw[e], total.to(t))
    assert not y[off[3]:].any() and not dx[off[3]:].any()


# ------------------------------------------------------- checkpoints and the gate

def repeated(base, times):
    return base.repeat(times, *[1] * (base.dim() - 1))


def check_repeats(got, times, what):
    """All rows repeat the first ones, to the bit."""
    got = got.view(torch.uint8).view(times, -1)
    for part in got[1:].split(1 << 12):
        assert bool((part == got[0]).all()), what


# (a thread of the kernels has 8 values: 4 threads a row, and 2^30 of them a grid)
@pytest.mark.parametrize("t,cols", [(BF, 3), (F32, 8)])
def test_gate_of_more_rows_than_a_grid(t, cols):
    n, times = 4099, 65500
    assert 4 * n * times > 2 ** 30
    g = torch.Generator("cuda").manual_seed(cols)
    base = torch.randn((n, 2 * cols), generator=g, device="cuda").to(t)
    d = torch.randn((n, cols), generator=g, device="cuda").to(t)
    acts, saved = ar.silu_gate(repeated(base, times))
    y, tol = ref.gate(base)
    ref.close(acts[:n], y, tol, "acts")
    codes, scales, _ = ref.save(base.view(n, 2, cols))
    assert torch.equal(saved.codes[:n].cpu(), codes) and torch.equal(saved.scales[:n].cpu(), scales)
    for v, what in ((acts, "acts"), (saved.codes, "codes"), (saved.scales, "scales")):
        check_repeats(v, times, what)
    dh, again = ar.silu_gate_backward(repeated(d, times), saved)
    want, tol = ref.gate_backward(d, codes, scales)
    for got, v, b, what in zip((dh, again), want, tol, ("dh", "again")):
        ref.close(got[:n], v, b, what)
        check_repeats(got, times, what)


@pytest.mark.parametrize("t,cols", [(BF, 3), (F32, 8)])
def test_checkpoint_of_more_rows_than_a_grid(t, cols):
    n, times = 4099, 65500
    base = torch.randn((n, cols), device="cuda").to(t)
    saved = ar.save_8bit(repeated(base, times))
    codes, scales, values = ref.save(base)
    assert torch.equal(saved.codes[:n].cpu(), codes) and torch.equal(saved.scales[:n].cpu(), scales)
    back = ar.restore_8bit(saved, t)
    ref.close(back[:n], values, 0.0)
    for v, what in ((saved.codes, "codes"), (saved.scales, "scales"), (back, "values")):
        check_repeats(v, times, what)
