"""The embedding, the experts' products and the gated activation through their C
entry points with guard regions around every output and the scratch, on another
stream, captured into graphs and replayed between eager calls, with scratch that
holds anything, and what the torch binding refuses of tensors on the GPU."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from ring_allreduce_rs_amd import _lib
from tests import model_refs as ref
from tests.test_gpu_operator_forms import BF, DT, F32, Guards, ctx, ok, p, same, scratch  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


# ---------------------------------------------------- the C entry points, with guards

@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("tokens,vocab,hidden,ib", [
    (1, 1, 1, 8), (16, 300, 7, 4), (17, 5, 64, 8), (700, 90, 771, 4), (5000, 20011, 40, 8),
    (33000, 40, 17, 4), (70000, 70001, 24, 8)])
def test_embedding_between_guards(ctx, tokens, vocab, hidden, ib, t):  # noqa: F811
    lib = _lib.lib
    table, dy = randn(vocab, hidden).to(t), randn(tokens, hidden, seed=1).to(t)
    ids = torch.randint(-1, vocab + 1, (tokens,), device="cuda",
                        dtype=torch.int64 if ib == 8 else torch.int32)
    want, back = ar.embedding(table, ids, 0.5), ar.embedding_backward(dy, ids, vocab, 0.5)
    for shift in (0, 1):
        g = Guards()
        gt, gd, gi = g.copy(table, shift), g.copy(dy, shift), g.copy(ids, shift)
        y, d = g(want.shape, t, shift), g(back.shape, t, shift)
        ok(ctx, lib.ar_embedding(ctx.handle, p(gt), p(gi), ib, tokens, vocab, hidden, DT[t], 0.5, p(y)))
        ws, n = scratch(g, lib.ar_embedding_backward_workspace, tokens, vocab, hidden, DT[t])
        ok(ctx, lib.ar_embedding_backward(ctx.handle, p(gd), hidden, p(gi), ib, tokens, vocab, hidden,
                                          DT[t], 0.5, p(d), p(ws), n))
        same((y, d), (want, back))
        ws.fill_(0xFF)
        ok(ctx, lib.ar_embedding_backward(ctx.handle, p(gd), hidden, p(gi), ib, tokens, vocab, hidden,
                                          DT[t], 0.5, p(d), p(ws), n))
        same((d,), (back,))
        g.check()
        same((gt, gd, gi), (table, dy, ids))


# (tiles of every shape, the depth in parts and not, widths that are and are not whole
# numbers of 4 and 16 bytes; shifts that put lines at every such address)
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("counts,hidden,out", [
    ((1,), 1, 1), ((0, 3, 1, 0), 4104, 24), ((1, 0, 1, 1), 2048, 520), ((70, 0, 131), 776, 264),
    ((70, 0, 131), 777, 265), ((129, 130), 640, 771), ((1100, 900), 520, 1032), ((1100, 900), 1024, 1032),
    ((1100, 900), 521, 1031), ((40,), 8200, 40), ((2500,), 72, 48)])
def test_products_between_guards(ctx, counts, hidden, out, t):  # noqa: F811
    lib = _lib.lib
    off = torch.tensor([0, *counts]).cumsum(0).int().cuda()
    n, experts = int(off[-1]), len(counts)
    rows, dout = randn(n, hidden).to(t), randn(n, out, seed=1).to(t)
    w = randn(experts, out, hidden, seed=2).to(t)
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    plan = ar.ExpertPlan(at.view(-1, 1), at, off)
    want = (ar.expert_matmul(rows, w, plan), ar.expert_matmul_drows(dout, w, plan),
            ar.expert_matmul_dweights(dout, rows, plan))
    tols = [ref.product(k, off, a, b) for k, a, b in (("out", rows, w), ("drows", dout, w),
                                                      ("dweights", dout, rows))]
    for v, (y, tol) in zip(want, tols):
        ref.close(v, y, tol)
    for shift in (0, 1, 2):
        g = Guards()
        gr, gd, gw, go = (g.copy(v, shift) for v in (rows, dout, w, off))
        y, dr, dw = (g(v.shape, t, shift) for v in want)
        sizes = (n, experts, hidden, out, DT[t])
        for _ in range(2):
            ws, b = scratch(g, lib.ar_expert_matmul_workspace, 0, *sizes)
            ok(ctx, lib.ar_expert_matmul(ctx.handle, p(gr), hidden, p(gw), p(go), *sizes, p(y), p(ws), b))
            ws, b = scratch(g, lib.ar_expert_matmul_workspace, 1, *sizes)
            ok(ctx, lib.ar_expert_matmul_drows(ctx.handle, p(gd), out, p(gw), p(go), *sizes, p(dr),
                                               p(ws), b))
            ws, b = scratch(g, lib.ar_expert_matmul_workspace, 2, *sizes)
            ok(ctx, lib.ar_expert_matmul_dweights(ctx.handle, p(gd), out, p(gr), hidden, p(go), *sizes,
                                                  p(dw), p(ws), b))
            # the order of a sum does not depend on where the arrays lie
            same((y, dr, dw), want)
        g.check()
        same((gr, gd, gw, go), (rows, dout, w, off))


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 33), (70, 771), (300, 1024), (17, 4104),
                                       (2, 70001)])
def test_gate_between_guards(ctx, rows, cols, t):  # noqa: F811
    lib = _lib.lib
    h, d = randn(rows, 2 * cols).to(t), randn(rows, cols, seed=1).to(t)
    acts, saved = ar.silu_gate(h)
    dh, again = ar.silu_gate_backward(d, saved)
    kept = ar.save_8bit(h)
    back = ar.restore_8bit(kept, t)
    for shift in (0, 1, 2, 3):
        g = Guards()
        gh, gd = g.copy(h, shift), g.copy(d, shift)
        ga, gdh, gagain, gback = (g(v.shape, t, shift) for v in (acts, dh, again, back))
        c, s = g(saved.codes.shape, torch.int8, shift), g(saved.scales.shape, torch.uint8, shift)
        kc, ks = g(kept.codes.shape, torch.int8, shift), g(kept.scales.shape, torch.uint8, shift)
        ok(ctx, lib.ar_silu_gate(ctx.handle, p(gh), 2 * cols, rows, cols, DT[t], p(ga), p(c), p(s)))
        ok(ctx, lib.ar_silu_gate_backward(ctx.handle, p(gd), cols, p(c), p(s), rows, cols, DT[t],
                                          p(gdh), p(gagain)))
        ok(ctx, lib.ar_save_8bit(ctx.handle, p(gh), 2 * cols, rows, 2 * cols, DT[t], p(kc), p(ks)))
        ok(ctx, lib.ar_restore_8bit(ctx.handle, p(kc), p(ks), rows, 2 * cols, DT[t], p(gback)))
        same((ga, c, s, gdh, gagain, kc, ks, gback), (acts, *saved, dh, again, *kept, back))
        g.check()
        same((gh, gd), (h, d))


# ------------------------------------------------------------------- streams and graphs

class Layer:
    """A layer of experts behind an embedding, forward and back; what its calls give."""

    def __init__(self, tokens, vocab, hidden, inner, experts, topk, t):
        self.vocab, self.experts, self.t, self.topk = vocab, experts, t, topk
        self.table = randn(vocab, hidden).to(t)
        self.w1 = (randn(experts, 2 * inner, hidden, seed=1) / hidden ** 0.5).to(t)
        self.w2 = (randn(experts, hidden, inner, seed=2) / inner ** 0.5).to(t)
        self.tokens = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        self.ids = torch.zeros((tokens, topk), dtype=torch.int32, device="cuda")
        self.gates = torch.zeros((tokens, topk), device="cuda")
        self.dy = torch.zeros((tokens, hidden), dtype=t, device="cuda")

    def draw(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.tokens.random_(0, self.vocab, generator=g)
        self.ids.random_(0, self.experts, generator=g)
        self.gates.uniform_(0, 1, generator=g)
        self.dy.copy_(torch.randn(self.dy.shape, generator=g, device="cuda"))

    def run(self):
        x = ar.embedding(self.table, self.tokens, 2.0)
        h, mean, rstd = ar.layer_norm(x)
        rows, plan = ar.expert_dispatch(h, self.ids, self.experts)
        a = ar.expert_matmul(rows, self.w1, plan)
        acts, saved = ar.silu_gate(a)
        out = ar.expert_matmul(acts, self.w2, plan)
        y = ar.expert_combine(out, self.gates, plan)
        dout, dgates = ar.expert_combine_backward(self.dy, out, self.gates, plan)
        dacts = ar.expert_matmul_drows(dout, self.w2, plan)
        da, again = ar.silu_gate_backward(dacts, saved)
        dw2 = ar.expert_matmul_dweights(dout, again, plan)
        dw1 = ar.expert_matmul_dweights(da, rows, plan)
        dh = ar.expert_dispatch_backward(ar.expert_matmul_drows(da, self.w1, plan), plan)
        dx = ar.layer_norm_backward(dh, x, mean, rstd)[0]
        dtable = ar.embedding_backward(dx, self.tokens, self.vocab, 2.0)
        return y, dgates, dw1, dw2, dtable, saved.codes, saved.scales


SIZES = [(3, 50, 64, 40, 4, 2), (600, 1000, 264, 200, 6, 2), (40000, 300, 64, 72, 3, 1)]


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("sizes", SIZES)
def test_graphs(sizes, t):
    """Two graphs of the same calls, replayed in turn between eager runs: each replay
    gives the eager results to the bit."""
    layers = [Layer(*sizes, t), Layer(*sizes, t)]
    captured = []
    side = torch.cuda.Stream()
    for i, layer in enumerate(layers):
        layer.draw(i)
        layer.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            results = layer.run()
        captured.append((graph, results))
    for seed in range(4):
        for layer, (graph, results) in zip(layers, captured):
            layer.draw(10 + seed)
            graph.replay()
            want = layer.run()
            torch.cuda.synchronize()
            same([r for r in results], want)
            layer.draw(50 + seed)
            layer.run()


@pytest.mark.parametrize("sizes", SIZES)
def test_two_streams(sizes):
    """The same calls on two streams at once."""
    layers = [Layer(*sizes, BF) for _ in range(2)]
    for i, layer in enumerate(layers):
        layer.draw(i)
    want = [layer.run() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        got = []
        for s, layer in zip(streams, layers):
            with torch.cuda.stream(s):
                got.append(layer.run())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            same(g, w)


# -------------------------------------------------------------------------- refusals

def test_refusals():
    x, ids = randn(6, 64), torch.zeros(6, dtype=torch.int64, device="cuda")
    w, off = randn(3, 32, 64), torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    at = torch.arange(6, dtype=torch.int32, device="cuda")
    plan, dout = ar.ExpertPlan(at.view(-1, 1), at, off), randn(6, 32)
    cpu = ar.ExpertPlan(*(v.cpu() for v in plan))
    saved = ar.silu_gate(x)[1]
    half = dout.contiguous()
    for match, call in (
            ("needs .vocab, hidden", lambda: ar.embedding(x[0], ids)),
            ("needs .vocab, hidden", lambda: ar.embedding(x[:0], ids)),
            ("not contiguous", lambda: ar.embedding(x[:, ::2], ids)),
            ("ids", lambda: ar.embedding(x, ids.float())),
            ("ids", lambda: ar.embedding(x, ids.cpu())),
            ("ids", lambda: ar.embedding(x, torch.zeros(12, dtype=torch.int64, device="cuda")[::2])),
            ("not finite", lambda: ar.embedding(x, ids, float("nan"))),
            ("not finite", lambda: ar.embedding_backward(x, ids, 9, float("inf"))),
            ("not finite", lambda: ar.embedding(x, ids, 1e39)),
            ("does not match ids", lambda: ar.embedding_backward(x, ids[:5], 9)),
            ("does not match ids", lambda: ar.embedding_backward(x, ids.view(2, 3), 9)),
            ("below 1", lambda: ar.embedding_backward(x, ids, 0)),
            ("does not match weights", lambda: ar.expert_matmul(x[:, :63], w, plan)),
            ("does not match weights", lambda: ar.expert_matmul_drows(x, w, plan)),
            ("needs .experts, out, hidden", lambda: ar.expert_matmul(x, w[0], plan)),
            ("needs .rows, width", lambda: ar.expert_matmul(x[0], w, plan)),
            ("are not of the plan's 3 experts", lambda: ar.expert_matmul(x, w[:2], plan)),
            ("weights", lambda: ar.expert_matmul(x, w.bfloat16(), plan)),
            ("weights", lambda: ar.expert_matmul(x, w.transpose(1, 2).contiguous().transpose(1, 2), plan)),
            ("weights", lambda: ar.expert_matmul(x, w.cpu(), plan)),
            ("plan.offsets", lambda: ar.expert_matmul(x, w, cpu)),
            ("plan.offsets", lambda: ar.expert_matmul(x, w, plan._replace(offsets=off.long()))),
            ("does not match rows", lambda: ar.expert_matmul_dweights(dout[:5], x, plan)),
            ("does not match rows", lambda: ar.expert_matmul_dweights(dout.bfloat16(), x, plan)),
            ("plan.offsets", lambda: ar.expert_matmul_dweights(dout, x, cpu)),
            ("no elements", lambda: ar.save_8bit(x[:, :0])),
            ("x", lambda: ar.save_8bit(x.t())),
            ("x", lambda: ar.save_8bit(x[:, ::2])),
            ("needs .*2 n", lambda: ar.silu_gate(x[:, :63])),
            ("needs .*2 n", lambda: ar.silu_gate(x[:, :0])),
            ("neither", lambda: ar.restore_8bit(saved, torch.float16)),
            ("saved.codes", lambda: ar.restore_8bit(saved._replace(codes=saved.codes.int()))),
            ("saved.scales", lambda: ar.restore_8bit(saved._replace(scales=saved.scales[..., :0]))),
            ("saved.scales", lambda: ar.restore_8bit(saved._replace(scales=saved.scales.cpu()))),
            ("does not match dacts", lambda: ar.silu_gate_backward(x, saved)),
            ("does not match dacts", lambda: ar.silu_gate_backward(half[:5], saved)),
            ("does not match dacts", lambda: ar.silu_gate_backward(half[:, :0], saved))):
        with pytest.raises(ValueError, match=match):
            call()
    # what the refused calls left behind does not stop a good one
    same((ar.silu_gate(x)[1].codes,), (saved.codes,))
    assert ar.embedding_backward(x[0], ids[0], 9).shape == (9, 64)
    torch.cuda.synchronize()
