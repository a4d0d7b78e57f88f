"""The training operators, measured: layer norm, tokens sorted by expert and back, distillation.

Each case is one pass through one operator in one direction, at sizes from a
single token to a training step's batch.  ``run`` computes it either in plain
form (elementary torch operations in 32 bits, rounded once) or, with ``own``
set, by the calls a user makes of ``ring_allreduce_rs_amd``.  ``exact`` gives
the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # --- layer norm ---------------------------------------------------------------------
        # one token in a decoding step: nothing but latency
        dict(name="norm_token", kind="norm_forward", rows=1, cols=4096, type="bf16", param="bf16"),
        # the norm of a training micro-batch of 16384 tokens
        dict(name="norm_batch", kind="norm_forward", rows=16384, cols=4096, type="bf16",
             param="bf16"),
        # a ragged tail batch in full precision, rows that start off every vector boundary
        dict(name="norm_grad_ragged", kind="norm_backward", rows=1021, cols=771, type="f32",
             param="f32"),
        # backward of a wide model's norm, weights kept in fp32 beside bf16 activations
        dict(name="norm_grad_batch", kind="norm_backward", rows=8192, cols=8192, type="bf16",
             param="f32"),
        # --- tokens sorted by expert and back -----------------------------------------------
        # four sequences decoding one token each
        dict(name="dispatch_tokens", kind="dispatch", tokens=4, topk=8, experts=64, hidden=2048,
             type="bf16", ids=64, pad=0.0),
        # a training micro-batch over many small experts
        dict(name="dispatch_batch", kind="dispatch", tokens=16384, topk=8, experts=128,
             hidden=2048, type="bf16", ids=64, pad=0.0),
        # the way back for a padded batch in full precision: a tenth of the tokens has no expert
        dict(name="combine_padded", kind="combine", tokens=4099, topk=6, experts=60, hidden=1000,
             type="f32", ids=32, pad=0.1),
        # both gradients of the way there and back, a training micro-batch
        dict(name="route_grad_batch", kind="route_backward", tokens=8192, topk=8, experts=64,
             hidden=4096, type="bf16", ids=64, pad=0.0),
        # --- distillation from a teacher's top logits ---------------------------------------
        # the loss of a single position, as an evaluation meets it
        dict(name="distill_token", kind="distill_loss", rows=1, vocab=131072, top=64, type="f32",
             ids=64, temperature=1.0, pad=0.0),
        # loss and gradient of a few positions
        dict(name="distill_few", kind="distill_step", rows=8, vocab=32000, top=16, type="bf16",
             ids=32, temperature=2.0, pad=0.0),
        # the gradient on its own, an odd vocabulary in full precision, padded positions
        dict(name="distill_grad_odd", kind="distill_backward", rows=2047, vocab=50021, top=100,
             type="f32", ids=64, temperature=2.0, pad=0.1),
        # the loss head of a training micro-batch: loss and gradient of every position
        dict(name="distill_batch", kind="distill_step", rows=4096, vocab=131072, top=64,
             type="bf16", ids=64, temperature=1.0, pad=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A row length: any number, or a multiple of 64, as models have it."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(64, n // 64 * 64)


def draw(rng):
    most = 1_000_000_000       # bytes of the largest tensor's worth of work, under the largest listed case
    kind = rng.choice(["norm_forward", "norm_backward", "dispatch", "combine", "route_backward",
                       "distill_loss", "distill_step", "distill_backward"])
    t = rng.choice(["bf16", "f32"])
    if kind.startswith("norm"):
        cols = _width(rng, 64, 16384)
        rows = min(_log(rng, 1, 16384), most // (3 * cols * SIZE[t]))
        return dict(kind=kind, rows=rows, cols=cols, type=t,
                    param="f32" if t == "f32" else rng.choice(["bf16", "f32"]))
    if kind.startswith("distill"):
        vocab = _width(rng, 1000, 200000)
        rows = max(1, min(_log(rng, 1, 8192), most // (2 * vocab * SIZE[t])))
        return dict(kind=kind, rows=rows, vocab=vocab, top=_log(rng, 1, 256), type=t,
                    ids=rng.choice([32, 64]), temperature=rng.choice([1.0, 2.0, 4.0]),
                    pad=rng.choice([0.0, 0.1]))
    experts, hidden = _log(rng, 4, 256), _width(rng, 64, 8192)
    topk = rng.randint(1, min(8, experts))
    each = (4 if kind == "route_backward" else 2) * topk * hidden * SIZE[t]
    return dict(kind=kind, tokens=max(1, min(_log(rng, 1, 16384), most // each)), topk=topk,
                experts=experts, hidden=hidden, type=t, ids=rng.choice([32, 64]),
                pad=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator("cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device=g.device).mul_(scale).add_(shift).to(dtype)


def _prepare_norm(c, g):
    t, p = DTYPES[c["type"]], DTYPES[c["param"]]
    # activations: another mean and spread in each row
    x = torch.randn((c["rows"], c["cols"]), generator=g, device=g.device)
    x = x.mul_(_normal(g, (c["rows"], 1), torch.float32, 0.3).exp_())
    x = x.add_(_normal(g, (c["rows"], 1), torch.float32, 0.5)).to(t)
    s = {"x": x, "weight": _normal(g, (c["cols"],), p, 0.2, 1.0),
         "bias": _normal(g, (c["cols"],), p, 0.1)}
    if c["kind"] == "norm_backward":
        s["dy"] = _normal(g, x.shape, t, 1e-2)
        wide = x.double()              # what the forward pass left
        mean = wide.mean(1, keepdim=True)
        s["rstd"] = ((wide - mean).square().mean(1) + EPS).rsqrt().float()
        s["mean"] = mean[:, 0].float()
    return s


def _prepare_route(c, g):
    t, n, k = DTYPES[c["type"]], c["tokens"], c["topk"]
    # a router's scores: some experts are more popular than others
    scores = _normal(g, (n, c["experts"]), torch.float32)
    scores += _normal(g, (1, c["experts"]), torch.float32, 0.5)
    top, ids = scores.topk(k, dim=1)
    weights = top.sub(top.amax(1, keepdim=True)).exp_()
    weights /= weights.sum(1, keepdim=True)
    padding = torch.rand((n, 1), generator=g, device=g.device) < c["pad"]
    ids = ids.masked_fill(padding, -1).to(torch.int64 if c["ids"] == 64 else torch.int32)
    s = {"ids": ids, "experts": c["experts"]}
    if c["kind"] == "dispatch":
        return {**s, "x": _normal(g, (n, c["hidden"]), t)}
    s["plan"] = _plan(ids, c["experts"])     # the dispatch's, from the forward pass
    live = torch.arange(n * k, device=g.device) < s["plan"][2][-1]
    s["weights"] = weights
    s["rows"] = _normal(g, (n * k, c["hidden"]), t).masked_fill_(~live[:, None], 0.0)
    if c["kind"] == "route_backward":
        s["dy"] = _normal(g, (n, c["hidden"]), t, 1e-2)
        # what the experts' own backward passes leave
        s["dx_rows"] = _normal(g, (n * k, c["hidden"]), t, 1e-2)
        s["dx_rows"].masked_fill_(~live[:, None], 0.0)
    return s


def _prepare_distill(c, g):
    t, i = DTYPES[c["type"]], torch.int64 if c["ids"] == 64 else torch.int32
    logits = _normal(g, (c["rows"], c["vocab"]), t, 2.5)
    # the teacher's choices lie among the places that the student likes too, in no order
    picks = torch.rand((c["rows"], c["top"]), generator=g, device=g.device)
    step = c["vocab"] // c["top"]
    at = (picks * step).long() + torch.arange(c["top"], device=g.device) * step
    at = at.clamp_(max=c["vocab"] - 1)
    teacher = logits.gather(1, at).float() * 0.5 + _normal(g, at.shape, torch.float32, 2.0, 4.0)
    padding = torch.rand((c["rows"], 1), generator=g, device=g.device) < c["pad"]
    short = torch.rand(at.shape, generator=g, device=g.device) < 0.5 * c["pad"]
    s = {"logits": logits, "indices": at.masked_fill(padding | short, -1).to(i),
         "teacher": teacher.to(t), "temperature": c["temperature"]}
    if c["kind"] != "distill_loss":
        # each position's share in the batch's loss
        s["dloss"] = torch.rand(c["rows"], generator=g, device=g.device).add_(0.5) / c["rows"]
    if c["kind"] == "distill_backward":
        s["lse"] = logits.double().div_(c["temperature"]).logsumexp(1).float()
    return s


def prepare(case, seed):
    g = _generator(seed)
    make = (_prepare_norm if case["kind"].startswith("norm") else
            _prepare_distill if case["kind"].startswith("distill") else _prepare_route)
    return {"kind": case["kind"], **make(case, g)}


# --------------------------------------------------------------------------- plain forms

def _norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _norm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    p = s["weight"].dtype
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(p),
            "dbias": dy.sum(0).to(p)}


def _plan(ids, experts):
    """Where each slot (token, choice) goes, which slot each sorted row is, where each
    expert's rows begin.  Slots without an expert come last."""
    flat = ids.reshape(-1).long()
    e = torch.where((flat >= 0) & (flat < experts), flat, experts)
    slot = e.argsort(stable=True)
    dest = torch.empty_like(slot)
    dest[slot] = torch.arange(e.numel(), device=e.device)
    of = torch.arange(experts, device=e.device)
    ends = torch.searchsorted(e[slot], of, right=True)
    offsets = torch.cat([ends.new_zeros(1), ends])
    return dest.int().view(ids.shape), slot.int(), offsets.int()


def _dispatch(s):
    dest, slot, offsets = _plan(s["ids"], s["experts"])
    rows = s["x"][slot.long() // s["ids"].shape[1]]
    live = torch.arange(slot.numel(), device=slot.device) < offsets[-1]
    return {"rows": torch.where(live[:, None], rows, torch.zeros((), dtype=rows.dtype,
                                                                 device=rows.device)),
            "dest": dest, "slot": slot, "offsets": offsets}


def _combine(s):
    dest, _, offsets = s["plan"]
    w = torch.where(dest < offsets[-1], s["weights"], 0.0)
    y = (s["rows"][dest.long()].float() * w[:, :, None]).sum(1)
    return {"y": y.to(s["rows"].dtype)}


def _route_backward(s):
    dest, slot, offsets = s["plan"]
    at, live = dest.long(), dest < offsets[-1]
    dy = s["dy"].float()
    dw = (s["rows"][at].float() * dy[:, None, :]).sum(2)
    w = torch.where(live, s["weights"], 0.0).reshape(-1)[slot.long()]
    drows = dy[slot.long() // dest.shape[1]] * w[:, None]
    dx = (s["dx_rows"][at].float() * live[:, :, None]).sum(1)
    return {"drows": drows.to(s["rows"].dtype), "dweights": torch.where(live, dw, 0.0),
            "dx": dx.to(s["rows"].dtype)}


def _teacher(s):
    """The teacher's distribution over its kept places (0 at entries left out), its
    logarithm, and the places."""
    live = s["indices"] >= 0
    z = torch.where(live, s["teacher"].float() / s["temperature"], -torch.inf)
    top = z.amax(1, keepdim=True)
    z = z - torch.where(top == -torch.inf, 0.0, top)
    total = z.exp().sum(1, keepdim=True)
    total = torch.where(total == 0, 1.0, total)
    return z.exp() / total, torch.where(live, z - total.log(), 0.0), s["indices"].clamp(min=0).long()


def _distill_loss(s):
    p, logp, at = _teacher(s)
    z = s["logits"].float() / s["temperature"]
    top = z.amax(1, keepdim=True)
    lse = top + (z - top).exp().sum(1, keepdim=True).log()
    logq = z.gather(1, at) - lse
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(1) * s["temperature"] ** 2
    return {"loss": loss, "lse": lse[:, 0]}


def _distill_backward(s):
    p, _, at = _teacher(s)
    some = (s["indices"] >= 0).any(1, keepdim=True)
    q = (s["logits"].float() / s["temperature"] - s["lse"][:, None]).exp() * some
    d = q.scatter_add_(1, at, -p) * (s["dloss"] * s["temperature"])[:, None]
    return {"dlogits": d.to(s["logits"].dtype)}


def _distill_step(s):
    f = _distill_loss(s)
    return {"loss": f["loss"], **_distill_backward({**s, "lse": f["lse"]})}


PLAIN = {"norm_forward": _norm_forward, "norm_backward": _norm_backward, "dispatch": _dispatch,
         "combine": _combine, "route_backward": _route_backward, "distill_loss": _distill_loss,
         "distill_backward": _distill_backward, "distill_step": _distill_step}


# ----------------------------------------------------------------- the framework's calls

def _own(s):
    import ring_allreduce_rs_amd as ar

    kind = s["kind"]
    if kind == "norm_forward":
        y, mean, rstd = ar.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_backward":
        dx, dweight, dbias = ar.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"],
                                                    s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if kind == "dispatch":
        rows, plan = ar.expert_dispatch(s["x"], s["ids"], s["experts"])
        return {"rows": rows, "dest": plan.dest, "slot": plan.slot, "offsets": plan.offsets}
    if kind == "combine":
        return {"y": ar.expert_combine(s["rows"], s["weights"], ar.ExpertPlan(*s["plan"]))}
    if kind == "route_backward":
        plan = ar.ExpertPlan(*s["plan"])
        drows, dweights = ar.expert_combine_backward(s["dy"], s["rows"], s["weights"], plan)
        return {"drows": drows, "dweights": dweights,
                "dx": ar.expert_dispatch_backward(s["dx_rows"], plan)}
    if kind == "distill_loss":
        loss, lse = ar.distill_loss(s["logits"], s["indices"], s["teacher"], s["temperature"])
        return {"loss": loss, "lse": lse}
    if kind == "distill_backward":
        return {"dlogits": ar.distill_backward(s["dloss"], s["logits"], s["indices"],
                                               s["teacher"], s["lse"], s["temperature"])}
    loss, dlogits = ar.distill_step(s["dloss"], s["logits"], s["indices"], s["teacher"],
                                    s["temperature"])
    return {"loss": loss, "dlogits": dlogits}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["kind"]](state)


# ---------------------------------------------------------------------------- least work

def work(case):
    c, e = case, SIZE[case["type"]]
    if c["kind"].startswith("norm"):
        n, p = c["rows"] * c["cols"], c["cols"] * SIZE[c["param"]]
        if c["kind"] == "norm_forward":      # x, y; weight, bias; mean, rstd
            return {"bytes": 2 * n * e + 2 * p + 8 * c["rows"], "flops": 8 * n}
        # x, dy, dx; weight, its gradient, the bias's; mean, rstd
        return {"bytes": 3 * n * e + 3 * p + 8 * c["rows"], "flops": 14 * n}
    if c["kind"].startswith("distill"):
        n, k = c["rows"] * c["vocab"], c["rows"] * c["top"]
        heads = k * (e + c["ids"] // 8)      # the teacher's logits and their places
        if c["kind"] == "distill_loss":      # logits; loss, lse
            return {"bytes": n * e + heads + 8 * c["rows"], "flops": 4 * n}
        # logits, their gradient; dloss and lse or loss
        return {"bytes": 2 * n * e + heads + 8 * c["rows"],
                "flops": (4 if c["kind"] == "distill_backward" else 8) * n}
    slots, h = c["tokens"] * c["topk"], c["hidden"] * e
    if c["kind"] == "dispatch":    # ids, x; rows, dest, slot, offsets
        return {"bytes": slots * (c["ids"] // 8 + 8) + 4 * c["experts"] + 4
                + (c["tokens"] + slots) * h, "flops": slots}
    if c["kind"] == "combine":     # dest, weights, rows; y
        return {"bytes": slots * 8 + (c["tokens"] + slots) * h,
                "flops": 2 * slots * c["hidden"]}
    # dest, weights, dy, rows, dx_rows; drows, dweights, dx
    return {"bytes": slots * 12 + (2 * c["tokens"] + 3 * slots) * h,
            "flops": 4 * slots * c["hidden"]}


# --------------------------------------------------- the definitions, in 64 bits

def _exact_norm(c, s):
    x, w = s["x"].double(), s["weight"].double()
    n = c["cols"]
    if c["kind"] == "norm_forward":
        mu = x.sum(1) / n
        var = (x - mu[:, None]).pow(2).sum(1) / n
        sd = torch.sqrt(var + EPS)
        return {"y": (x - mu[:, None]) / sd[:, None] * w + s["bias"].double(), "mean": mu,
                "rstd": 1 / sd}
    # the chain rule through the statistics that the pass is given
    r, dy = s["rstd"].double(), s["dy"].double()
    xc = x - s["mean"].double()[:, None]
    a = (dy @ w) / n
    b = torch.matmul(dy * xc, w) * r * r / n
    dx = r[:, None] * (dy * w - a[:, None] - xc * b[:, None])
    return {"dx": dx, "dweight": torch.matmul(r, dy * xc),
            "dbias": torch.matmul(torch.ones_like(r), dy)}


def _exact_route(c, s):
    ids, k = s["ids"].cpu().numpy().astype(np.int64), c["topk"]
    key = np.where((ids < 0) | (ids >= c["experts"]), c["experts"], ids).reshape(-1)
    slot = np.lexsort((np.arange(key.size), key))
    dest = np.empty(key.size, np.int64)
    dest[slot] = np.arange(key.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=c["experts"] + 1))[:-1]])
    dev, live = s["ids"].device, int(offsets[-1])
    token = torch.from_numpy(slot[:live] // k).to(dev)
    if c["kind"] == "dispatch":
        rows = torch.zeros((key.size, c["hidden"]), dtype=torch.float64, device=dev)
        rows[:live] = s["x"].double()[token]
        return {"rows": rows, "dest": dest.reshape(ids.shape).astype(np.int32),
                "slot": slot.astype(np.int32), "offsets": offsets.astype(np.int32)}
    at = torch.from_numpy(slot[:live]).to(dev)
    w = s["weights"].double().reshape(-1)[at][:, None]

    def back(rows):
        y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=dev)
        return y.index_add_(0, token, rows)

    if c["kind"] == "combine":
        return {"y": back(s["rows"][:live].double() * w)}
    dy = s["dy"].double()[token]
    drows = torch.zeros((key.size, c["hidden"]), dtype=torch.float64, device=dev)
    drows[:live] = dy * w
    dweights = torch.zeros(key.size, dtype=torch.float64, device=dev)
    dweights[at] = (dy * s["rows"][:live].double()).sum(1)
    return {"drows": drows, "dweights": dweights.view(ids.shape),
            "dx": back(s["dx_rows"][:live].double())}


def _exact_distill(c, s):
    tau = c["temperature"]
    at = s["indices"].long()
    live = at >= 0
    t = s["teacher"].double() / tau
    t = torch.where(live, t, torch.full_like(t, -math.inf))
    some = live.any(1)
    logp = torch.log_softmax(torch.where(some[:, None], t, torch.zeros_like(t)), 1)
    p = torch.where(live, logp.exp(), torch.zeros_like(t))
    z = s["logits"].double() / tau
    lse = torch.logsumexp(z, 1)
    terms = p * (logp - z.gather(1, at.clamp(min=0)) + lse[:, None])
    loss = tau * tau * torch.where(p > 0, terms, torch.zeros_like(terms)).sum(1)
    if c["kind"] == "distill_loss":
        return {"loss": loss, "lse": lse}
    given = s["lse"].double() if c["kind"] == "distill_backward" else lse
    d = z.sub_(given[:, None]).exp_().mul_(some[:, None])
    i = torch.arange(c["rows"], device=at.device)[:, None].expand_as(at)
    d.index_put_((i, at.clamp(min=0)), -p, accumulate=True)
    d.mul_(tau * s["dloss"].double()[:, None])
    return {"dlogits": d} if c["kind"] == "distill_backward" else {"loss": loss, "dlogits": d}


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    return (_exact_norm if kind.startswith("norm") else _exact_distill
            if kind.startswith("distill") else _exact_route)(case, state)
