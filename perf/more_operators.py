"""More training operators, measured: the embedding and its gradient, the experts' products and
their gradients, and the experts' gated activation with its checkpoint in 8 bits.

Each case is one pass through one operator in one direction, at sizes from a few tokens to a
training step's batch.  ``run`` computes it either in plain form (elementary torch operations in
32 bits, rounded once) or, with ``own`` set, by the calls a user makes of
``ring_allreduce_rs_amd``.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
GROUP = 32          # values of a checkpoint that share a scale


def listed():
    return [
        # --- embedding ----------------------------------------------------------------------
        # four sequences decoding one token each: nothing but latency
        dict(name="embed_tokens", kind="embed", tokens=4, vocab=131072, hidden=4096, type="bf16",
             ids=64, scale=64.0, pad=0.0),
        # the first operator of a training micro-batch
        dict(name="embed_batch", kind="embed", tokens=16384, vocab=131072, hidden=4096,
             type="bf16", ids=64, scale=64.0, pad=0.0),
        # the gradient of a ragged batch in full precision, a tenth of it padding
        dict(name="embed_grad_ragged", kind="embed_backward", tokens=2047, vocab=50021, hidden=771,
             type="f32", ids=32, scale=1.0, pad=0.1),
        # the gradient bucket of a training micro-batch: some tokens come hundreds of times
        dict(name="embed_grad_batch", kind="embed_backward", tokens=16384, vocab=131072,
             hidden=4096, type="bf16", ids=64, scale=64.0, pad=0.0),
        # --- the experts' products ----------------------------------------------------------
        # four sequences decoding one token each: the chosen experts' weights are the work
        dict(name="expert_tokens", kind="product", tokens=4, topk=8, experts=64, hidden=2048,
             out=2048, type="bf16", pad=0.0),
        # the first product of a training micro-batch
        dict(name="expert_batch", kind="product", tokens=8192, topk=8, experts=64, hidden=4096,
             out=2048, type="bf16", pad=0.0),
        # the rows' gradient of a small padded batch in full precision, odd widths
        dict(name="expert_drows_ragged", kind="drows", tokens=513, topk=6, experts=60, hidden=1000,
             out=771, type="f32", pad=0.1),
        # the weights' gradient of a training micro-batch over many small experts
        dict(name="expert_dweights_batch", kind="dweights", tokens=16384, topk=8, experts=128,
             hidden=2048, out=1024, type="bf16", pad=0.0),
        # --- the gated activation and its checkpoint -----------------------------------------
        # the rows of four decoded tokens
        dict(name="gate_tokens", kind="gate", rows=32, cols=2048, type="bf16"),
        # the experts' rows of a training micro-batch, and the checkpoint's values read back
        dict(name="gate_batch", kind="gate", rows=65536, cols=2048, type="bf16"),
        # the backward pass from the checkpoint, for the same rows
        dict(name="gate_grad_batch", kind="gate_backward", rows=65536, cols=2048, type="bf16"),
        # a checkpoint of rows in full precision, odd width, written and read back
        dict(name="save_ragged", kind="save", rows=4099, cols=1001, type="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A row length: any number, or a multiple of 64, as models have it."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(64, n // 64 * 64)


def draw(rng):
    most = 1_000_000_000       # bytes of the largest tensor, under the largest listed case's
    kind = rng.choice(["embed", "embed_backward", "product", "drows", "dweights", "gate",
                       "gate_backward", "save"])
    t = rng.choice(["bf16", "f32"])
    if kind.startswith("embed"):
        vocab = _width(rng, 1000, 200000)
        hidden = min(_width(rng, 64, 8192), max(64, most // (vocab * SIZE[t])))
        return dict(kind=kind, tokens=_log(rng, 1, 16384), vocab=vocab, hidden=hidden, type=t,
                    ids=rng.choice([32, 64]), scale=rng.choice([1.0, math.sqrt(hidden)]),
                    pad=rng.choice([0.0, 0.1]))
    if kind in ("product", "drows", "dweights"):
        experts = _log(rng, 4, 256)
        hidden, out = _width(rng, 64, 8192), _width(rng, 64, 8192)
        experts = max(1, min(experts, most // (hidden * out * SIZE[t])))
        topk = rng.randint(1, min(8, experts))
        # multiplications and additions: full precision has a sixteenth of the matrix rate
        ops = 1.0e12 if t == "bf16" else 6.0e10
        tokens = min(_log(rng, 1, 16384), int(ops / (2.0 * topk * hidden * out)))
        return dict(kind=kind, tokens=max(1, tokens), topk=topk, experts=experts, hidden=hidden,
                    out=out, type=t, pad=rng.choice([0.0, 0.1]))
    cols = _width(rng, 32, 8192)
    rows = max(1, min(_log(rng, 1, 131072), most // (4 * cols * SIZE[t])))
    return dict(kind=kind, rows=rows, cols=cols, type=t)


# ------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator("cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device=g.device).mul_(scale).add_(shift).to(dtype)


def _prepare_embed(c, g):
    t = DTYPES[c["type"]]
    # a text's tokens: the one at place r of the order comes about 1 / r as often as the first
    u = torch.rand(c["tokens"], generator=g, device=g.device, dtype=torch.float64)
    place = u.mul_(math.log(c["vocab"] + 1)).exp_().sub_(1).long().clamp_(0, c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=g, device=g.device)[place]
    padding = torch.rand(c["tokens"], generator=g, device=g.device) < c["pad"]
    ids = ids.masked_fill(padding, -1).to(torch.int64 if c["ids"] == 64 else torch.int32)
    s = {"ids": ids, "scale": c["scale"], "vocab": c["vocab"]}
    if c["kind"] == "embed":
        return {**s, "table": _normal(g, (c["vocab"], c["hidden"]), t, c["hidden"] ** -0.5)}
    return {**s, "dy": _normal(g, (c["tokens"], c["hidden"]), t, 1e-2)}


def _plan(ids, experts):
    """Where each slot (token, choice) goes, which slot each sorted row is, where each
    expert's rows begin.  Slots without an expert come last."""
    flat = ids.reshape(-1)
    e = torch.where((flat >= 0) & (flat < experts), flat, experts)
    slot = e.argsort(stable=True)
    dest = torch.empty_like(slot)
    dest[slot] = torch.arange(e.numel(), device=e.device)
    ends = torch.searchsorted(e[slot], torch.arange(experts, device=e.device), right=True)
    offsets = torch.cat([ends.new_zeros(1), ends])
    return dest.int().view(ids.shape), slot.int(), offsets.int()


def _prepare_product(c, g):
    t, n, k = DTYPES[c["type"]], c["tokens"], c["topk"]
    # a router's choices: some experts are more popular than others
    scores = _normal(g, (n, c["experts"]), torch.float32)
    scores += _normal(g, (1, c["experts"]), torch.float32, 0.5)
    ids = scores.topk(k, dim=1)[1]
    padding = torch.rand((n, 1), generator=g, device=g.device) < c["pad"]
    plan = _plan(ids.masked_fill(padding, -1), c["experts"])
    live = (torch.arange(n * k, device=g.device) < plan[2][-1])[:, None]
    s = {"plan": plan, "ends": plan[2].tolist()}    # the plain form's loop goes by the latter
    if c["kind"] != "dweights":
        s["weights"] = _normal(g, (c["experts"], c["out"], c["hidden"]), t, c["hidden"] ** -0.5)
    if c["kind"] != "drows":
        s["rows"] = _normal(g, (n * k, c["hidden"]), t).masked_fill_(~live, 0.0)
    if c["kind"] != "product":
        s["dout"] = _normal(g, (n * k, c["out"]), t, 1e-2).masked_fill_(~live, 0.0)
    return s


def _quantise(x):
    """x in 8 bits: whole numbers in [-127, 127], and for each group of 32 along the last
    dimension the biased exponent of its scale, the least power of two s with
    127 s >= the group's largest magnitude (2^-126 at least)."""
    cols = x.shape[-1]
    groups = (cols + GROUP - 1) // GROUP
    wide = torch.nn.functional.pad(x.float(), (0, groups * GROUP - cols))
    wide = wide.view(*x.shape[:-1], groups, GROUP)
    bits = wide.abs().amax(-1).view(torch.int32)
    e = ((bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).int()).clamp_(min=1)
    scale = (e << 23).view(torch.float32)
    codes = (wide / scale[..., None]).round_()
    return codes.to(torch.int8).flatten(-2)[..., :cols].contiguous(), e.to(torch.uint8)


def _values(codes, scales):
    """What the codes stand for, in 32 bits."""
    s = (scales.int() << 23).view(torch.float32)
    return codes.float() * s.repeat_interleave(GROUP, -1)[..., :codes.shape[-1]]


def _prepare_gate(c, g):
    t = DTYPES[c["type"]]
    if c["kind"] == "save":      # a norm's outputs: a few columns much larger than the rest
        loud = _normal(g, (1, c["cols"]), torch.float32).exp_()
        return {"x": _normal(g, (c["rows"], c["cols"]), torch.float32).mul_(loud).to(t)}
    h = _normal(g, (c["rows"], 2 * c["cols"]), t)
    if c["kind"] == "gate":
        return {"h": h}
    codes, scales = _quantise(h.view(c["rows"], 2, c["cols"]))      # the forward pass's
    return {"codes": codes, "scales": scales, "dacts": _normal(g, (c["rows"], c["cols"]), t, 1e-2)}


def prepare(case, seed):
    g = _generator(seed)
    make = (_prepare_embed if case["kind"].startswith("embed") else
            _prepare_product if "experts" in case else _prepare_gate)
    return {"kind": case["kind"], **make(case, g)}


# --------------------------------------------------------------------------- plain forms

def _embed(s):
    known = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    rows = s["table"][torch.where(known, s["ids"], 0).long()].float() * s["scale"]
    return {"y": torch.where(known[:, None], rows, 0.0).to(s["table"].dtype)}


def _embed_backward(s):
    known = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    dy = torch.where(known[:, None], s["dy"].float(), 0.0)
    total = torch.zeros((s["vocab"], dy.shape[1]), device=dy.device)
    total.index_add_(0, torch.where(known, s["ids"], 0).long(), dy)
    return {"dtable": total.mul_(s["scale"]).to(s["dy"].dtype)}


def _by_expert(s):
    ends = s["ends"]
    return [(e, slice(ends[e], ends[e + 1])) for e in range(len(ends) - 1) if ends[e + 1] > ends[e]]


def _product(s):
    rows, w = s["rows"], s["weights"]
    out = rows.new_zeros((rows.shape[0], w.shape[1]))
    for e, at in _by_expert(s):
        out[at] = (rows[at].float() @ w[e].float().t()).to(rows.dtype)
    return {"out": out}


def _drows(s):
    dout, w = s["dout"], s["weights"]
    drows = dout.new_zeros((dout.shape[0], w.shape[2]))
    for e, at in _by_expert(s):
        drows[at] = (dout[at].float() @ w[e].float()).to(dout.dtype)
    return {"drows": drows}


def _dweights(s):
    dout, rows = s["dout"], s["rows"]
    dw = rows.new_zeros((len(s["ends"]) - 1, dout.shape[1], rows.shape[1]))
    for e, at in _by_expert(s):
        dw[e] = (dout[at].float().t() @ rows[at].float()).to(rows.dtype)
    return {"dweights": dw}


def _gate(s):
    h = s["h"].float()
    n = h.shape[1] // 2
    a, u = h[:, :n], h[:, n:]
    codes, scales = _quantise(s["h"].view(h.shape[0], 2, n))
    return {"acts": (a * torch.sigmoid(a) * u).to(s["h"].dtype),
            "saved": _values(codes, scales).to(s["h"].dtype)}


def _gate_backward(s):
    v = _values(s["codes"], s["scales"])
    a, u, d = v[:, 0], v[:, 1], s["dacts"].float()
    q = torch.sigmoid(a)
    t = s["dacts"].dtype
    da = d * u * q * (1.0 + a * (1.0 - q))
    return {"dh": torch.cat([da, d * a * q], 1).to(t), "acts": (a * q * u).to(t)}


def _save(s):
    return {"saved": _values(*_quantise(s["x"])).to(s["x"].dtype)}


PLAIN = {"embed": _embed, "embed_backward": _embed_backward, "product": _product, "drows": _drows,
         "dweights": _dweights, "gate": _gate, "gate_backward": _gate_backward, "save": _save}


# ----------------------------------------------------------------- the framework's calls

def _own(s):
    import ring_allreduce_rs_amd as ar

    kind = s["kind"]
    if kind == "embed":
        return {"y": ar.embedding(s["table"], s["ids"], s["scale"])}
    if kind == "embed_backward":
        return {"dtable": ar.embedding_backward(s["dy"], s["ids"], s["vocab"], s["scale"])}
    if kind == "product":
        return {"out": ar.expert_matmul(s["rows"], s["weights"], ar.ExpertPlan(*s["plan"]))}
    if kind == "drows":
        return {"drows": ar.expert_matmul_drows(s["dout"], s["weights"],
                                                ar.ExpertPlan(*s["plan"]))}
    if kind == "dweights":
        return {"dweights": ar.expert_matmul_dweights(s["dout"], s["rows"],
                                                      ar.ExpertPlan(*s["plan"]))}
    if kind == "gate":
        acts, saved = ar.silu_gate(s["h"])
        return {"acts": acts, "saved": ar.restore_8bit(saved, s["h"].dtype)}
    if kind == "gate_backward":
        dh, acts = ar.silu_gate_backward(s["dacts"], ar.Saved8(s["codes"], s["scales"]))
        return {"dh": dh, "acts": acts}
    return {"saved": ar.restore_8bit(ar.save_8bit(s["x"]), s["x"].dtype)}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["kind"]](state)


# ---------------------------------------------------------------------------- least work

def _distinct(tokens, vocab):
    """How many tokens of the vocabulary a batch holds, on average."""
    r = np.arange(1, vocab + 1, dtype=np.float64)
    p = np.log1p(1.0 / r) / math.log(vocab + 1)
    return int(-np.expm1(tokens * np.log1p(-p)).sum())


def work(case):
    c, e = case, SIZE[case["type"]]
    if c["kind"] == "embed":             # ids, the table's rows that occur; y
        rows = _distinct(c["tokens"], c["vocab"]) + c["tokens"]
        return {"bytes": c["tokens"] * c["ids"] // 8 + rows * c["hidden"] * e,
                "flops": c["tokens"] * c["hidden"]}
    if c["kind"] == "embed_backward":    # ids, dy; the table's gradient
        return {"bytes": c["tokens"] * c["ids"] // 8 + (c["tokens"] + c["vocab"]) * c["hidden"] * e,
                "flops": c["tokens"] * c["hidden"]}
    if "experts" in c:
        slots = c["tokens"] * c["topk"]
        used = c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** c["tokens"])
        if c["kind"] == "dweights":      # every expert's gradient is written
            used = c["experts"]
        return {"bytes": int(e * (slots * (c["hidden"] + c["out"]) + used * c["hidden"] * c["out"]))
                + 4 * c["experts"] + 4, "flops": 2 * slots * c["hidden"] * c["out"]}
    n = c["rows"] * c["cols"]
    codes = c["rows"] * (c["cols"] + (c["cols"] + GROUP - 1) // GROUP)
    if c["kind"] == "gate":              # h; acts, the checkpoint's values
        return {"bytes": 5 * n * e, "flops": 12 * n}
    if c["kind"] == "gate_backward":     # the checkpoint, dacts; dh, acts
        return {"bytes": 4 * n * e + 2 * codes, "flops": 16 * n}
    return {"bytes": 2 * n * e, "flops": 4 * n}      # x; the checkpoint's values


# --------------------------------------------------- the definitions, in 64 bits

def _exact_embed(c, s):
    at = s["ids"].long()
    keep = ((at >= 0) & (at < c["vocab"])).nonzero()[:, 0]
    if c["kind"] == "embed":
        y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=at.device)
        y[keep] = c["scale"] * s["table"].index_select(0, at[keep]).double()
        return {"y": y}
    # sorted by token: the sum of each run of equal ones
    order = keep[at[keep].argsort(stable=True)]
    which, counts = torch.unique_consecutive(at[order], return_counts=True)
    run_of = torch.repeat_interleave(torch.arange(which.numel(), device=at.device), counts)
    sums = torch.zeros((which.numel(), c["hidden"]), dtype=torch.float64, device=at.device)
    sums.index_add_(0, run_of, s["dy"][order].double())
    d = torch.zeros((c["vocab"], c["hidden"]), dtype=torch.float64, device=at.device)
    d[which] = c["scale"] * sums
    return {"dtable": d}


def _exact_product(c, s):
    begin = s["plan"][2].cpu().numpy()
    like = s["rows"] if "rows" in s else s["dout"]
    shape = {"product": (like.shape[0], c["out"]), "drows": (like.shape[0], c["hidden"]),
             "dweights": (c["experts"], c["out"], c["hidden"])}[c["kind"]]
    r = torch.zeros(shape, dtype=torch.float64, device=like.device)
    for e in range(c["experts"]):
        lo, hi = int(begin[e]), int(begin[e + 1])
        if lo == hi:
            continue
        if c["kind"] == "dweights":
            r[e] = torch.mm(s["dout"][lo:hi].double().t().contiguous(), s["rows"][lo:hi].double())
        elif c["kind"] == "drows":
            r[lo:hi] = torch.mm(s["dout"][lo:hi].double(), s["weights"][e].double())
        else:
            r[lo:hi] = torch.mm(s["weights"][e].double(), s["rows"][lo:hi].double().t()).t()
    return {{"product": "out"}.get(c["kind"], c["kind"]): r}


def _powers(device):
    """2^-127 .. 2^128, exactly."""
    return torch.tensor([math.ldexp(1.0, k) for k in range(-127, 129)], dtype=torch.float64,
                        device=device)


def _exact_saved(x):
    """The values of x's checkpoint, group by group: x to the nearest multiple of the scale."""
    x, power = x.double(), _powers(x.device)
    r = torch.empty_like(x)
    for lo in range(0, x.shape[-1], GROUP):
        g = x[..., lo:lo + GROUP]
        m, e = torch.frexp(g.abs().amax(-1, keepdim=True))     # amax = m 2^e, m in [1/2, 1)
        e = torch.where(m * 128 <= 127, e - 7, e - 6).clamp(min=-126)
        step = power[e.long() + 127]
        r[..., lo:lo + GROUP] = torch.round(g / step) * step
    return r


def _exact_gate(c, s):
    if c["kind"] == "save":
        return {"saved": _exact_saved(s["x"])}
    n = c["cols"]
    if c["kind"] == "gate":
        a, u = s["h"][:, :n].double(), s["h"][:, n:].double()
        return {"acts": a * u / (1 + torch.exp(-a)),
                "saved": _exact_saved(s["h"].view(c["rows"], 2, n))}
    step = _powers(s["codes"].device)[s["scales"].long()]
    at = torch.arange(n, device=step.device) // GROUP
    a, u = (s["codes"][:, i].double() * step[:, i].index_select(1, at) for i in (0, 1))
    d, w = s["dacts"].double(), 1 + torch.exp(-a)
    return {"dh": torch.cat([d * u * (w + a * (w - 1)) / (w * w), d * a / w], 1),
            "acts": a * u / w}


def exact(case, seed):
    state = prepare(case, seed)
    make = (_exact_embed if case["kind"].startswith("embed") else
            _exact_product if "experts" in case else _exact_gate)
    return make(case, state)
