"""The training operators by their definitions in 64 bits, and the error
bounds that the GPU tests hold the kernels to.

Bounds, with u = 2^-24 (half a step of fp32): a sum of n terms that every lane
of a wavefront takes part in has at most ceil(n / 64) + 24 additions behind
one another (each lane's share, then the joins over lanes and wavefronts), so
it is off by at most (ceil(n / 64) + 24) u times the sum of the terms'
magnitudes; each product or difference adds u of its own size.  The last
rounding, to an output of type t, adds torch.finfo(t).eps / 2 of the value.
Second-order terms are covered by the factor 1.01.
"""

import math

import torch

U = 2.0 ** -24


def depth(n):
    return math.ceil(n / 64) + 24


def half_step(t):
    return torch.finfo(t).eps / 2


def close(got, want, tol, what=""):
    """|got - want| <= tol elementwise; non-finite values have to agree."""
    g, w = got.detach().double().cpu(), want.double().cpu()
    t = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(w)
    assert g.shape == w.shape, f"{what}: shape {tuple(g.shape)} != {tuple(w.shape)}"
    odd = ~torch.isfinite(w)
    same = torch.where(torch.isnan(w), torch.isnan(g), g == w)
    assert bool(same[odd].all()), f"{what}: non-finite values differ"
    err = torch.where(odd, 0.0, (g - w).abs())
    bad = ~(err <= t) & ~odd
    if bad.any():
        i = tuple(int(k[0]) for k in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {w.numel()} off; first at {i}: got "
                             f"{g[i]:.9g} want {w[i]:.9g} bound {t[i]:.3g}")


# ------------------------------------------------------------------------ layer norm

def norm(x, weight, bias, eps):
    """(y, mean, rstd) and their bounds."""
    t = x.dtype
    x = x.double()
    w = weight.double() if weight is not None else torch.ones(x.shape[-1], dtype=torch.float64,
                                                              device=x.device)
    b = bias.double() if bias is not None else torch.zeros_like(w)
    n = x.shape[-1]
    k = depth(n)
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    var = d.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    y = d * rstd * w + b
    tmean = 1.01 * (k + 1) * U * x.abs().mean(-1, keepdim=True)
    # each centred value is off by the mean's error and its own rounding; the
    # mean's error enters the variance squared (the centred values add up to 0)
    drel = (k + 4) * U + 2 * U * d.abs().mean(-1, keepdim=True) / var.sqrt().clamp(min=1e-300)
    tvar = var * 2 * drel + tmean.square()
    trstd = 1.01 * (rstd * (0.5 * tvar / (var + eps) + 3 * U))
    ty = 1.01 * (w.abs() * (rstd * (tmean + U * d.abs()) + d.abs() * trstd
                            + 3 * U * d.abs() * rstd) + 2 * U * (y.abs() + b.abs())) \
        + half_step(t) * y.abs() + 1e-40
    return (y, mean[..., 0], rstd[..., 0]), (ty, (tmean + U * mean.abs())[..., 0] + 1e-40,
                                             (trstd + U * rstd)[..., 0])


def norm_backward(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) and their bounds, from the statistics given."""
    t = x.dtype
    p = weight.dtype if weight is not None else t
    n = x.shape[-1]
    k = depth(n)
    x, dy = x.double().reshape(-1, n), dy.double().reshape(-1, n)
    mean, rstd = mean.double().reshape(-1, 1), rstd.double().reshape(-1, 1)
    w = weight.double() if weight is not None else torch.ones(n, dtype=torch.float64,
                                                              device=x.device)
    xh = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    tc1 = (k + 2) * U * g.abs().mean(1, keepdim=True)
    tc2 = (k + 6) * U * (g * xh).abs().mean(1, keepdim=True)
    tdx = 1.01 * rstd * (4 * U * (g.abs() + c1.abs() + (xh * c2).abs()) + tc1 + xh.abs() * tc2
                         + 3 * U * (xh * c2).abs()) + half_step(t) * dx.abs() + 1e-40
    dw, db = (dy * xh).sum(0), dy.sum(0)
    m = x.shape[0] + 8    # any order of the rows
    tdw = 1.01 * (m + 4) * U * (dy * xh).abs().sum(0) + half_step(p) * dw.abs() + 1e-40
    tdb = 1.01 * m * U * dy.abs().sum(0) + half_step(p) * db.abs() + 1e-40
    return (dx, dw, db), (tdx, tdw, tdb)


# -------------------------------------------------------- tokens by expert and back

def plan(ids, experts):
    """(dest, slot, offsets) by a stable sort on the host."""
    flat = ids.reshape(-1).long().cpu()
    e = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    slot = torch.argsort(e, stable=True)
    dest = torch.empty_like(slot)
    dest[slot] = torch.arange(slot.numel())
    count = torch.bincount(e, minlength=experts + 1)[:experts]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)])
    return dest.view(ids.shape).int(), slot.int(), offsets.int()


def combine(rows, weights, dest, live):
    """y and its bound; slots whose dest is not below `live` count for nothing."""
    t = rows.dtype
    ok = (dest >= 0) & (dest < live)
    at = torch.where(ok, dest, torch.zeros_like(dest)).long()
    w = torch.where(ok, weights.double(), 0.0)[:, :, None]
    r = torch.where(ok[:, :, None], rows.double()[at], 0.0)
    y = (w * r).sum(1)
    ty = 1.01 * (dest.shape[1] + 1) * U * (w * r).abs().sum(1) + half_step(t) * y.abs() + 1e-40
    return y, ty


def combine_backward(dy, rows, weights, dest, live):
    """(drows, dweights) and their bounds."""
    t = rows.dtype
    n, h = rows.shape
    ok = (dest >= 0) & (dest < live)
    at = torch.where(ok, dest, torch.zeros_like(dest)).long()
    g = dy.double()[:, None, :].expand(-1, dest.shape[1], -1)
    r = torch.where(ok[:, :, None], rows.double()[at], 0.0)
    dw = (g * r).sum(2)
    tdw = 1.01 * (depth(h) + 2) * U * (g * r).abs().sum(2) + 1e-40
    drows = torch.zeros((n, h), dtype=torch.float64, device=rows.device)
    drows[at[ok]] = (g * weights.double()[:, :, None])[ok]
    return (drows, torch.where(ok, dw, 0.0)), (1.01 * U * drows.abs() + half_step(t) * drows.abs()
                                               + 1e-40, tdw)


# ---------------------------------------------------------------------- distillation

EXP = 2.0 ** -22      # what an exponential may be off, relative


def distill(logits, indices, teacher, temperature, dloss=None, lse=None):
    """(loss, lse, dlogits) and their bounds; dlogits from `lse` where given."""
    t, T = logits.dtype, temperature
    v = logits.shape[1]
    at = indices.long()
    live = (at >= 0) & (at < v)
    at = torch.where(live, at, torch.zeros_like(at))
    s = torch.where(live, teacher.double() / T, -math.inf)
    smax = s.amax(1, keepdim=True)
    some = torch.isfinite(smax)
    smax = torch.where(some, smax, 0.0)
    total = (s - smax).exp().sum(1, keepdim=True)
    p = torch.where(some, (s - smax).exp() / torch.where(some, total, 1.0), 0.0)
    logp = torch.where(p > 0, s - smax - torch.where(some, total, 1.0).log(), 0.0)
    # relative error of an exponential of a rounded argument, of p, and of log p
    rp = EXP + 4 * U * (1 + torch.where(p > 0, (s - smax).abs() + s.abs(), 0.0))
    rtot = (p * rp).sum(1, keepdim=True) + depth(at.shape[1]) * U
    z = logits.double() / T
    m = z.amax(1, keepdim=True)
    m0 = torch.where(torch.isfinite(m), m, 0.0)
    e = (z - m0).exp()
    big = e.sum(1, keepdim=True)
    out_lse = m0 + big.log()
    far = torch.where(e > 0, (z - m0).abs(), 0.0)
    rbig = (e * (EXP + 4 * U * (1 + far))).sum(1, keepdim=True) / big + depth(v) * U
    tlse = 1.01 * (rbig + 2 * U * (m0.abs() + out_lse.abs() + big.log().abs())) + 1e-40
    logq = z.gather(1, at) - out_lse
    terms = torch.where(p > 0, p * (logp - logq), 0.0)
    loss = T * T * terms.sum(1)
    zabs = torch.where(p > 0, z.gather(1, at).abs(), 0.0)
    per = torch.where(p > 0, p * ((rp + rtot) * (logp - logq).abs() + 2 * U * (s.abs() + logp.abs())
                                  + rtot + 4 * U * (zabs + logq.abs()) + tlse), 0.0)
    tloss = 1.01 * T * T * (per.sum(1) + (depth(at.shape[1]) + 4) * U * terms.abs().sum(1)) + 1e-40
    if dloss is None:
        return (loss, out_lse[:, 0]), (tloss, tlse[:, 0])
    scale = (dloss.double() * T)[:, None]
    if lse is None:
        q, rq = e / big, EXP + 4 * U * (1 + far) + rbig
    else:
        a = z - lse.double()[:, None]
        q = a.exp()
        rq = EXP + 4 * U * (1 + torch.where(q > 0, z.abs() + a.abs(), 0.0))
    q = torch.where(some, q, 0.0)
    d = q.clone().scatter_add_(1, at, -torch.where(live, p, 0.0)) * scale
    td = (q * rq).scatter_add_(1, at, torch.where(live, p * (rp + rtot + 2 * U), 0.0))
    # sums of duplicates, the difference and the product round once each
    td = td + (at.shape[1] + 4) * U * q.clone().scatter_add_(1, at, torch.where(live, p, 0.0))
    td = 1.01 * td * scale.abs() + half_step(t) * d.abs() + 1e-40
    if t == torch.bfloat16:
        td = td + 2.0 ** -133      # a step of bf16's subnormals
    else:
        td = td + 2.0 ** -126      # (an exponential may flush below the normal numbers)
    td = torch.where(some, td, 0.0)
    d = torch.where(some, d, 0.0)
    return (loss, out_lse[:, 0], d), (tloss, tlse[:, 0], td)
