"""The embedding, the experts' products and the gated activation with its 8-bit
checkpoint by their definitions in 64 bits, and the error bounds that the GPU
tests hold the kernels to (u = 2^-24, half a step of fp32; the last rounding to
a type t adds torch.finfo(t).eps / 2 of the value).

- A sum of n terms in any order is off by at most n u times the sum of their
  magnitudes.  A matrix instruction may cut what it adds instead of rounding,
  so a product over n terms is given 2 (n + 8) u.
- A checkpoint's codes, scales and values are exact.
- The sigmoid is off by RS = 2^-21 of its value: an exponential good to 2^-22,
  a reciprocal good to 2^-23, two roundings.  Below fp32's normal numbers it may
  be 0.
"""

import torch

from tests.operator_refs import U, close, half_step  # noqa: F401

RS = 2.0 ** -21
TINY = 2.0 ** -126
GROUP = 32


def floor_of(t):
    """What an output of type t may lose below the normal numbers."""
    return 2.0 ** -133 if t == torch.bfloat16 else TINY


# ------------------------------------------------------------------------- embedding

def embedding(table, ids, scale):
    known = (ids >= 0) & (ids < table.shape[0])
    rows = table.double()[torch.where(known, ids, 0).long()] * float(torch.tensor(scale))
    y = torch.where(known[..., None], rows, 0.0)
    return y, (U + half_step(table.dtype)) * y.abs() * 1.01 + floor_of(table.dtype)


def embedding_backward(dy, ids, vocab, scale):
    t, scale = dy.dtype, float(torch.tensor(scale))
    ids, dy = ids.reshape(-1).cpu(), dy.double().reshape(-1, dy.shape[-1]).cpu()
    known = ((ids >= 0) & (ids < vocab)).nonzero()[:, 0]
    at = ids[known].long()
    total = torch.zeros((vocab, dy.shape[1]), dtype=torch.float64, device=dy.device)
    size, count = total.clone(), torch.zeros(vocab, dtype=torch.float64, device=dy.device)
    total.index_add_(0, at, dy[known])
    size.index_add_(0, at, dy[known].abs())
    count.index_add_(0, at, torch.ones(at.numel(), dtype=torch.float64, device=dy.device))
    d = scale * total
    tol = 1.01 * (abs(scale) * (count[:, None] + 2) * U * size + half_step(t) * d.abs())
    return d, torch.where(count[:, None] > 0, tol + floor_of(t), 0.0)


# ---------------------------------------------------------------- the experts' products

def groups(offsets, n):
    """The experts' rows, from offsets as they may come: inside [0, n], the first 0,
    none where the end lies before the beginning."""
    o = [0, *(min(max(int(v), 0), n) for v in offsets.tolist()[1:])]
    return [(b, max(b, e)) for b, e in zip(o[:-1], o[1:])]


def _mm(a, b, t):
    y = a.double() @ b.double()
    tol = 2.02 * (a.shape[1] + 8) * U * (a.double().abs() @ b.double().abs())
    return y, tol + half_step(t) * y.abs() + floor_of(t)


def product(kind, offsets, a, b):
    """kind "out": a = rows, b = weights; "drows": a = dout, b = weights;
    "dweights": a = dout, b = rows."""
    t, n = a.dtype, a.shape[0]
    g = groups(offsets, n)
    shape = {"out": (n, b.shape[1]), "drows": (n, b.shape[-1]),
             "dweights": (len(g), a.shape[1], b.shape[-1])}[kind]
    y = torch.zeros(shape, dtype=torch.float64, device=a.device)
    tol = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(g):
        if lo == hi:
            continue
        if kind == "dweights":
            y[e], tol[e] = _mm(a[lo:hi].double().t().contiguous(), b[lo:hi], t)
        else:
            w = b[e].double().t().contiguous() if kind == "out" else b[e]
            y[lo:hi], tol[lo:hi] = _mm(a[lo:hi], w, t)
    return y, tol


# ------------------------------------------------------------- checkpoints and the gate

def save(x):
    """(codes, scales, values) of a checkpoint; the values NaN where a group is not
    finite."""
    x = x.double().cpu()
    n = x.shape[-1]
    codes, values = torch.zeros_like(x), torch.empty_like(x)
    scales = torch.zeros((*x.shape[:-1], (n + GROUP - 1) // GROUP), dtype=torch.float64)
    for i in range(scales.shape[-1]):
        s = slice(GROUP * i, GROUP * i + GROUP)
        big = x[..., s].abs().amax(-1, keepdim=True)
        fine = torch.isfinite(x[..., s]).all(-1, keepdim=True)
        m, e = torch.frexp(torch.where(fine, big, 1.0))
        # big = m 2^e, m in [1/2, 1): the least power of two with 127 of it >= big
        e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(min=-126)
        e = torch.where(m > 0, e, -126)       # (a group of zeros)
        step = torch.tensor([2.0 ** k for k in range(-126, 128)], dtype=torch.float64)[e + 126]
        most = torch.where(e == 122, 63.0, 127.0)      # 64 * 2^122 is past fp32's numbers
        codes[..., s] = torch.where(fine, torch.round(x[..., s] / step).clamp(-most, most), 0.0)
        values[..., s] = torch.where(fine, codes[..., s] * step, torch.nan)
        scales[..., i] = torch.where(fine, e + 127, 255)[..., 0]
    return codes.to(torch.int8), scales.to(torch.uint8), values


def values(codes, scales):
    step = 2.0 ** (torch.arange(256, dtype=torch.float64) - 127)
    at = torch.arange(codes.shape[-1]) // GROUP
    return codes.double().cpu() * step[scales.long().cpu()][..., at]


def gate(h):
    t, n = h.dtype, h.shape[-1] // 2
    h = h.double().cpu()
    a, u = h[..., :n], h[..., n:]
    y = a * torch.sigmoid(a) * u
    # (where the sigmoid or a product falls below the normal numbers, it may be 0)
    return y, 1.01 * (RS + 2 * U + half_step(t)) * y.abs() + floor_of(t) \
        + TINY * ((a * u).abs() + u.abs())


def gate_backward(dacts, codes, scales):
    """(dh, acts) and their bounds."""
    t = dacts.dtype
    v, d = values(codes, scales), dacts.double().cpu()
    a, u = v[..., 0, :], v[..., 1, :]
    s = torch.sigmoid(a)
    f = 1 + a * (1 - s)
    tf = a.abs() * (RS * s + 2 * U) + 3 * U * (1 + (a * (1 - s)).abs())
    da, du, acts = d * u * s * f, d * a * s, a * s * u
    low = TINY * (1 + (d * u).abs() * (1 + f.abs()) + d.abs() + (d * a).abs())
    tda = 1.01 * ((d * u * s).abs() * (tf + (RS + 4 * U) * f.abs()) + half_step(t) * da.abs())
    tdu = 1.01 * (RS + 3 * U + half_step(t)) * du.abs()
    ta = 1.01 * (RS + 2 * U + half_step(t)) * acts.abs() + TINY * ((a * u).abs() + u.abs())
    low = low + floor_of(t)
    return (torch.cat([da, du], -1), acts), (torch.cat([tda + low, tdu + low], -1),
                                             ta + floor_of(t))
