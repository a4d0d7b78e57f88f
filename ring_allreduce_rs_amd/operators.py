"""Training operators on torch tensors: layer norm, tokens sorted by expert and
back, and distillation from a teacher's top logits, each with its gradient.

They are the operators beside the collectives in a data-parallel training
step: what the forward and backward passes run between two AllReduces of the
gradient buckets.  Each function checks its tensors, allocates its outputs (and
scratch, where an operator needs some) from torch's allocator on torch's
current stream, and enqueues the HIP kernels of libar.so there (include/ar.h
holds the formulas and limits).  Nothing is recorded for torch's autograd: the
gradients are the ``*_backward`` functions (and ``distill_step``).

Activations are bfloat16 or float32, with rows at any stride; weights and
biases of a norm may be of the other type than its input.  Statistics, expert
weights and losses are float32.  Every argument is on one GPU; there is no CPU
fallback.

As with any kernel on torch's current stream, a tensor made on another stream
has to be ready (``wait_stream``) before the call.
"""

from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

import torch

from . import _lib
from ._lib import AR_DISTILL_MAX_TOP, AR_MAX_EXPERTS, ArError, Context

_FLOATS = {torch.float32: _lib.DTYPES["float32"], torch.bfloat16: _lib.DTYPES["bfloat16"]}
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}
_local = threading.local()


class ExpertPlan(NamedTuple):
    """Where the tokens of one dispatch went (all int32, on the GPU).

    dest     (tokens, topk): the sorted row of each choice of each token
    slot     (tokens * topk,): the choice (token * topk + k) of each sorted row
    offsets  (experts + 1,): the first sorted row of each expert; the last is
             the number of rows in use
    """

    dest: torch.Tensor
    slot: torch.Tensor
    offsets: torch.Tensor


def _context(device: torch.device) -> Context:
    """This thread's context on `device`, bound to torch's current stream.  Its
    arrays come from tensors that were looked at here, so the library does not
    ask the runtime about them again."""
    index = device.index
    try:
        c = _local.contexts[index]
    except (AttributeError, KeyError):
        c = Context(index, torch.cuda.current_stream(index).cuda_stream)
        c.set_operator_checks(False)
        if not hasattr(_local, "contexts"):
            _local.contexts = {}
        _local.contexts[index] = c
    c.set_stream(torch.cuda.current_stream(index).cuda_stream)
    return c


def _float_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is not a tensor")
    dt = _FLOATS.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}; use float32 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a GPU")
    return dt


def _like(t, name, dtype, shape, device):
    """t is dense, of this dtype and shape, on this device."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is not a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, needs {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, needs {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t.data_ptr()


def _row_stride(t, name):
    """Elements from one row (the last dimension) to the next."""
    if t.dim() == 0:
        raise ValueError(f"{name} has no dimensions")
    cols = t.shape[-1]
    if t.is_contiguous():
        return cols
    if t.dim() == 2 and (t.stride(1) == 1 or cols == 1):
        s = t.stride(0)
    else:
        try:
            if cols > 1 and t.stride(-1) != 1:
                raise RuntimeError
            s = t.view(-1, cols).stride(0)
        except RuntimeError:
            raise ValueError(f"{name}: the rows of {tuple(t.shape)} with strides "
                             f"{tuple(t.stride())} are not evenly spaced dense rows") from None
    if s < cols and t.numel() > cols:
        raise ValueError(f"{name}: rows {s} elements apart overlap (broadcast?)")
    return s


def _scratch(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _size(fn, *args):
    out = ctypes.c_size_t()
    st = fn(*args, ctypes.byref(out))
    if st != _lib.AR_OK:
        raise ArError(st, fn.__name__, f"sizes {args}")
    return out.value


# ------------------------------------------------------------------------ layer norm

def _param(t, name, cols, device):
    """(pointer, dtype) of a norm's weight or bias."""
    if t is None:
        return None, None
    dt = _float_tensor(t, name)
    return _like(t, name, t.dtype, (cols,), device), dt


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension: (y, mean, rstd), the last two float32
    of x's leading shape, as ``layer_norm_backward`` takes them."""
    dt = _float_tensor(x, "x")
    stride, dev = _row_stride(x, "x"), x.device
    cols = x.shape[-1]
    if cols == 0:
        raise ValueError("x has rows of no elements")
    w, wdt = _param(weight, "weight", cols, dev)
    b, bdt = _param(bias, "bias", cols, dev)
    if w is not None and b is not None and wdt != bdt:
        raise ValueError("weight and bias need one dtype")
    if not 0.0 <= eps < float("inf"):
        raise ValueError(f"eps {eps} is negative or not finite")
    lead = x.shape[:-1]
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    mean = torch.empty(lead, dtype=torch.float32, device=dev)
    rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    pdt = wdt if wdt is not None else bdt if bdt is not None else dt
    c = _context(dev)
    c.call(_lib.lib.ar_layer_norm, x.data_ptr(), stride, w, b, pdt, y.data_ptr(),
           mean.data_ptr(), rstd.data_ptr(), mean.numel(), cols, dt, eps)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """Gradients of ``layer_norm``: (dx, dweight, dbias).  dweight and dbias have
    the weight's dtype (x's without a weight)."""
    dt = _float_tensor(x, "x")
    _float_tensor(dy, "dy")
    dev, shape = x.device, x.shape
    if dy.dtype != x.dtype or dy.shape != shape or dy.device != dev:
        raise ValueError(f"dy ({dy.dtype}, {tuple(dy.shape)}, {dy.device}) does not match x "
                         f"({x.dtype}, {tuple(shape)}, {dev})")
    xs, gs = _row_stride(x, "x"), _row_stride(dy, "dy")
    cols = shape[-1]
    if cols == 0:
        raise ValueError("x has rows of no elements")
    lead = shape[:-1]
    m = _like(mean, "mean", torch.float32, lead, dev)
    r = _like(rstd, "rstd", torch.float32, lead, dev)
    w, wdt = _param(weight, "weight", cols, dev)
    pdt = dt if w is None else wdt
    ptype = x.dtype if w is None else weight.dtype
    rows = mean.numel()
    dx = torch.empty(shape, dtype=x.dtype, device=dev)
    dweight = torch.empty(cols, dtype=ptype, device=dev)
    dbias = torch.empty(cols, dtype=ptype, device=dev)
    nbytes = _size(_lib.lib.ar_layer_norm_backward_workspace, rows, cols, dt)
    ws = _scratch(nbytes, dev)
    _context(dev).call(_lib.lib.ar_layer_norm_backward, dy.data_ptr(), gs, x.data_ptr(), xs, m, r,
                       w, pdt, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), rows, cols, dt,
                       _ptr(ws), nbytes)
    return dx, dweight, dbias


# -------------------------------------------------------- tokens by expert and back

def expert_dispatch(x, ids, experts: int):
    """The tokens x (tokens, hidden) sorted by the experts ids (tokens, topk;
    int32 or int64) chose: (rows, plan).

    rows (tokens * topk, hidden) holds each token once per choice, expert by
    expert and in token order within one; plan says where each went.  Choices
    outside [0, experts) have no expert: they come last, as rows of zeros."""
    dt = _float_tensor(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, needs (tokens, hidden)")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError("ids needs shape (tokens, topk) with x's tokens")
    ib = _INDEX_BYTES.get(ids.dtype)
    if ib is None:
        raise ValueError(f"ids: unsupported dtype {ids.dtype}; use int32 or int64")
    tokens, hidden = x.shape
    topk, dev = ids.shape[1], x.device
    i = _like(ids, "ids", ids.dtype, ids.shape, dev)
    if topk == 0 or hidden == 0:
        raise ValueError("topk and hidden have to be positive")
    if not 1 <= experts <= AR_MAX_EXPERTS:
        raise ValueError(f"experts {experts} outside [1, {AR_MAX_EXPERTS}]")
    stride = _row_stride(x, "x")
    slots = tokens * topk
    rows = torch.empty((slots, hidden), dtype=x.dtype, device=dev)
    dest = torch.empty((tokens, topk), dtype=torch.int32, device=dev)
    slot = torch.empty(slots, dtype=torch.int32, device=dev)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    nbytes = _size(_lib.lib.ar_expert_dispatch_workspace, tokens, topk, experts)
    ws = _scratch(nbytes, dev)
    _context(dev).call(_lib.lib.ar_expert_dispatch, x.data_ptr(), stride, i, ib, tokens, topk,
                       experts, hidden, dt, rows.data_ptr(), dest.data_ptr(), slot.data_ptr(),
                       offsets.data_ptr(), _ptr(ws), nbytes)
    return rows, ExpertPlan(dest, slot, offsets)


def _plan(plan, rows, name):
    """Sizes and pointers that the calls after a dispatch take."""
    dt = _float_tensor(rows, name)
    dest, _, offsets = plan
    dev = rows.device
    if not isinstance(dest, torch.Tensor) or dest.dim() != 2 or dest.shape[1] == 0:
        raise ValueError("plan.dest needs shape (tokens, topk)")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("plan.offsets needs shape (experts + 1,)")
    experts = offsets.shape[0] - 1
    if experts > AR_MAX_EXPERTS:
        raise ValueError(f"experts {experts} above {AR_MAX_EXPERTS}")
    d = _like(dest, "plan.dest", torch.int32, dest.shape, dev)
    o = _like(offsets, "plan.offsets", torch.int32, offsets.shape, dev)
    tokens, topk = dest.shape
    if rows.dim() != 2 or rows.shape[0] != tokens * topk or rows.shape[1] == 0:
        raise ValueError(f"{name} has shape {tuple(rows.shape)}, needs "
                         f"({tokens * topk}, hidden)")
    if not rows.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return dt, d, o, tokens, topk, experts, rows.shape[1]


def expert_dispatch_backward(drows, plan: ExpertPlan):
    """Gradient of ``expert_dispatch``'s x: each token's choices added up."""
    dt, d, o, tokens, topk, experts, hidden = _plan(plan, drows, "drows")
    dx = torch.empty((tokens, hidden), dtype=drows.dtype, device=drows.device)
    _context(drows.device).call(_lib.lib.ar_expert_dispatch_backward, drows.data_ptr(), d, o,
                                tokens, topk, experts, hidden, dt, dx.data_ptr())
    return dx


def expert_combine(rows, weights, plan: ExpertPlan):
    """The way back: y[t] = sum over k of weights[t, k] * rows[dest[t, k]], with
    the experts' outputs in the rows of a dispatch.  weights: float32."""
    dt, d, o, tokens, topk, experts, hidden = _plan(plan, rows, "rows")
    w = _like(weights, "weights", torch.float32, (tokens, topk), rows.device)
    y = torch.empty((tokens, hidden), dtype=rows.dtype, device=rows.device)
    _context(rows.device).call(_lib.lib.ar_expert_combine, rows.data_ptr(), w, d, o, tokens, topk,
                               experts, hidden, dt, y.data_ptr())
    return y


def expert_combine_backward(dy, rows, weights, plan: ExpertPlan):
    """Gradients of ``expert_combine``: (drows, dweights)."""
    dt, d, o, tokens, topk, experts, hidden = _plan(plan, rows, "rows")
    dev = rows.device
    w = _like(weights, "weights", torch.float32, (tokens, topk), dev)
    _float_tensor(dy, "dy")
    if dy.dtype != rows.dtype or dy.shape != (tokens, hidden) or dy.device != dev:
        raise ValueError(f"dy ({dy.dtype}, {tuple(dy.shape)}, {dy.device}) does not match rows: "
                         f"needs ({rows.dtype}, {(tokens, hidden)}, {dev})")
    stride = _row_stride(dy, "dy")
    drows = torch.empty(rows.shape, dtype=rows.dtype, device=dev)
    dweights = torch.empty((tokens, topk), dtype=torch.float32, device=dev)
    _context(dev).call(_lib.lib.ar_expert_combine_backward, dy.data_ptr(), stride, rows.data_ptr(),
                       w, d, o, tokens, topk, experts, hidden, dt, drows.data_ptr(),
                       dweights.data_ptr())
    return drows, dweights


# ---------------------------------------------------------------------- distillation

def _distill(logits, indices, teacher, temperature):
    """What the three calls share: (device, sizes and the leading arguments)."""
    dt = _float_tensor(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits has shape {tuple(logits.shape)}, needs (rows, vocab)")
    rows, vocab = logits.shape
    dev = logits.device
    if not isinstance(indices, torch.Tensor) or indices.dim() != 2 or indices.shape[0] != rows:
        raise ValueError("indices needs shape (rows, top) with the logits' rows")
    ib = _INDEX_BYTES.get(indices.dtype)
    if ib is None:
        raise ValueError(f"indices: unsupported dtype {indices.dtype}; use int32 or int64")
    top = indices.shape[1]
    i = _like(indices, "indices", indices.dtype, indices.shape, dev)
    t = _like(teacher, "teacher", logits.dtype, indices.shape, dev)
    if vocab == 0 or not 1 <= top <= AR_DISTILL_MAX_TOP:
        raise ValueError(f"vocab {vocab} is 0 or top {top} outside [1, {AR_DISTILL_MAX_TOP}]")
    if not 0.0 < temperature < float("inf"):
        raise ValueError(f"temperature {temperature} is not positive and finite")
    return dev, rows, vocab, top, dt, (logits.data_ptr(), _row_stride(logits, "logits"), i, ib, t)


def distill_loss(logits, indices, teacher, temperature: float = 1.0):
    """Distillation from a teacher's top logits: (loss, lse), float32, a value
    per row; lse is what ``distill_backward`` takes.

    logits (rows, vocab) are the student's; teacher (rows, top) holds the
    teacher's logits at the places indices (rows, top; int32 or int64).  A
    negative index leaves its entry out (an index past the vocabulary too); a
    row without entries has loss 0.  With p and q the two softmaxes at this
    temperature, loss = temperature^2 * sum(p * (log p - log q))."""
    dev, rows, vocab, top, dt, args = _distill(logits, indices, teacher, temperature)
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    lse = torch.empty(rows, dtype=torch.float32, device=dev)
    nbytes = _size(_lib.lib.ar_distill_workspace, rows, vocab, dt, 0)
    ws = _scratch(nbytes, dev)
    _context(dev).call(_lib.lib.ar_distill_loss, *args, rows, vocab, top, dt, temperature,
                       loss.data_ptr(), lse.data_ptr(), _ptr(ws), nbytes)
    return loss, lse


def distill_backward(dloss, logits, indices, teacher, lse, temperature: float = 1.0):
    """Gradient of ``distill_loss`` by the logits, given dloss (rows, float32)."""
    dev, rows, vocab, top, dt, args = _distill(logits, indices, teacher, temperature)
    g = _like(dloss, "dloss", torch.float32, (rows,), dev)
    e = _like(lse, "lse", torch.float32, (rows,), dev)
    dlogits = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
    _context(dev).call(_lib.lib.ar_distill_backward, g, *args, e, rows, vocab, top, dt,
                       temperature, dlogits.data_ptr())
    return dlogits


def distill_step(dloss, logits, indices, teacher, temperature: float = 1.0):
    """Loss and gradient at once, where each row's dloss is known beforehand (a
    mean over the batch, say): (loss, dlogits)."""
    dev, rows, vocab, top, dt, args = _distill(logits, indices, teacher, temperature)
    g = _like(dloss, "dloss", torch.float32, (rows,), dev)
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    dlogits = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
    nbytes = _size(_lib.lib.ar_distill_workspace, rows, vocab, dt, 1)
    ws = _scratch(nbytes, dev)
    _context(dev).call(_lib.lib.ar_distill_step, g, *args, rows, vocab, top, dt, temperature,
                       loss.data_ptr(), dlogits.data_ptr(), _ptr(ws), nbytes)
    return loss, dlogits
