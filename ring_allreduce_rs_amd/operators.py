"""Training operators on torch tensors: layer norm, tokens sorted by expert and
back, and distillation from a teacher's top logits, each with its gradient.

They are the operators beside the collectives in a data-parallel training
step: what the forward and backward passes run between two AllReduces of the
gradient buckets.  Each function checks its tensors (ValueError), allocates its
outputs (and scratch, where an operator needs some) from torch's allocator, and
enqueues the HIP kernels of libar.so on torch's current stream (include/ar.h
holds the formulas and limits; csrc/torch_ops.cpp is the binding).  Nothing is
recorded for torch's autograd: the gradients are the ``*_backward`` functions
(and ``distill_step``).  A tensor that requires grad is therefore refused
(ValueError) unless it is detached or the call runs under ``torch.no_grad()``,
and one with a forward-mode tangent always.

Activations are bfloat16 or float32, with rows at any stride; weights and
biases of a norm may be of the other type than its input.  Statistics, expert
weights and losses are float32.  Every argument is on one GPU; there is no CPU
fallback.

As with any kernel on torch's current stream, a tensor made on another stream
has to be ready (``wait_stream``) before the call.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib  # noqa: F401  (libar.so first: the binding links against it)

try:
    from . import _torch_ops as _ops
except ImportError as e:
    raise ImportError(f"{_lib.TORCH_OPS_PATH} is not built or does not load ({e}); run "
                      "`python ring_allreduce_rs_amd/_build.py` (or __graft_entry__.build()) "
                      "first") from e


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


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension: (y, mean, rstd), the last two float32
    of x's leading shape, as ``layer_norm_backward`` takes them."""
    return _ops.layer_norm(x, weight, bias, eps)


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """Gradients of ``layer_norm``: (dx, dweight, dbias).  dweight and dbias have
    the weight's dtype (x's without a weight)."""
    return _ops.layer_norm_backward(dy, x, mean, rstd, weight)


def expert_dispatch(x, ids, experts: int):
    """The tokens x (tokens, hidden) sorted by the experts ids (tokens, topk;
    int32 or int64) chose: (rows, plan).

    rows (tokens * topk, hidden) holds each token once per choice, expert by
    expert and in token order within one; plan says where each went.  Choices
    outside [0, experts) have no expert: they come last, as rows of zeros."""
    rows, dest, slot, offsets = _ops.expert_dispatch(x, ids, experts)
    return rows, ExpertPlan(dest, slot, offsets)


def expert_dispatch_backward(drows, plan: ExpertPlan):
    """Gradient of ``expert_dispatch``'s x: each token's choices added up."""
    return _ops.expert_dispatch_backward(drows, plan[0], plan[2])


def expert_combine(rows, weights, plan: ExpertPlan):
    """The way back: y[t] = sum over k of weights[t, k] * rows[dest[t, k]], with
    the experts' outputs in the rows of a dispatch.  weights: float32."""
    return _ops.expert_combine(rows, weights, plan[0], plan[2])


def expert_combine_backward(dy, rows, weights, plan: ExpertPlan):
    """Gradients of ``expert_combine``: (drows, dweights)."""
    return _ops.expert_combine_backward(dy, rows, weights, plan[0], plan[2])


def distill_loss(logits, indices, teacher, temperature: float = 1.0):
    """Distillation from a teacher's top logits: (loss, lse), float32, a value
    per row; lse is what ``distill_backward`` takes.

    logits (rows, vocab) are the student's; teacher (rows, top) holds the
    teacher's logits at the places indices (rows, top; int32 or int64).  A
    negative index leaves its entry out (an index past the vocabulary too); a
    row without entries has loss 0.  With p and q the two softmaxes at this
    temperature, loss = temperature^2 * sum(p * (log p - log q))."""
    return _ops.distill_loss(logits, indices, teacher, temperature)


def distill_backward(dloss, logits, indices, teacher, lse, temperature: float = 1.0):
    """Gradient of ``distill_loss`` by the logits, given dloss (rows, float32)."""
    return _ops.distill_backward(dloss, logits, indices, teacher, lse, temperature)


def distill_step(dloss, logits, indices, teacher, temperature: float = 1.0):
    """Loss and gradient at once, where each row's dloss is known beforehand (a
    mean over the batch, say): (loss, dlogits)."""
    return _ops.distill_step(dloss, logits, indices, teacher, temperature)
