"""What a training step runs around the head: the teacher-forced loss with its
gradient, and the global gradient norm with clipping.

A step of one process is ``apply_block_logits`` -> ``block_cross_entropy`` ->
``apply_block_logits_backward`` -> ``GradientClipper.clip``;
``VanillaMarkov.teacher_forced_gradients`` runs it. With several ranks a program
calls the parts: the all-reduce of ``sharding`` stands between the backward and
the clipping, and a mean over all ranks takes ``reduction="sum"`` and a division
by the sum of all ranks' weights.
"""
from __future__ import annotations

import bisect
import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from . import _native as N
from .head import _DT, _check_cuda, _device_guard, _ranged, _stream_ptr


@_ranged
def block_cross_entropy(logits: torch.Tensor, targets: torch.Tensor, *, weights: Optional[torch.Tensor] = None,
                        ignore_index: int = -100, reduction: str = "mean", want_grad: bool = True,
                        out_grad: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Cross entropy of corrected ``logits`` (..., V) against ``targets`` (...)
    int64, with its gradient. Returns (loss, row_losses, grad):

        row_losses[i] = logsumexp(logits[i]) - logits[i, targets[i]]           fp32 (...)
        loss          = sum_i weights[i] row_losses[i] / N                     fp32 scalar
        grad[i]       = weights[i] / N (softmax(logits[i]) - onehot(targets[i]))

    N is the sum of the weights of the rows that count ("mean") or 1 ("sum").
    ``weights`` (...) fp32 (default all 1; a block's later positions or other
    losses' shares). A row whose target is ``ignore_index`` or whose weight is
    zero does not count: its logits are not read, its loss and gradient are 0.
    A target outside the vocabulary does the same and sets the TOKEN_RANGE
    status bit. With no row left the loss is 0. ``out_grad`` takes the gradient
    (the logits' shape and dtype) and may be ``logits`` (in place); the
    gradient is the ``grad_out`` of ``apply_block_logits_backward``."""
    if logits.dim() < 1:
        raise ValueError("logits must be (..., V)")
    dtype, device = logits.dtype, logits.device
    if dtype not in _DT:
        raise ValueError("logits must be float32 or bfloat16")
    if reduction not in ("mean", "sum"):
        raise ValueError("reduction must be 'mean' or 'sum'")
    vocab = logits.shape[-1]
    if vocab == 0:
        raise ValueError("logits must have a vocabulary")
    lead = logits.shape[:-1]
    if targets.shape != lead:
        raise ValueError("targets must match logits without its last dim")
    ids = targets if targets.dtype == torch.int64 else targets.long()
    _check_cuda(logits, "logits", device)
    _check_cuda(ids, "targets", device)
    if weights is not None:
        if weights.shape != lead or weights.dtype != torch.float32:
            raise ValueError("weights must be fp32 with the shape of targets")
        _check_cuda(weights, "weights", device)
    grad = None
    if out_grad is not None:
        if out_grad is not logits:
            if out_grad.shape != logits.shape or out_grad.dtype != dtype:
                raise ValueError("out_grad must match logits in shape and dtype")
            _check_cuda(out_grad, "out_grad", device)
        grad = out_grad
    elif want_grad:
        grad = torch.empty_like(logits)
    rows = ids.numel()
    lib = N.load()
    with _device_guard(device):
        loss = torch.empty((), dtype=torch.float32, device=device)
        row_losses = torch.empty_like(ids, dtype=torch.float32)
        code = lib.dspark_markov_block_cross_entropy(
            logits.data_ptr(), ids.data_ptr(), weights.data_ptr() if weights is not None else None, rows, vocab,
            ignore_index, reduction == "mean", loss.data_ptr(), row_losses.data_ptr(),
            grad.data_ptr() if grad is not None else None, _DT[dtype], _stream_ptr(device))
    if code:
        N.check(code, "dspark_markov_block_cross_entropy")
    return loss, row_losses, grad


class GradientClipper:
    """The global norm over ``grads`` and clipping by it, for buffers that stay
    where they are from step to step (a flat bucket's views, the head's dW1 and
    dW2).

    ``grads``: contiguous fp32 or bf16 CUDA tensors on one device that do not
    overlap. ``out``: tensors of the same shapes and dtypes that take the
    clipped gradients (each its gradient itself or memory that overlaps none of
    them); None: in place. Creating the object lays the tensors out as a plan
    in device memory: a host-to-device copy for which the host waits, and with
    it for the work before it on the stream. During a graph capture that is
    refused; create the object before. ``clip`` reads what the tensors hold at each call. Calls of one object are
    ordered on one stream or by events, as anything that writes the same
    tensors is; the object is kept until they have run.
    """

    def __init__(self, grads: Sequence[torch.Tensor], *, out: Optional[Sequence[torch.Tensor]] = None):
        grads = list(grads)
        outs = grads if out is None else list(out)
        if len(outs) != len(grads):
            raise ValueError("out must have one tensor for each gradient")
        self.device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
        for i, (g, o) in enumerate(zip(grads, outs)):
            if g.dtype not in _DT:
                raise ValueError("gradients must be float32 or bfloat16")
            if o.shape != g.shape or o.dtype != g.dtype:
                raise ValueError("out must match the gradients in shape and dtype")
            _check_cuda(g, f"grads[{i}]", self.device)
            if o is not g:
                _check_cuda(o, f"out[{i}]", self.device)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a GradientClipper is created before a graph capture, not during it")
        self.grads, self.outs = grads, outs
        self._starts = sorted((g.data_ptr(), i) for i, g in enumerate(grads) if g.numel())
        lib = N.load()
        n = len(grads)
        args = ((ctypes.c_void_p * n)(*[g.data_ptr() for g in grads]), (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs]),
                (ctypes.c_int64 * n)(*[g.numel() for g in grads]), (ctypes.c_int32 * n)(*[_DT[g.dtype] for g in grads]), n)
        pieces = ctypes.c_int64(0)
        self._checked(lib.dspark_markov_clip_plan(*args, None, 0, ctypes.byref(pieces)))
        self._pieces = pieces.value
        plan = (N.ClipPiece * max(1, self._pieces))()
        self._checked(lib.dspark_markov_clip_plan(*args, plan, self._pieces, ctypes.byref(pieces)))
        self._plan = torch.frombuffer(plan, dtype=torch.uint8).to(self.device)
        # Calls of one object write one set of outputs, so they are ordered and can share this.
        self._work = torch.empty(N.DSPARK_CLIP_SCRATCH_BYTES, dtype=torch.uint8, device=self.device)
        self._call = lib.dspark_markov_clip_grad_norm
        self._fixed = (self._plan.data_ptr(), self._work.data_ptr())

    @staticmethod
    def _checked(code: int) -> None:
        if code == N.DSPARK_ERR_INVALID_ARG:
            raise ValueError("gradients and outputs must not overlap one another")
        N.check(code, "dspark_markov_clip_plan")

    def clipped(self, grad: torch.Tensor) -> torch.Tensor:
        """Where ``clip`` leaves ``grad``, which is one of ``grads`` or a contiguous
        part of one: ``grad`` itself, or its place in ``out``."""
        at, size = grad.data_ptr(), grad.element_size()
        k = bisect.bisect_right(self._starts, (at, len(self.grads))) - 1
        if k >= 0 and grad.is_contiguous() and grad.device == self.device:
            start, i = self._starts[k]
            g, o = self.grads[i], self.outs[i]
            if g.dtype == grad.dtype and at + grad.numel() * size <= start + g.numel() * size:
                if o.data_ptr() == start:
                    return grad
                return o.view(-1)[(at - start) // size:][: grad.numel()].view(grad.shape)
        raise ValueError("not one of the clipper's gradients")

    @_ranged
    def clip(self, max_norm: float) -> torch.Tensor:
        """Scales by min(1, max_norm / (norm + 1e-6)) and returns the norm before
        it, an fp32 scalar on the device. ``max_norm`` inf only measures (and
        copies to ``out``), whatever the norm; otherwise an infinite norm
        scales by 0 and a NaN norm by NaN."""
        max_norm = float(max_norm)
        if math.isnan(max_norm) or max_norm < 0.0:
            raise ValueError("max_norm must not be negative or NaN")
        device = self.device
        plan, work = self._fixed
        with _device_guard(device):
            norm = torch.empty((), dtype=torch.float32, device=device)
            code = self._call(plan, self._pieces, max_norm, norm.data_ptr(), work, _stream_ptr(device))
        if code:
            N.check(code, "dspark_markov_clip_grad_norm")
        return norm


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, *,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """``GradientClipper(grads, out=out).clip(max_norm)`` for buffers that are
    clipped once. Making the object stops the host until the stream's work so
    far has run, and is refused during a graph capture; buffers that are clipped
    again and again want an object that is kept."""
    return GradientClipper(grads, out=out).clip(max_norm)
