"""Token constraints on corrected logits: penalties for repeated tokens,
additive biases and grammar masks.

They stand between the head's corrected logits and the token. A serving loop
keeps one ``TokenConstraints`` for its batch, appends the accepted tokens to
the history behind it, and passes it to ``VanillaMarkov.sample_block_tokens``
(drafting) and to ``process_logits`` (single positions, or a drafted block
that is being verified). For row (b, k) with logit x of id v, n generated
occurrences of v (the history past the prompt, and the drafted tokens before
position k), in fp32 and in this order:

    seen (n > 0 or v in the prompt):  x = x / repetition if x > 0 else x * repetition
    n > 0:                            x = (x - frequency * n) - presence
    biased:                           x = x + bias
    not allowed:                      x = -inf

with one rounding to the logits' dtype at the end.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple, Union

import torch

from . import _native as N
from .head import _DT, _check_cuda, _device_guard, _ranged, _stream_ptr

Penalty = Union[float, torch.Tensor]


class TokenConstraints:
    """The constraints of one batch of sequences, over caller-owned buffers.

    history         [B, L] int64, rows contiguous along L: each sequence's tokens, of which the first
                    ``history_lens[b]`` ([B] int64, default L; clamped to [0, L]) count and the first
                    ``prompt_lens[b]`` ([B] int64, default 0) are its prompt. Prompt tokens count for
                    the repetition penalty only, the others for all three.
    repetition_penalty, frequency_penalty, presence_penalty
                    a number for all sequences or a [B] fp32 tensor (1, 0 and 0 change nothing; the
                    repetition penalty is positive).
    bias_ids, bias_values
                    [B, K] or [K] (for all sequences) int64 and fp32. A negative id is an unused entry;
                    of several entries with one id the last counts.

    The object keeps the tensors and reads what they hold at each call, so a
    loop updates them in place. Ids outside the vocabulary are left out and set
    the TOKEN_RANGE status bit.
    """

    def __init__(self, vocab_size: int, *, history: Optional[torch.Tensor] = None,
                 history_lens: Optional[torch.Tensor] = None, prompt_lens: Optional[torch.Tensor] = None,
                 repetition_penalty: Penalty = 1.0, frequency_penalty: Penalty = 0.0,
                 presence_penalty: Penalty = 0.0, bias_ids: Optional[torch.Tensor] = None,
                 bias_values: Optional[torch.Tensor] = None):
        self.vocab_size = int(vocab_size)
        if self.vocab_size <= 0:
            raise ValueError("vocab_size must be positive")
        self.batch: Optional[int] = None  # None: any (nothing here belongs to one sequence)
        self.device: Optional[torch.device] = None
        self._kept = []
        c = N.Constraints()
        if history is None and (history_lens is not None or prompt_lens is not None):
            raise ValueError("history_lens and prompt_lens need history")
        if history is not None:
            if history.dim() != 2 or history.dtype != torch.int64:
                raise ValueError("history must be int64 [B, L]")
            if history.shape[1] > 1 and history.stride(1) != 1:
                raise ValueError("history's rows must be contiguous")
            self._take(history, "history", history.shape[0], strided=True)
            c.history, c.history_cap, c.history_stride = history.data_ptr(), history.shape[1], history.stride(0)
        for name, t in (("history_lens", history_lens), ("prompt_lens", prompt_lens)):
            if t is not None:
                if t.dim() != 1 or t.dtype != torch.int64:
                    raise ValueError(f"{name} must be int64 [B]")
                self._take(t, name, t.shape[0])
                setattr(c, name, t.data_ptr())
        for name, x in (("repetition", repetition_penalty), ("frequency", frequency_penalty),
                        ("presence", presence_penalty)):
            if isinstance(x, torch.Tensor):
                if x.dim() != 1 or x.dtype != torch.float32:
                    raise ValueError(f"{name}_penalty must be a number or fp32 [B]")
                self._take(x, f"{name}_penalty", x.shape[0])
                setattr(c, name, x.data_ptr())
            else:
                x = ctypes.c_float(float(x)).value  # as the kernel gets it
                if not math.isfinite(x) or (name == "repetition" and x <= 0.0):
                    raise ValueError(f"{name}_penalty must be finite" + (" and positive" if name == "repetition" else ""))
                setattr(c, name + "_value", x)
        if (bias_ids is None) != (bias_values is None):
            raise ValueError("bias_ids and bias_values come together")
        if bias_ids is not None:
            if bias_ids.dim() not in (1, 2) or bias_ids.shape != bias_values.shape:
                raise ValueError("bias_ids and bias_values must both be [K] or [B, K]")
            if bias_ids.dtype != torch.int64 or bias_values.dtype != torch.float32:
                raise ValueError("bias_ids must be int64 and bias_values float32")
            rows = bias_ids.shape[0] if bias_ids.dim() == 2 else None
            self._take(bias_ids, "bias_ids", rows)
            self._take(bias_values, "bias_values", rows)
            c.bias_count = bias_ids.shape[-1]
            c.bias_stride = c.bias_count if rows is not None else 0
            c.bias_ids, c.bias_values = bias_ids.data_ptr(), bias_values.data_ptr()
        self._c = c
        self._ref = ctypes.byref(c)
        self._sizes = {}

    def _scratch(self, device: torch.device, batch: int, block: int, drafted: int, choose: bool) -> Optional[torch.Tensor]:
        """Working memory of one call, its size kept by the call's sizes."""
        key = (batch, block, drafted, choose)
        size = self._sizes.get(key)
        if size is None:
            size = N.load().dspark_markov_constrain_scratch_bytes(
                batch, block, self.vocab_size, self._c.history_cap, self._c.bias_count, drafted, choose)
            if len(self._sizes) < 256:
                self._sizes[key] = size
        return torch.empty(size, dtype=torch.uint8, device=device) if size else None

    def _take(self, t: torch.Tensor, name: str, rows: Optional[int], strided: bool = False) -> None:
        if not t.is_cuda or (self.device is not None and t.device != self.device):
            raise ValueError(f"{name} must be a CUDA tensor" + (f" on {self.device}" if self.device else ""))
        if not strided and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if rows is not None:
            if self.batch is not None and rows != self.batch:
                raise ValueError(f"{name} is for {rows} sequences, not {self.batch}")
            self.batch = rows
        self.device = t.device
        self._kept.append(t)

    def _check(self, batch: int, vocab: int, device: torch.device) -> None:
        if vocab != self.vocab_size:
            raise ValueError(f"vocab mismatch: logits {vocab} vs constraints {self.vocab_size}")
        if self.batch is not None and batch != self.batch:
            raise ValueError(f"batch mismatch: logits {batch} vs constraints {self.batch}")
        if self.device is not None and device != self.device:
            raise ValueError(f"the constraints are on {self.device}")


def _allowed_args(allowed: Optional[torch.Tensor], batch: int, block: int, vocab: int,
                  device: torch.device) -> Tuple[Optional[int], int, int]:
    """(pointer, sequence stride, row stride) of a bit mask [B, W] or [B, M, W]."""
    if allowed is None:
        return None, 0, 0
    words = (vocab + 31) // 32
    if allowed.dtype != torch.int32:
        raise ValueError("allowed must be int32 words of 32 bits")
    if allowed.device != device:
        raise ValueError(f"allowed must be a CUDA tensor on {device}")
    shape, stride = allowed.shape, allowed.stride()
    if tuple(shape) not in ((batch, words), (batch, block, words)):
        raise ValueError(f"allowed must be [{batch}, {words}] or [{batch}, {block}, {words}]")
    if words > 1 and stride[-1] != 1:
        raise ValueError("allowed's rows must be contiguous")
    return allowed.data_ptr(), stride[0], stride[1] if len(shape) == 3 else 0


@_ranged
def process_logits(logits: torch.Tensor, constraints: TokenConstraints, *,
                   draft_tokens: Optional[torch.Tensor] = None, allowed: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, out_tokens: Optional[torch.Tensor] = None,
                   return_tokens: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Constrained logits and the greedy token of every row.

    ``logits`` (B, V) (one position of each sequence) or (B, M, V) (a block),
    fp32 or bf16, unit stride along V and any strides before it.
    ``draft_tokens`` (B, M) int64: position k's history is its sequence's and
    the first k of these (a negative id is padding); None: no drafted tokens.
    ``allowed`` int32 (B, W) or (B, M, W), W = ceil(V / 32): token v is allowed
    where bit v % 32 of word v // 32 is set; a row that allows nothing becomes
    all -inf and its token 0. ``out`` may be ``logits`` (in place). Returns
    (logits, tokens): the constrained logits in the same dtype and, unless
    ``return_tokens`` is False, the lowest index of each row's largest value
    (NaN counts as the largest), int64 (B,) or (B, M)."""
    dim = logits.dim()
    if dim == 2:
        batch, vocab = logits.shape
        block = 1
    elif dim == 3:
        batch, block, vocab = logits.shape
    else:
        raise ValueError("logits must be (B, V) or (B, M, V)")
    dtype, device = logits.dtype, logits.device
    if dtype not in _DT:
        raise ValueError("logits must be float32 or bfloat16")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    constraints._check(batch, vocab, device)
    istride = logits.stride()
    if out is None:
        out = torch.empty(logits.shape, dtype=dtype, device=device)
        ostride = out.stride()
    elif out is logits:
        ostride = istride
    else:
        ostride = out.stride()
        if out.shape != logits.shape or out.dtype != dtype or out.device != device:
            raise ValueError("out must match logits in shape, dtype and device")
    if vocab > 1 and (istride[-1] != 1 or ostride[-1] != 1):
        raise ValueError("logits and out need unit stride along the vocabulary")
    draft = None
    if draft_tokens is not None:
        if dim != 3 or tuple(draft_tokens.shape) != (batch, block) or draft_tokens.dtype != torch.int64:
            raise ValueError("draft_tokens must be int64 (B, M) beside (B, M, V) logits")
        _check_cuda(draft_tokens, "draft_tokens", device)
        draft = draft_tokens.data_ptr()
    mask, mask_batch, mask_row = _allowed_args(allowed, batch, block, vocab, device)
    tokens = None
    if return_tokens or out_tokens is not None:
        if out_tokens is None:
            tokens = torch.empty(logits.shape[:-1], dtype=torch.int64, device=device)
        else:
            tokens = out_tokens
            if tokens.shape != logits.shape[:-1] or tokens.dtype != torch.int64:
                raise ValueError("out_tokens must be int64 (B,) or (B, M)")
            _check_cuda(tokens, "out_tokens", device)
    if batch == 0 or block == 0:
        return out, tokens
    lib = N.load()
    with _device_guard(device):
        scratch = constraints._scratch(device, batch, block, block - 1 if draft is not None else 0, tokens is not None)
        code = lib.dspark_markov_process_logits(
            logits.data_ptr(), out.data_ptr(), batch, block, vocab, istride[0], istride[1] if dim == 3 else vocab,
            ostride[0], ostride[1] if dim == 3 else vocab, constraints._ref, draft, block, 0, mask, mask_batch,
            mask_row, tokens.data_ptr() if tokens is not None else None, block, 0.0, 0,
            scratch.data_ptr() if scratch is not None else None, _DT[dtype], _stream_ptr(device))
    if code:
        N.check(code, "dspark_markov_process_logits")
    return out, tokens
