"""What stands around the head, in 64 bits: token constraints, the training
loss with its gradient, and gradient clipping.

TEST INFRASTRUCTURE. Plain numpy from the formulas, one row or token at a time,
with the error bounds that the tests hold the kernels to. u = 2^-24 is half a
step of binary32: one rounding moves a value by at most u relative to it.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
# exp evaluated as ex2 of a product by log2 e: CUDA states 2 ulp + floor(abs(1.16 x)) ulp for expf's fast form,
# that is (2 + 1.16 |x|) 2^-23 relative.
EXP_ULPS, EXP_ULPS_PER_X = 2.0, 1.16
# Sums of non-negative terms in any tree or chain of at most n additions err by n u relative to the sum.


def allowed_from_words(words: np.ndarray, vocab: int) -> np.ndarray:
    """Truth values [..., vocab] of bit masks [..., ceil(vocab / 32)] (int32)."""
    w = np.ascontiguousarray(words).astype(np.int64) & 0xFFFFFFFF
    v = np.arange(vocab)
    return ((w[..., v // 32] >> (v % 32)) & 1).astype(bool)


def constrain_row(row, prompt, generated, repetition, frequency, presence, biases, allowed):
    """One row: (exact values, absolute error bound before the last rounding).

    Each fp32 operation rounds once: with the intermediate values x1 = x rho or
    x / rho, t = f n, x2 = x1 - t, x3 = x2 - p, x4 = x3 + beta the error is at
    most u (|x1| + |t| + |x2| + |x3| + |x4|) (1 + small), doubled here to cover
    the second-order terms."""
    x = np.array(row, dtype=np.float64)
    err = np.zeros_like(x)
    counts = {}
    for t in generated:
        counts[int(t)] = counts.get(int(t), 0) + 1
    last = {}
    for i, b in biases:
        last[int(i)] = float(b)
    seen = set(int(t) for t in prompt) | set(counts)
    with np.errstate(invalid="ignore", over="ignore"):
        for v in seen | set(i for i in last if i >= 0):
            if not 0 <= v < len(x):
                continue
            e = 0.0
            if v in seen:
                x[v] = x[v] / repetition if x[v] > 0 else x[v] * repetition
                e += abs(x[v])
            n = counts.get(v, 0)
            if n:
                e += abs(frequency * n)
                x[v] -= frequency * n
                e += abs(x[v])
                x[v] -= presence
                e += abs(x[v])
            if v in last:
                x[v] += last[v]
                e += abs(x[v])
            err[v] = 2 * U32 * e if np.isfinite(e) else 0.0
    if allowed is not None:
        x[~allowed] = -np.inf
        err[~allowed] = 0.0
    return x, err


def choose(row) -> int:
    """The lowest index of the largest value; NaN counts as the largest."""
    row = np.asarray(row, dtype=np.float64)
    if np.isnan(row).any():
        return int(np.flatnonzero(np.isnan(row))[0])
    return int(np.flatnonzero(row == row.max())[0])


def cross_entropy(logits, targets, weights, ignore_index, mean, out_dtype):
    """(loss, row losses, gradient) in 64 bits, and the bounds of their errors."""
    c = np.asarray(logits, dtype=np.float64)
    rows, vocab = c.shape
    w = np.ones(rows) if weights is None else np.asarray(weights, dtype=np.float64)
    live = [i for i in range(rows) if targets[i] != ignore_index and 0 <= targets[i] < vocab and w[i] != 0]
    total = float(sum(w[i] for i in live)) if mean else 1.0
    inv = 1.0 / total if total != 0 else 0.0
    row = np.zeros(rows)
    row_err = np.zeros(rows)
    grad = np.zeros_like(c)
    grad_err = np.zeros_like(c)
    for i in live:
        x, t = c[i], int(targets[i])
        m = x.max()
        if np.isnan(x).any() or not np.isfinite(m):
            row[i] = np.nan
            grad[i] = np.nan
            continue
        d = x - m
        e = np.exp(d)
        s = e.sum()
        row[i] = np.log(s) - d[t]
        p = e / s
        one = np.zeros(vocab)
        one[t] = 1.0
        grad[i] = w[i] * inv * (p - one)
        # exp's own error and the rounding of its argument (|d| u, as an absolute error of the exponent), doubled for
        # the rescaling of a partial sum by another such exp; weighted as the terms are. Then the sum's additions: at
        # most `vocab` one after another.
        fin = np.where(np.isfinite(d), d, 0.0)
        rel = 2 * (EXP_ULPS + (EXP_ULPS_PER_X + 1) * np.abs(fin)) * 2 * U32
        depth = min(vocab, 1024) * U32
        rel_s = float((p * rel).sum()) + depth
        row_err[i] = rel_s + 4 * U32 * (abs(np.log(s)) + abs(fin[t]) + 1.0)
        if not np.isfinite(d[t]):
            row_err[i] = 0.0
        perr = p * (rel + rel_s + 4 * U32)
        grad_err[i] = abs(w[i] * inv) * (perr + 4 * U32 * np.abs(p - one)) + HALF_STEP[out_dtype] * np.abs(grad[i])
    loss = float(sum(w[i] * row[i] for i in live) * inv)
    loss_err = float(sum(abs(w[i]) * row_err[i] for i in live) * abs(inv)) + 4 * U32 * float(
        sum(abs(w[i] * row[i]) for i in live) * abs(inv))
    # Where a gradient lies below the smallest normal number a step is absolute.
    tiny = {"bf16": 2.0 ** -126, "fp32": 2.0 ** -126}[out_dtype]
    return (loss, loss_err), (row, row_err), (grad, grad_err + tiny)


def clip(grads, max_norm):
    """(norm, factor) of the global norm in 64 bits."""
    total = 0.0
    for g in grads:
        g = np.asarray(g, dtype=np.float64)
        total += float((g * g).sum())
    norm = float(np.sqrt(total))
    return norm, min(1.0, max_norm / (norm + 1e-6))


# The clipper forms squares of four elements and their sum in 32 bits, three roundings one after another at most (a
# square, the multiply-add of another one, the sum of two such), halved by the root; the root is rounded once. The rest
# is 64-bit: up to 2^17 additions in a row of 2^-53 each, halved too.
CLIP_NORM_REL = 3 * U32 / 2 + U32 + 2.0 ** -37
