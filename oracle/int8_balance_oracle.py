"""Plain float64 oracle (numpy) of the 8-bit integer rows and products, of the norm in
front of them, and of the router's balance loss.

TEST INFRASTRUCTURE, written from the definitions; it shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def int8_scales(v):
    """float32 scales of the rows of float64 values; NaN for a row that is not finite."""
    top = np.where(np.isfinite(v).all(-1), np.abs(np.where(np.isfinite(v), v, 0)).max(-1), np.nan)
    return (top / 127.0).astype(np.float32)


def int8_quotients(v, scales):
    """What is rounded to codes: the quotients of v and the scales, 0 where codes are 0."""
    s = np.asarray(scales, dtype=np.float64)[..., None]
    ok = s > 0
    with np.errstate(invalid="ignore"):
        return np.where(ok, np.where(np.isfinite(v), v, 0) / np.where(ok, s, 1.0), 0.0)


def int8_quantize(v):
    """(codes int8, scales float32) of the rows of float64 values."""
    v = np.asarray(v, dtype=np.float64)
    scales = int8_scales(v)
    codes = np.clip(np.rint(int8_quotients(v, scales)), -127, 127).astype(np.int8)
    return codes, scales


def rms_norm(x, weight, eps, residual=None):
    """(h, n) in float64."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + residual
    with np.errstate(invalid="ignore", divide="ignore"):
        return h, h * weight / np.sqrt((h * h).sum(-1, keepdims=True) / h.shape[-1] + eps)


def int8_sums(x, w, row_expert=None):
    """Integer sums [M, N] (int64) of codes; rows with a negative expert get zeros."""
    x, w = x.astype(np.int64), w.astype(np.int64)
    if row_expert is None:
        return x @ w.T
    out = np.zeros((x.shape[0], w.shape[1]), dtype=np.int64)
    for e in range(w.shape[0]):
        at = np.asarray(row_expert) == e
        out[at] = x[at] @ w[e].T
    return out


def int8_product(x, x_scales, w, w_scales, row_expert=None):
    """y [M, N]: the sums and the two products by scales, each rounded to fp32."""
    s = int8_sums(x, w, row_expert).astype(np.float32)
    ws = w_scales[None, :] if row_expert is None else w_scales[np.maximum(row_expert, 0)]
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        return s * np.asarray(x_scales, dtype=np.float32)[:, None] * ws.astype(np.float32)


def softmax(logits):
    """Probabilities [T, E] in float64; zeros for a row of -inf alone."""
    z = np.asarray(logits, dtype=np.float64)
    top = z.max(1, keepdims=True)
    p = np.exp(z - np.where(np.isneginf(top), 0, top))
    total = p.sum(1, keepdims=True)
    return np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))


def balance_loss(logits, topk_ids, mask=None):
    """(loss, counts, mean_probs, n, p of the tokens that take part)."""
    T, E = logits.shape
    keep = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    p = softmax(logits[keep])
    ids = np.asarray(topk_ids)[keep]
    counts = np.array([(ids == e).sum() for e in range(E)], dtype=np.int64)
    n = int(keep.sum())
    mean = p.sum(0) / max(n, 1)
    loss = E / (max(n, 1) * ids.shape[1]) * float(counts @ mean)
    return loss, counts, mean, n, p


def balance_loss_backward(d_loss, logits, counts, n, top_k, mask=None):
    """(d_logits, its magnitude before the difference) in float64; zeros for masked tokens."""
    T, E = logits.shape
    keep = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    p = softmax(logits[keep])
    c = np.asarray(counts, dtype=np.float64)
    dot = p @ c
    g = d_loss * E / (float(max(n, 1)) ** 2 * top_k) if n else 0.0
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    d[keep] = g * p * (c[None, :] - dot[:, None])
    mag[keep] = abs(g) * p * (np.abs(c[None, :] - dot[:, None]) + dot[:, None])
    return d, mag
