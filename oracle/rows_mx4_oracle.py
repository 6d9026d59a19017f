"""Plain float64 oracle (numpy) of the rows in expert order, of MX4 quantisation
and of the products with MX4 weights.

TEST INFRASTRUCTURE, written from the definitions: pairs are visited one at a
time, blocks of 32 are quantised by comparing with the e2m1 grid, products are
dot products of decoded rows.  It shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------------------
# rows in expert order
# ---------------------------------------------------------------------------
def pair_rows_of(sorted_pair_ids, num_pairs):
    """Row of each pair in a layout, -1 where it has none."""
    rows = np.full(num_pairs, -1, dtype=np.int64)
    for r, p in enumerate(np.asarray(sorted_pair_ids)):
        if 0 <= p < num_pairs:
            assert rows[p] == -1, "a pair has two rows"
            rows[p] = r
    return rows


def permute(x, pair_rows, top_k, num_rows):
    """(rows, written): rows[r(t, j)] = x[t]; `written` marks rows that have a pair."""
    rows = np.zeros((num_rows, x.shape[1]), dtype=x.dtype)
    written = np.zeros(num_rows, dtype=bool)
    for p, r in enumerate(pair_rows):
        if r >= 0:
            rows[r] = x[p // top_k]
            written[r] = True
    return rows, written


def unpermute(rows, pair_rows, top_k, weights=None):
    """(y, sum of magnitudes) in float64."""
    T = len(pair_rows) // top_k
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for p, r in enumerate(pair_rows):
        if r < 0:
            continue
        w = 1.0 if weights is None else float(np.asarray(weights).reshape(-1)[p])
        term = w * rows[r].astype(np.float64)
        y[p // top_k] += term
        mag[p // top_k] += np.abs(term)
    return y, mag


def unpermute_backward(dy, rows, pair_rows, top_k, weights, num_rows):
    """(d_rows, d_weights, magnitudes of the d_weights sums) in float64."""
    T = len(pair_rows) // top_k
    w = np.asarray(weights, dtype=np.float64).reshape(-1)
    d_rows = np.zeros((num_rows, dy.shape[1]))
    d_w = np.zeros(T * top_k)
    mag = np.zeros(T * top_k)
    for p, r in enumerate(pair_rows):
        if r < 0:
            continue
        g = dy[p // top_k].astype(np.float64)
        d_rows[r] = w[p] * g
        prod = g * rows[r].astype(np.float64)
        d_w[p], mag[p] = prod.sum(), np.abs(prod).sum()
    return d_rows, d_w.reshape(T, top_k), mag.reshape(T, top_k)


# ---------------------------------------------------------------------------
# MX4
# ---------------------------------------------------------------------------
def mx4_quantize(x):
    """(codes, scales) of float values [.., K]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(-1, 32)
    codes = np.zeros(b.shape, dtype=np.uint8)
    scales = np.zeros(b.shape[0], dtype=np.uint8)
    for i, blk in enumerate(b):
        if not np.all(np.isfinite(blk)):
            scales[i] = 255
            continue
        a = np.max(np.abs(blk))
        e = -127
        while e < 127 and a >= 2.0 ** (e + 3):     # largest e with 2^(e + 2) <= a
            e += 1
        scales[i] = e + 127
        m = np.abs(blk) / 2.0 ** e
        dist = np.abs(m[:, None] - E2M1[None, :])
        best = dist.min(axis=1, keepdims=True)
        for q in range(32):
            near = np.nonzero(dist[q] == best[q])[0]
            even = [c for c in near if c % 2 == 0]
            c = near[0] if len(near) == 1 else even[0]
            codes[i, q] = c | (8 if np.signbit(blk[q]) else 0)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    lead = x.shape[:-1]
    return (packed.reshape(*lead, x.shape[-1] // 2).astype(np.uint8),
            scales.reshape(*lead, x.shape[-1] // 32))


def mx4_values(codes, scales):
    """Values of MX4 bytes in float64."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def mx4_gemm(x, w, row_expert, silu_mul=False):
    """(out, magnitudes of the product sums) of x [M, K] and w [E, N, K] float64;
    rows whose expert is -1 give NaN (they have no result)."""
    M, N = x.shape[0], w.shape[1]
    y = np.full((M, N), np.nan)
    mag = np.full((M, N), np.nan)
    row_expert = np.asarray(row_expert)
    for e in range(w.shape[0]):
        at = np.nonzero(row_expert == e)[0]
        y[at] = x[at] @ w[e].T
        mag[at] = np.abs(x[at]) @ np.abs(w[e]).T
    if not silu_mul:
        return y, mag
    h = N // 2
    g, u = y[:, :h], y[:, h:]
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    return s * u, (g, u, s, mag[:, :h], mag[:, h:])
