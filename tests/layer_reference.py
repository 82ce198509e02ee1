"""Plain 64-bit statements of the calls between cache and experts (shared by
their tests, not a test module): products with packed weights, norm and
rotation of heads, routing and the rows' order, on NumPy arrays."""
from __future__ import annotations

import numpy as np

import oracle


def weights(fmt, packed, scales5d, rows, cols, sf=1.0):
    """float64 (rows, cols): what codes and 5D scales stand for."""
    s = cols // oracle.block_size(fmt)
    return oracle.dequantize(fmt, packed, oracle.layout.scales_from_5d_view(scales5d, rows, s)[:rows, :s], np.float32(1)).astype(np.float64) / float(sf)


def half_step(y, dtype):
    """Rounding of y to the type: half a unit in the last place, or half the least subnormal."""
    rel, low = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 2.0 ** -150)}[dtype]
    return np.abs(y) * rel + low


def linear(x, w, add, out):
    """y and its tolerance.  FP32 sums of exact products: a sum of k products is off by at most one unit (2^-23) of the
    magnitudes' sum per step, 16 products make a step, and up to 64 warps' and blocks' sums are added to that.  BF16 values
    below 2^-31 of the token's largest may be off by 2^-39 of it.  Then the division by the tensor scale, add, and rounding."""
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = mag * ((x.shape[1] / 16 + 64) * 2.0 ** -23) + np.abs(x).max(1, keepdims=True, initial=0) * 2.0 ** -39 * np.abs(w).sum(1)[None]
    if add is not None:
        y = y + add
        tol = tol + np.abs(y) * 2.0 ** -23
    return y, tol + np.abs(y) * 2.0 ** -23 + half_step(y, out)


def rope(x, w, positions, inv_freq, eps, interleaved, dtype):
    """One of q, k: float64 result and tolerance.  Relative to the pair's sides: sum of squares 13 steps / 2, its root 2, the
    factors 3, the angle (a fraction of a turn rounded to 24 bits, at most pi 2^-24) 4, sine and cosine 2, the two
    products and their sum 3: 21 units of 2^-24, taken as 32."""
    n, dim = len(inv_freq), x.shape[2]
    u = x if w is None else x / np.sqrt((x ** 2).mean(2, keepdims=True) + eps) * w
    y, size = u.copy(), np.abs(u)
    a = positions.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    y[..., i] = u[..., i] * np.cos(a) - u[..., j] * np.sin(a)
    y[..., j] = u[..., j] * np.cos(a) + u[..., i] * np.sin(a)
    size[..., i] = size[..., j] = np.abs(u[..., i]) + np.abs(u[..., j])
    return y, size * 2.0 ** -19 + half_step(y, dtype)


def route(z, top_k, sigmoid, bias, groups, top_groups, group_top, renormalize, scale):
    """ids and weights in float64; logits that are NaN or +inf count as -inf."""
    z = np.where(z < np.inf, z, -np.inf).astype(np.float64)
    tokens, experts = z.shape
    per = experts // groups
    ids, weights = np.zeros((tokens, top_k), np.int32), np.zeros((tokens, top_k))
    for t in range(tokens):
        some = z[t].max() > -np.inf
        with np.errstate(over="ignore"):
            if sigmoid:
                p = 1 / (1 + np.exp(-z[t]))
            else:
                p = np.exp(z[t] - z[t].max()) if some else np.zeros(experts)
                p = p / p.sum() if some else p
        p = np.where(z[t] > -np.inf, p, 0)
        value = z[t] if bias is None else np.where(z[t] > -np.inf, p + bias, -np.inf)
        if groups > 1:
            of = p if bias is None and group_top == 2 else value
            score = np.sort(of.reshape(groups, per), 1)[:, ::-1][:, :group_top].sum(1)
            kept = np.argsort(-score, kind="stable")[:top_groups]
            value = np.where(np.isin(np.arange(experts) // per, kept), value, -np.inf)
        ids[t] = np.argsort(-value, kind="stable")[:top_k]
        # of logarithms: ratios of scores that are below 64 bits' range stay what they are
        log = np.where(z[t] > -np.inf, np.minimum(z[t], 0) - np.log1p(np.exp(-np.abs(z[t]))) if sigmoid else z[t], -np.inf)[ids[t]]
        w = np.exp(log - log.max()) if renormalize and log.max() > -np.inf else p[ids[t]]
        weights[t] = (w / w.sum() if renormalize and w.sum() > 0 else w) * scale
    return ids, weights


def rows(ids, experts):
    """row_offsets, scales_offsets, row_indices, positions."""
    flat = ids.ravel()
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(experts)])
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    indices, positions = np.zeros(flat.size, np.int32), np.full(flat.size, -1, np.int32)
    indices[:order.size] = order // ids.shape[1]
    positions[order] = np.arange(order.size)
    cut = lambda c: np.concatenate([[0], np.cumsum(c)]).astype(np.int32)  # noqa: E731
    return cut(counts), cut(-(-counts // 128) * 128), indices, positions.reshape(ids.shape)
