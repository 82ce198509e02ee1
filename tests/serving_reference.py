"""Plain 64-bit statements of the serving operators (shared by their tests,
not a test module): the append of keys and values, attention over the cache,
and the expert layer, written from their formulas on NumPy arrays."""
from __future__ import annotations

import numpy as np

import oracle
from oracle.formats import e4m3_decode, e4m3_encode, e8m0_ceil_exponent

MIN_EXP = -32


def append(x, cache, scales, table, offsets, lens):
    """x float (total, heads, dim); cache uint8 (pages, heads, page, dim) and
    scales uint8 (pages, heads), changed in place."""
    page = cache.shape[2]
    for b in range(len(lens)):
        t0, n = offsets[b], offsets[b + 1] - offsets[b]
        start = lens[b] - n
        for pos in sorted({(start + i) // page for i in range(n)}):
            lo, hi = max(start, pos * page), min(lens[b], (pos + 1) * page)
            pid, first = table[b][pos], lo - pos * page
            for h in range(cache.shape[1]):
                new = x[t0 + lo - start:t0 + hi - start, h].astype(np.float32)
                amax = np.float32(np.abs(new).max())
                e = MIN_EXP if amax == 0 else max(MIN_EXP, int(e8m0_ceil_exponent(amax / np.float32(448))))
                if first > 0:
                    old = int(scales[pid, h]) - 127
                    if e > old:
                        kept = e4m3_decode(cache[pid, h, :first]) * 2.0 ** (old - e)
                        cache[pid, h, :first] = e4m3_encode(kept.astype(np.float32))
                    e = max(e, old)
                cache[pid, h, first:first + hi - lo] = e4m3_encode((new.astype(np.float64) * 2.0 ** -e).astype(np.float32))
                scales[pid, h] = e + 127


def attention(q, k_cache, v_cache, k_scales, v_scales, table, offsets, lens, sm_scale, causal, window):
    """In float64: out, lse, sum_j p_j |v_j|, the row's largest sm_scale sum
    |q||k|, and what an absolute error of 1 in every weight relative to the
    largest could add: 2^ev* sum_j |c_j| (v = c 2^ev; ev* of the key with
    the largest weight 2^(score log2 e + ev))."""
    total, heads, dim = q.shape
    kv_heads, page = k_cache.shape[1], k_cache.shape[2]
    group = heads // kv_heads
    out, mag, low = np.zeros((3, total, heads, dim))
    lse, size = np.full((total, heads), -np.inf), np.zeros((total, heads))
    for b in range(len(lens)):
        t0, n, length = offsets[b], offsets[b + 1] - offsets[b], lens[b]
        if length == 0 or n == 0:
            continue
        ids = [table[b][i] for i in range(-(-length // page))]
        for h in range(kv_heads):
            k, v = (np.concatenate([e4m3_decode(c[i, h]) * 2.0 ** (int(s[i, h]) - 127) for i in ids])[:length]
                    for c, s in ((k_cache, k_scales), (v_cache, v_scales)))
            ev = np.repeat([int(v_scales[i, h]) - 127 for i in ids], page)[:length]
            j = np.arange(length)[None]
            pos = (length - n + np.arange(n))[:, None]
            see = np.ones((n, length), bool)
            if causal:
                see &= j <= pos
            if window:
                see &= pos - j < window
            for g in range(h * group, (h + 1) * group):
                qq = q[t0:t0 + n, g].astype(np.float64)
                s = np.where(see, qq @ k.T * sm_scale, -np.inf)
                top = s.max(1, initial=-np.inf)
                ok = top > -np.inf
                p = np.exp(s - np.where(ok, top, 0)[:, None])
                l = p.sum(1)
                with np.errstate(divide="ignore"):
                    lse[t0:t0 + n, g] = np.where(ok, top + np.log(l), -np.inf)
                p /= np.where(ok, l, 1)[:, None]
                out[t0:t0 + n, g] = p @ v
                mag[t0:t0 + n, g] = p @ np.abs(v)
                star = ev[np.argmax(s * np.log2(np.e) + ev, axis=1)].astype(np.float64)
                low[t0:t0 + n, g] = 2.0 ** star[:, None] * (see @ (np.abs(v) * 2.0 ** -ev.astype(np.float64)[:, None]))
                size[t0:t0 + n, g] = np.where(see, np.abs(qq) @ np.abs(k).T * abs(sm_scale), 0).max(1, initial=0)
    return out, lse, mag, size, low


def quantized_values(fmt, rows_f32, tsf):
    """What FP32 rows (exact BF16 values) stand for once quantized."""
    bits = (np.ascontiguousarray(rows_f32, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return oracle.dequantize(fmt, *oracle.quantize_rank2(fmt, bits, tsf), tsf)


def bf16(x):
    """float64 -> nearest BF16 (through FP32), as float32."""
    u = np.ascontiguousarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def moe(fmt, x, logits, w13, w2, top_k, x_sf, h_sf, renormalize):
    """y and its tolerance.  w13 (experts, 2*inter, hidden), w2 (experts, hidden,
    inter): the weights' values.

    The kernel sums in FP32, so g and u are off by at most e = K 2^-24 sum
    |x||w|; h then may fall on the other side of a BF16 or code boundary.  The
    codes at the corners g +- e, u +- e bound by how much each value of Q(h)
    can differ, and |w2| carries that to y.  To it come the FP32 sums of the
    second product and the rounding of y to BF16."""
    tokens, hidden = x.shape
    inter = w2.shape[2]
    y, tol = np.zeros((2, tokens, hidden))
    for t in range(tokens):
        z = logits[t].astype(np.float64)
        ids = np.argsort(-z, kind="stable")[:top_k]
        if not np.isfinite(z.max()):
            continue
        p = np.exp(z - z.max())
        p /= p.sum()
        w = p[ids] / (p[ids].sum() if renormalize else 1)
        for e, pe in zip(ids, w):
            xq = quantized_values(fmt, x[t:t + 1], x_sf[e])[0]
            gu = w13[e] @ xq
            err = np.abs(w13[e]) @ np.abs(xq) * hidden * 2.0 ** -24

            def codes(sg, su):
                g, u = gu[:inter] + sg * err[:inter], gu[inter:] + su * err[inter:]
                with np.errstate(over="ignore"):
                    h = g / (1 + np.exp(-g)) * u
                return quantized_values(fmt, bf16(h)[None], h_sf[e])[0]

            hq = codes(0, 0)
            off = np.max([np.abs(codes(a, b) - hq) for a in (-1, 1) for b in (-1, 1)], axis=0)
            y[t] += pe * (w2[e] @ hq)
            tol[t] += pe * (np.abs(w2[e]) @ (off + np.abs(hq) * (inter + 16) * 2.0 ** -24))
    return y, tol * 1.01 + np.abs(y) * 2.0 ** -8 + 1e-30
