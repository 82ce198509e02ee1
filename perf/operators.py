"""Cases of the serving operators over block-scaled storage: an 8-bit paged
key/value cache (append, attention) and a mixture-of-experts layer for a few
tokens over packed weights.

``listed()`` and ``draw()`` give cases, ``prepare`` a user's tensors, ``run``
one pass (the plain FP32 form, or the library's calls where ``own`` is set),
``work`` the bytes and operations that the pass cannot do without and
``exact`` the result in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
FMT_SF = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the step of every generated token: one new key and value per sequence of a batch
        dict(name="append decode", op="append", batch=64, new_max=1, ragged=False, past_max=900, kv_heads=8, dim=128,
             page=64, dtype="bf16"),
        # a few prompts of different lengths enter the cache at once
        dict(name="append prompt", op="append", batch=6, new_max=4500, ragged=True, past_max=100, kv_heads=8, dim=128,
             page=64, dtype="bf16"),
        # one user's next token over a short context: latency
        dict(name="attn one short", op="attn", batch=1, q_max=1, ragged=False, ctx_min=777, ctx_max=777, heads=32,
             kv_heads=8, dim=128, page=16, dtype="bf16", causal=True, window=0, empty=False),
        # the next token of a full batch with contexts of every length
        dict(name="attn decode batch", op="attn", batch=64, q_max=1, ragged=False, ctx_min=1000, ctx_max=8192, heads=64,
             kv_heads=8, dim=128, page=64, dtype="bf16", causal=True, window=0, empty=False),
        # the next token of two very long contexts
        dict(name="attn decode long", op="attn", batch=2, q_max=1, ragged=False, ctx_min=120001, ctx_max=131072, heads=32,
             kv_heads=4, dim=128, page=64, dtype="bf16", causal=True, window=0, empty=False),
        # checking a few guessed tokens per sequence, sliding window, narrow heads, one sequence without a cache yet
        dict(name="attn verify window", op="attn", batch=33, q_max=5, ragged=True, ctx_min=300, ctx_max=4000, heads=24,
             kv_heads=8, dim=64, page=32, dtype="f16", causal=True, window=1024, empty=True),
        # a chunk of a prompt over what is in the cache so far
        dict(name="attn prompt chunk", op="attn", batch=1, q_max=2048, ragged=False, ctx_min=16384, ctx_max=16384,
             heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", causal=True, window=0, empty=False),
        # one user's next token through an expert layer
        dict(name="moe one nvfp4", op="moe", fmt="nvfp4", tokens=1, hidden=7168, inter=2048, experts=256, top_k=8,
             renorm=True),
        # a small layer of odd sizes
        dict(name="moe odd mxfp4", op="moe", fmt="mxfp4", tokens=7, hidden=2912, inter=640, experts=33, top_k=3,
             renorm=False),
        # a small batch, 8-bit weights
        dict(name="moe small batch mxfp8", op="moe", fmt="mxfp8", tokens=16, hidden=4096, inter=2048, experts=64, top_k=4,
             renorm=True),
        # a full decode batch: nearly every expert is read
        dict(name="moe batch nvfp4", op="moe", fmt="nvfp4", tokens=64, hidden=7168, inter=2048, experts=256, top_k=8,
             renorm=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "moe"])
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128])
        new_max = _log_int(rng, 1, 4000)
        return dict(op=op, batch=max(1, min(_log_int(rng, 1, 64), 24000 // new_max)), new_max=new_max,
                    ragged=rng.random() < 0.7, past_max=_log_int(rng, 1, 1200), kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]))
    if op == "attn":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
        q_max = rng.choice([1, 1, _log_int(rng, 2, 8), _log_int(rng, 9, 1500)])
        ctx_max = _log_int(rng, max(q_max, 40), 60000)
        # bounded by the largest listed cases: cache bytes, and operations
        most = 8.0e8 / (2.0 * ctx_max * kv_heads * dim)
        most = min(most, 4.0e11 / (4.0 * heads * dim * q_max * ctx_max), 4.0e9 / (4.0 * heads * q_max * ctx_max))
        batch = max(1, min(_log_int(rng, 1, 96), int(most)))
        if q_max * ctx_max * heads > 1.0e9:
            q_max = max(1, int(1.0e9 / (ctx_max * heads)))
        return dict(op=op, batch=batch, q_max=q_max, ragged=rng.random() < 0.6, ctx_min=max(1, ctx_max // rng.choice([1, 2, 5])),
                    ctx_max=ctx_max, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "f16"]), causal=rng.random() < 0.85,
                    window=rng.choice([0, 0, 0, _log_int(rng, 16, 5000)]), empty=rng.random() < 0.3)
    hidden, inter = 32 * _log_int(rng, 8, 224), 128 * _log_int(rng, 1, 16)
    experts = _log_int(rng, 2, 256)
    return dict(op=op, fmt=rng.choice(["nvfp4", "mxfp4", "mxfp8"]), tokens=_log_int(rng, 1, 64), hidden=hidden, inter=inter,
                experts=experts, top_k=rng.randint(1, min(8, experts)), renorm=rng.random() < 0.7)


def _spread(n, lo, hi, ragged):
    """n lengths from lo to hi, in no order, the same for every seed."""
    if not ragged:
        return [hi] * n
    return [lo + int((hi - lo) * ((i * 0.6180339887 + 0.37) % 1.0)) for i in range(n - 1)] + [hi]


def _append_lens(c):
    new = _spread(c["batch"], max(1, c["new_max"] // 3), c["new_max"], c["ragged"])
    past = [int(c["past_max"] * ((i * 0.7548776662 + 0.11) % 1.0)) for i in range(c["batch"])]
    return new, [p + n for p, n in zip(past, new)]


def _attn_lens(c):
    q = _spread(c["batch"], 1, c["q_max"], c["ragged"])
    ctx = _spread(c["batch"], c["ctx_min"], c["ctx_max"], True)
    ctx = [max(a, b) for a, b in zip(ctx, q)]
    if c["empty"] and c["batch"] > 1:
        ctx[c["batch"] // 2] = 0
    return q, ctx


# ---------------------------------------------------------------- prepare --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(lens, page, g):
    """Block table over shuffled pages; -1 where a sequence has none."""
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(1, max(need))
    perm = torch.randperm(total + 3, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(DEV), total + 3


def _cache(pages, heads, page, dim, g):
    """Codes and scale bytes as kept for values of unit scale."""
    codes = (torch.randn((pages, heads, page, dim), generator=g, device=DEV, dtype=torch.bfloat16) * 64).clamp_(-448, 448)
    scales = torch.randint(120, 123, (pages, heads), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), scales


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "moe":
        return _prepare_moe(case, g)
    dt = DTYPES[case["dtype"]]
    new, lens = _append_lens(case) if case["op"] == "append" else _attn_lens(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    table, pages = _table(lens, case["page"], g)
    s = dict(case=case, offsets=_i32(starts), seq_lens=_i32(lens), table=table)
    s["k_cache"], s["k_scales"] = _cache(pages, case["kv_heads"], case["page"], case["dim"], g)
    s["v_cache"], s["v_scales"] = _cache(pages, case["kv_heads"], case["page"], case["dim"], g)
    if case["op"] == "append":
        shape = (starts[-1], case["kv_heads"], case["dim"])
        s["k"] = torch.randn(shape, generator=g, device=DEV).to(dt)
        s["v"] = (torch.randn(shape, generator=g, device=DEV) * 2).to(dt)
    else:
        s["q"] = torch.randn((starts[-1], case["heads"], case["dim"]), generator=g, device=DEV).to(dt)
        s["max_q"] = max(new)
    return s


def _normal_codes(shape, bits, g):
    """Codes of normally distributed weights: uniform draws through the
    quantiles of the block-scaled normal distribution."""
    u = (torch.arange(256, device=DEV, dtype=torch.float64) + 0.5) / 256
    z = torch.erfinv(2 * u - 1) * math.sqrt(2.0)
    if bits == 8:
        table = (z * 130).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
        near = ((z * 2.4).abs()[:, None] - mags[None]).abs().argmin(1)
        nib = (near + 8 * (z < 0)).to(torch.uint8)
        table = nib | (nib[torch.randperm(256, generator=g, device=DEV)] << 4)
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for part in out.view(shape[0], -1).split(max(1, (1 << 28) // (out.numel() // shape[0])), 0):
        part.copy_(table[torch.randint(0, 256, part.shape, generator=g, device=DEV, dtype=torch.uint8).int()])
    return out


def _weight(fmt, experts, rows, cols, g):
    """Packed codes (E, rows, bytes), scales (E, 5D bytes) and the tensor scale (E)."""
    codes = _normal_codes((experts, rows, cols if fmt == "mxfp8" else cols // 2), 8 if fmt == "mxfp8" else 4, g)
    s = cols // FMT_SF[fmt]
    tiles = -(-rows // 128) * -(-s // 4) * 512
    if fmt == "nvfp4":  # E4M3 bytes from 64 to 224, weights of about 1/sqrt(cols) once divided by the tensor scale
        scales = torch.randint(0x68, 0x77, (experts, tiles), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        tsf = torch.full((experts,), 280.0 * math.sqrt(cols), device=DEV) * (0.8 + 0.4 * torch.rand(experts, generator=g, device=DEV))
    else:
        mid = 127 - round(math.log2(math.sqrt(cols) * (130 if fmt == "mxfp8" else 2.4)))
        scales = torch.randint(mid - 1, mid + 2, (experts, tiles), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        tsf = torch.ones(experts, device=DEV)
    return codes, scales, tsf


def _prepare_moe(c, g):
    t, h, i, e = c["tokens"], c["hidden"], c["inter"], c["experts"]
    s = dict(case=c)
    s["x"] = torch.randn((t, h), generator=g, device=DEV).bfloat16()
    s["logits"] = torch.randn((t, e), generator=g, device=DEV) + 0.5 * torch.randn((1, e), generator=g, device=DEV)
    s["w13"], s["w13_scales"], s["w13_sf"] = _weight(c["fmt"], e, 2 * i, h, g)
    s["w2"], s["w2_scales"], s["w2_sf"] = _weight(c["fmt"], e, h, i, g)
    # calibrated activation scales, 448*6 / amax with some room
    s["x_sf"] = (448.0 * 6.0) / (4.0 + 2.0 * torch.rand(e, generator=g, device=DEV))
    s["h_sf"] = (448.0 * 6.0) / (6.0 + 6.0 * torch.rand(e, generator=g, device=DEV))
    return s


# -------------------------------------------------------------------- run --

_workspaces = {}


def _workspace(op, nbytes):
    """The program's workspace of an operator, kept between its calls."""
    ws = _workspaces.get(op)
    if ws is None or ws.numel() < nbytes:
        ws = _workspaces[op] = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    return ws


def run(s):
    c = s["case"]
    if own:
        import fp8_activation_quantization_bsq_gb300 as bsq
        if c["op"] == "append":
            bsq.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["offsets"],
                          s["seq_lens"])
            return _append_out(s)
        if c["op"] == "attn":
            q = s["q"]
            ws = _workspace("attn", bsq.kv_attention_workspace_bytes(q.shape[0], c["heads"], c["kv_heads"], c["dim"], c["batch"],
                                                                     s["max_q"]))
            return bsq.kv_attention(q, s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["offsets"],
                                    s["seq_lens"], s["max_q"], causal=c["causal"], window=c["window"], return_lse=True,
                                    workspace=ws)
        ws = _workspace("moe", bsq.moe_layer_workspace_bytes(c["fmt"], c["tokens"], c["hidden"], c["inter"], c["experts"],
                                                             c["top_k"]))
        return bsq.moe_layer(s["x"], s["logits"], s["w13"], s["w13_scales"], s["w2"], s["w2_scales"], c["fmt"], c["top_k"],
                             x_sf=s["x_sf"], w13_sf=s["w13_sf"], h_sf=s["h_sf"], w2_sf=s["w2_sf"], renormalize=c["renorm"],
                             workspace=ws)
    if c["op"] == "append":
        _plain_append(s, s["k"], s["k_cache"], s["k_scales"])
        _plain_append(s, s["v"], s["v_cache"], s["v_scales"])
        return _append_out(s)
    return _plain_attention(s) if c["op"] == "attn" else _plain_moe(s)


def _append_out(s):
    return dict(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn), k_scales=s["k_scales"],
                v_scales=s["v_scales"])


def _token_places(s, total):
    """Sequence and position of every new token."""
    t = torch.arange(total, device=DEV)
    off, lens = s["offsets"].long(), s["seq_lens"].long()
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return b, t - off[b], lens[b] - (off[b + 1] - off[b]) + t - off[b]


def _over(v, d):
    """v / d, rounded once (a plain number as divisor may become a product with its reciprocal)."""
    return v / torch.full_like(v, d)


def _ceil_exponent(v):
    """Smallest whole e with 2^e >= v > 0."""
    f, e = torch.frexp(v)
    return torch.where(f == 0.5, e - 1, e)


def _plain_append(s, x, cache, scales):
    page = s["case"]["page"]
    pages, heads = scales.shape
    b, _, pos = _token_places(s, x.shape[0])
    pid, slot = s["table"][b, pos // page].long(), pos % page
    xf = x.float()
    amax = torch.zeros((pages, heads), device=DEV).index_reduce_(0, pid, xf.abs().amax(2), "amax")
    first = torch.full((pages,), page, device=DEV, dtype=torch.long).index_reduce_(0, pid, slot, "amin")
    e_new = torch.where(amax == 0, -32, _ceil_exponent(_over(amax, 448.0)).clamp(-32, 127))
    e_old = scales.int() - 127
    keep = ((first > 0) & (first < page))[:, None]
    touched = (first < page)[:, None]
    e = torch.where(touched, torch.where(keep, torch.maximum(e_new, e_old), e_new), e_old)
    old = cache.view(torch.float8_e4m3fn).float() * torch.exp2((e_old - e).float())[:, :, None, None]
    keep_rows = ~touched[:, :, None] | (torch.arange(page, device=DEV)[None, None] < first[:, None, None])
    codes = torch.where(keep_rows[..., None], old.to(torch.float8_e4m3fn).view(torch.uint8), cache)
    codes[pid, :, slot] = (xf * torch.exp2(-e[pid].float())[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.copy_(codes)
    scales.copy_((e + 127).to(torch.uint8))


def _plain_attention(s):
    c, q = s["case"], s["q"]
    batch, group, page = c["batch"], c["heads"] // c["kv_heads"], c["page"]
    off, lens, table = s["offsets"].long(), s["seq_lens"].long(), s["table"].clamp(min=0).long()
    span = table.shape[1] * page

    def gathered(cache, scales):
        x = cache[table].view(torch.float8_e4m3fn).float() * torch.exp2(scales[table].float() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(batch, c["kv_heads"], span, c["dim"])

    place = torch.arange(s["max_q"], device=DEV)
    n = off[1:] - off[:-1]
    rows = (off[:-1, None] + place[None]).clamp(max=q.shape[0] - 1)
    qb = q.float()[rows].reshape(batch, s["max_q"], c["kv_heads"], group, c["dim"]).permute(0, 2, 3, 1, 4)
    qb = qb.reshape(batch, c["kv_heads"], group * s["max_q"], c["dim"])
    score = torch.matmul(qb, gathered(s["k_cache"], s["k_scales"]).transpose(2, 3)) / math.sqrt(c["dim"])
    score = score.view(batch, c["kv_heads"], group, s["max_q"], span)
    at = (lens - n)[:, None, None] + place[None, :, None]
    key = torch.arange(span, device=DEV)[None, None]
    ok = key < lens[:, None, None]
    if c["causal"]:
        ok = ok & (key <= at)
    if c["window"]:
        ok = ok & (at - key < c["window"])
    score.masked_fill_(~ok[:, None, None], -math.inf)
    top = score.amax(4, keepdim=True).clamp(min=-3.0e38)
    p = score.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    v = torch.where((torch.arange(span, device=DEV)[None] < lens[:, None])[:, None, :, None], gathered(s["v_cache"], s["v_scales"]), 0.0)
    out = torch.matmul(p.view(batch, c["kv_heads"], group * s["max_q"], span), v).view(batch, c["kv_heads"], group, s["max_q"], c["dim"])
    out = torch.where(total > 0, out / total, 0.0)
    lse = (torch.log(total) + torch.where(total > 0, top, 0.0)).squeeze(4)
    b, i, _ = _token_places(s, q.shape[0])
    out = out.permute(0, 3, 1, 2, 4)[b, i].reshape(q.shape[0], c["heads"], c["dim"])
    return out.to(q.dtype), lse.permute(0, 3, 1, 2)[b, i].reshape(q.shape[0], c["heads"])


def _values(fmt):
    """The value of every code byte (of every nibble for 4 bits)."""
    if fmt == "mxfp8":
        return torch.arange(256, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    return torch.tensor(mags + [-m for m in mags], device=DEV)


def _decoded(fmt, packed, scales, sf):
    """FP32 weights (N, rows, cols) of N experts' codes, 5D scales and tensor scales."""
    n, rows, nbytes = packed.shape
    if fmt == "mxfp8":
        w = packed.view(torch.float8_e4m3fn).float()
    else:
        pairs = torch.arange(256, device=DEV)
        pairs = torch.stack([_values(fmt)[pairs & 15], _values(fmt)[pairs >> 4]], 1)
        w = pairs[packed.int()].view(n, rows, nbytes * 2)
    sc = w.shape[2] // FMT_SF[fmt]
    mt, kt = -(-rows // 128), -(-sc // 4)
    sb = scales.view(n, mt, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, mt * 128, kt * 4)[:, :rows, :sc]
    f = sb.contiguous().view(torch.float8_e4m3fn).float() / sf[:, None, None] if fmt == "nvfp4" else torch.exp2(sb.float() - 127)
    w.view(n, rows, sc, FMT_SF[fmt]).mul_(f[..., None])
    return w


def _rounded(v, bits, low, most):
    """v on the grid of floats with `bits` fraction bits and least exponent `low`, ties to even, at most `most`."""
    _, e = torch.frexp(v)
    step = torch.exp2(((e - 1).clamp(min=low) - bits).float())
    return (torch.round(v / step) * step).clamp(-most, most)


def _quantized(x, fmt, sf):
    """The values that rows x (N, K) stand for once block-quantized, tensor scale sf (N)."""
    blocks = x.float().view(x.shape[0], -1, FMT_SF[fmt])
    amax = blocks.abs().amax(2, keepdim=True)
    if fmt == "nvfp4":
        sf = sf[:, None, None]
        ds = _rounded(_over(amax, 6.0) * sf, 3, -6, 448.0)
        f = torch.where(ds == 0, 0.0, sf / torch.where(ds == 0, 1.0, ds))
        return (_rounded(blocks * f, 1, 0, 6.0) * (ds / sf)).view(x.shape)
    e = torch.where(amax == 0, -127, _ceil_exponent(_over(amax, 448.0 if fmt == "mxfp8" else 6.0)).clamp(-127, 127)).float()
    y = blocks * torch.exp2(-e)
    y = _rounded(y, 3, -6, 448.0) if fmt == "mxfp8" else _rounded(y, 1, 0, 6.0)
    return (y * torch.exp2(e)).view(x.shape)


def _plain_moe(s):
    c = s["case"]
    p = s["logits"] - s["logits"].amax(1, keepdim=True)
    p = p.exp()
    p = p / p.sum(1, keepdim=True)
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = p.gather(1, order)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros((c["tokens"], c["hidden"]), device=DEV)
    for k in range(c["top_k"]):  # a choice at a time: all of them at once would not fit
        e = order[:, k]
        xq = _quantized(s["x"], c["fmt"], s["x_sf"][e])
        gu = torch.matmul(_decoded(c["fmt"], s["w13"][e], s["w13_scales"][e], s["w13_sf"][e]), xq[:, :, None])[:, :, 0]
        gate, up = gu[:, :c["inter"]], gu[:, c["inter"]:]
        h = (gate / (1 + torch.exp(-gate)) * up).bfloat16()
        hq = _quantized(h, c["fmt"], s["h_sf"][e])
        y += w[:, k, None] * torch.matmul(_decoded(c["fmt"], s["w2"][e], s["w2_scales"][e], s["w2_sf"][e]), hq[:, :, None])[:, :, 0]
    return y.bfloat16()


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "append":
        new, lens = _append_lens(case)
        n = sum(new) * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * 3, "flops": 2 * n * 2}
    if case["op"] == "attn":
        q, ctx = _attn_lens(case)
        keys, pairs = 0, 0
        for n, length in zip(q, ctx):
            lo, hi = length, 0
            for i in range(n):
                at = length - n + i
                top = min(length, at + 1) if case["causal"] else length
                bottom = max(0, at - case["window"] + 1) if case["window"] else 0
                if top > bottom:
                    pairs += top - bottom
                    lo, hi = min(lo, bottom), max(hi, top)
            keys += max(0, hi - lo)
        return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] + 4 * sum(q) * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    t, h, i, e, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "top_k"))
    # distinct experts that the tokens' choices reach, on average, were all experts as likely
    reached = e * (1 - (1 - k / e) ** t)
    per = {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32}[case["fmt"]]
    return {"bytes": reached * 3 * i * h * per + 4 * t * h + 4 * t * e, "flops": 6 * t * k * i * h}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        new, lens = _append_lens(case)
        k, ks = _exact_append(case, s, s["k"], s["k_cache"], s["k_scales"], new, lens)
        v, vs = _exact_append(case, s, s["v"], s["v_cache"], s["v_scales"], new, lens)
        return dict(k=k, v=v, k_scales=ks, v_scales=vs)
    return _exact_attention(case, s) if case["op"] == "attn" else _exact_moe(case, s)


def _e4m3_values():
    c = torch.arange(256, device=DEV)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(c >= 128, -mag, mag)


def _exact_exponent(amax, most):
    """The least whole e with most * 2^e >= amax, -127 for zero."""
    e = torch.floor(torch.log2(amax.clamp(min=1e-300) / most)) - 1
    for _ in range(3):  # products with powers of two are exact, the logarithm is not
        e = torch.where(most * torch.exp2(e) < amax, e + 1, e)
    return torch.where(amax == 0, -127.0, e)


def _nearest(v, grid):
    """The nearest value of an increasing grid of magnitudes, ties to the even place, with v's sign."""
    a = v.abs()
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    at = torch.where(a >= grid[-1], grid.numel() - 1, at)
    return torch.where(v < 0, -grid[at], grid[at])


def _exact_append(c, s, x, cache, scales, new, lens):
    values = _e4m3_values()
    grid = values[:127].contiguous()
    out, sc, table = values[cache.long()], scales.clone(), s["table"].cpu()
    at, page = 0, c["page"]
    for b, n in enumerate(new):
        start = lens[b] - n
        for pg in range(start // page, (lens[b] - 1) // page + 1):
            lo, hi = max(start, pg * page), min(lens[b], (pg + 1) * page)
            rows = x[at + lo - start:at + hi - start].double().transpose(0, 1)
            pid, first = int(table[b, pg]), lo - pg * page
            e = _exact_exponent(rows.abs().amax((1, 2)), 448.0).clamp(-32, 127)
            if first:
                was = sc[pid].double() - 127
                e = torch.maximum(e, was)
                out[pid, :, :first] = _nearest(out[pid, :, :first] * torch.exp2(was - e)[:, None, None], grid)
            out[pid, :, first:first + hi - lo] = _nearest(rows * torch.exp2(-e)[:, None, None], grid)
            sc[pid] = (e + 127).to(torch.uint8)
        at += n
    return out, sc


def _exact_attention(c, s):
    values = _e4m3_values()
    q, ctx = _attn_lens(c)
    group, page = c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, length) in enumerate(zip(q, ctx)):
        if length:
            ids = s["table"][b, :-(-length // page)].long()
            for h in range(c["kv_heads"]):
                k, v = ((values[x[ids, h].long()] * torch.exp2(y[ids, h].double() - 127)[:, None, None]).reshape(-1, c["dim"])[:length]
                        for x, y in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
                where = length - n + torch.arange(n, device=DEV)[:, None]
                j = torch.arange(length, device=DEV)[None]
                bad = torch.zeros((n, length), dtype=torch.bool, device=DEV)
                if c["causal"]:
                    bad |= j > where
                if c["window"]:
                    bad |= where - j >= c["window"]
                for g in range(h * group, (h + 1) * group):
                    z = (s["q"][at:at + n, g].double() @ k.T) / math.sqrt(c["dim"])
                    z = z.masked_fill(bad, -math.inf)
                    some = ~bad.all(1)
                    l = torch.logsumexp(z, 1)
                    lse[at:at + n, g] = l
                    out[at:at + n, g] = torch.where(some[:, None], torch.exp(z - torch.where(some, l, 0.0)[:, None]) @ v, 0.0)
        at += n
    return out, lse


def _exact_decoded(fmt, packed, scales, sf):
    rows = packed.shape[0]
    if fmt == "mxfp8":
        w = _e4m3_values()[packed.long()]
    else:
        c = torch.stack([packed & 15, packed >> 4], 2).view(rows, -1)
        e, m = ((c >> 1) & 3).double(), (c & 1).double()
        w = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1)) * torch.where(c >= 8, -1.0, 1.0)
    n = w.shape[1] // FMT_SF[fmt]
    r, col = torch.arange(rows, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
    b = scales[((r // 128) * -(-n // 4) + col // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + col % 4]
    f = _e4m3_values()[b.long()] / sf.double() if fmt == "nvfp4" else torch.exp2(b.double() - 127)
    return w * f.repeat_interleave(FMT_SF[fmt], 1)


def _exact_quantized(x, fmt, sf):
    """Like the definition: the scale steps that it does in 32 bits are done there, the rest in 64."""
    b = x.double().view(x.shape[0], -1, FMT_SF[fmt])
    amax = b.abs().amax(2, keepdim=True)
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
    e4m3 = _e4m3_values()[:127].contiguous()
    if fmt == "nvfp4":
        t = ((amax.float() / torch.tensor(6.0, device=DEV)) * sf.float()).double()
        ds = _nearest(t, e4m3)
        f = torch.where(ds == 0, 0.0, (sf.float() / torch.where(ds == 0, 1.0, ds).float()).double())
        return (_nearest((b * f).float().double(), e2m1) * ds / sf.double()).view(x.shape)
    e = _exact_exponent(amax, 448.0 if fmt == "mxfp8" else 6.0)
    return (_nearest(b * torch.exp2(-e), e4m3 if fmt == "mxfp8" else e2m1) * torch.exp2(e)).view(x.shape)


def _exact_moe(c, s):
    z = s["logits"].double()
    ids = torch.argsort(z, dim=1, descending=True, stable=True)[:, :c["top_k"]]
    w = torch.softmax(z, 1).gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=DEV)
    for e in torch.unique(ids).tolist():
        t, k = (ids == e).nonzero(as_tuple=True)
        xq = _exact_quantized(s["x"][t], c["fmt"], s["x_sf"][e])
        gu = xq @ _exact_decoded(c["fmt"], s["w13"][e], s["w13_scales"][e], s["w13_sf"][e]).T
        gate, up = gu[:, :c["inter"]], gu[:, c["inter"]:]
        h = (gate * torch.sigmoid(gate) * up).bfloat16()
        hq = _exact_quantized(h, c["fmt"], s["h_sf"][e])
        y[t] += w[t, k, None] * (hq @ _exact_decoded(c["fmt"], s["w2"][e], s["w2_scales"][e], s["w2_sf"][e]).T)
    return y
