"""Cases of the operators between the block-scaled calls of a decoder layer:
products with packed weights, norm and rotation of queries and keys, and
routing to experts with the rows' order for grouped calls.

``listed()`` and ``draw()`` give cases, ``prepare`` a user's tensors, ``run``
one pass (the plain form, or the library's calls where ``own`` is set),
``work`` the bytes and operations that the pass cannot do without and
``exact`` the result in 64 bits."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FMT_SF = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a few guessed tokens through a small projection of odd sizes: latency
        dict(name="linear guessed mxfp4", op="linear", fmt="mxfp4", tokens=5, rows=1000, cols=2912, dtype="f16", out="f16", add=False),
        # one user's next token through a query/key/value projection (64 and 2 x 8 heads of 128)
        dict(name="linear one nvfp4", op="linear", fmt="nvfp4", tokens=1, rows=10240, cols=7168, dtype="bf16", out="bf16", add=False),
        # router logits of a small batch, in FP32
        dict(name="linear router mxfp8", op="linear", fmt="mxfp8", tokens=16, rows=256, cols=7168, dtype="bf16", out="f32", add=False),
        # the output projection of a full decode batch, added to the residual stream
        dict(name="linear batch nvfp4", op="linear", fmt="nvfp4", tokens=64, rows=7168, cols=8192, dtype="bf16", out="bf16", add=True),
        # a chunk of a prompt through the query/key/value projection
        dict(name="linear prompt nvfp4", op="linear", fmt="nvfp4", tokens=2048, rows=10240, cols=7168, dtype="bf16", out="bf16",
             add=False),
        # one user's next token, far into a context: latency
        dict(name="rope one", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, pairs=64, dtype="bf16", interleaved=False, norm=True,
             pos_max=131072),
        # guessed tokens of a batch, part of an odd head rotated, neighbouring pairs
        dict(name="rope guessed partial", op="rope", tokens=257, heads=24, kv_heads=8, dim=96, pairs=32, dtype="f16", interleaved=True,
             norm=True, pos_max=9000),
        # a prompt
        dict(name="rope prompt", op="rope", tokens=4096, heads=64, kv_heads=8, dim=128, pairs=64, dtype="bf16", interleaved=False,
             norm=True, pos_max=40000),
        # one user's next token: sigmoid scores, balance bias, 4 of 8 groups: latency
        dict(name="route one", op="route", tokens=1, experts=256, top_k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, scale=2.5, dtype="f32", rows=False),
        # a full decode batch, plain softmax of BF16 logits (equal ones among them)
        dict(name="route batch", op="route", tokens=64, experts=256, top_k=8, scoring="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, dtype="bf16", rows=False),
        # a small layer of odd sizes, with the rows' order for the grouped calls
        dict(name="route odd rows", op="route", tokens=333, experts=33, top_k=3, scoring="softmax", bias=True, groups=3, top_groups=2,
             group_top=1, renorm=False, scale=1.0, dtype="f16", rows=True),
        # a prompt, with the rows' order for the grouped calls
        dict(name="route prompt rows", op="route", tokens=4096, experts=256, top_k=8, scoring="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", rows=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "route"])
    if op == "linear":
        rows, cols = _log_int(rng, 20, 16000), 32 * _log_int(rng, 2, 256)
        most = min(1.5e11 / (rows * cols), 2.0e7 / rows, 2.0e7 / cols)
        dtype = rng.choice(["bf16", "bf16", "f16"])
        return dict(op=op, fmt=rng.choice(["nvfp4", "mxfp4", "mxfp8"]), tokens=max(1, min(_log_int(rng, 1, 2048), int(most))), rows=rows,
                    cols=cols, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]), add=rng.random() < 0.4)
    if op == "rope":
        dim, kv_heads = rng.choice([64, 80, 96, 128, 256]), rng.choice([1, 2, 4, 5, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        most = 4096 * 72 * 128 // ((heads + kv_heads) * dim)
        return dict(op=op, tokens=min(_log_int(rng, 1, 4096), most), heads=heads, kv_heads=kv_heads, dim=dim,
                    pairs=rng.choice([dim // 2, dim // 2, dim // 4, 5, rng.randint(1, dim // 2)]), dtype=rng.choice(["bf16", "f16"]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, pos_max=_log_int(rng, 1, 1000000))
    per, groups = _log_int(rng, 2, 64), rng.choice([1, 1, 2, 3, 4, 8])
    experts, top_groups = per * groups, rng.randint(1, groups)
    return dict(op=op, tokens=_log_int(rng, 1, 4096), experts=experts, top_k=rng.randint(1, min(8, per * top_groups)),
                scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                dtype=rng.choice(["f32", "f32", "bf16", "f16"]), rows=rng.random() < 0.5)


# ---------------------------------------------------------------- prepare --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal_codes(rows, nbytes, bits, g):
    """Codes of normally distributed weights: uniform draws through the quantiles of the block-scaled normal distribution."""
    u = (torch.arange(256, device=DEV, dtype=torch.float64) + 0.5) / 256
    z = torch.erfinv(2 * u - 1) * math.sqrt(2.0)
    if bits == 8:
        table = (z * 130).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
        near = ((z * 2.4).abs()[:, None] - mags[None]).abs().argmin(1)
        nib = (near + 8 * (z < 0)).to(torch.uint8)
        table = nib | (nib[torch.randperm(256, generator=g, device=DEV)] << 4)
    return table[torch.randint(0, 256, (rows, nbytes), generator=g, device=DEV, dtype=torch.uint8).int()]


def prepare(case, seed):
    return {"linear": _prepare_linear, "rope": _prepare_rope, "route": _prepare_route}[case["op"]](case, _gen(seed))


def _prepare_linear(c, g):
    fmt, rows, cols = c["fmt"], c["rows"], c["cols"]
    s = dict(case=c, x=torch.randn((c["tokens"], cols), generator=g, device=DEV).to(DTYPES[c["dtype"]]))
    s["w"] = _normal_codes(rows, cols if fmt == "mxfp8" else cols // 2, 8 if fmt == "mxfp8" else 4, g)
    tiles = -(-rows // 128) * -(-(cols // FMT_SF[fmt]) // 4) * 512
    s["w_sf"] = None
    if fmt == "nvfp4":  # E4M3 bytes from 64 to 224, weights of about 1/sqrt(cols) once divided by the tensor scale
        s["w_scales"] = torch.randint(0x68, 0x77, (tiles,), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        s["w_sf"] = 280.0 * math.sqrt(cols) * (0.8 + 0.4 * torch.rand(1, generator=g, device=DEV))
    else:
        mid = 127 - round(math.log2(math.sqrt(cols) * (130 if fmt == "mxfp8" else 2.4)))
        s["w_scales"] = torch.randint(mid - 1, mid + 2, (tiles,), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    s["add"] = torch.randn((c["tokens"], rows), generator=g, device=DEV).to(DTYPES[c["out"]]) if c["add"] else None
    return s


def _prepare_rope(c, g):
    t, h, kv, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn((t, h + 2 * kv, d), generator=g, device=DEV).to(DTYPES[c["dtype"]])  # a projection's output; q and k are views
    s = dict(case=c, q=qkv[:, :h], k=qkv[:, h:h + kv])
    s["positions"] = torch.randint(0, c["pos_max"], (t,), generator=g, device=DEV, dtype=torch.int32)
    s["inv_freq"] = torch.pow(10000.0, -torch.arange(c["pairs"], device=DEV, dtype=torch.float64) / c["pairs"]).float()
    for name in ("q_weight", "k_weight"):
        s[name] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(DTYPES[c["dtype"]]) if c["norm"] else None
    return s


def _prepare_route(c, g):
    t, e = c["tokens"], c["experts"]
    z = torch.randn((t, e), generator=g, device=DEV) + 0.5 * torch.randn((1, e), generator=g, device=DEV)
    s = dict(case=c, logits=z.to(DTYPES[c["dtype"]]), bias=None)
    if c["bias"]:
        s["bias"] = (0.05 if c["scoring"] == "sigmoid" else 0.5 / e) * torch.randn(e, generator=g, device=DEV)
    return s


# -------------------------------------------------------------------- run --

def run(s):
    c = s["case"]
    if own:
        import fp8_activation_quantization_bsq_gb300 as bsq
        if c["op"] == "linear":
            return bsq.packed_linear(s["x"], s["w"], s["w_scales"], c["fmt"], w_sf=s["w_sf"], add=s["add"], out_dtype=DTYPES[c["out"]])
        if c["op"] == "rope":
            return bsq.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                    eps=1e-6, interleaved=c["interleaved"])
        ids, weights = bsq.moe_route(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"],
                                     top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
        out = dict(ids=ids, weights=weights)
        if c["rows"]:
            out["row_offsets"], out["scales_offsets"], out["row_indices"], out["positions"] = bsq.moe_rows(ids, c["experts"])
        return out
    return {"linear": _plain_linear, "rope": _plain_rope, "route": _plain_route}[c["op"]](s)


def _values(fmt):
    """The value of every code byte (of every nibble for 4 bits)."""
    if fmt == "mxfp8":
        return torch.arange(256, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    return torch.tensor(mags + [-m for m in mags], device=DEV)


def _plain_linear(s):
    c = s["case"]
    fmt, rows, cols = c["fmt"], c["rows"], c["cols"]
    w = s["w"]
    w = _values(fmt)[w.int()] if fmt == "mxfp8" else _values(fmt)[torch.stack([w & 15, w >> 4], 2).int()].view(rows, cols)
    n = cols // FMT_SF[fmt]
    mt, kt = -(-rows // 128), -(-n // 4)
    b = s["w_scales"].view(mt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(mt * 128, kt * 4)[:rows, :n]
    f = b.contiguous().view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(b.float() - 127)
    w = (w.view(rows, n, FMT_SF[fmt]) * f[..., None]).view(rows, cols)
    y = torch.matmul(s["x"].float(), w.t())
    if fmt == "nvfp4":
        y = y / s["w_sf"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(DTYPES[c["out"]])


def _plain_rope(s):
    c = s["case"]
    r = c["pairs"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + 1e-6) * w.float()
        a, b = (y[..., 0:2 * r:2], y[..., 1:2 * r:2]) if c["interleaved"] else (y[..., :r], y[..., r:2 * r])
        a, b = a * cos - b * sin, b * cos + a * sin
        head = torch.stack([a, b], 3).flatten(2) if c["interleaved"] else torch.cat([a, b], 2)
        out.append(torch.cat([head, y[..., 2 * r:]], 2).to(x.dtype))
    return tuple(out)


def _plain_route(s):
    c = s["case"]
    t, e, groups = c["tokens"], c["experts"], c["groups"]
    z = s["logits"].double()
    if c["scoring"] == "softmax":
        p = (z - z.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + (-z).exp())
    value = z if s["bias"] is None else p + s["bias"].double()
    if groups > 1:
        by_group = (z if s["bias"] is None and c["group_top"] == 1 else p if s["bias"] is None else value).view(t, groups, -1)
        score = by_group.sort(dim=2, descending=True)[0][..., :c["group_top"]].sum(2)
        kept = score.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        ok = torch.zeros((t, groups), dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        value = torch.where(ok[:, :, None], value.view(t, groups, -1), -math.inf).view(t, e)
    ids = value.sort(dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = dict(ids=ids.int(), weights=(w * c["scale"]).float())
    if c["rows"]:
        flat = ids.flatten()
        order = flat.sort(stable=True)[1]
        counts = (flat[:, None] == torch.arange(e, device=DEV)[None]).sum(0)
        zero = torch.zeros(1, dtype=torch.long, device=DEV)
        out["row_offsets"] = torch.cat([zero, counts.cumsum(0)]).int()
        out["scales_offsets"] = torch.cat([zero, ((counts + 127) // 128 * 128).cumsum(0)]).int()
        out["row_indices"] = (order // c["top_k"]).int()
        out["positions"] = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=DEV)).view(t, -1).int()
    return out


# ------------------------------------------------------------------- work --

def work(case):
    c, t = case, case["tokens"]
    if c["op"] == "linear":
        per = {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32}[c["fmt"]]
        wide = 4 if c["out"] == "f32" else 2
        return {"bytes": c["rows"] * c["cols"] * per + 2 * t * c["cols"] + wide * t * c["rows"] * (2 if c["add"] else 1),
                "flops": 2 * t * c["rows"] * c["cols"]}
    if c["op"] == "rope":
        n = t * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 4 * n + 4 * t, "flops": n * (7 if c["norm"] else 3)}
    wide = 4 if c["dtype"] == "f32" else 2
    pairs = t * c["top_k"]
    return {"bytes": wide * t * c["experts"] + 8 * pairs + (8 * pairs + 8 * (c["experts"] + 1) if c["rows"] else 0),
            "flops": 8 * t * c["experts"]}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "route": _exact_route}[case["op"]](case, s)


def _e4m3_values():
    c = torch.arange(256, device=DEV)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(c >= 128, -mag, mag)


def _exact_linear(c, s):
    fmt, rows, cols = c["fmt"], c["rows"], c["cols"]
    n = cols // FMT_SF[fmt]
    x, y = s["x"].double(), torch.empty((c["tokens"], rows), dtype=torch.float64, device=DEV)
    for lo in range(0, rows, 1024):
        r = torch.arange(lo, min(rows, lo + 1024), device=DEV)[:, None]
        if fmt == "mxfp8":
            w = _e4m3_values()[s["w"][r[:, 0]].long()]
        else:
            byte = s["w"][r[:, 0]].long()
            code = torch.stack([byte % 16, byte // 16], 2).view(-1, cols)
            e, m = (code % 8) // 2, (code % 2).double()
            w = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e.double() - 1)) * (1 - 2 * (code // 8)).double()
        col = torch.arange(n, device=DEV)[None]
        b = s["w_scales"][((r // 128) * -(-n // 4) + col // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + col % 4].long()
        f = _e4m3_values()[b] / s["w_sf"].double() if fmt == "nvfp4" else 2.0 ** (b.double() - 127)
        y[:, lo:lo + 1024] = x @ (w * f.repeat_interleave(FMT_SF[fmt], 1)).T
    return y if s["add"] is None else y + s["add"].double()


def _exact_rope(c, s):
    r = c["pairs"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["inv_freq"].double()))
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if w is not None:
            y = w.double() * y / torch.sqrt((y ** 2).sum(2, keepdim=True) / c["dim"] + 1e-6)
        at = torch.arange(r, device=DEV)
        first, second = (2 * at, 2 * at + 1) if c["interleaved"] else (at, at + r)
        v = torch.complex(y[:, :, first], y[:, :, second]) * turn[:, None]
        y[:, :, first], y[:, :, second] = v.real, v.imag
        out.append(y)
    return tuple(out)


def _exact_route(c, s):
    z = s["logits"].double().cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    t, e, k, per = c["tokens"], c["experts"], c["top_k"], c["experts"] // c["groups"]
    ids, weights = np.zeros((t, k), np.int32), np.zeros((t, k))
    for i in range(t):
        if c["scoring"] == "softmax":
            p = np.exp(z[i] - z[i].max())
            p /= p.sum()
        else:
            p = 1 / (1 + np.exp(-z[i]))
        value = z[i] if bias is None else p + bias
        open_to = np.arange(e)
        if c["groups"] > 1:
            of = p if bias is None and c["group_top"] == 2 else value
            score = [sum(sorted(of[g * per:(g + 1) * per], reverse=True)[:c["group_top"]]) for g in range(c["groups"])]
            kept = sorted(range(c["groups"]), key=lambda g: (-score[g], g))[:c["top_groups"]]
            open_to = np.concatenate([np.arange(g * per, (g + 1) * per) for g in sorted(kept)])
        ids[i] = open_to[np.argsort(-value[open_to], kind="stable")[:k]]
        weights[i] = p[ids[i]] / (p[ids[i]].sum() if c["renorm"] else 1) * c["scale"]
    out = dict(ids=ids, weights=weights)
    if c["rows"]:
        lists = [[] for _ in range(e)]
        for place, x in enumerate(ids.ravel().tolist()):
            lists[x].append(place)
        out["row_offsets"] = np.cumsum([0] + [len(v) for v in lists]).astype(np.int32)
        out["scales_offsets"] = np.cumsum([0] + [-(-len(v) // 128) * 128 for v in lists]).astype(np.int32)
        order = np.array([p for v in lists for p in v])
        out["row_indices"] = (order // k).astype(np.int32)
        out["positions"] = np.empty(t * k, np.int32)
        out["positions"][order] = np.arange(t * k, dtype=np.int32)
        out["positions"] = out["positions"].reshape(t, k)
    return {name: torch.from_numpy(v).to(DEV) for name, v in out.items()}
