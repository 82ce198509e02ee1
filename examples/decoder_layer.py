#!/usr/bin/env python3
"""One decoder layer served from block-scaled storage: prompts enter an 8-bit
paged key/value cache in chunks, then tokens are generated one per sequence,
with attention over the cache and a mixture of experts over packed weights.

    python examples/decoder_layer.py [--fmt nvfp4] [--batch 4] [--prompt 300] [--steps 8]

Weights are random; the layer's projections are plain matmuls.  A whole
decoding step can be captured in a CUDA graph: every call is asynchronous on
the current stream and keeps its workspace."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_activation_quantization_bsq_gb300 as bsq  # noqa: E402


class Cache:
    """Pages for `batch` sequences of at most `most` tokens, given out in order."""

    def __init__(self, batch, most, kv_heads, dim, page=64, device="cuda"):
        per = -(-most // page)
        shape = (batch * per, kv_heads, page, dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(shape[:2], dtype=torch.uint8, device=device) for _ in range(2))
        self.table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def tensors(self):
        return self.k, self.v, self.k_scales, self.v_scales, self.table


class Layer:
    def __init__(self, fmt, hidden=1024, heads=16, kv_heads=2, dim=128, inter=512, experts=16, top_k=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g, device=device) / s[-1] ** 0.5).bfloat16()  # noqa: E731
        self.fmt, self.hidden, self.heads, self.kv_heads, self.dim, self.top_k = fmt, hidden, heads, kv_heads, dim, top_k
        self.w_qkv, self.w_out, self.w_router = rand((heads + 2 * kv_heads) * dim, hidden), rand(hidden, heads * dim), rand(experts, hidden)
        self.moe = []
        self.kw = dict(x_sf=torch.full((experts,), 2688 / 8.0, device=device), h_sf=torch.full((experts,), 2688 / 8.0, device=device))
        for name, rows, cols in (("w13_sf", 2 * inter, hidden), ("w2_sf", hidden, inter)):
            w = [rand(rows, cols) for _ in range(experts)]
            sf = torch.stack([bsq.tensor_sf(m)[1] for m in w])
            q = [bsq.quantize_dynamic(m, fmt, s[None]) for m, s in zip(w, sf)]
            self.moe += [torch.stack([a for a, _ in q]), torch.stack([b for _, b in q])]
            self.kw[name] = sf
        if fmt != "nvfp4":
            self.kw = {}
        self.workspaces = {}

    def workspace(self, name, nbytes):
        """Zeroed once, kept between calls (each leaves it ready for the next); a smaller one that a larger
        replaces is kept too, for a captured step goes on using it."""
        kept = self.workspaces.setdefault(name, [])
        if not kept or kept[-1].numel() < nbytes:
            kept.append(torch.zeros(nbytes, dtype=torch.uint8, device=self.w_out.device))
        return kept[-1]

    def attend(self, x, cache, offsets, max_q):
        """x: (tokens, hidden), rows offsets[b]:offsets[b+1] new in sequence b, which cache.lens already counts."""
        qkv = (torch.nn.functional.rms_norm(x, (self.hidden,)) @ self.w_qkv.t()).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)  # strided views: taken as they are
        bsq.kv_append(k, v, *cache.tensors(), offsets, cache.lens)
        ws = self.workspace("attention", bsq.kv_attention_workspace_bytes(x.shape[0], self.heads, self.kv_heads, self.dim,
                                                                          cache.lens.numel(), max_q))
        out = bsq.kv_attention(q, *cache.tensors(), offsets, cache.lens, max_q, workspace=ws)
        return x + out.view(x.shape[0], -1) @ self.w_out.t()

    def experts(self, x):
        x = x.contiguous()
        y = torch.nn.functional.rms_norm(x, (self.hidden,))
        logits = (y @ self.w_router.t()).float()
        ws = self.workspace("moe", bsq.moe_layer_workspace_bytes(self.fmt, x.shape[0], self.hidden, self.moe[2].shape[2] * (1 if self.fmt == "mxfp8" else 2),
                                                                 logits.shape[1], self.top_k))
        return x + bsq.moe_layer(y, logits, *self.moe, self.fmt, self.top_k, workspace=ws, **self.kw)

    def __call__(self, x, cache, offsets, max_q):
        x = self.attend(x, cache, offsets, max_q)
        return torch.cat([self.experts(part) for part in x.split(64)])  # the expert layer takes a few tokens at a time


def serve(fmt="nvfp4", batch=4, prompt=300, steps=8, chunk=128, seed=0):
    """(outputs of the prompts' last tokens and of each step, the cache)."""
    layer = Layer(fmt, seed=seed)
    cache = Cache(batch, prompt + steps, layer.kv_heads, layer.dim)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompts = torch.randn((batch, prompt, layer.hidden), generator=g, device="cuda").bfloat16()
    x = None
    for start in range(0, prompt, chunk):
        n = min(chunk, prompt - start)
        cache.lens += n
        offsets = torch.arange(0, batch * n + 1, n, dtype=torch.int32, device="cuda")
        x = layer(prompts[:, start:start + n].reshape(batch * n, -1), cache, offsets, n).view(batch, n, -1)[:, -1]
    one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    outs = [x]
    for _ in range(steps):
        cache.lens += 1
        x = layer(x, cache, one, 1)
        outs.append(x)
    return torch.stack(outs), cache


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=sorted(bsq.FORMATS), default="nvfp4")
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    outs, cache = serve(a.fmt, a.batch, a.prompt, a.steps)
    torch.cuda.synchronize()
    assert bsq.device_error() == 0
    print(f"{a.fmt}: {a.batch} prompts of {a.prompt} tokens and {a.steps} steps; cache lengths {cache.lens.tolist()}, "
          f"last output rms {outs[-1].float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
