"""Binding of the serving calls: the 8-bit paged key/value cache
(``bsq_kv_append``, ``bsq_kv_attention``) and the few-token expert layer
(``bsq_moe_layer``).  As in the package's other calls, work is enqueued on the
current stream (or ``stream``), outputs are allocated with torch when not
passed in, and a refused argument raises ValueError or BsqError."""
from __future__ import annotations

import math

import torch

from . import FORMATS, _check, _fmt, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _on(device, stream):
    """The raw stream of a call on `device`, which has to be current where no stream is given."""
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _call(name, device, args):
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    _check(rc, name)


def _check_rows(x, what):
    """A (tokens, heads, dim) 16-bit CUDA tensor with unit inner stride: its dtype code."""
    code = _DTYPES.get(x.dtype)
    if code is None or x.dim() != 3 or not x.is_cuda or x.stride(2) != 1:
        raise ValueError(f"{what} must be a (tokens, heads, dim) bfloat16 or float16 CUDA tensor with unit inner stride")
    return code


def _cache_args(rows, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens):
    """Checks the cache tensors of a call for `rows`; (kv_heads, dim, page, batch)."""
    if k_cache.dtype != torch.uint8 or k_cache.dim() != 4 or k_cache.stride(3) != 1 or v_cache.dtype != torch.uint8 or \
            k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must be uint8 (pages, kv_heads, page, dim) tensors of equal strides, unit inner stride")
    pages, heads, page, dim = k_cache.shape
    for s in (k_scales, v_scales):
        if s.dtype != torch.uint8 or s.dim() != 2 or s.shape[0] != pages or s.shape[1] != heads or not s.is_contiguous():
            raise ValueError("k_scales and v_scales must be contiguous uint8 (pages, kv_heads) tensors")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 (batch, pages per sequence) tensor with unit inner stride")
    batch = block_table.shape[0]
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] != batch + 1 or not offsets.is_contiguous() or \
            seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or seq_lens.shape[0] != batch or not seq_lens.is_contiguous():
        raise ValueError("offsets and seq_lens must be contiguous int32 tensors of batch + 1 and batch entries")
    device = rows.device
    for t in (k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens):
        if t.device != device:
            raise ValueError("all tensors of a cache call must be on one CUDA device")
    if rows.shape[2] != dim:
        raise ValueError("the rows' dim must be the cache's")
    return heads, dim, page, batch


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
              v_scales: torch.Tensor, block_table: torch.Tensor, offsets: torch.Tensor, seq_lens: torch.Tensor,
              stream=None) -> None:
    """Write new keys and values into the 8-bit paged cache, in place.

    ``k``, ``v``: (tokens, kv_heads, dim) BF16 or FP16 of equal strides, the
    rows of sequence b at ``offsets[b]:offsets[b+1]`` (int32, batch + 1).
    ``k_cache``, ``v_cache``: uint8 (pages, kv_heads, page, dim) E4M3 codes in
    any order of equal strides (e.g. a transposed view of (pages, page,
    kv_heads, dim)); ``k_scales``, ``v_scales``: uint8 (pages, kv_heads), the
    E8M0 byte e + 127 of each page and head.  ``block_table``: int32 (batch,
    pages per sequence); ``seq_lens``: int32 (batch), each sequence's length
    with the new tokens.  A page that earlier tokens share keeps the larger
    of its scale and the new tokens', and its codes are rewritten when it grows."""
    dt = _check_rows(k, "k")
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride() or v.device != k.device:
        raise ValueError("k and v must have equal shapes, types and strides")
    heads, dim, page, batch = _cache_args(k, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens)
    if k.shape[1] != heads:
        raise ValueError("k must have the cache's kv_heads")
    cs = k_cache.stride()
    _call("bsq_kv_append", k.device,
          (dt, k.data_ptr(), v.data_ptr(), k.shape[0], heads, dim, k.stride(0), k.stride(1), k_cache.data_ptr(),
           v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), k_cache.shape[0], page, cs[0], cs[1], cs[2],
           block_table.data_ptr(), block_table.stride(0), block_table.shape[1], offsets.data_ptr(), seq_lens.data_ptr(), batch,
           _on(k.device, stream)))


def kv_attention_workspace_bytes(total: int, heads: int, kv_heads: int, dim: int, batch: int, max_q: int) -> int:
    """Bytes of the ``workspace`` of :func:`kv_attention` for `total` query rows."""
    return lib().bsq_kv_attention_workspace_bytes(total, heads, kv_heads, dim, batch, max_q)


def kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, block_table: torch.Tensor, offsets: torch.Tensor, seq_lens: torch.Tensor, max_q: int,
                 sm_scale: float | None = None, causal: bool = True, window: int = 0, out=None, return_lse: bool = False,
                 lse=None, workspace=None, stream=None):
    """Attention of ``q`` (tokens, heads, dim) over the 8-bit paged cache (its
    tensors as for :func:`kv_append`; ``seq_lens`` count the rows of ``q``).

    ``max_q``: the most rows of any sequence.  ``causal``: a sequence's last
    row sits at its last position and each row sees the keys up to its own.
    ``window`` > 0: only the last ``window`` of those.  ``sm_scale``: 1 /
    sqrt(dim) when None.  A row without keys gives zeros and an lse of -inf.
    ``workspace``: uint8, zeroed once (``torch.zeros``), left ready for the
    next call; allocated when None.  Returns ``out`` (contiguous, q's type),
    or (out, float32 lse (tokens, heads)) with ``return_lse``."""
    dt = _check_rows(q, "q")
    kv_heads, dim, page, batch = _cache_args(q, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens)
    total, heads = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((total, heads, dim), dtype=q.dtype, device=q.device)
    elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous() or out.device != q.device:
        raise ValueError("out must be a contiguous tensor of q's shape, type and device")
    if return_lse and lse is None:
        lse = torch.empty((total, heads), dtype=torch.float32, device=q.device)
    elif lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (total, heads) or not lse.is_contiguous() or
                              lse.device != q.device):
        raise ValueError("lse must be a contiguous float32 (tokens, heads) tensor on q's device")
    if workspace is None:
        workspace = torch.zeros(kv_attention_workspace_bytes(total, heads, kv_heads, dim, batch, max_q), dtype=torch.uint8,
                                device=q.device)
    cs = k_cache.stride()
    _call("bsq_kv_attention", q.device,
          (dt, q.data_ptr(), total, heads, kv_heads, dim, q.stride(0), q.stride(1), k_cache.data_ptr(), v_cache.data_ptr(),
           k_scales.data_ptr(), v_scales.data_ptr(), k_cache.shape[0], page, cs[0], cs[1], cs[2], block_table.data_ptr(),
           block_table.stride(0), block_table.shape[1], offsets.data_ptr(), seq_lens.data_ptr(), batch, max_q,
           1.0 / math.sqrt(dim) if sm_scale is None else sm_scale, 1 if causal else 0, window, out.data_ptr(),
           None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _on(q.device, stream)))
    return (out, lse) if return_lse else out


def moe_layer_workspace_bytes(fmt, tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    """Bytes of the ``workspace`` of :func:`moe_layer`."""
    return lib().bsq_moe_layer_workspace_bytes(_fmt(fmt), tokens, hidden, inter, experts, top_k)


def moe_layer(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
              w2_scales: torch.Tensor, fmt, top_k: int, x_sf=None, w13_sf=None, h_sf=None, w2_sf=None,
              renormalize: bool = True, out=None, workspace=None, stream=None) -> torch.Tensor:
    """A mixture-of-experts layer for at most 64 tokens.

    ``x``: BF16 (tokens, hidden); ``logits``: float32 (tokens, experts) of the
    router.  ``w13``: packed codes (experts, 2*inter, row bytes), gate rows
    first, and ``w2`` (experts, hidden, row bytes), as :func:`quantize` gives
    them for each expert's BF16 rows, with their 5D scales (experts, bytes).
    NVFP4 also takes the float32 (experts) tensor scales of x, w13, the inner
    activation and w2.  The ``top_k`` experts of the softmax over the logits are
    weighted by their probabilities (divided by their sum with
    ``renormalize``).  Activations are quantized to ``fmt`` as by
    :func:`quantize`, x before the first product and bf16(silu(g) * u) before the second.
    ``workspace``: uint8, zeroed once, left ready for the next call; allocated when None."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    tokens, hidden = x.shape
    if logits.dtype != torch.float32 or logits.dim() != 2 or logits.shape[0] != tokens or logits.stride(1) != 1:
        raise ValueError("logits must be a float32 (tokens, experts) tensor with unit inner stride")
    experts = logits.shape[1]
    f = _fmt(fmt)
    bits = 8 if f == FORMATS["mxfp8"] else 4
    if w13.dtype != torch.uint8 or w13.dim() != 3 or w2.dtype != torch.uint8 or w2.dim() != 3 or not w13.is_contiguous() or \
            not w2.is_contiguous():
        raise ValueError("w13 and w2 must be contiguous uint8 (experts, rows, row bytes) tensors")
    inter = w13.shape[1] // 2
    if w13.shape[0] != experts or w13.shape[1] % 2 or w13.shape[2] * 8 != hidden * bits or w2.shape[0] != experts or \
            w2.shape[1] != hidden or w2.shape[2] * 8 != inter * bits:
        raise ValueError("w13 must be (experts, 2*inter, row bytes of hidden) and w2 (experts, hidden, row bytes of inter)")
    for s, rows, cols in ((w13_scales, 2 * inter, hidden), (w2_scales, hidden, inter)):
        if s.dtype != torch.uint8 or not s.is_contiguous() or s.numel() != experts * lib().bsq_scales5d_bytes(f, rows, cols):
            raise ValueError("w13_scales and w2_scales must be contiguous uint8 tensors of each expert's 5D scales")
    sfs = (x_sf, w13_sf, h_sf, w2_sf)
    if f == FORMATS["nvfp4"]:
        for s in sfs:
            if s is None or s.dtype != torch.float32 or s.numel() != experts or not s.is_contiguous():
                raise ValueError("nvfp4 needs contiguous float32 (experts) tensors x_sf, w13_sf, h_sf and w2_sf")
    else:
        sfs = (None,) * 4
    device = x.device
    for t in (logits, w13, w13_scales, w2, w2_scales, *sfs):
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on one CUDA device")
    if out is None:
        out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=device)
    elif out.dtype != torch.bfloat16 or out.shape != x.shape or out.stride(1) != 1 or out.device != device:
        raise ValueError("out must be a (tokens, hidden) bfloat16 tensor with unit inner stride on x's device")
    if workspace is None:
        workspace = torch.zeros(lib().bsq_moe_layer_workspace_bytes(f, tokens, hidden, inter, experts, top_k),
                                dtype=torch.uint8, device=device)
    _call("bsq_moe_layer", device,
          (f, x.data_ptr(), x.stride(0), logits.data_ptr(), logits.stride(0), w13.data_ptr(), w13_scales.data_ptr(),
           w2.data_ptr(), w2_scales.data_ptr(), *(None if s is None else s.data_ptr() for s in sfs), out.data_ptr(),
           out.stride(0), tokens, hidden, inter, experts, top_k, 1 if renormalize else 0, workspace.data_ptr(),
           workspace.numel(), _on(device, stream)))
    return out
