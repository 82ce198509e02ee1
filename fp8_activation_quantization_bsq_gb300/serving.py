"""Binding of the serving calls: the 8-bit paged key/value cache
(``bsq_kv_append``, ``bsq_kv_attention``) and the few-token expert layer
(``bsq_moe_layer``).  As in the package's other calls, work is enqueued on the
current stream (or ``stream``), outputs are allocated with torch when not
passed in (under the given stream, so that their memory is free in its order),
and a refused argument raises ValueError or BsqError."""
from __future__ import annotations

import math

import torch

from . import FORMATS, _check, _fmt, lib

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_MXFP8, _NVFP4 = FORMATS["mxfp8"], FORMATS["nvfp4"]

# A call of these costs the host about as much as the GPU for a single token,
# so each attribute of a tensor is read once and the checks are plain expressions.


def _call(name, index, stream, args):
    """Call the library on device `index` and the given or current stream."""
    fn = getattr(lib(), name)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        _check(rc, name)


def _new(stream, make, shape, dtype, device):
    """make(shape) on the stream that the call runs on."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _own_workspace(stream, index, nbytes, counter_bytes, device):
    """A workspace for one call: its counters have to be zero, the rest may hold anything."""
    ws = _new(stream, torch.empty, nbytes, _U8, device)
    _call("bsq_workspace_zero", index, stream, (ws.data_ptr(), min(nbytes, counter_bytes)))
    return ws


def _rows(x, what):
    """(dtype code, shape, strides, device index) of a (tokens, heads, dim) 16-bit CUDA tensor."""
    code, shape = _DTYPES.get(x.dtype), x.shape
    if code is None or len(shape) != 3 or not x.is_cuda or (stride := x.stride())[2] != 1:
        raise ValueError(f"{what} must be a (tokens, heads, dim) bfloat16 or float16 CUDA tensor with unit inner stride")
    return code, shape, stride, x.get_device()


def _cache(dim, index, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens):
    """Checks the cache tensors of a call; the library's arguments from the cache to the batch."""
    shape, cs = k_cache.shape, k_cache.stride()
    if k_cache.dtype is not _U8 or v_cache.dtype is not _U8 or len(shape) != 4 or v_cache.shape != shape or \
            v_cache.stride() != cs or cs[3] != 1:
        raise ValueError("k_cache and v_cache must be uint8 (pages, kv_heads, page, dim) tensors of equal strides, unit inner stride")
    pages, heads, page, cache_dim = shape
    if k_scales.dtype is not _U8 or v_scales.dtype is not _U8 or k_scales.shape != (pages, heads) or \
            v_scales.shape != (pages, heads) or not k_scales.is_contiguous() or not v_scales.is_contiguous():
        raise ValueError("k_scales and v_scales must be contiguous uint8 (pages, kv_heads) tensors")
    tshape = block_table.shape
    if block_table.dtype is not _I32 or len(tshape) != 2 or ((ts := block_table.stride())[1] != 1 and tshape[1] > 1):
        raise ValueError("block_table must be an int32 (batch, pages per sequence) tensor with unit inner stride")
    batch, width = tshape
    if offsets.dtype is not _I32 or offsets.shape != (batch + 1,) or not offsets.is_contiguous() or \
            seq_lens.dtype is not _I32 or seq_lens.shape != (batch,) or not seq_lens.is_contiguous():
        raise ValueError("offsets and seq_lens must be contiguous int32 tensors of batch + 1 and batch entries")
    if not (k_cache.get_device() == v_cache.get_device() == k_scales.get_device() == v_scales.get_device() ==
            block_table.get_device() == offsets.get_device() == seq_lens.get_device() == index):
        raise ValueError("all tensors of a cache call must be on one CUDA device")
    if dim != cache_dim:
        raise ValueError("the rows' dim must be the cache's")
    return heads, (k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), pages, page, cs[0], cs[1], cs[2],
                   block_table.data_ptr(), ts[0], width, offsets.data_ptr(), seq_lens.data_ptr(), batch)


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
              v_scales: torch.Tensor, block_table: torch.Tensor, offsets: torch.Tensor, seq_lens: torch.Tensor,
              stream=None) -> None:
    """Write new keys and values into the 8-bit paged cache, in place.

    ``k``, ``v``: (tokens, kv_heads, dim) BF16 or FP16, each with strides of its own, the
    rows of sequence b at ``offsets[b]:offsets[b+1]`` (int32, batch + 1).
    ``k_cache``, ``v_cache``: uint8 (pages, kv_heads, page, dim) E4M3 codes in
    any order of equal strides (e.g. a transposed view of (pages, page,
    kv_heads, dim)); ``k_scales``, ``v_scales``: uint8 (pages, kv_heads), the
    E8M0 byte e + 127 of each page and head.  ``block_table``: int32 (batch,
    pages per sequence); ``seq_lens``: int32 (batch), each sequence's length
    with the new tokens.  A page that earlier tokens share keeps the larger
    of its scale and the new tokens', and its codes are rewritten when it grows."""
    dt, shape, stride, index = _rows(k, "k")
    vs = v.stride()
    if v.dtype != k.dtype or v.shape != shape or vs[2] != 1 or v.get_device() != index:
        raise ValueError("k and v must have equal shapes and types, unit inner strides and one device")
    heads, cache = _cache(shape[2], index, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens)
    if shape[1] != heads:
        raise ValueError("k must have the cache's kv_heads")
    _call("bsq_kv_append_strided", index, stream,
          (dt, k.data_ptr(), v.data_ptr(), shape[0], heads, shape[2], stride[0], stride[1], vs[0], vs[1], *cache))


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
    next call (but for one after which :func:`device_error` reports
    BSQ_ERR_TIMEOUT: then zeroed again); allocated when None.  Returns ``out`` (contiguous, q's type),
    or (out, float32 lse (tokens, heads)) with ``return_lse``."""
    dt, shape, stride, index = _rows(q, "q")
    total, heads, dim = shape
    kv_heads, cache = _cache(dim, index, k_cache, v_cache, k_scales, v_scales, block_table, offsets, seq_lens)
    if out is None:
        out = _new(stream, torch.empty, shape, q.dtype, q.device)
    elif out.dtype != q.dtype or out.shape != shape or not out.is_contiguous() or out.get_device() != index:
        raise ValueError("out must be a contiguous tensor of q's shape, type and device")
    if lse is None:
        if return_lse:
            lse = _new(stream, torch.empty, (total, heads), _F32, q.device)
    elif lse.dtype is not _F32 or lse.shape != (total, heads) or not lse.is_contiguous() or lse.get_device() != index:
        raise ValueError("lse must be a contiguous float32 (tokens, heads) tensor on q's device")
    if workspace is None:
        workspace = _own_workspace(stream, index, kv_attention_workspace_bytes(total, heads, kv_heads, dim, cache[-1], max_q),
                                   lib().bsq_kv_attention_counter_bytes(), q.device)
    elif workspace.dtype is not _U8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    _call("bsq_kv_attention", index, stream,
          (dt, q.data_ptr(), total, heads, kv_heads, dim, stride[0], stride[1], *cache, max_q,
           1.0 / math.sqrt(dim) if sm_scale is None else sm_scale, 1 if causal else 0, window, out.data_ptr(),
           None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel()))
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
    ``workspace``: uint8, zeroed once, left ready for the next call (but for one
    after which :func:`device_error` reports BSQ_ERR_TIMEOUT: then zeroed
    again); allocated when None."""
    shape = x.shape
    if x.dtype is not _BF16 or len(shape) != 2 or not x.is_cuda or (xs := x.stride())[1] != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    tokens, hidden = shape
    index = x.get_device()
    lshape = logits.shape
    if logits.dtype is not _F32 or len(lshape) != 2 or lshape[0] != tokens or (ls := logits.stride())[1] != 1:
        raise ValueError("logits must be a float32 (tokens, experts) tensor with unit inner stride")
    experts = lshape[1]
    f = _fmt(fmt)
    s13, s2 = w13.shape, w2.shape
    if w13.dtype is not _U8 or len(s13) != 3 or w2.dtype is not _U8 or len(s2) != 3 or not w13.is_contiguous() or \
            not w2.is_contiguous():
        raise ValueError("w13 and w2 must be contiguous uint8 (experts, rows, row bytes) tensors")
    inter = s13[1] // 2
    per = 1 if f == _MXFP8 else 2  # values per byte
    if s13 != (experts, 2 * inter, hidden // per) or s2 != (experts, hidden, inter // per) or hidden % per or inter % per:
        raise ValueError("w13 must be (experts, 2*inter, row bytes of hidden) and w2 (experts, hidden, row bytes of inter)")
    sf = 16 if f == _NVFP4 else 32
    n13 = experts * -(-2 * inter // 128) * -(-hidden // (4 * sf)) * 512
    n2 = experts * -(-hidden // 128) * -(-inter // (4 * sf)) * 512
    if w13_scales.dtype is not _U8 or w13_scales.numel() != n13 or not w13_scales.is_contiguous() or \
            w2_scales.dtype is not _U8 or w2_scales.numel() != n2 or not w2_scales.is_contiguous():
        raise ValueError("w13_scales and w2_scales must be contiguous uint8 tensors of each expert's 5D scales")
    if not (logits.get_device() == w13.get_device() == w2.get_device() == w13_scales.get_device() == w2_scales.get_device() == index):
        raise ValueError("all tensors must be on one CUDA device")
    if f == _NVFP4:
        for t in (x_sf, w13_sf, h_sf, w2_sf):
            if t is None or t.dtype is not _F32 or t.numel() != experts or not t.is_contiguous() or t.get_device() != index:
                raise ValueError("nvfp4 needs contiguous float32 (experts) tensors x_sf, w13_sf, h_sf and w2_sf on x's device")
        sfs = (x_sf.data_ptr(), w13_sf.data_ptr(), h_sf.data_ptr(), w2_sf.data_ptr())
    else:
        sfs = (None, None, None, None)
    if out is None:
        out = _new(stream, torch.empty, shape, _BF16, x.device)
    elif out.dtype is not _BF16 or out.shape != shape or out.stride(1) != 1 or out.get_device() != index:
        raise ValueError("out must be a (tokens, hidden) bfloat16 tensor with unit inner stride on x's device")
    if workspace is None:
        workspace = _own_workspace(stream, index, moe_layer_workspace_bytes(f, tokens, hidden, inter, experts, top_k),
                                   lib().bsq_moe_layer_counter_bytes(), x.device)
    elif workspace.dtype is not _U8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    _call("bsq_moe_layer", index, stream,
          (f, x.data_ptr(), xs[0], logits.data_ptr(), ls[0], w13.data_ptr(), w13_scales.data_ptr(), w2.data_ptr(),
           w2_scales.data_ptr(), *sfs, out.data_ptr(), out.stride(0), tokens, hidden, inter, experts, top_k,
           1 if renormalize else 0, workspace.data_ptr(), workspace.numel()))
    return out
