"""Binding of the calls between cache and experts of a decoder layer:
projections over packed weights (``bsq_packed_linear``), norm and rotation of
query and key heads (``bsq_qk_norm_rope``), routing to experts
(``bsq_moe_route``) and the rows' order for the grouped calls
(``bsq_moe_rows``).  Streams, outputs and errors are as in serving.py."""
from __future__ import annotations

import torch

from . import FORMATS, _fmt
from .serving import _BF16, _DTYPES, _F32, _I32, _U8, _call, _new, _rows

_ALL_DTYPES = {**_DTYPES, torch.float32: 2}
_NVFP4, _MXFP8 = FORMATS["nvfp4"], FORMATS["mxfp8"]
_SCORING = {"softmax": 0, "sigmoid": 1}


def packed_linear(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, fmt, w_sf=None, add=None, out_dtype=None, out=None,
                  stream=None) -> torch.Tensor:
    """``x @ W.T`` (+ ``add``) over packed weights, x as it is (not quantized).

    ``x``: BF16 or FP16 (tokens, cols), cols a multiple of 32.  ``w``, ``w_scales``: uint8 codes (rows, row
    bytes) and 5D scales of the weights, as :func:`quantize` gives them for a (rows, cols) matrix; ``w_sf``
    (NVFP4): a float32 tensor of one element, the tensor scale that they were quantized with (e.g.
    ``tensor_sf(W)[1:]``).  ``add``: a residual (tokens, rows) with unit inner stride or a bias (rows), of the
    output's type; may be ``out``.  Returns ``out`` (tokens, rows) in ``out_dtype``: x's type (None) or float32."""
    shape, dt = x.shape, _DTYPES.get(x.dtype)
    if dt is None or len(shape) != 2 or not x.is_cuda or ((xs := x.stride())[1] != 1 and shape[0]):
        raise ValueError("x must be a 2-D bfloat16 or float16 CUDA tensor with unit inner stride")
    tokens, cols = shape
    index = x.get_device()
    f = _fmt(fmt)
    wshape = w.shape
    if w.dtype is not _U8 or len(wshape) != 2 or not w.is_contiguous() or wshape[1] != (cols if f == _MXFP8 else cols // 2) or cols % 32:
        raise ValueError("w must be a contiguous uint8 (rows, row bytes of cols) tensor, cols a multiple of 32")
    rows = wshape[0]
    if w_scales.dtype is not _U8 or not w_scales.is_contiguous() or \
            w_scales.numel() != -(-rows // 128) * -(-cols // (64 if f == _NVFP4 else 128)) * 512:
        raise ValueError("w_scales must be a contiguous uint8 tensor of the weights' 5D scales")
    if w.get_device() != index or w_scales.get_device() != index:
        raise ValueError("all tensors must be on one CUDA device")
    sf = None
    if f == _NVFP4:
        if w_sf is None or w_sf.dtype is not _F32 or w_sf.numel() != 1 or w_sf.get_device() != index:
            raise ValueError("nvfp4 needs w_sf, a float32 tensor of one element on x's device")
        sf = w_sf.data_ptr()
    if out is None:
        out_dtype = x.dtype if out_dtype is None else out_dtype
        od = _ALL_DTYPES.get(out_dtype)
        out = _new(stream, torch.empty, (tokens, rows), out_dtype, x.device)
        ld_out = rows
    else:
        od, os = _ALL_DTYPES.get(out.dtype), out.stride()
        if out.shape != (tokens, rows) or os[1] != 1 or out.get_device() != index or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must be a (tokens, rows) tensor of out_dtype with unit inner stride on x's device")
        ld_out = os[0]
    if od != dt and od != 2:
        raise ValueError("out_dtype must be x's type or float32")
    ap, ld_add = None, 0
    if add is not None:
        if add.dtype != out.dtype or add.get_device() != index or add.stride(-1) != 1 or add.shape[-1] != rows or \
                (add.shape != (tokens, rows) and add.shape != (rows,)):
            raise ValueError("add must be a (tokens, rows) or (rows) tensor of the output's type with unit inner stride on x's device")
        ap = add.data_ptr()
        ld_add = add.stride(0) if len(add.shape) == 2 else 0
    _call("bsq_packed_linear", index, stream, (f, dt, x.data_ptr(), tokens, cols, xs[0] if tokens > 1 else cols, w.data_ptr(),
                                               w_scales.data_ptr(), rows, sf, ap, ld_add, od, out.data_ptr(), ld_out))
    return out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Norm of query and key heads and their rotation by position, in one pass.

    ``q`` (tokens, heads, dim) and ``k`` (tokens, kv_heads, dim): BF16 or FP16 with any strides that are multiples of
    8 (views of a projection's output), dim a multiple of 8 up to 256.  ``positions``: int32 (tokens); a token at a
    negative one is left out (its rows of given outputs stay as they are).  ``inv_freq``: float32, at most dim / 2
    frequencies: pair i of a row, elements (i, i + n) of n frequencies or (2i, 2i + 1) with ``interleaved``, turns by
    position * inv_freq[i]; the row's other elements pass.  ``q_weight``, ``k_weight``: dim weights (q's type or
    float32) of a root-mean-square norm before that; None: no norm.  Returns (q_out, k_out), contiguous when not given;
    each may be its input itself."""
    dt, qshape, qs, index = _rows(q, "q")
    kshape, ks = k.shape, k.stride()
    tokens, heads, dim = qshape
    if k.dtype != q.dtype or len(kshape) != 3 or kshape[0] != tokens or kshape[2] != dim or ks[2] != 1 or k.get_device() != index:
        raise ValueError("k must be a (tokens, kv_heads, dim) tensor of q's type and device with unit inner stride")
    if positions.dtype is not _I32 or positions.shape != (tokens,) or not positions.is_contiguous() or \
            inv_freq.dtype is not _F32 or len(inv_freq.shape) != 1 or not inv_freq.is_contiguous() or \
            positions.get_device() != index or inv_freq.get_device() != index:
        raise ValueError("positions must be an int32 (tokens) and inv_freq a float32 (pairs) contiguous tensor on q's device")
    wd, weights = dt, [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is not None:
            if (w.dtype != q.dtype and w.dtype is not _F32) or w.shape != (dim,) or not w.is_contiguous() or w.get_device() != index:
                raise ValueError("q_weight and k_weight must be contiguous (dim) tensors of q's type or float32 on q's device")
            wd, weights[i] = _ALL_DTYPES[w.dtype], w.data_ptr()
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have one type")
    if q_out is None:
        q_out = _new(stream, torch.empty, qshape, q.dtype, q.device)
        qos = (heads * dim, dim)
    else:
        qos = _out_strides(q_out, q)
    if k_out is None:
        k_out = _new(stream, torch.empty, kshape, q.dtype, q.device)
        kos = (kshape[1] * dim, dim)
    else:
        kos = _out_strides(k_out, k)
    _call("bsq_qk_norm_rope", index, stream,
          (dt, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], tokens, heads, kshape[1], dim, positions.data_ptr(),
           inv_freq.data_ptr(), inv_freq.shape[0], 1 if interleaved else 0, weights[0], weights[1], wd, eps, q_out.data_ptr(), qos[0], qos[1],
           k_out.data_ptr(), kos[0], kos[1]))
    return q_out, k_out


def _out_strides(out, x):
    stride = out.stride()
    if out.dtype != x.dtype or out.shape != x.shape or stride[2] != 1 or out.get_device() != x.get_device():
        raise ValueError("q_out and k_out must have their inputs' shapes, types and device and unit inner strides")
    return stride


def moe_route(logits: torch.Tensor, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_top: int = 2, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """Experts of each token and their weights: (int32 ids, float32 weights), both (tokens, top_k).

    ``logits``: (tokens, experts) float32, BF16 or FP16, at most 1024 experts.  ``scoring``: "softmax" or "sigmoid".
    An expert's value is its score plus ``bias`` (float32, experts), or its logit without a bias.  With ``groups`` > 1
    only the ``top_groups`` groups of consecutive experts with the largest sums of their ``group_top`` (1 or 2) largest
    values take part.  The ``top_k`` (at most 16) largest values are chosen, equal ones lowest expert first; weights are
    their scores without the bias, divided by their sum with ``renormalize``, times ``scale``.  Logits of -inf exclude an
    expert.  The choice is that of exact arithmetic (see bsq.h)."""
    dt, shape = _ALL_DTYPES.get(logits.dtype), logits.shape
    if dt is None or len(shape) != 2 or not logits.is_cuda or ((ls := logits.stride())[1] != 1 and shape[1] > 1):
        raise ValueError("logits must be a 2-D float32, bfloat16 or float16 CUDA tensor with unit inner stride")
    sigmoid = _SCORING.get(scoring)
    if sigmoid is None:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}")
    tokens, experts = shape
    index = logits.get_device()
    if bias is not None and (bias.dtype is not _F32 or bias.shape != (experts,) or not bias.is_contiguous() or bias.get_device() != index):
        raise ValueError("bias must be a contiguous float32 (experts) tensor on the logits' device")
    pair = (tokens, top_k)
    if ids is None:
        ids = _new(stream, torch.empty, pair, _I32, logits.device)
    elif ids.dtype is not _I32 or ids.shape != pair or not ids.is_contiguous() or ids.get_device() != index:
        raise ValueError("ids must be a contiguous int32 (tokens, top_k) tensor on the logits' device")
    if weights is None:
        weights = _new(stream, torch.empty, pair, _F32, logits.device)
    elif weights.dtype is not _F32 or weights.shape != pair or not weights.is_contiguous() or weights.get_device() != index:
        raise ValueError("weights must be a contiguous float32 (tokens, top_k) tensor on the logits' device")
    _call("bsq_moe_route", index, stream,
          (dt, logits.data_ptr(), ls[0] if tokens > 1 else experts, tokens, experts, top_k, sigmoid, None if bias is None else bias.data_ptr(),
           groups, top_groups, group_top, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr()))
    return ids, weights


def moe_rows(ids: torch.Tensor, experts: int, stream=None):
    """The rows of routed pairs, sorted by expert, for the grouped calls with one group per expert.

    ``ids``: contiguous int32 (tokens, top_k); a negative id has no row.  Returns int32 tensors (row_offsets
    (experts + 1), scales_offsets (experts + 1), row_indices (tokens * top_k), positions (tokens, top_k)): the first two and
    row_indices are :func:`grouped_quantize`'s, with ``expert_ids`` 0 to experts - 1, ``total_rows`` tokens * top_k and
    ``total_scale_rows`` of :func:`moe_rows_scale_rows`; ``positions`` is each pair's row (-1 without one)."""
    shape = ids.shape
    if ids.dtype is not _I32 or len(shape) != 2 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 (tokens, top_k) CUDA tensor")
    index, device = ids.get_device(), ids.device
    offsets = _new(stream, torch.empty, (2, experts + 1), _I32, device)
    places = _new(stream, torch.empty, (2, shape[0] * shape[1]), _I32, device)
    row_offsets, scales_offsets = offsets.unbind()
    row_indices, positions = places.unbind()
    _call("bsq_moe_rows", index, stream, (ids.data_ptr(), shape[0], shape[1], experts, row_offsets.data_ptr(), scales_offsets.data_ptr(),
                                          row_indices.data_ptr(), positions.data_ptr()))
    return row_offsets, scales_offsets, row_indices, positions.view(shape)


def moe_rows_scale_rows(pairs: int, experts: int) -> int:
    """Scale rows that `pairs` rows of `experts` experts take at most, each expert's count rounded up to 128."""
    few = min(pairs, experts)  # experts with rows
    return (pairs + 127 * few) // 128 * 128
