"""Binding of the calls between cache and experts of a decoder layer:
projections over packed weights (``bsq_packed_linear``), norm and rotation of
query and key heads (``bsq_qk_norm_rope``), routing to experts
(``bsq_moe_route``) and the rows' order for the grouped calls
(``bsq_moe_rows``).  Streams, outputs and errors are as in serving.py."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import BsqError, _fmt, lib
from ._build import BINDING_PATH

_SCORING = {"softmax": 0, "sigmoid": 1}
_ext = None


def _binding():
    """The compiled binding (checks, allocations and calls; raises if it has not been built)."""
    global _ext
    if _ext is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"the binding is not built ({BINDING_PATH} missing); build it with "
                               "python -m fp8_activation_quantization_bsq_gb300._build")
        lib()
        loader = importlib.machinery.ExtensionFileLoader("_bsq_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_bsq_binding", loader))
        loader.exec_module(module)
        module.set_error(BsqError)
        _ext = module
    return _ext


def packed_linear(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, fmt, w_sf=None, add=None, out_dtype=None, out=None,
                  stream=None) -> torch.Tensor:
    """``x @ W.T`` (+ ``add``) over packed weights, x as it is (not quantized).

    ``x``: BF16 or FP16 (tokens, cols), cols a multiple of 32.  ``w``, ``w_scales``: uint8 codes (rows, row
    bytes) and 5D scales of the weights, as :func:`quantize` gives them for a (rows, cols) matrix; ``w_sf``
    (NVFP4): a float32 tensor of one element, the tensor scale that they were quantized with (e.g.
    ``tensor_sf(W)[1:]``).  ``add``: a residual (tokens, rows) with unit inner stride or a bias (rows), of the
    output's type; may be ``out``.  Returns ``out`` (tokens, rows) in ``out_dtype``: x's type (None) or float32."""
    return (_ext or _binding()).packed_linear(x, w, w_scales, _fmt(fmt), w_sf, add, out_dtype, out, stream)


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
    return (_ext or _binding()).qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)


def moe_route(logits: torch.Tensor, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_top: int = 2, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """Experts of each token and their weights: (int32 ids, float32 weights), both (tokens, top_k).

    ``logits``: (tokens, experts) float32, BF16 or FP16, at most 1024 experts.  ``scoring``: "softmax" or "sigmoid".
    An expert's value is its score plus ``bias`` (float32, experts), or its logit without a bias.  With ``groups`` > 1
    only the ``top_groups`` groups of consecutive experts with the largest sums of their ``group_top`` (1 or 2) largest
    values take part.  The ``top_k`` (at most 16) largest values are chosen, equal ones lowest expert first; weights are
    their scores without the bias, divided by their sum with ``renormalize``, times ``scale``.  Logits of -inf exclude an
    expert.  The choice is that of exact arithmetic (see bsq.h)."""
    sigmoid = _SCORING.get(scoring)
    if sigmoid is None:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}")
    return (_ext or _binding()).moe_route(logits, top_k, sigmoid, bias, groups, top_groups, group_top, renormalize, scale, ids, weights, stream)


def moe_rows(ids: torch.Tensor, experts: int, stream=None):
    """The rows of routed pairs, sorted by expert, for the grouped calls with one group per expert.

    ``ids``: contiguous int32 (tokens, top_k); a negative id has no row.  Returns int32 tensors (row_offsets
    (experts + 1), scales_offsets (experts + 1), row_indices (tokens * top_k), positions (tokens, top_k)): the first two and
    row_indices are :func:`grouped_quantize`'s, with ``expert_ids`` 0 to experts - 1, ``total_rows`` tokens * top_k and
    ``total_scale_rows`` of :func:`moe_rows_scale_rows`; ``positions`` is each pair's row (-1 without one)."""
    return (_ext or _binding()).moe_rows(ids, experts, stream)


def moe_rows_scale_rows(pairs: int, experts: int) -> int:
    """Scale rows that `pairs` rows of `experts` experts take at most, each expert's count rounded up to 128."""
    few = min(pairs, experts)  # experts with rows
    return (pairs + 127 * few) // 128 * 128
