"""Refusals of the append with strides of its own for keys and values, and of the workspace calls, on the CPU."""
import pytest

from test_serving_args import ALIGN, APPEND, ATTN, CACHE_BAD, NULL, P, SHAPE, bsq  # noqa: F401

STRIDED = {}
for key, value in APPEND.items():
    STRIDED[key] = value
    if key == "src_head":
        STRIDED |= dict(v_tok=192, v_head=64)


@pytest.mark.parametrize("change,code", CACHE_BAD + [
    (dict(k=None), NULL), (dict(v=P + 2), ALIGN), (dict(src_tok=132), ALIGN), (dict(src_head=60), ALIGN), (dict(v_tok=196), ALIGN),
    (dict(v_head=68), ALIGN)])
def test_strided_append_refusals(bsq, change, code):  # noqa: F811
    assert bsq.lib().bsq_kv_append_strided(*{**STRIDED, **change}.values()) == code


def test_workspace_zero_refusals(bsq):  # noqa: F811
    lib = bsq.lib()
    assert lib.bsq_workspace_zero(None, 16, None) == NULL
    assert lib.bsq_workspace_zero(P, -1, None) == SHAPE
    assert lib.bsq_workspace_zero(None, 0, None) == 0
    assert lib.bsq_kv_attention_counter_bytes() > 0 and lib.bsq_moe_layer_counter_bytes() > 0
    assert bsq.moe_layer_workspace_bytes("mxfp8", 1, 64, 128, 1, 1) > lib.bsq_moe_layer_counter_bytes()
    assert bsq.kv_attention_workspace_bytes(1, 1, 1, 64, 1, 1) > lib.bsq_kv_attention_counter_bytes()


def test_more_sequences_than_a_grid_holds(bsq):  # noqa: F811
    for batch in (1 << 30, (1 << 31) - 1):
        assert bsq.lib().bsq_kv_append(*{**APPEND, "batch": batch}.values()) == SHAPE
        assert bsq.lib().bsq_kv_attention(*{**ATTN, "batch": batch}.values()) == SHAPE
