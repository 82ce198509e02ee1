"""Refusals of the append with strides of their own for keys and values, on the CPU."""
import pytest

from test_serving_args import ALIGN, APPEND, CACHE_BAD, NULL, P, bsq  # noqa: F401

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
