"""Refusals of the serving calls, on the CPU: the C entry points return the
documented status before anything is enqueued, the binding raises."""
import pytest
import torch

P = 0x10000  # a fake, aligned, never dereferenced pointer
OK, NULL, SHAPE, ALIGN, VALUE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def bsq():
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    import fp8_activation_quantization_bsq_gb300 as m
    return m


APPEND = dict(dtype=0, k=P, v=P, total=4, kv_heads=2, dim=64, src_tok=128, src_head=64, kc=P, vc=P, ks=P, vs=P, pages=8, page=16,
              cs_page=2048, cs_head=1024, cs_tok=64, table=P, table_ld=4, width=4, offsets=P, lens=P, batch=2, stream=None)
ATTN = dict(dtype=0, q=P, total=4, heads=4, kv_heads=2, dim=64, q_tok=256, q_head=64, kc=P, vc=P, ks=P, vs=P, pages=8, page=16,
            cs_page=2048, cs_head=1024, cs_tok=64, table=P, table_ld=4, width=4, offsets=P, lens=P, batch=2, max_q=2, sm_scale=1.0,
            causal=1, window=0, out=P, lse=None, ws=P, ws_bytes=1 << 40, stream=None)
CACHE_BAD = [(dict(dtype=2), VALUE), (dict(dtype=-1), VALUE), (dict(total=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(kv_heads=0), SHAPE),
             (dict(dim=96), SHAPE), (dict(dim=256), SHAPE), (dict(page=8), SHAPE), (dict(page=256), SHAPE), (dict(pages=0), SHAPE),
             (dict(width=-1), SHAPE), (dict(width=(1 << 26) + 1, table_ld=1 << 27), SHAPE), (dict(table_ld=3), SHAPE), (dict(cs_tok=48), SHAPE), (dict(cs_page=-16), SHAPE),
             (dict(kc=None), NULL), (dict(vs=None), NULL), (dict(table=None), NULL), (dict(offsets=None), NULL), (dict(lens=None), NULL),
             (dict(kc=P + 8), ALIGN), (dict(cs_page=2056), ALIGN), (dict(cs_head=1032), ALIGN), (dict(cs_tok=72), ALIGN),
             (dict(table=P + 2), ALIGN), (dict(total=0), OK), (dict(batch=0), OK)]


@pytest.mark.parametrize("change,code", CACHE_BAD + [
    (dict(k=None), NULL), (dict(v=P + 2), ALIGN), (dict(src_tok=132), ALIGN), (dict(src_head=60), ALIGN)])
def test_append_refusals(bsq, change, code):
    assert bsq.lib().bsq_kv_append(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", CACHE_BAD + [
    (dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(heads=130, kv_heads=2), SHAPE), (dict(window=-1), SHAPE), (dict(max_q=0), SHAPE),
    (dict(sm_scale=float("inf")), VALUE), (dict(sm_scale=float("nan")), VALUE), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(ws_bytes=64), SHAPE), (dict(out=P + 4), ALIGN), (dict(lse=P + 2), ALIGN), (dict(q_tok=252), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(total=(1 << 29) + 1), SHAPE)])
def test_attention_refusals(bsq, change, code):
    assert bsq.lib().bsq_kv_attention(*{**ATTN, **change}.values()) == code


MOE = dict(fmt=2, x=P, ld_x=64, logits=P, ld_logits=4, w13=P, w13_s=P, w2=P, w2_s=P, x_sf=None, w13_sf=None, h_sf=None, w2_sf=None, y=P,
           ld_y=64, tokens=2, hidden=64, inter=128, experts=4, top_k=2, renorm=1, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(fmt=3), VALUE), (dict(tokens=-1), SHAPE), (dict(tokens=65), SHAPE), (dict(hidden=48), SHAPE), (dict(hidden=0), SHAPE),
    (dict(inter=96), SHAPE), (dict(inter=0), SHAPE), (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE), (dict(top_k=0), SHAPE),
    (dict(top_k=5), SHAPE), (dict(experts=20, ld_logits=20, top_k=17), SHAPE), (dict(ld_x=56), SHAPE), (dict(ld_y=32), SHAPE),
    (dict(ld_logits=3), SHAPE), (dict(x=None), NULL), (dict(logits=None), NULL), (dict(w2_s=None), NULL), (dict(y=None), NULL),
    (dict(ws=None), NULL), (dict(fmt=0), NULL), (dict(ws_bytes=100), SHAPE), (dict(x=P + 2), ALIGN), (dict(w13=P + 8), ALIGN),
    (dict(ld_x=68), ALIGN), (dict(ld_y=68), ALIGN), (dict(ws=P + 16), ALIGN), (dict(tokens=0), OK)])
def test_moe_refusals(bsq, change, code):
    assert bsq.lib().bsq_moe_layer(*{**MOE, **change}.values()) == code


def test_workspace_sizes(bsq):
    assert bsq.kv_attention_workspace_bytes(1, 8, 2, 64, 1, 1) > 0
    assert bsq.kv_attention_workspace_bytes(1, 8, 3, 64, 1, 1) == 0 and bsq.kv_attention_workspace_bytes(1, 8, 2, 96, 1, 1) == 0
    assert bsq.moe_layer_workspace_bytes("nvfp4", 1, 64, 128, 4, 2) > 0
    assert bsq.moe_layer_workspace_bytes("nvfp4", 65, 64, 128, 4, 2) == 0 and bsq.moe_layer_workspace_bytes("mxfp8", 1, 64, 100, 4, 2) == 0


def test_binding_rejects_host_and_mistyped_tensors(bsq):
    b16, u8, i32, f32 = (lambda *s, t=t: torch.zeros(s, dtype=t) for t in (torch.bfloat16, torch.uint8, torch.int32, torch.float32))
    cache = (u8(2, 1, 16, 64), u8(2, 1, 16, 64), u8(2, 1), u8(2, 1), i32(1, 1), i32(2), i32(1))
    with pytest.raises(ValueError, match="CUDA"):
        bsq.kv_append(b16(1, 1, 64), b16(1, 1, 64), *cache)
    with pytest.raises(ValueError, match="CUDA"):
        bsq.kv_attention(f32(1, 1, 64), *cache, 1)
    with pytest.raises(ValueError, match="CUDA"):
        bsq.moe_layer(b16(1, 64), f32(1, 4), u8(4, 256, 64), u8(4, 1024), u8(4, 64, 128), u8(4, 512), "mxfp8", 2)
