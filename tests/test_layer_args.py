"""Refusals of the calls between cache and experts, on the CPU: the C entry
points return the documented status before anything is enqueued, the binding
raises."""
import pytest
import torch

P = 0x10000  # a fake, aligned, never dereferenced pointer
OK, NULL, SHAPE, ALIGN, VALUE = 0, 1, 2, 3, 4
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def bsq():
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    import fp8_activation_quantization_bsq_gb300 as m
    return m


LINEAR = dict(fmt=0, dtype=0, x=P, tokens=2, cols=64, ld_x=64, w=P, ws=P, rows=100, sf=P, add=None, ld_add=0, out_dtype=0, out=P, ld_out=100,
              stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(fmt=3), VALUE), (dict(fmt=-1), VALUE), (dict(dtype=2), VALUE), (dict(dtype=-1), VALUE), (dict(out_dtype=1), VALUE), (dict(out_dtype=3), VALUE),
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 20) + 1), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 20) + 1, ld_out=1 << 21), SHAPE),
    (dict(cols=0), SHAPE), (dict(cols=48), SHAPE), (dict(cols=(1 << 20) + 32, ld_x=1 << 21), SHAPE), (dict(ld_x=56), SHAPE), (dict(ld_x=-64), SHAPE),
    (dict(ld_out=99), SHAPE), (dict(ld_out=-100), SHAPE), (dict(add=P, ld_add=99), SHAPE), (dict(add=P, ld_add=-1), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(sf=None), NULL), (dict(out=None), NULL),
    (dict(x=P + 8), ALIGN), (dict(ld_x=68), ALIGN), (dict(w=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(sf=P + 2), ALIGN), (dict(out=P + 1), ALIGN),
    (dict(out_dtype=2, out=P + 2), ALIGN), (dict(add=P + 1), ALIGN), (dict(tokens=0), OK), (dict(rows=0), OK), (dict(tokens=0, x=None, out=None), OK)])
def test_linear_refusals(bsq, change, code):
    assert bsq.lib().bsq_packed_linear(*{**LINEAR, **change}.values()) == code


def test_linear_mx_needs_no_tensor_scale(bsq):
    assert bsq.lib().bsq_packed_linear(*{**LINEAR, "fmt": 1, "sf": None, "out": P + 1}.values()) == ALIGN


ROPE = dict(dtype=0, q=P, q_tok=512, q_head=64, k=P, k_tok=128, k_head=64, tokens=3, heads=8, kv_heads=2, dim=64, pos=P, freq=P, pairs=32,
            interleaved=0, qw=P, kw=P, wd=0, eps=1e-6, qo=P, qo_tok=512, qo_head=64, ko=P, ko_tok=128, ko_head=64, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), VALUE), (dict(wd=1), VALUE), (dict(wd=3), VALUE), (dict(eps=-1.0), VALUE), (dict(eps=NAN), VALUE), (dict(eps=INF), VALUE),
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(heads=-1), SHAPE), (dict(heads=4097), SHAPE), (dict(kv_heads=-1), SHAPE),
    (dict(dim=0), SHAPE), (dict(dim=60), SHAPE), (dict(dim=264), SHAPE), (dict(pairs=33), SHAPE), (dict(pairs=-1), SHAPE), (dict(q_tok=-8), SHAPE),
    (dict(ko_head=1 << 31), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL), (dict(freq=None), NULL), (dict(qo=None), NULL),
    (dict(ko=None), NULL), (dict(q=P + 8), ALIGN), (dict(k_tok=132), ALIGN), (dict(qo_head=68), ALIGN), (dict(ko=P + 2), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(freq=P + 1), ALIGN), (dict(qw=P + 1), ALIGN), (dict(wd=2, kw=P + 2), ALIGN), (dict(tokens=0), OK), (dict(heads=0, kv_heads=0), OK)])
def test_rope_refusals(bsq, change, code):
    assert bsq.lib().bsq_qk_norm_rope(*{**ROPE, **change}.values()) == code


ROUTE = dict(dtype=2, z=P, ld=64, tokens=3, experts=64, top_k=4, sigmoid=0, bias=P, groups=8, top_groups=2, group_top=2, renorm=1, scale=1.0, ids=P,
             weights=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), VALUE), (dict(scale=INF), VALUE), (dict(scale=NAN), VALUE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(experts=0), SHAPE), (dict(experts=1032, ld=1032), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=17), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=7), SHAPE), (dict(groups=64, top_groups=8), SHAPE), (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE),
    (dict(group_top=0), SHAPE), (dict(group_top=3), SHAPE), (dict(top_k=9, top_groups=1), SHAPE), (dict(ld=63), SHAPE), (dict(ld=-1), SHAPE),
    (dict(z=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(z=P + 2), ALIGN), (dict(bias=P + 2), ALIGN),
    (dict(ids=P + 1), ALIGN), (dict(weights=P + 2), ALIGN), (dict(tokens=0), OK)])
def test_route_refusals(bsq, change, code):
    assert bsq.lib().bsq_moe_route(*{**ROUTE, **change}.values()) == code


ROWS = dict(ids=P, tokens=3, top_k=2, experts=5, ro=P, so=P, idx=P, pos=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 30), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=1025), SHAPE), (dict(experts=0), SHAPE),
    (dict(experts=1025), SHAPE), (dict(ids=None), NULL), (dict(ro=None), NULL), (dict(so=None), NULL), (dict(idx=None), NULL), (dict(pos=None), NULL),
    (dict(ids=P + 2), ALIGN), (dict(ro=P + 1), ALIGN), (dict(idx=P + 2), ALIGN)])
def test_rows_refusals(bsq, change, code):
    assert bsq.lib().bsq_moe_rows(*{**ROWS, **change}.values()) == code


def test_scale_rows_bound(bsq):
    assert bsq.moe_rows_scale_rows(0, 8) == 0 and bsq.moe_rows_scale_rows(1, 8) == 128 and bsq.moe_rows_scale_rows(16, 4) == 512
    assert bsq.moe_rows_scale_rows(32768, 256) >= 32768 // 256 // 128 * 128 * 256


def test_binding_rejects_host_and_mistyped_tensors(bsq):
    b16, u8, i32, f32 = (lambda *s, t=t: torch.zeros(s, dtype=t) for t in (torch.bfloat16, torch.uint8, torch.int32, torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        bsq.packed_linear(b16(1, 64), u8(100, 32), u8(512), "nvfp4", w_sf=f32(1))
    with pytest.raises(ValueError, match="CUDA"):
        bsq.qk_norm_rope(f32(1, 2, 64), f32(1, 1, 64), i32(1), f32(32))
    with pytest.raises(ValueError, match="CUDA"):
        bsq.moe_route(f32(1, 8), 2)
    with pytest.raises(ValueError, match="CUDA"):
        bsq.moe_rows(i32(1, 2), 8)


ROUTED = dict(fmt=2, x=P, ld_x=64, ids=P, weights=P, w13=P, w13_s=P, w2=P, w2_s=P, x_sf=None, w13_sf=None, h_sf=None, w2_sf=None, y=P, ld_y=64,
              tokens=2, hidden=64, inter=128, experts=4, top_k=2, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(fmt=3), VALUE), (dict(tokens=65), SHAPE), (dict(top_k=5), SHAPE), (dict(ld_x=56), SHAPE), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(x=None), NULL), (dict(fmt=0), NULL), (dict(ids=P + 2), ALIGN), (dict(weights=P + 1), ALIGN), (dict(ws=P + 16), ALIGN),
    (dict(ws_bytes=100), SHAPE), (dict(tokens=0), OK)])
def test_routed_moe_refusals(bsq, change, code):
    assert bsq.lib().bsq_moe_layer_routed(*{**ROUTED, **change}.values()) == code


BIG = 0x100000


@pytest.mark.parametrize("change,refused", [
    (dict(out=P), True), (dict(out=P + 64), True), (dict(out=P, tokens=1), True), (dict(out=P + 128, ld_out=128, ld_x=256), True),
    (dict(out=P + 128, ld_out=256, ld_x=256), False), (dict(out=P + 126, ld_out=256, ld_x=256), True),
    (dict(out=P + 312, ld_out=256, ld_x=256), False), (dict(out=P + 314, ld_out=256, ld_x=256), True), (dict(out=P - 200, ld_out=256, ld_x=256), False),
    (dict(out=P - 198, ld_out=256, ld_x=256), True), (dict(out=P + 192, tokens=2), True), (dict(out=P + 256, tokens=2), False),
    (dict(out=BIG, add=BIG, ld_add=100), False), (dict(out=BIG, add=BIG, ld_add=0), True), (dict(out=BIG, add=BIG, ld_add=108), True),
    (dict(out=BIG, add=BIG + 2, ld_add=100), True), (dict(out=BIG, add=BIG + 200, ld_add=100), True), (dict(out=BIG, add=BIG + 400, ld_add=0), False),
    (dict(out=BIG, add=BIG, ld_add=0, tokens=1), False)])
def test_linear_refuses_overlaps(bsq, change, refused):
    if not refused and torch.cuda.is_available():
        pytest.skip("would run")  # without a device such a call ends where that is looked for
    got = bsq.lib().bsq_packed_linear(*{**LINEAR, **change}.values())
    assert got == VALUE if refused else got not in (OK, NULL, SHAPE, ALIGN, VALUE)


@pytest.mark.parametrize("change,code", [
    (dict(qo=P, ko=3 * BIG, qo_tok=520), VALUE), (dict(qo=P, ko=3 * BIG, qo_head=72), VALUE), (dict(ko=BIG, ko_tok=136), VALUE), (dict(qo=BIG), VALUE),
    (dict(ko=P), VALUE), (dict(qo=2 * BIG, ko=2 * BIG), VALUE), (dict(qo_head=56), SHAPE), (dict(ko_tok=0), SHAPE), (dict(qo_tok=0), SHAPE)])
def test_rope_refuses_overlaps(bsq, change, code):
    assert bsq.lib().bsq_qk_norm_rope(*{**ROPE, "k": BIG, "qo": 2 * BIG, "ko": 3 * BIG, **change}.values()) == code
