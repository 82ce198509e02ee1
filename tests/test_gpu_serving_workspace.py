"""The serving calls' workspaces: parts and counters that blocks share."""
import pytest

from test_gpu_kv_cache import Case
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


# 4, 16, 32 and 160 rows of a kv head
@pytest.mark.parametrize("group,new", [(4, 1), (8, 2), (8, 4), (4, 40)])
@pytest.mark.parametrize("lens", [[30011], [4000, 777, 9000]])
def test_parts_meet_in_any_order(bsq, group, new, lens):
    """Items joined by whichever block comes last, beside work on other streams that delays some of the blocks: the
    same bits each time, and the counters are down again."""
    case = Case(lens, [new] * len(lens), 2, 128, 64, seed=new)
    q, _ = case.rows(2 * group)
    args = case.device()
    ws = torch.zeros(bsq.kv_attention_workspace_bytes(q.shape[0], 2 * group, 2, 128, len(lens), new), dtype=torch.uint8, device="cuda")
    expect, lse = bsq.kv_attention(q, *args, new, return_lse=True, workspace=ws)
    other = torch.cuda.Stream()
    rows = torch.randn((8192, 4096), device="cuda").bfloat16()
    torch.cuda.synchronize()
    for k in range(30):
        with torch.cuda.stream(other):
            for _ in range(k % 4):
                bsq.quantize(rows, "mxfp8")
        got, got_lse = bsq.kv_attention(q, *args, new, return_lse=True, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, expect) and torch.equal(got_lse, lse)
        assert not ws[:4096].any()


@pytest.mark.parametrize("group,new", [(4, 1), (8, 4), (4, 40)])
def test_spoiled_attention_workspace_is_reported(bsq, group, new):
    """Counters that do not hold (as after a wait that gave up): nothing is written, each call says so, zeros mend it."""
    case = Case([3000, 100], [new, new], 1, 64, 16, seed=new)
    q, _ = case.rows(group)
    args = case.device()
    ws = torch.zeros(bsq.kv_attention_workspace_bytes(q.shape[0], group, 1, 64, 2, new), dtype=torch.uint8, device="cuda")
    expect = bsq.kv_attention(q, *args, new, workspace=ws)
    ws.fill_(255)
    out = torch.full_like(expect, 7.0)
    for _ in range(2):
        bsq.kv_attention(q, *args, new, out=out, workspace=ws)
        assert bsq.device_error() == 6 and (out == 7.0).all()
    ws.zero_()
    assert torch.equal(bsq.kv_attention(q, *args, new, workspace=ws), expect) and bsq.device_error() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_spoiled_expert_workspace_is_reported(bsq, fmt):
    layer = Layer(bsq, fmt, 128, 128, 6, seed=1)
    x, _, z = layer.inputs(5, 2)
    zl = torch.from_numpy(z).cuda()
    ws = torch.zeros(bsq.moe_layer_workspace_bytes(fmt, 5, 128, 128, 6, 2), dtype=torch.uint8, device="cuda")
    expect = bsq.moe_layer(x, zl, *layer.args, fmt, 2, workspace=ws, **layer.kw)
    ws.fill_(255)
    out = torch.full_like(expect, 7.0)
    for _ in range(2):
        bsq.moe_layer(x, zl, *layer.args, fmt, 2, out=out, workspace=ws, **layer.kw)
        assert bsq.device_error() == 6 and (out == 7.0).all()
    ws.zero_()
    assert torch.equal(bsq.moe_layer(x, zl, *layer.args, fmt, 2, workspace=ws, **layer.kw), expect) and bsq.device_error() == 0


@pytest.mark.parametrize("group,new", [(4, 1), (8, 4), (4, 40)])
def test_only_attention_counters_have_to_be_zero(bsq, group, new):
    """A workspace of anything but for its counters, passed in or (from memory of that kind) the call's own."""
    case = Case([5000, 100], [new, new], 1, 64, 16, seed=new)
    q, _ = case.rows(group)
    args = case.device()
    nbytes, counters = bsq.kv_attention_workspace_bytes(q.shape[0], group, 1, 64, 2, new), bsq.lib().bsq_kv_attention_counter_bytes()
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    expect = bsq.kv_attention(q, *args, new, workspace=ws)
    ws.fill_(255)[:counters].zero_()
    assert torch.equal(bsq.kv_attention(q, *args, new, workspace=ws), expect)
    assert not ws[:counters].any()
    ws.fill_(255)
    del ws
    assert torch.equal(bsq.kv_attention(q, *args, new), expect) and bsq.device_error() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_only_expert_counters_have_to_be_zero(bsq, fmt):
    layer = Layer(bsq, fmt, 288, 256, 6, seed=1)
    x, _, z = layer.inputs(5, 2)
    zl = torch.from_numpy(z).cuda()
    nbytes, counters = bsq.moe_layer_workspace_bytes(fmt, 5, 288, 256, 6, 2), bsq.lib().bsq_moe_layer_counter_bytes()
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    expect = bsq.moe_layer(x, zl, *layer.args, fmt, 2, workspace=ws, **layer.kw)
    ws.fill_(255)[:counters].zero_()
    assert torch.equal(bsq.moe_layer(x, zl, *layer.args, fmt, 2, workspace=ws, **layer.kw), expect)
    assert not ws[:counters].any()
    ws.fill_(255)
    del ws
    assert torch.equal(bsq.moe_layer(x, zl, *layer.args, fmt, 2, **layer.kw), expect) and bsq.device_error() == 0


def test_waits_end_and_the_context_stays_usable(bsq):
    """The kernels' waits on barriers and counters that nothing completes give up at their limit."""
    assert bsq.lib().bsq_selftest_serving_waits(torch.cuda.current_stream().cuda_stream) == 0
    assert bsq.device_error() == 6 and bsq.device_error() == 0
    case = Case([100], [1], 1, 64, 16, seed=1)
    q, _ = case.rows(2)
    assert torch.isfinite(bsq.kv_attention(q, *case.device(), 1)).all() and bsq.device_error() == 0
