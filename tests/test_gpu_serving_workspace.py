"""The serving calls' workspaces: parts and counters that blocks share."""
import pytest

from test_gpu_kv_cache import Case

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
