"""kv_append and kv_attention at the ends of what include/bsq.h allows: scale
bytes 1 to 254, query rows of any finite size, softmax weights far below a
row's largest, NaN queries."""
import pytest

from test_gpu_kv_cache import Case, check_append

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


def test_append_under_the_largest_scale(bsq):
    """New tokens in a page whose earlier tokens brought it to byte 254."""
    case = Case([20, 40, 7], [3, 1, 7], 2, 64, 32, seed=5)
    for s in case.scales:
        s[:] = 254
    check_append(bsq, case, 2.0 ** 126, 2.0 ** 125)
