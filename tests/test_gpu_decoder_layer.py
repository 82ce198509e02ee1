"""The decoder-layer example: it runs with each format, its outputs do not
depend on how the prompt was cut, beyond what quantization leaves open, and
repeat bit for bit."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")


@pytest.fixture(scope="module")
def example():
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_serves(example, fmt):
    outs, cache = example.serve(fmt, batch=3, prompt=150, steps=4)
    again, _ = example.serve(fmt, batch=3, prompt=150, steps=4)
    assert example.bsq.device_error() == 0
    assert torch.isfinite(outs).all() and torch.equal(outs, again)
    assert cache.lens.tolist() == [154] * 3


def test_chunks_agree(example):
    """The prompt in one piece and in pieces: the same keys and values up to the
    page scales' growth, so the first output agrees closely."""
    whole, a = example.serve("mxfp8", batch=2, prompt=192, steps=1, chunk=192)
    parts, b = example.serve("mxfp8", batch=2, prompt=192, steps=1, chunk=50)
    x, y = whole[0].float(), parts[0].float()
    assert (x - y).norm() <= 0.1 * x.norm()
    assert torch.equal(a.k_scales[:, :], b.k_scales) and torch.equal(a.v_scales, b.v_scales)


def test_main(example, capsys):
    example.main(["--batch", "1", "--prompt", "20", "--steps", "2"])
    assert "cache lengths [22]" in capsys.readouterr().out
