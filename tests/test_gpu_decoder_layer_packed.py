"""The decoder layer over packed projections: the calls as they are used
together.  It runs with each format and repeats bit for bit, eagerly and
captured; its attention half and its routing agree with their formulas."""
import importlib.util
import os

import numpy as np
import pytest

import layer_reference as ref
import oracle

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
    outs, cache = example.serve(fmt, batch=3, prompt=150, steps=4, packed=True)
    again, _ = example.serve(fmt, batch=3, prompt=150, steps=4, packed=True)
    assert example.bsq.device_error() == 0
    assert torch.isfinite(outs).all() and torch.equal(outs, again)
    assert cache.lens.tolist() == [154] * 3


def test_main(example, capsys):
    example.main(["--batch", "1", "--prompt", "20", "--steps", "2", "--packed"])
    assert "cache lengths [22]" in capsys.readouterr().out


def test_captured_step_equals_eager(example):
    layer = example.PackedLayer("nvfp4", seed=3)
    caches = [example.Cache(5, 80, layer.kv_heads, layer.dim) for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(4)
    prompt = torch.randn((5 * 30, layer.hidden), generator=g, device="cuda").bfloat16()
    one = torch.arange(6, dtype=torch.int32, device="cuda")
    for c in caches:
        c.lens += 30
        layer(prompt, c, 30 * one, 30)
    x = torch.randn((5, layer.hidden), generator=g, device="cuda").bfloat16()

    def step(c):
        c.lens += 1
        return layer(x, c, one, 1)

    step(caches[1])                        # set-up before the capture, undone
    caches[1].lens -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[1])
    for i in range(3):
        x.copy_(torch.randn((5, layer.hidden), generator=g, device="cuda").bfloat16())
        expect = step(caches[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect) and caches[0].lens.tolist() == caches[1].lens.tolist()
    assert example.bsq.device_error() == 0


def _values(projection, rows, cols):
    packed, scales, fmt, sf = projection
    return ref.weights(fmt, packed.cpu().numpy(), scales.cpu().numpy(), rows, cols, 1.0 if sf is None else float(sf))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_attention_half_agrees_with_its_formula(example, fmt):
    """In 64 bits from the layer's input, over the keys and values that its cache holds.  BF16 roundings of qkv, of the rotated
    queries, of attention's output and of the sum, 2^-9 each; the queries' 2^-8 moves scores of a size up to about 8 by 2^-5
    at most, and the weights by as much, so by far the largest part is that: 0.05 of the attention's share."""
    layer = example.PackedLayer(fmt, seed=5)
    cache = example.Cache(2, 70, layer.kv_heads, layer.dim)
    g = torch.Generator(device="cuda").manual_seed(6)
    one = torch.arange(3, dtype=torch.int32, device="cuda")
    cache.lens += 60
    layer(torch.randn((120, layer.hidden), generator=g, device="cuda").bfloat16(), cache, 60 * one, 60)
    x = torch.randn((2, layer.hidden), generator=g, device="cuda").bfloat16()
    cache.lens += 1
    y = layer.attend(x, cache, one, 1).double().cpu().numpy()
    xn = x.double().cpu().numpy()
    h = xn / np.sqrt((xn ** 2).mean(1, keepdims=True) + 2.0 ** -52)
    heads, kv, dim = layer.heads, layer.kv_heads, layer.dim
    qkv = (h @ _values(layer.projections["w_qkv"], (heads + 2 * kv) * dim, layer.hidden).T).reshape(2, -1, dim)
    q, _ = ref.rope(qkv[:, :heads], layer.q_weight.double().cpu().numpy(), np.array([60, 60]), layer.inv_freq.cpu().numpy(), 1e-6, False, "bf16")
    k, _ = ref.rope(qkv[:, heads:heads + kv], layer.k_weight.double().cpu().numpy(), np.array([60, 60]), layer.inv_freq.cpu().numpy(), 1e-6, False, "bf16")
    ids = cache.table.cpu().numpy()
    kc, vc = (np.stack([np.concatenate([oracle.formats.e4m3_decode(c[p]) * 2.0 ** (s[p].astype(int) - 127)[:, None, None] for p in row], 1)[:, :61]
                        for row in ids]) for c, s in ((cache.k.cpu().numpy(), cache.k_scales.cpu().numpy()), (cache.v.cpu().numpy(), cache.v_scales.cpu().numpy())))
    # the cache's last key is this step's, rotated: E4M3 rounds by 2^-4 at most, BF16 before that by 2^-8
    assert np.abs(kc[:, :, 60] - k).max() <= (2.0 ** -4 + 2.0 ** -6) * np.abs(k).max()
    s = np.einsum("bhgd,bhtd->bhgt", q.reshape(2, kv, heads // kv, dim), kc) / np.sqrt(dim)
    p = np.exp(s - s.max(3, keepdims=True))
    o = np.einsum("bhgt,bhtd->bhgd", p / p.sum(3, keepdims=True), vc).reshape(2, -1)
    share = o @ _values(layer.projections["w_out"], layer.hidden, heads * dim).T
    assert np.linalg.norm(y - xn - share) <= 0.05 * np.linalg.norm(share) + 2.0 ** -8 * np.linalg.norm(xn + share)


def test_routing_agrees_with_its_formula(example):
    layer = example.PackedLayer("nvfp4", seed=7)
    y = torch.randn((33, layer.hidden), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    logits = example.bsq.packed_linear(y, *layer.projections["w_router"], out_dtype=torch.float32)
    expect, tol = ref.linear(y.double().cpu().numpy(), _values(layer.projections["w_router"], 16, layer.hidden), None, "f32")
    assert (np.abs(logits.double().cpu().numpy() - expect) <= tol).all()
    ids, weights = layer.route(y)
    eids, ew = ref.route(logits.double().cpu().numpy(), layer.top_k, True, layer.bias.double().cpu().numpy(), 4, 2, 2, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), eids)
    assert np.abs(weights.cpu().numpy() - ew).max() <= 2.0 ** -18
