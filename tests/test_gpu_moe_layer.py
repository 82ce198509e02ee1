"""moe_layer on the GPU against its 64-bit statement (serving_reference.moe,
which derives the tolerance: FP32 sums, codes that they can move, one BF16
rounding)."""
import numpy as np
import pytest

import oracle
import serving_reference as ref

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


class Layer:
    """Random weights quantized by the library, and what they stand for."""

    def __init__(self, bsq, fmt, hidden, inter, experts, seed):
        self.fmt, self.hidden, self.inter, self.experts = fmt, hidden, inter, experts
        rng = np.random.default_rng(seed)
        nv = fmt == "nvfp4"
        sf = lambda top: rng.uniform(0.5, 1.0, experts).astype(np.float32) * np.float32(2688 / top)  # noqa: E731
        self.x_sf, self.h_sf = (sf(6.0), sf(20.0)) if nv else (np.ones(experts, np.float32),) * 2
        self.w, packed, scales, sfs = [], [], [], []
        for rows, cols in ((2 * inter, hidden), (hidden, inter)):
            w = torch.from_numpy(rng.standard_normal((experts, rows, cols)) / np.sqrt(cols)).bfloat16().cuda()
            tsf = [float(bsq.tensor_sf(m)[1]) if nv else 1.0 for m in w]
            q = [bsq.quantize(m, fmt, t) for m, t in zip(w, tsf)]
            packed.append(torch.stack([a for a, _ in q]))
            scales.append(torch.stack([b for _, b in q]))
            sfs.append(np.asarray(tsf, np.float32))
            s = cols // oracle.block_size(fmt)
            self.w.append(np.stack([oracle.dequantize(fmt, a.cpu().numpy(), oracle.layout.scales_from_5d_view(b.cpu().numpy(), rows, s)[:rows, :s], t)
                                    for (a, b), t in zip(q, tsf)]))
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.args = (packed[0], scales[0], packed[1], scales[1])
        self.kw = dict(x_sf=dev(self.x_sf), w13_sf=dev(sfs[0]), h_sf=dev(self.h_sf), w2_sf=dev(sfs[1])) if nv else {}

    def inputs(self, tokens, seed):
        rng = np.random.default_rng(seed)
        x = torch.from_numpy(rng.standard_normal((tokens, self.hidden))).bfloat16()
        return x.cuda(), x.float().numpy(), rng.standard_normal((tokens, self.experts)).astype(np.float32)

    def check(self, bsq, tokens, top_k, renormalize=True, logits=None, seed=1, **kw):
        x, xn, z = self.inputs(tokens, seed)
        z = z if logits is None else logits
        y = bsq.moe_layer(x, torch.from_numpy(z).cuda(), *self.args, self.fmt, top_k, renormalize=renormalize, **self.kw, **kw)
        expect, tol = ref.moe(self.fmt, xn, z, *self.w, top_k, self.x_sf, self.h_sf, renormalize)
        err = np.abs(y.double().cpu().numpy() - expect)
        assert np.isfinite(err).all()
        assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
        return x, z, y


FORMATS = ["nvfp4", "mxfp4", "mxfp8"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden,inter,experts,top_k,tokens", [
    (32, 128, 1, 1, 1),       # less than a stage, one expert
    (96, 128, 3, 3, 2),       # every expert chosen
    (288, 256, 5, 2, 17),     # columns and rows that end inside a stage and a tile half
    (544, 128, 33, 4, 33),    # more than 32 experts, 16 and 32 tokens passed
    (160, 384, 2, 1, 64),     # all tokens on two experts
    (1056, 128, 40, 16, 5),   # the most choices
])
def test_sizes(bsq, fmt, hidden, inter, experts, top_k, tokens):
    layer = Layer(bsq, fmt, hidden, inter, experts, seed=hidden + tokens)
    layer.check(bsq, tokens, top_k)
    layer.check(bsq, tokens, top_k, renormalize=False)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_experts_and_one_workspace_for_all_sizes(bsq, fmt):
    big = Layer(bsq, fmt, 64, 128, 300, seed=1)
    small = Layer(bsq, fmt, 192, 128, 4, seed=2)
    ws = torch.zeros(max(bsq.moe_layer_workspace_bytes(fmt, 64, 64, 128, 300, 8), bsq.moe_layer_workspace_bytes(fmt, 3, 192, 128, 4, 2)),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        x, z, y = big.check(bsq, 64, 8, workspace=ws)
        small.check(bsq, 3, 2, workspace=ws)
    for _ in range(3):  # no sum's order depends on timing
        assert torch.equal(bsq.moe_layer(x, torch.from_numpy(z).cuda(), *big.args, fmt, 8, workspace=ws, **big.kw), y)


def test_ties_and_excluded_experts(bsq):
    layer = Layer(bsq, "mxfp8", 64, 128, 40, seed=3)
    z = np.zeros((6, 40), np.float32)
    z[0] = 1.0                                   # all equal: the lowest experts
    z[1, ::2] = -np.inf                          # half of them excluded
    z[2] = -np.inf                               # all but two, of three choices
    z[2, [7, 31]] = [0.5, 2.0]
    z[3] = -np.inf                               # nothing left: zeros
    z[4, 33:] = 5.0                              # ties past the first 32
    z[5] = np.where(np.arange(40) % 2, 0.0, -0.0)  # equal zeros of both signs
    for renormalize in (True, False):
        _, _, y = layer.check(bsq, 6, 3, renormalize, logits=z)
        assert not y[3].any()


def test_weights_of_an_excluded_expert_do_not_matter(bsq):
    layer = Layer(bsq, "mxfp8", 64, 128, 4, seed=8)
    x, _, z = layer.inputs(2, 4)
    z[:] = -np.inf
    z[0, :2] = [0.5, 1.0]
    z[1, 1] = 0.0
    zl = torch.from_numpy(z).cuda()
    expect = bsq.moe_layer(x, zl, *layer.args, "mxfp8", 4)
    bad = [t.clone() for t in layer.args]
    for t in bad:
        t[2:] = 0x7F                                 # NaN codes (weights), 2^0 (scales)
    assert torch.isfinite(expect).all() and torch.equal(bsq.moe_layer(x, zl, *bad, "mxfp8", 4), expect)


def test_nan_logits_are_reported(bsq):
    layer = Layer(bsq, "mxfp4", 64, 128, 8, seed=4)
    x, _, z = layer.inputs(3, 5)
    clean = z.copy()
    z[1, 2] = np.nan
    clean[1, 2] = -np.inf
    y = bsq.moe_layer(x, torch.from_numpy(z).cuda(), *layer.args, "mxfp4", 2)
    assert bsq.device_error() == 4
    assert torch.equal(y, bsq.moe_layer(x, torch.from_numpy(clean).cuda(), *layer.args, "mxfp4", 2))


def test_strides_streams_graphs(bsq):
    layer = Layer(bsq, "nvfp4", 128, 128, 12, seed=6)
    x, z, y = layer.check(bsq, 9, 4)
    zl = torch.from_numpy(z).cuda()
    wide_x, wide_z = torch.zeros((9, 192), dtype=torch.bfloat16, device="cuda"), torch.zeros((9, 16), device="cuda")
    wide_x[:, 64:], wide_z[:, 1:13] = x, zl
    out = torch.zeros((9, 256), dtype=torch.bfloat16, device="cuda")[:, 8:136]
    ws = torch.zeros(bsq.moe_layer_workspace_bytes("nvfp4", 9, 128, 128, 12, 4), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    bsq.moe_layer(wide_x[:, 64:], wide_z[:, 1:13], *layer.args, "nvfp4", 4, out=out, workspace=ws, stream=stream, **layer.kw)
    stream.synchronize()
    assert torch.equal(out, y)
    graph = torch.cuda.CUDAGraph()
    out2 = torch.empty_like(y)
    with torch.cuda.graph(graph):
        bsq.moe_layer(x, zl, *layer.args, "nvfp4", 4, out=out2, workspace=ws, **layer.kw)
    for _ in range(3):
        out2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, y)


def test_no_tokens_is_a_no_op(bsq):
    layer = Layer(bsq, "mxfp8", 64, 128, 4, seed=7)
    y = bsq.moe_layer(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 4), device="cuda"), *layer.args, "mxfp8", 2,
                      workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    assert y.shape == (0, 64)
