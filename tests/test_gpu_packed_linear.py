"""packed_linear on the GPU against its 64-bit statement (layer_reference.linear
derives the tolerance), and bit for bit where every sum is a whole number."""
import numpy as np
import pytest

import layer_reference as ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FORMATS = ["nvfp4", "mxfp4", "mxfp8"]


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


class Weights:
    """Random weights quantized by the library, and what they stand for."""

    def __init__(self, bsq, fmt, rows, cols, seed, spread=0.0):
        rng = np.random.default_rng(seed)
        w = rng.standard_normal((rows, cols)) / np.sqrt(cols) * np.exp2(np.round(spread * rng.standard_normal((rows, cols // 32, 1)))
                                                                       ).repeat(32, 2).reshape(rows, cols)
        w = torch.from_numpy(w).bfloat16().cuda()
        self.fmt, self.rows, self.cols = fmt, rows, cols
        self.sf = bsq.tensor_sf(w)[1:] if fmt == "nvfp4" else None
        self.packed, self.scales = bsq.quantize_dynamic(w, fmt, self.sf)
        self.values = ref.weights(fmt, self.packed.cpu().numpy(), self.scales.cpu().numpy(), rows, cols,
                                  1.0 if self.sf is None else float(self.sf))

    def call(self, bsq, x, **kw):
        return bsq.packed_linear(x, self.packed, self.scales, self.fmt, w_sf=self.sf, **kw)

    def check(self, bsq, x, add=None, out="x", **kw):
        name = {torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype] if out == "x" else out
        y = self.call(bsq, x, add=add, out_dtype=DT[name], **kw)
        expect, tol = ref.linear(x.double().cpu().numpy(), self.values, None if add is None else add.double().cpu().numpy(), name)
        err = np.abs(y.double().cpu().numpy() - expect)
        assert y.dtype == DT[name] and np.isfinite(err).all()
        assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
        return y


def inputs(tokens, cols, dtype, seed=1):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((tokens, cols))).to(DT[dtype]).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 32),          # less than a piece, one row
    (1, 129, 96),        # a row past a band, columns that end inside a piece
    (3, 100, 1056),      # columns that end inside a scale atom
    (8, 257, 4128),      # a full tile of tokens, several blocks along K
    (9, 33, 160),        # a token past a tile
    (16, 640, 2080),
    (17, 70, 544),
    (33, 130, 320),      # tokens past the tiles of the kernel for few
    (64, 384, 1184),
    (65, 96, 2048),
    (200, 300, 288),
    (300, 129, 64),
])
def test_sizes(bsq, fmt, dtype, tokens, rows, cols):
    w = Weights(bsq, fmt, rows, cols, seed=rows + cols)
    x = inputs(tokens, cols, dtype)
    w.check(bsq, x)
    w.check(bsq, x, out="f32")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 300, 7168), (7, 96, 4096), (30, 200, 2048), (64, 300, 4096), (150, 520, 1024)])
def test_whole_numbers_are_exact(bsq, fmt, dtype, tokens, rows, cols):
    """Codes under scales 1 or 2, whole values of x: every sum is a multiple of 1/2 below 2^23, so FP32 holds it in any order."""
    rng = np.random.default_rng(tokens + cols)
    if fmt == "mxfp8":
        codes = np.arange(256, dtype=np.uint8)
        vals = oracle.formats.e4m3_decode(codes)
        codes = codes[(np.abs(vals) <= 8) & (vals * 2 == np.round(vals * 2))]
        packed = rng.choice(codes, (rows, cols))
        per = 32
    else:
        packed = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
        per = 16 if fmt == "nvfp4" else 32
    tiles = -(-rows // 128) * -(-(cols // per) // 4) * 512
    scales = rng.choice(np.array([0x38, 0x40] if fmt == "nvfp4" else [127, 128], np.uint8), tiles)
    x = torch.from_numpy(rng.integers(-4, 5, (tokens, cols))).to(DT[dtype]).cuda()
    sf = torch.tensor([0.5], device="cuda") if fmt == "nvfp4" else None
    w = ref.weights(fmt, packed, scales, rows, cols, 0.5 if fmt == "nvfp4" else 1.0)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y = bsq.packed_linear(x, dev(packed), dev(scales), fmt, w_sf=sf, out_dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), x.double().cpu().numpy() @ w.T)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 12, 40, 130])
def test_add_residual_bias_and_in_place(bsq, fmt, tokens):
    rows, cols = 200, 352
    w = Weights(bsq, fmt, rows, cols, seed=3)
    x = inputs(tokens, cols, "bf16")
    residual, bias = inputs(tokens, rows, "bf16", 5), inputs(1, rows, "f16", 6)[0]
    y = w.check(bsq, x, add=residual)
    w.check(bsq, x.half(), add=bias)
    w.check(bsq, x, add=inputs(tokens, rows, "f32", 7), out="f32")
    w.check(bsq, x, add=inputs(1, rows, "f32", 7)[0], out="f32")
    inplace = residual.clone()
    assert w.call(bsq, x, add=inplace, out=inplace) is inplace
    assert torch.equal(inplace, y)


@pytest.mark.parametrize("tokens", [2, 20, 100])
def test_strides(bsq, tokens):
    rows, cols = 150, 224
    w = Weights(bsq, "nvfp4", rows, cols, seed=4)
    wide = inputs(tokens, 3 * cols, "bf16", 8)
    x = wide[:, cols:2 * cols]
    frame = torch.full((tokens, rows + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    out = frame[:, 3:3 + rows]
    res = inputs(tokens, rows + 1, "bf16", 9)[:, 1:]
    w.call(bsq, x, add=res, out=out)
    assert torch.equal(out, w.check(bsq, x.contiguous(), add=res.contiguous()))
    assert (frame[:, :3] == 7).all() and (frame[:, 3 + rows:] == 7).all()   # what lies beside the rows stays


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_wide_ranges(bsq, fmt, tokens):
    """Scales that differ by many powers of two within a row, tokens of very different sizes, tiny and huge ones."""
    w = Weights(bsq, fmt, 140, 1024, seed=5, spread=8.0 if fmt != "nvfp4" else 1.0)
    x = inputs(tokens, 1024, "bf16").float()
    x = x * torch.exp2(torch.linspace(-90, 60, tokens, device="cuda").round())[:, None]
    x[:, ::7] *= 2.0 ** -20
    w.check(bsq, x.bfloat16(), out="f32")
    h = inputs(tokens, 1024, "f16", 2)
    h[:, ::5] *= 2.0 ** -14   # subnormal numbers of FP16 are exact
    w.check(bsq, h, out="f32")


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_blocks_along_k_of_very_different_tokens(bsq, tokens):
    """The power of two that a token is held times follows its largest value, wherever along K that lies."""
    w = Weights(bsq, "mxfp8", 64, 8192, seed=6)
    x = inputs(tokens, 8192, "bf16").float()
    for i, f in enumerate((2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** -100)):
        x[i % tokens, 2048 * i:2048 * (i + 1)] *= f
    x[-1, 100:8000] = 0
    w.check(bsq, x.bfloat16(), out="f32")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [3, 40])
def test_nan_and_inf_stay_with_their_token(bsq, fmt, tokens):
    w = Weights(bsq, fmt, 130, 256, seed=7)
    for dtype in ("bf16", "f16"):
        x = inputs(tokens, 256, dtype)
        clean = w.call(bsq, x)
        x[1, 7], x[2, 200] = float("nan"), float("inf")
        y = w.call(bsq, x)
        assert torch.equal(y[0], clean[0]) and torch.equal(y[3:], clean[3:])
        assert y[1].isnan().all() and not torch.isfinite(y[2]).any()


def test_scale_extremes(bsq):
    """E8M0 bytes 0 (a block of zeros, and 2^-127) and 246; E4M3 scales from the least subnormal to 448."""
    rows, cols = 128, 128
    x = torch.ones((1, cols), dtype=torch.bfloat16, device="cuda")
    packed = torch.full((rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda")   # every code 1.0
    for byte, value in ((0, 2.0 ** -127), (1, 2.0 ** -126), (127, 1.0), (246, 2.0 ** 119)):
        scales = torch.full((512,), byte, dtype=torch.uint8, device="cuda")
        for tokens in (1, 33):
            y = bsq.packed_linear(x.expand(tokens, cols).contiguous(), packed, scales, "mxfp4", out_dtype=torch.float32)
            assert (y.double() == 128 * value).all(), byte
    one = torch.ones(1, device="cuda")
    for byte, value in ((1, 2.0 ** -9), (0x38, 1.0), (0x7E, 448.0)):
        scales = torch.full((1024,), byte, dtype=torch.uint8, device="cuda")
        for tokens in (1, 33):
            y = bsq.packed_linear(x.expand(tokens, cols).contiguous(), packed, scales, "nvfp4", w_sf=one, out_dtype=torch.float32)
            assert (y.double() == 128 * value).all(), byte


def test_no_tokens_and_no_rows(bsq):
    w = Weights(bsq, "mxfp4", 64, 64, seed=8)
    assert w.call(bsq, inputs(0, 64, "bf16")).shape == (0, 64)
    empty = bsq.packed_linear(inputs(2, 64, "bf16"), w.packed[:0], w.scales[:0], "mxfp4")
    assert empty.shape == (2, 0)


@pytest.mark.parametrize("tokens", [1, 16, 64, 300])
def test_graph_streams_and_repeats(bsq, tokens):
    """Captured, replayed on new inputs, on another stream, twice at once: the same bits each time."""
    w = Weights(bsq, "nvfp4", 500, 1536, seed=9)
    x, out = inputs(tokens, 1536, "bf16"), torch.empty((tokens, 500), dtype=torch.bfloat16, device="cuda")
    w.call(bsq, x, out=out)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        w.call(bsq, x, out=out)
    for seed in (11, 12):
        x.copy_(inputs(tokens, 1536, "bf16", seed))
        expect = w.check(bsq, x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = [w.call(bsq, x, stream=s) for s in (stream, other) * 4]
    torch.cuda.synchronize()
    assert all(torch.equal(y, expect) for y in ys)


@pytest.mark.parametrize("fmt,dtype", [("nvfp4", "bf16"), ("mxfp4", "f16"), ("mxfp8", "bf16"), ("mxfp8", "f16")])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 10000, 1024),    # more blocks than SMs, none along K
    (2, 5000, 4096),     # four sets of rows per block, eight blocks along K, more of them than fit at once
    (5, 20000, 256),
    (16, 100, 16384),    # tokens in more than one segment, one set of rows per block
    (16, 1000, 16384),   # the same with four
    (17, 9750, 1024),    # two tiles of rows per block, three blocks along K, the last tile behind the last row
    (100, 19580, 512),   # two tiles, one block along K
    (33, 60000, 96),     # the same, several tiles one after the other
    (300, 20000, 96),    # one tile of rows, several one after the other
    (250, 129, 8192),    # eight blocks along K and the largest tile of tokens, one tile of rows
    (112, 7000, 16384),  # five, and two
])
def test_splits(bsq, fmt, dtype, tokens, rows, cols):
    """The ways in which rows, K and tokens are shared out, with a residual; the rows at both ends and some between are checked."""
    w = Weights(bsq, fmt, 1, 32, seed=0)  # for its call
    rng = np.random.default_rng(rows)
    full = torch.from_numpy(rng.standard_normal((rows, cols), np.float32) / np.float32(np.sqrt(cols))).bfloat16().cuda()
    w.sf = bsq.tensor_sf(full)[1:] if fmt == "nvfp4" else None
    w.packed, w.scales = bsq.quantize_dynamic(full, fmt, w.sf)
    bands = sorted({0, 128 * int(rng.integers(0, -(-rows // 128))), (rows - 1) // 256 * 256, (rows - 1) // 128 * 128})
    x = inputs(tokens, cols, dtype)
    add = torch.from_numpy(rng.standard_normal((tokens, rows), np.float32)).to(DT[dtype]).cuda()
    y = w.call(bsq, x, add=add).double().cpu().numpy()
    atom_row = w.scales.numel() // -(-rows // 128)  # bytes of a band's scales
    for r0 in bands:
        r1 = min(r0 + 128, rows)
        values = ref.weights(fmt, w.packed[r0:r1].cpu().numpy(), w.scales.reshape(-1)[r0 // 128 * atom_row:][:atom_row].cpu().numpy(), r1 - r0, cols,
                             1.0 if w.sf is None else float(w.sf))
        expect, tol = ref.linear(x.double().cpu().numpy(), values, add[:, r0:r1].double().cpu().numpy(), dtype)
        err = np.abs(y[:, r0:r1] - expect)
        assert (err <= tol).all(), f"rows from {r0}: {(err / tol).max():.3f} of the tolerance"
