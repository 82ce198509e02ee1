"""packed_linear at the ends of the scales' range, in every kernel: bit for bit
where sums are whole multiples of one number, else against the 64-bit
statement."""
import numpy as np
import pytest

import layer_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(128, 128), (300, 1056), (100, 8192)])  # the last with several blocks along K
def test_rows_of_very_small_scales(bsq, fmt, dtype, rows, cols):
    """Codes 1.0, tokens 1.0, one E8M0 byte: every sum is cols 2^(byte - 127), from the least byte on."""
    packed = torch.full((rows, cols if fmt == "mxfp8" else cols // 2), 0x38 if fmt == "mxfp8" else 0x22, dtype=torch.uint8, device="cuda")
    tiles = -(-rows // 128) * -(-cols // 128)
    for tokens in (1, 16, 17, 33, 130):
        x = torch.ones((tokens, cols), dtype=DT[dtype], device="cuda")
        for byte in (0, 1, 6, 7, 8, 12, 13, 14, 40):
            scales = torch.full((512 * tiles,), byte, dtype=torch.uint8, device="cuda")
            y = bsq.packed_linear(x, packed, scales, fmt, out_dtype=torch.float32)
            assert (y.double() == cols * 2.0 ** (byte - 127)).all(), (tokens, byte, y[0, 0].item())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("tokens,rows,cols", [(17, 200, 4096), (33, 130, 224), (300, 129, 512)])
def test_rows_of_small_and_ordinary_scales(bsq, fmt, tokens, rows, cols):
    """FP16 tokens, random codes, each row's scales between byte 0 and one of its own.  Beyond what layer_reference.linear allows, values
    are off by at most 2^-35 (E2M1) or 2^-23 (E4M3) of their row's largest scale, and up to eight blocks' sums along K are rounded where FP32
    has subnormal numbers."""
    rng = np.random.default_rng(rows)
    if fmt == "mxfp8":
        packed = rng.integers(0, 127, (rows, cols), dtype=np.uint8) | rng.integers(0, 2, (rows, cols), dtype=np.uint8) << 7
    else:
        packed = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    blocks = cols // 32
    top = rng.integers(0, 24, rows)
    top[:24] = np.arange(24)
    by_row = rng.integers(0, top[:, None] + 1, (rows, blocks))
    scales = np.zeros(-(-rows // 128) * -(-blocks // 4) * 512, np.uint8)
    r, c = np.arange(rows)[:, None], np.arange(blocks)[None]
    scales[((r // 128) * -(-blocks // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = by_row
    w = ref.weights(fmt, packed, scales, rows, cols)
    x = torch.from_numpy(rng.standard_normal((tokens, cols))).half().cuda()
    y = bsq.packed_linear(x, torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), fmt, out_dtype=torch.float32).double().cpu().numpy()
    xn = x.double().cpu().numpy()
    expect, tol = ref.linear(xn, w, None, "f32")
    largest = 2.0 ** (by_row.max(1) - 127.0)
    tol = tol + np.abs(xn).sum(1)[:, None] * largest[None] * 2.0 ** (-35 if fmt == "mxfp4" else -23) + 8 * 2.0 ** -149
    err = np.abs(y - expect)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows", [(1, 1), (16, 129), (17, 1), (17, 128), (33, 129), (300, 2), (257, 257)])
def test_one_block_of_columns(bsq, fmt, dtype, tokens, rows):
    """32 columns, less than any kernel's step: whole numbers, so the sums are exact."""
    rng = np.random.default_rng(tokens + rows)
    packed = rng.choice(np.array([0x00, 0x30, 0x38, 0x40, 0xB8, 0xC4], np.uint8), (rows, 32)) if fmt == "mxfp8" else rng.integers(0, 256, (rows, 16), dtype=np.uint8)
    scales = np.zeros(-(-rows // 128) * 512, np.uint8)  # what lies past the last row and column
    r = np.arange(rows)
    for c in range(2 if fmt == "nvfp4" else 1):
        scales[r // 128 * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c] = rng.choice([0x38, 0x40] if fmt == "nvfp4" else [127, 128], rows)
    x = torch.from_numpy(rng.integers(-4, 5, (tokens, 32))).to(DT[dtype]).cuda()
    sf = torch.tensor([0.5], device="cuda") if fmt == "nvfp4" else None
    w = ref.weights(fmt, packed, scales, rows, 32, 0.5 if fmt == "nvfp4" else 1.0)
    y = bsq.packed_linear(x, torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), fmt, w_sf=sf, out_dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), x.double().cpu().numpy() @ w.T)
