"""kv_append and kv_attention at the ends of what include/bsq.h allows: scale
bytes 1 to 254, query rows of any finite size, softmax weights far below a
row's largest, NaN queries."""
import numpy as np
import pytest

import serving_reference as ref
from test_gpu_kv_cache import HALF_ULP, SUBNORMAL, Case, check_append

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# query heads per kv head, rows: 4, 16, 32 and 160 rows of a kv head, each in a kernel of its own
ROWS = [(4, 1), (8, 2), (8, 4), (4, 40)]


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


def small_codes(case, top=1.0):
    """Codes of magnitudes up to `top`, so that values under the largest scale stay finite."""
    mags = np.arange(0x7F, dtype=np.uint8)
    mags = mags[ref.e4m3_decode(mags) <= top]
    for c in case.cache:
        c[:] = case.rng.choice(mags, c.shape) | (case.rng.integers(0, 2, c.shape).astype(np.uint8) << 7)


def close(case, got, got_lse, out, lse, mag, size, low, weight=2.0 ** -25):
    """As test_gpu_kv_cache.compare, without a floor for the smallest outputs.
    A score and the value scale's exponent meet in one FP32 number, and references of both are subtracted
    from such numbers: four roundings of up to 2^-24 of the exponent each.  `weight`: error of the smallest weights, of the largest."""
    ev = max(abs(int(b) - 127) for b in case.scales[1].ravel())
    score = (case.dim + 4) * 2.0 ** -24 * size + 2.0 ** -22 * ev
    tol = HALF_ULP[case.dtype] * np.abs(out) + (2.0 ** -11 + 2 * score + 2.0 ** -19)[..., None] * mag + weight * low + SUBNORMAL[case.dtype]
    err = np.abs(got.double().cpu().numpy() - out)
    assert np.isfinite(err).all()
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
    g = got_lse.double().cpu().numpy()
    some = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(g), ~some)
    assert (np.abs(g[some] - lse[some]) <= 2 * score[some] + 2.0 ** -20 * (1 + np.abs(lse[some]))).all()


def attend(bsq, case, heads, q_scale=1.0, **kw):
    q, qn = case.rows(heads, q_scale)
    got = bsq.kv_attention(q, *case.device(), int(np.max(np.diff(case.offsets))), return_lse=True)
    close(case, *got, *ref.attention(qn, *case.cache, *case.scales, case.table, case.offsets, case.lens, case.dim ** -0.5, True, 0), **kw)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
@pytest.mark.parametrize("value_bytes", [(1,), (254,), (1, 254), (1, 127, 254), (95, 247), (20, 100, 127), (87, 167), (86, 127, 168)])
def test_value_scales_from_end_to_end(bsq, group, new, q_scale, value_bytes):
    """The lse does not depend on the values' scales, and the output is their weighted mean, however far apart they are."""
    case = Case([777, 130, new], [new] * 3, 2, 128, 16, seed=len(value_bytes) + new)
    small_codes(case)
    case.scales = [case.rng.integers(124, 130, case.scales[0].shape).astype(np.uint8),
                   case.rng.choice(np.array(value_bytes, np.uint8), case.scales[1].shape)]
    attend(bsq, case, 2 * group, q_scale)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("byte", [1, 12])
def test_small_value_scales_over_many_tokens(bsq, group, new, byte):
    case = Case([40000], [new], 1, 64, 64, seed=byte)
    small_codes(case)
    case.scales[1][:] = byte
    attend(bsq, case, group, 0.1)


def test_append_under_the_largest_scale(bsq):
    """New tokens in a page whose earlier tokens brought it to byte 254."""
    case = Case([20, 40, 7], [3, 1, 7], 2, 64, 32, seed=5)
    for s in case.scales:
        s[:] = 254
    check_append(bsq, case, 2.0 ** 126, 2.0 ** 125)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("q_exp,key_byte", [(-113, 233), (-116, 236), (-122, 242), (-129, 249)])
def test_smallest_query_rows(bsq, group, new, q_exp, key_byte):
    """Rows below 2^-114, down to subnormal numbers, against keys large enough for scores of about 1."""
    case = Case([300, 77], [new, new], 2, 128, 16, seed=new)
    case.scales[0][:] = key_byte
    attend(bsq, case, 2 * group, 2.0 ** q_exp)


@pytest.mark.parametrize("group,new", ROWS)
def test_zero_keys_under_any_scale(bsq, group, new):
    """Scores of 0, where the factors of the row and of the page together pass FP32."""
    case = Case([300, 77], [new, new], 2, 64, 16, seed=new)
    case.cache[0][:] = case.rng.choice(np.array([0x00, 0x80], np.uint8), case.cache[0].shape)
    case.scales[0][:] = 254
    attend(bsq, case, 2 * group, 2.0 ** 100)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,new", ROWS)
def test_one_heavy_key_and_a_flat_tail(bsq, group, new, dtype):
    """A first key 26 ln 2 above all others, with values of 0: what is left comes from 4000 weights of 2^-26, of
    which no more than 2^-32 of the first key's weight may be lost each.  Enough heads that a block meets many keys of one."""
    heads = 152
    case = Case([4000], [new], heads, 64, 64, seed=new, dtype=dtype)
    case.cache[0][:] = 0
    case.cache[0][case.table[0, 0], :, 0] = 0x38         # the first key: ones, all others zeros
    case.cache[1][:] = 0x38
    case.cache[1][case.table[0, 0], :, 0] = 0
    for s in case.scales:
        s[:] = 127
    q = torch.full((new, heads * group, 64), 26 * np.log(2) / 8).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    got = bsq.kv_attention(q.cuda(), *case.device(), new, return_lse=True)
    expect = ref.attention(q.double().numpy(), *case.cache, *case.scales, case.table, case.offsets, case.lens, 1 / 8, True, 0)
    close(case, *got, *expect, weight=2.0 ** -32)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("length", [90, 5000])
def test_nan_query_rows_stay_nan(bsq, group, new, length):
    """The output and the lse of such a row are NaN (an lse of -inf marks a row without keys); other rows do not change."""
    case = Case([length, 40], [new, new], 1, 128, 64, seed=new)
    q, _ = case.rows(group)
    expect, lse = bsq.kv_attention(q, *case.device(), new, return_lse=True)
    bad = q.clone()
    bad[0, 0] = float("nan")
    bad[-1, -1, 5] = float("nan")
    got, got_lse = bsq.kv_attention(bad, *case.device(), new, return_lse=True)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[0, 0] = hit[-1, -1] = True
    assert got[hit].isnan().all() and got_lse[hit].isnan().all()
    assert torch.equal(got[~hit], expect[~hit]) and torch.equal(got_lse[~hit], lse[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 40])
def test_append_keys_and_values_of_different_strides(bsq, new, dtype):
    """Keys contiguous (as after a rotary embedding), values a view of the fused projection, and the other way round."""
    for turn in (False, True):
        case = Case([70, new + 3], [new, new], 3, 64, 32, seed=8, dtype=dtype)
        args = case.device()
        (k, kn), (v, vn) = case.rows(3), case.rows(3)
        fused = torch.cat([k, v, k], 1)
        bsq.kv_append(*((fused[:, :3], v) if turn else (k, fused[:, 3:6])), *args)
        for x, cache, scales, got_c, got_s in ((kn, case.cache[0], case.scales[0], args[0], args[2]),
                                               (vn, case.cache[1], case.scales[1], args[1], args[3])):
            ref.append(x, cache, scales, case.table, case.offsets, case.lens)
            np.testing.assert_array_equal(got_s.cpu().numpy(), scales)
            np.testing.assert_array_equal(got_c.cpu().numpy(), cache)
