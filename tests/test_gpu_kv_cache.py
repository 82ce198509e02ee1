"""kv_append and kv_attention on the GPU against their 64-bit statements.

Append is exact: every code and scale byte.  Attention's tolerance: a softmax
weight enters the product with the values rounded to FP16 (2^-11 of it at
most), a score is off by the FP32 rounding of its products and sums
((dim + 4) 2^-24 of sm_scale sum |q||k|), which moves its weight by that much
relatively, and exp2, sums and quotient add less than 2^-19; all of it is
relative to sum p |v|.  A weight below 2^-14 of the row's largest is an FP16
subnormal, off by up to 2^-25 of the largest weight whatever its own size.  The
output is rounded once to its type."""
import numpy as np
import pytest

import serving_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SUBNORMAL = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the spacing of the type's least numbers


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


class Case:
    """Sequences in a shuffled page pool; unused table entries are -1."""

    def __init__(self, lens, new, heads, dim, page, seed, dtype="bf16", order="hnd", spare=2):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.page, self.heads, self.dim, self.dtype = lens, page, heads, dim, dtype
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(int)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, heads, page, dim)
        self.cache = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
        for c in self.cache:
            c[(c & 0x7F) == 0x7F] = 0x38  # no NaN where values count
        self.scales = [rng.integers(118, 130, shape[:2]).astype(np.uint8) for _ in range(2)]
        self.order = order

    def poison(self):
        """NaN codes wherever no sequence has a token."""
        used = np.zeros((self.pages, self.page), bool)
        for b, n in enumerate(self.lens):
            for i in range(n):
                used[self.table[b, i // self.page], i % self.page] = True
        for c in self.cache:
            c.transpose(0, 2, 1, 3)[~used] = 0x7F

    def device(self):
        if self.order == "hnd":
            c = [torch.from_numpy(x.copy()).cuda() for x in self.cache]
        else:  # (pages, page, heads, dim) in memory
            c = [torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).cuda().permute(0, 2, 1, 3) for x in self.cache]
        s = [torch.from_numpy(x.copy()).cuda() for x in self.scales]
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
        return (*c, *s, i32(self.table), i32(self.offsets), i32(self.lens))

    def rows(self, heads, scale=1.0):
        x = torch.from_numpy(self.rng.standard_normal((int(self.offsets[-1]), heads, self.dim)) * scale).to(DT[self.dtype])
        return x.cuda(), x.double().numpy()


def check_append(bsq, case, k_scale=1.0, v_scale=3.0, strided=False):
    args = case.device()
    (k, kn), (v, vn) = case.rows(case.heads, k_scale), case.rows(case.heads, v_scale)
    if strided:  # parts of one projection's output
        both = torch.cat([k, v, k], 2).contiguous()
        k, v = both[:, :, :case.dim], both[:, :, case.dim:2 * case.dim]
    bsq.kv_append(k, v, *args)
    for x, cache, scales, got_c, got_s in ((kn, case.cache[0], case.scales[0], args[0], args[2]),
                                           (vn, case.cache[1], case.scales[1], args[1], args[3])):
        ref.append(x, cache, scales, case.table, case.offsets, case.lens)
        np.testing.assert_array_equal(got_s.cpu().numpy(), scales)
        np.testing.assert_array_equal(got_c.cpu().numpy(), cache)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_bytes(bsq, dtype, dim, page):
    # single tokens, a whole page, one that ends and one that begins a page, nothing, many pages
    new = [1, page, 1, 1, 0, 3 * page + 5, 2]
    past = [0, 0, page - 1, page, 7, 9, page - 1]
    case = Case([a + b for a, b in zip(new, past)], new, 3, dim, page, seed=page + dim, dtype=dtype)
    check_append(bsq, case)


@pytest.mark.parametrize("scale", [1e-12, 1e-3, 1.0, 1e4])
def test_append_scale_growth_and_floor(bsq, scale):
    """New tokens far below, near and above what the page holds; below the least scale."""
    case = Case([20, 40, 33], [3, 1, 33], 2, 128, 32, seed=5)
    check_append(bsq, case, scale, scale)


def test_append_zeros_and_token_by_token(bsq):
    """A page filled one token at a time, with zero tokens among them."""
    case = Case([1], [1], 2, 64, 16, seed=6)
    args = case.device()
    for length in range(1, 20):
        case.lens = [length]
        if length == 17:
            case.table = np.array([[case.table[0, 0], (case.table[0, 0] + 1) % case.pages]], np.int32)
        x = case.rng.standard_normal((1, 2, 64)) * (0 if length in (1, 5) else 2.0 ** (length % 7))
        t = torch.from_numpy(x).bfloat16()
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
        args = (*args[:4], i32(case.table), i32([0, 1]), i32(case.lens))
        bsq.kv_append(t.cuda(), t.cuda(), *args)
        for c, s, gc, gs in ((case.cache[0], case.scales[0], args[0], args[2]), (case.cache[1], case.scales[1], args[1], args[3])):
            ref.append(t.double().numpy(), c, s, case.table, [0, 1], case.lens)
            np.testing.assert_array_equal(gs.cpu().numpy(), s)
            np.testing.assert_array_equal(gc.cpu().numpy(), c)


def test_append_strides(bsq):
    check_append(bsq, Case([70, 5], [40, 5], 5, 128, 32, seed=8, order="nhd"), strided=True)


def check_attention(bsq, case, heads, causal=True, window=0, sm_scale=None, **kw):
    q, qn = case.rows(heads)
    max_q = int(np.max(np.diff(case.offsets)))
    scale = 1 / np.sqrt(case.dim) if sm_scale is None else sm_scale
    args = case.device()
    got, got_lse = bsq.kv_attention(q, *args, max_q, causal=causal, window=window, sm_scale=sm_scale, return_lse=True, **kw)
    expect = ref.attention(qn, *case.cache, *case.scales, case.table, case.offsets, case.lens, scale, causal, window)
    compare(case, got, got_lse, *expect)
    return q, args, got, got_lse


def compare(case, got, got_lse, out, lse, mag, size, low):
    score = (case.dim + 4) * 2.0 ** -24 * size
    tol = HALF_ULP[case.dtype] * np.abs(out) + (2.0 ** -11 + 2 * score + 2.0 ** -19)[..., None] * mag + 2.0 ** -25 * low + SUBNORMAL[case.dtype] + 1e-30
    err = np.abs(got.double().cpu().numpy() - out)
    assert np.isfinite(err).all()
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
    g = got_lse.double().cpu().numpy()
    some = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(g), ~some)
    assert (np.abs(g[some] - lse[some]) <= 2 * score[some] + 2.0 ** -20 * (1 + np.abs(lse[some]))).all()


# rows per kv head: 1..8, 9..16, 17..32 and many take kernels of their own
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group,new", [(1, 1), (5, 1), (8, 1), (3, 5), (16, 1), (8, 3), (8, 4), (5, 7), (1, 130), (4, 70)])
def test_attention_rows(bsq, dim, page, group, new):
    # lengths around pages and tiles, one of them shorter than its rows
    lens = [max(1, new - 1), new, 63 + new, 64, 65, 128, 129 + new, 300]
    case = Case([max(n, 1) for n in lens], [min(new, n) if i else new for i, n in enumerate(lens)], 2, dim, page,
                seed=group * 100 + new, dtype="bf16" if page != 32 else "f16")
    case.poison()
    check_attention(bsq, case, 2 * group)


@pytest.mark.parametrize("group,new", [(4, 1), (4, 3), (4, 7), (4, 40)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 50, 64, 129])
def test_attention_masks(bsq, group, new, causal, window):
    case = Case([400, 64, 77, new], [new, new, 1, new], 1, 128, 64, seed=window + new)
    check_attention(bsq, case, group, causal, window)


@pytest.mark.parametrize("group,new", [(2, 1), (8, 2), (3, 9), (2, 90)])
def test_attention_empty_sequences(bsq, group, new):
    """No keys at all, no rows at all, rows before the first key."""
    case = Case([0, 50, 200, 1, 0, 30], [new, 0, new, new, 1, new], 2, 64, 16, seed=3)
    check_attention(bsq, case, 2 * group)


@pytest.mark.parametrize("group,new", [(8, 1), (16, 1), (4, 8), (8, 20)])
def test_attention_long_context_is_joined(bsq, group, new):
    """One item over all blocks, joined in one and in two levels."""
    for length in (3000, 30011):
        case = Case([length], [new], 1, 128, 64, seed=length)
        q, args, out, lse = check_attention(bsq, case, group)
        for _ in range(3):  # the order of the sums does not depend on timing
            again = bsq.kv_attention(q, *args, new, return_lse=True)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("group,new", [(8, 1), (4, 20)])
def test_attention_many_sequences(bsq, group, new):
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(0, 120, 700)]
    check_attention(bsq, Case(lens, [min(new, n) for n in lens], 1, 64, 16, seed=2), group)


@pytest.mark.parametrize("group,new", [(4, 4), (3, 5), (8, 4), (5, 5)])
def test_attention_many_items_share_query_memory(bsq, group, new):
    """Rows in shared memory that the items of a block use one after the other."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 300, 500)]
    check_attention(bsq, Case(lens, [min(new, n) for n in lens], 2, 128, 16, seed=6), 2 * group)


@pytest.mark.parametrize("group,new", [(4, 1), (8, 3), (4, 33)])
def test_attention_scales_and_sharpness(bsq, group, new):
    """Page scales far apart, and one key that takes all of the weight."""
    case = Case([333, 128], [new, new], 2, 128, 16, seed=9)
    case.scales = [case.rng.integers(100, 126, (case.pages, 2)).astype(np.uint8), case.rng.integers(97, 150, (case.pages, 2)).astype(np.uint8)]
    for s in (None, 4.0, -1.0, 0.0):
        check_attention(bsq, case, 2 * group, sm_scale=s)


@pytest.mark.parametrize("group,new", [(4, 1), (4, 5), (2, 70)])
def test_attention_strides_streams_graphs(bsq, group, new):
    case = Case([150, 31, 260], [new, new, new], 2, 128, 64, seed=4, order="nhd")
    case.poison()
    q, qn = case.rows(2 * group)
    fused = torch.cat([q, q], 1)[:, :2 * group]          # row stride of a fused projection
    args = case.device()
    expect = bsq.kv_attention(q, *args, new)
    ws = torch.zeros(bsq.kv_attention_workspace_bytes(q.shape[0], 2 * group, 2, 128, 3, new), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(expect)
    got = bsq.kv_attention(fused, *args, new, out=out, workspace=ws, stream=stream)
    stream.synchronize()
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, expect)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsq.kv_attention(q, *args, new, out=out, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, expect)
    assert not ws[:4096].any()                            # flags are down again
    check_attention(bsq, case, 2 * group)


def test_append_then_attention_past_32_bit_offsets(bsq):
    """Pages at the end of pools of more than 4 GB."""
    pages = (5 << 30) // (64 * 128 * 2)
    cache = [torch.empty((pages, 2, 64, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = 150
    ids = [pages - 1, pages - 7, pages - 3]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens = i32([ids]), i32([n])
    rng = np.random.default_rng(0)
    k, v = (torch.from_numpy(rng.standard_normal((n, 2, 128))).bfloat16().cuda() for _ in range(2))
    bsq.kv_append(k, v, *cache, *scales, table, i32([0, n]), lens)
    case = Case([n], [1], 2, 128, 64, seed=0, spare=0)
    case.table = np.array([[0, 1, 2]], np.int32)
    case.cache = [c[ids].cpu().numpy() for c in cache]
    case.scales = [s[ids].cpu().numpy() for s in scales]
    q, qn = case.rows(8)
    out, lse = bsq.kv_attention(q, *cache, *scales, table, i32([0, 1]), lens, 1, return_lse=True)
    compare(case, out, lse, *ref.attention(qn, *case.cache, *case.scales, case.table, [0, 1], [n], 128 ** -0.5, True, 0))


def test_bad_metadata_is_reported_and_skipped(bsq):
    case = Case([40, 40, 40], [1, 1, 1], 1, 64, 16, seed=11)
    good = case.device()
    q, qn = case.rows(4)
    before = bsq.kv_attention(q, *good, 1)
    for entry in (-1, case.pages, 1 << 30):
        bad = list(case.device())
        bad[4][1, 1] = entry                              # a page that sequence 1 needs
        out = bsq.kv_attention(q, *bad, 1)
        assert bsq.device_error() == 4
        assert torch.equal(out[0], before[0]) and torch.equal(out[2], before[2]) and torch.isfinite(out).all()
        k, _ = case.rows(1)
        bad[4][1] = entry
        kept = bad[0].clone()
        bsq.kv_append(k, k, *bad)
        assert bsq.device_error() == 4
        ids = [i for i in range(case.pages) if i not in (case.table[0, 2], case.table[2, 2])]
        assert torch.equal(bad[0][ids], kept[ids])        # sequence 1 wrote nowhere
    bad = list(case.device())
    bad[6][0] = 16 * bad[4].shape[1] + 1                  # longer than its table
    out = bsq.kv_attention(q, *bad, 1)
    assert bsq.device_error() == 4
    assert not out[0].any() and torch.equal(out[1:], before[1:])


def test_falling_offsets_reach_nothing_else(bsq):
    case = Case([200] * 3, [100] * 3, 1, 64, 16, seed=13)
    k, _ = case.rows(1)
    q, _ = case.rows(2)
    for offsets in ([0, 200, 100, 300], [0, 300, 300, 100], [200, 0, 100, 300], [-20, 0, 100, 200], [0, 100, 200, 1 << 30],
                    [160, 176, 0, 300]):
        args = list(case.device())
        args[5] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        used = set(case.table.ravel().tolist())
        others = [i for i in range(case.pages) if i not in used]
        kept = args[0].clone()
        bsq.kv_append(k, k, *args)
        assert torch.equal(args[0][others], kept[others])  # nothing outside the sequences' pages
        bsq.device_error()
        out = bsq.kv_attention(q, *case.device()[:5], args[5], args[6], 100)
        assert out.shape == q.shape
        bsq.device_error()


@pytest.mark.parametrize("new", [1, 40])
def test_widest_window_is_none(bsq, new):
    case = Case([300, 20], [new, min(new, 20)], 1, 64, 16, seed=14)
    q, _ = case.rows(2)
    args = case.device()
    for causal in (True, False):
        expect = bsq.kv_attention(q, *args, new, causal=causal)
        for window in (1 << 20, (1 << 30) - 1, 1 << 30, (1 << 31) - 1):
            assert torch.equal(bsq.kv_attention(q, *args, new, causal=causal, window=window), expect)


def test_own_workspace_on_another_stream(bsq):
    """What the call allocates belongs to the stream it runs on: the current one is busy, and its free memory is not zero."""
    case = Case([3000], [1], 1, 128, 64, seed=15)
    q, _ = case.rows(8)
    args = case.device()
    expect = bsq.kv_attention(q, *args, 1)
    stale = torch.full((bsq.kv_attention_workspace_bytes(1, 8, 1, 128, 1, 1),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del stale
    stream = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got, lse = bsq.kv_attention(q, *args, 1, return_lse=True, stream=stream)
    stream.synchronize()
    assert torch.equal(got.cpu(), expect.cpu()) and bsq.device_error() == 0


def test_no_rows_is_a_no_op(bsq):
    case = Case([5], [1], 1, 64, 16, seed=12)
    args = case.device()
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    zero = (*args[:5], torch.zeros(2, dtype=torch.int32, device="cuda"), args[6])
    kept = args[0].clone()
    bsq.kv_append(none, none, *zero)
    assert bsq.kv_attention(none, *zero, 1).shape == (0, 1, 64)
    assert torch.equal(args[0], kept)
