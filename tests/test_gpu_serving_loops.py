"""The serving kernels where their rings go round many times: long runs of
units per block, full-size weights; and the cache's metadata where every
attention kernel meets it."""
import numpy as np
import pytest

import serving_reference as ref
from test_gpu_kv_cache import Case, check_attention, compare
from test_gpu_moe_layer import FORMATS

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


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16)])
def test_attention_runs_of_many_units(bsq, group, new, dim, page):
    """At least 12 units per block, with 152 blocks or 2 or 3 times that, over rings of 3 to 6; items of uneven lengths."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(new, 2 * 2300, 40)]
    case = Case(lens, [new] * len(lens), 4, dim, page, seed=dim + new)
    case.poison()
    keys, blocks = {4: (64, 456), 16: (64, 304), 32: (64, 152), 160: (128, 152)}[group * new]
    assert sum(n // keys for n in lens) * 4 >= 12 * blocks
    check_attention(bsq, case, 4 * group)


def moe_expected(fmt, x, logits, w13, w2, top_k, x_sf, h_sf):
    """serving_reference.moe for many tokens of few experts: the products as matrix products in float64 on the GPU.
    To its tolerance comes the error of silu: the exponential's argument makes it grow with |g|, to (4 + 1.2 |g|) 2^-23."""
    tokens, hidden = x.shape
    inter = w2[0].shape[1]
    y, tol = (torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda") for _ in range(2))
    ids = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :top_k]
    p = np.exp(np.take_along_axis(logits.astype(np.float64), ids, 1) - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float64)).cuda()  # noqa: E731
    for e in range(logits.shape[1]):
        t, k = np.nonzero(ids == e)
        if not len(t):
            continue
        a13, a2 = dev(w13[e]), dev(w2[e])
        xq = dev(ref.quantized_values(fmt, x[t], x_sf[e]))
        gu = (xq @ a13.T).cpu().numpy()
        err = (xq.abs() @ a13.abs().T).cpu().numpy() * hidden * 2.0 ** -24

        def codes(sg, su, sh):
            g, u = gu[:, :inter] + sg * err[:, :inter], gu[:, inter:] + su * err[:, inter:]
            with np.errstate(over="ignore"):
                h = g / (1 + np.exp(-g)) * u * (1 + sh * (4 + 1.2 * np.abs(g)) * 2.0 ** -23)
            return ref.quantized_values(fmt, ref.bf16(h), h_sf[e])

        hq = codes(0, 0, 0)
        off = np.max([np.abs(codes(a, b, c) - hq) for a in (-1, 1) for b in (-1, 1) for c in (-1, 1)], axis=0)
        pe, rows = dev(p[t, k])[:, None], torch.from_numpy(t).cuda()
        y.index_add_(0, rows, pe * (dev(hq) @ a2.T))
        tol.index_add_(0, rows, pe * (dev(off + np.abs(hq) * (inter + 16) * 2.0 ** -24) @ a2.abs().T))
    y, tol = y.cpu().numpy(), tol.cpu().numpy()
    return y, tol * 1.01 + np.abs(y) * 2.0 ** -8 + 1e-30


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [16, 64])
def test_expert_layer_runs_of_many_stages(bsq, fmt, tokens):
    """Two experts of 4096 x 6144: 15 stages (4-bit formats) or 30 per block, over rings of 4 to 6; 16 and 64 tokens each."""
    import oracle
    hidden, inter, experts = 4096, 6144, 2
    rng = np.random.default_rng(tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    nv = fmt == "nvfp4"
    sf = lambda top: rng.uniform(0.5, 1.0, experts).astype(np.float32) * np.float32(2688 / top)  # noqa: E731
    x_sf, h_sf = (sf(6.0), sf(20.0)) if nv else (np.ones(experts, np.float32),) * 2
    args, values, sfs = [], [], []
    for rows, cols in ((2 * inter, hidden), (hidden, inter)):
        w = [(torch.randn((rows, cols), generator=g, device="cuda") / cols ** 0.5).bfloat16() for _ in range(experts)]
        tsf = [float(bsq.tensor_sf(m)[1]) if nv else 1.0 for m in w]
        q = [bsq.quantize(m, fmt, t) for m, t in zip(w, tsf)]
        args += [torch.stack([a for a, _ in q]), torch.stack([b for _, b in q])]
        s = cols // oracle.block_size(fmt)
        values.append([oracle.dequantize(fmt, a.cpu().numpy(), oracle.layout.scales_from_5d_view(b.cpu().numpy(), rows, s)[:rows, :s], t)
                       for (a, b), t in zip(q, tsf)])
        sfs.append(np.asarray(tsf, np.float32))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    kw = dict(x_sf=dev(x_sf), w13_sf=dev(sfs[0]), h_sf=dev(h_sf), w2_sf=dev(sfs[1])) if nv else {}
    x = torch.from_numpy(rng.standard_normal((tokens, hidden))).bfloat16()
    z = rng.standard_normal((tokens, experts)).astype(np.float32)
    y = bsq.moe_layer(x.cuda(), dev(z), *args, fmt, 2, **kw)
    expect, tol = moe_expected(fmt, x.float().numpy(), z, *values, 2, x_sf, h_sf)
    err = np.abs(y.double().cpu().numpy() - expect)
    assert np.isfinite(err).all()
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
    for _ in range(3):
        assert torch.equal(bsq.moe_layer(x.cuda(), dev(z), *args, fmt, 2, **kw), y)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("page", [16, 128])
def test_missing_pages_count_as_no_keys(bsq, group, new, page):
    """A page id outside the pool is reported; its tokens are no keys, whatever the ring's memory holds, and other sequences do not change."""
    case = Case([400, 700, 300], [new] * 3, 2, 64, page, seed=11)
    case.poison()
    q, qn = case.rows(2 * group)
    good = bsq.kv_attention(q, *case.device(), new, return_lse=True)
    for entry in (-1, case.pages, 1 << 30):
        bad = list(case.device())
        bad[4][1, 2] = entry
        out, lse = bsq.kv_attention(q, *bad, new, return_lse=True)
        assert bsq.device_error() == 4
        rows = np.r_[0:new, 2 * new:3 * new]
        assert torch.equal(out[rows], good[0][rows]) and torch.equal(lse[rows], good[1][rows])
        # sequence 1 without those tokens: the same keys in a shorter context, all of them before the first row
        kept = np.r_[0:2 * page, 3 * page:700]
        less = Case([len(kept)], [new], 2, 64, page, seed=1, spare=0)
        for c in range(2):
            flat = np.concatenate([case.cache[c][i] for i in case.table[1, :-(-700 // page)]], axis=1)[:, kept]
            ids = less.table[0]
            for i, pid in enumerate(ids[:-(-len(kept) // page)]):
                part = flat[:, i * page:(i + 1) * page]
                less.cache[c][pid][:, :part.shape[1]] = part
        # the kept tokens' pages are whole, so each page of `less` has the scale of one of them
        for c in range(2):
            src = [i for i in range(-(-700 // page)) if i != 2]
            for i, at in enumerate(src):
                less.scales[c][less.table[0, i]] = case.scales[c][case.table[1, at]]
        expect = ref.attention(qn[new:2 * new], *less.cache, *less.scales, less.table, less.offsets, less.lens, 1 / 8, True, 0)
        less.dtype = case.dtype
        compare(less, out[new:2 * new], lse[new:2 * new], *expect)


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("page", [16, 64])
def test_pages_before_the_window_need_no_entry(bsq, group, new, page):
    case = Case([1500, 300, 90], [new] * 3, 2, 64, page, seed=12)
    window = 100
    q, qn = case.rows(2 * group)
    for b, length in enumerate(case.lens):
        first = max(0, length - new - window + 1)        # of the first row
        case.cache[0][case.table[b, :first // page]] = 0x7F
        case.cache[1][case.table[b, :first // page]] = 0x7F
    args = list(case.device())
    expect, lse = bsq.kv_attention(q, *args, new, window=window, return_lse=True)
    for b, length in enumerate(case.lens):
        args[4][b, :max(0, length - new - window + 1) // page] = -1
    got, got_lse = bsq.kv_attention(q, *args, new, window=window, return_lse=True)
    assert torch.equal(got, expect) and torch.equal(got_lse, lse) and bsq.device_error() == 0
    case.cache = [np.where((c & 0x7F) == 0x7F, 0, c) for c in case.cache]
    compare(case, got, got_lse, *ref.attention(qn, *case.cache, *case.scales, case.table, case.offsets, case.lens, 1 / 8, True, window))


def test_falling_offsets_leave_other_rows_right(bsq):
    """Sequence 0 has no rows (its offsets fall); attention gives the others all of theirs."""
    case = Case([200] * 3, [100] * 3, 1, 64, 16, seed=13)
    case.offsets = np.array([200, 0, 100, 300])
    args = case.device()
    for group, max_q in ((2, 100), (1, 16)):
        q = torch.from_numpy(case.rng.standard_normal((300, group, 64))).bfloat16()
        got, lse = bsq.kv_attention(q.cuda(), *args, max_q, return_lse=True)
        bsq.device_error()
        compare(case, got, lse, *ref.attention(q.double().numpy(), *case.cache, *case.scales, case.table[1:], case.offsets[1:], case.lens[1:], 1 / 8,
                                               True, 0))
