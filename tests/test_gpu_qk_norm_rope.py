"""qk_norm_rope on the GPU against its 64-bit statement (layer_reference.rope derives the tolerance)."""
import numpy as np
import pytest

import layer_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def bsq():
    import fp8_activation_quantization_bsq_gb300 as m
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert m.device_error() == 0
    yield m
    assert m.device_error() == 0


def make(tokens, heads, kv_heads, dim, pairs, dtype, seed=0, most=100000, base=10000.0):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((tokens, heads + 2 * kv_heads, dim))).to(DT[dtype]).cuda()
    pos = torch.from_numpy(rng.integers(0, most, tokens).astype(np.int32)).cuda()
    freq = torch.from_numpy((base ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)).cuda()
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DT[dtype]).cuda() for _ in range(2)]
    return qkv[:, :heads], qkv[:, heads:heads + kv_heads], pos, freq, w[0], w[1]


def check(q, k, pos, freq, qw, kw, got, dtype, interleaved, eps=1e-6):
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        expect, tol = ref.rope(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), pos.cpu().numpy(), freq.cpu().numpy(),
                               eps, interleaved, dtype)
        err = np.abs(y.double().cpu().numpy() - expect)
        assert y.shape == x.shape and y.dtype == x.dtype
        assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,pairs", [
    (1, 1, 1, 8, 4), (1, 32, 8, 128, 64), (3, 7, 1, 64, 32), (2, 5, 2, 80, 40), (5, 6, 3, 96, 32), (4, 3, 3, 128, 5), (2, 4, 2, 256, 128),
    (3, 2, 1, 256, 33), (9, 4, 4, 72, 1), (2, 3, 1, 64, 0), (700, 3, 2, 64, 16), (65, 24, 8, 40, 19), (2, 1, 1, 24, 12), (1000, 1, 1, 16, 7)])
def test_sizes(bsq, dtype, interleaved, tokens, heads, kv_heads, dim, pairs):
    q, k, pos, freq, qw, kw = make(tokens, heads, kv_heads, dim, pairs, dtype, seed=dim + pairs)
    for a, b in ((qw, kw), (None, None), (qw, None), (None, kw), (qw.float() * 1.001, kw.float())):
        got = bsq.qk_norm_rope(q, k, pos, freq, a, b, interleaved=interleaved)
        assert got[0].is_contiguous() and got[1].is_contiguous()
        check(q, k, pos, freq, a, b, got, dtype, interleaved)


@pytest.mark.parametrize("pairs", [64, 6])
def test_far_positions(bsq, pairs):
    """Angles of positions up to 2^31 - 1, frequencies above 1, negative and tiny ones."""
    q, k, pos, freq, qw, kw = make(64, 2, 1, 128, pairs, "f16", seed=3, most=2 ** 31 - 1)
    pos[0], pos[1] = 2 ** 31 - 1, 0
    check(q, k, pos, freq, qw, kw, bsq.qk_norm_rope(q, k, pos, freq, qw, kw), "f16", False)
    freq[0], freq[1], freq[2], freq[3] = 12345.678, -0.37, 1e-30, 2.0 ** 20
    pos %= 1000000
    check(q, k, pos, freq, None, None, bsq.qk_norm_rope(q, k, pos, freq), "f16", False)


def test_in_place_strided_outputs_and_negative_positions(bsq):
    q, k, pos, freq, qw, kw = make(40, 4, 2, 128, 64, "bf16", seed=4)
    pos[7], pos[39] = -1, -2 ** 31
    v = q.as_strided((40, 2, 128), q.stride(), q.storage_offset() + 6 * 128).clone()
    expect = bsq.qk_norm_rope(q, k, pos, freq, qw, kw, q_out=torch.full_like(q, 3).contiguous(), k_out=torch.full_like(k, 3).contiguous())
    assert (expect[0][7] == 3).all() and (expect[1][39] == 3).all()
    keep = [q[7].clone(), k[39].clone()]
    frame = torch.full((40, 4, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    a, b = bsq.qk_norm_rope(q, k, pos, freq, qw, kw, q_out=frame[..., 128:], k_out=k)
    assert b is k and (frame[..., :128] == 5).all() and (frame[7] == 5).all()
    ok = pos >= 0
    assert torch.equal(a[ok], expect[0][ok]) and torch.equal(k[ok], expect[1][ok]) and torch.equal(k[39], keep[1])
    bsq.qk_norm_rope(q, k, pos, freq, qw, None, q_out=q)
    assert torch.equal(q[ok], expect[0][ok]) and torch.equal(q[7], keep[0])
    assert torch.equal(q.as_strided((40, 2, 128), q.stride(), q.storage_offset() + 6 * 128), v)  # the values beside them stay


def test_transposed_heads_and_no_keys(bsq):
    q, k, pos, freq, qw, kw = make(6, 8, 2, 64, 32, "f16", seed=5)
    t = q.transpose(0, 1).contiguous().transpose(0, 1)   # (heads, tokens, dim) in memory
    assert torch.equal(bsq.qk_norm_rope(t, k, pos, freq, qw, kw)[0], bsq.qk_norm_rope(q, k, pos, freq, qw, kw)[0])
    a, b = bsq.qk_norm_rope(q, k[:, :0], pos, freq, qw, kw)
    assert b.shape == (6, 0, 64) and torch.equal(a, bsq.qk_norm_rope(q, k, pos, freq, qw, kw)[0])
    a, b = bsq.qk_norm_rope(q[:0], k[:0], pos[:0], freq, qw, kw)
    assert a.shape == (0, 8, 64) and b.shape == (0, 2, 64)


def test_extreme_values(bsq):
    """Rows whose squares pass FP32, zeros, and rows with inf or NaN, which stay with their row and their pair."""
    q, k, pos, freq, qw, kw = make(6, 2, 1, 128, 32, "bf16", seed=6)
    q[0] *= 1e25
    q[1] *= 1e-30
    q[2] = 0
    q[3] *= 3e37
    got = bsq.qk_norm_rope(q, k, pos, freq, qw, kw)
    check(q, k, pos, freq, qw, kw, got, "bf16", False)
    q[4, 0, 5], q[5, 1, 100] = float("inf"), float("nan")
    a, _ = bsq.qk_norm_rope(q, k, pos, freq)
    assert torch.equal(a[:4], bsq.qk_norm_rope(q[:4], k[:4], pos[:4], freq)[0])
    assert not torch.isfinite(a[4, 0, [5, 37]]).any() and torch.isfinite(a[4, 0]).sum() == 126
    assert a[5, 1, 100].isnan() and a[5, 1].isnan().sum() == 1
    b, _ = bsq.qk_norm_rope(q, k, pos, freq, qw, kw)
    assert torch.equal(b[4, 1], got[0][4, 1]) and b[5, 1].isnan().all()


def test_graph_and_streams(bsq):
    q, k, pos, freq, qw, kw = make(50, 8, 2, 128, 64, "bf16", seed=7)
    expect = bsq.qk_norm_rope(q, k, pos, freq, qw, kw)
    outs = [torch.empty_like(x) for x in expect]
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        bsq.qk_norm_rope(q, k, pos, freq, qw, kw, q_out=outs[0], k_out=outs[1])
    for shift in (0, 100):
        pos += shift
        expect = bsq.qk_norm_rope(q, k, pos, freq, qw, kw)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, expect))
    got = bsq.qk_norm_rope(q, k, pos, freq, qw, kw, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, expect))
