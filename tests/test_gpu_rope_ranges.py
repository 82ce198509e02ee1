"""qk_norm_rope where its parts meet and at the ends of its ranges, against the
64-bit statement."""
import numpy as np
import pytest

from test_gpu_qk_norm_rope import DT, bsq, check, make  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("norm", [None, "q", "k"])
def test_queries_and_keys_of_every_number_of_steps(bsq, dim, norm):  # noqa: F811
    """A warp takes a token's queries, then its keys, through one ring of shared memory, without anything between but what the passes
    themselves wait for: every number of steps that leaves the ring at another place, each way of pairing."""
    at_once = 256 // dim if dim < 256 else 1
    for steps in range(1, 10):
        for pairs, interleaved in ((dim // 2, False), (dim // 2, True), (dim // 2 - 1, False)):
            # so many tokens that a warp takes all rows of one
            q, k, pos, freq, qw, kw = make(2600, steps * at_once, 2 * at_once, dim, pairs, "bf16", seed=steps)
            a, b = qw if norm == "q" else None, kw if norm == "k" else None
            got = bsq.qk_norm_rope(q, k, pos, freq, a, b, interleaved=interleaved)
            part = slice(None, None, 97)
            check(q[part], k[part], pos[part], freq, a, b, (got[0][part], got[1][part]), "bf16", interleaved)
            # the same rows one pass at a time
            assert torch.equal(got[0], bsq.qk_norm_rope(q, k[:, :0], pos, freq, a, b, interleaved=interleaved)[0])
            assert torch.equal(got[1], bsq.qk_norm_rope(q[:, :0], k, pos, freq, a, b, interleaved=interleaved)[1])


@pytest.mark.parametrize("size,weight,eps", [(1e18, 1e-25, 1e-6), (1e-12, 1e30, 0.0), (1e10, 1e-36, 1e-6), (1e-10, 1e28, 1e-30)])
def test_weights_far_from_one(bsq, size, weight, eps):  # noqa: F811
    """The norm's factor times the weight may lie outside FP32 where the result does not."""
    q, k, pos, freq, qw, kw = make(20, 3, 2, 128, 64, "bf16", seed=8)
    q, k, qw, kw = q.float().mul(size).bfloat16(), k.float().mul(size).bfloat16(), qw.float() * weight, kw.float() * weight
    got = bsq.qk_norm_rope(q, k, pos, freq, qw, kw, eps=eps)
    check(q, k, pos, freq, qw, kw, got, "bf16", False, float(np.float32(eps)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-36, 1e-30, 1e-24, 1e-21, 1e-20, 1e-12, 1e-6, 1.0, 1e20, 3.4e38])
def test_every_size_of_rows_with_every_eps(bsq, dtype, eps):  # noqa: F811
    """Rows whose squares leave FP32 at either end, with an eps that matters beside them, far above or not at all; elements of very different
    sizes in one row."""
    q, k, pos, freq, qw, kw = make(60, 3, 1, 128, 64, dtype, seed=9)
    low, high = (-130, 126) if dtype == "bf16" else (-20, 14)
    size = torch.exp2(torch.linspace(low, high, 60, device="cuda").round()).double()[:, None, None]
    q, k = ((x.double().clamp(-1.9, 1.9) * size).to(DT[dtype]) for x in (q, k))
    q[:, 1, ::5] = (q[:, 1, ::5].double() * 2.0 ** -60).to(DT[dtype])
    q[:, 2, 1:] = 0  # one element alone
    got = bsq.qk_norm_rope(q, k, pos, freq, qw, kw, eps=eps)
    check(q, k, pos, freq, qw, kw, got, dtype, False, float(np.float32(eps)))


@pytest.mark.parametrize("tokens,heads,kv_heads,dim", [(1, 4096, 4096, 8), (2, 300, 37, 64), (3, 1, 500, 128), (1, 2, 1, 256)])
def test_many_heads(bsq, tokens, heads, kv_heads, dim):  # noqa: F811
    q, k, pos, freq, qw, kw = make(tokens, heads, kv_heads, dim, dim // 2, "f16", seed=10)
    check(q, k, pos, freq, qw, kw, bsq.qk_norm_rope(q, k, pos, freq, qw, kw), "f16", False)
