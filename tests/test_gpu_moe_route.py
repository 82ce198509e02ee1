"""moe_route and moe_rows on the GPU: the experts equal the 64-bit statement's,
weights agree to FP32, rows are equal; and the run into the grouped quantize
and the expert layer."""
import numpy as np
import pytest

import layer_reference as ref
import oracle

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


def check(bsq, z, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    ids, weights = bsq.moe_route(z, top_k, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                                 renormalize=renormalize, scale=scale)
    zn = z.double().cpu().numpy()
    eids, ew = ref.route(zn, top_k, scoring == "sigmoid", None if bias is None else bias.double().cpu().numpy(), groups, top_groups, group_top,
                         renormalize, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), eids)
    # the exponent's argument is off by half a unit of |z - max| or |z|, the exponential and the division by 2 units each,
    # sums over choices (5 steps) or experts (10 steps of a tree, 32 in a lane), the scale one more
    finite = np.where(np.isfinite(zn), np.abs(zn), 0).max(1, keepdims=True)
    tol = ew * (2 * finite + 64) * 2.0 ** -24 + 2.0 ** -120
    err = np.abs(weights.double().cpu().numpy() - ew)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
    return ids, weights


def logits(tokens, experts, dtype, seed=0, size=1.5):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((tokens, experts)) * size).to(DT[dtype]).cuda()


def biases(experts, size, seed=1):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(experts) * size).astype(np.float32)).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups", [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 2, 2, 2, 2), (5, 33, 3, 3, 2), (130, 64, 6, 1, 1), (7, 65, 16, 5, 2), (300, 256, 8, 8, 3),
    (4, 1024, 16, 32, 4), (9, 96, 4, 32, 5), (2, 257, 8, 1, 1), (6, 30, 5, 30, 7), (1, 40, 16, 2, 1)])
def test_sizes(bsq, dtype, scoring, tokens, experts, top_k, groups, top_groups):
    z = logits(tokens, experts, dtype, seed=experts + tokens)
    for bias in (None, biases(experts, 0.1 if scoring == "sigmoid" else 1.0 / experts)):
        for group_top in (1, 2):
            check(bsq, z, top_k, scoring, bias, groups, top_groups, group_top)
    check(bsq, z, top_k, scoring, None, groups, top_groups, 1, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_values_closer_than_fp32(bsq, scoring):
    """Biases that make up for the scores' differences: the values lie 2^-30 to 2^-40 apart, in an order that FP32 cannot see."""
    rng = np.random.default_rng(2)
    tokens, experts = 16, 64
    z = rng.standard_normal(experts).astype(np.float32)
    p = 1 / (1 + np.exp(-z.astype(np.float64))) if scoring == "sigmoid" else np.exp(z.astype(np.float64)) / np.exp(z.astype(np.float64)).sum()
    bias = (1.0 - p).astype(np.float32)                 # p + bias = 1 up to the bias's rounding
    gap = np.diff(np.sort(p + bias.astype(np.float64)))
    assert gap.max() < 2.0 ** -23 and np.median(gap) > 2.0 ** -40
    both = torch.from_numpy(np.tile(z, (tokens, 1))).cuda()
    check(bsq, both, 16, scoring, torch.from_numpy(bias).cuda())
    check(bsq, both, 8, scoring, torch.from_numpy(bias).cuda(), 8, 3, 2)


def test_ties_go_to_the_lowest_expert(bsq):
    z = torch.zeros((4, 48), device="cuda")
    z[1, 40:] = 1
    z[2, ::3] = -0.0
    z[3] = torch.arange(48, device="cuda") // 5
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(48, device="cuda")):
            check(bsq, z, 10, scoring, bias)
            check(bsq, z, 10, scoring, bias, 4, 2, 2)
            check(bsq, z, 10, scoring, bias, 4, 2, 1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_excluded_experts(bsq, scoring):
    """Logits of -inf: fewer than top_k left, whole groups, whole rows; and the type's lowest value."""
    z = logits(7, 40, "f32", seed=3)
    z[1, 3:] = -np.inf                  # three left
    z[2, :20] = -np.inf                 # two groups out
    z[3] = -np.inf                      # nothing left
    z[4, ::2] = torch.finfo(torch.float32).min
    z[5, 10:] = -1e30
    z[6, 1:] = -np.inf
    for bias in (None, biases(40, 0.3)):
        check(bsq, z, 6, scoring, bias)
        check(bsq, z, 6, scoring, bias, renormalize=False)
        check(bsq, z, 6, scoring, bias, 4, 2, 2)
        check(bsq, z, 6, scoring, bias, 4, 1, 1)
    bias = biases(40, 0.3)
    bias[:30] = -np.inf
    ids, w = check(bsq, z[:1], 8, scoring, bias)
    assert (ids >= 30).all() and (w > 0).all()


def test_large_logits_and_biases(bsq):
    z = logits(50, 128, "f32", seed=4, size=30.0)
    check(bsq, z, 8, "softmax")
    check(bsq, z, 8, "sigmoid")
    check(bsq, z, 8, "softmax", biases(128, 1000.0), 8, 3, 2)
    check(bsq, z, 8, "sigmoid", biases(128, 1e6), 8, 3, 2)


def test_nan_and_inf_are_reported(bsq):
    z = logits(3, 20, "f32", seed=5)
    z[1, 4], z[2, 5] = float("nan"), float("inf")
    ids, _ = check(bsq, z, 4)
    assert bsq.device_error() == 4 and bsq.device_error() == 0
    bias = torch.zeros(20, device="cuda")
    bias[3] = float("nan")
    ids, w = bsq.moe_route(z[:1], 4, bias=bias)
    assert bsq.device_error() == 4 and 3 not in ids.tolist()[0] and torch.isfinite(w).all()


def test_strided_logits_and_given_outputs(bsq):
    wide = logits(9, 100, "bf16", seed=6)
    z = wide[:, 10:74]
    ids, w = torch.full((9, 4), -7, dtype=torch.int32, device="cuda"), torch.zeros((9, 4), device="cuda")
    got = bsq.moe_route(z, 4, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    a, b = check(bsq, z.contiguous(), 4)
    assert torch.equal(ids, a) and torch.equal(w, b)
    e, f = bsq.moe_route(z[:0], 4)
    assert e.shape == (0, 4) and f.shape == (0, 4)


@pytest.mark.parametrize("tokens,top_k,experts", [(0, 4, 8), (1, 1, 1), (1, 8, 256), (37, 3, 5), (512, 2, 1000), (129, 8, 256), (700, 16, 1024),
                                                  (5000, 8, 256), (33, 1, 3), (20000, 2, 7), (9000, 40, 64)])
def test_rows(bsq, tokens, top_k, experts):
    rng = np.random.default_rng(tokens + experts)
    ids = np.minimum(rng.zipf(1.3, (tokens, top_k)) - 1, experts - 1).astype(np.int32)
    for drop in (0.0, 0.2, 1.0):
        x = np.where(rng.random(ids.shape) < drop, -1, ids).astype(np.int32)
        got = bsq.moe_rows(torch.from_numpy(x).cuda(), experts)
        for a, b in zip(got, ref.rows(x, experts)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        assert int(got[1][-1]) <= bsq.moe_rows_scale_rows(x.size, experts)


def test_rows_report_ids_past_the_last(bsq):
    ids = torch.tensor([[0, 3], [2, 2], [-5, 1]], dtype=torch.int32, device="cuda")
    got = bsq.moe_rows(ids, 3)
    assert bsq.device_error() == 4
    expect = ref.rows(np.array([[0, -1], [2, 2], [-1, 1]]), 3)
    for a, b in zip(got, expect):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("tokens,kernel", [(200, "token"), (200, "stream"), (40, "latency"), (200, "auto")])
def test_route_rows_and_grouped_quantize(bsq, tokens, kernel):
    """Routing, rows and the grouped quantize one after the other, nothing on the host in between, some tokens dropped as padding."""
    experts, top_k, K = 24, 4, 256
    x = torch.from_numpy(np.random.default_rng(8).standard_normal((tokens, K))).bfloat16().cuda()
    ids, _ = bsq.moe_route(logits(tokens, experts, "f32", seed=9), top_k, "sigmoid", biases(experts, 0.2), 4, 2)
    ids[tokens - 10:] = -1
    ro, so, idx, pos = bsq.moe_rows(ids, experts)
    scale_rows = bsq.moe_rows_scale_rows(tokens * top_k, experts)
    every = torch.arange(experts, dtype=torch.int32, device="cuda")
    sf = bsq.grouped_tensor_sf(x, ro, every, experts, idx, total_rows=tokens * top_k)
    packed, scales = bsq.grouped_quantize(x, "nvfp4", ro, so, every, sf, idx, total_rows=tokens * top_k, total_scale_rows=scale_rows,
                                          k_tiles_per_block=0, kernel=kernel)
    assert bsq.device_error() == 0
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    u32 = lambda a: a.cpu().numpy().astype(np.uint32)  # noqa: E731
    _, sf_ref = oracle.expert_tensor_sf(bits, u32(ro), every.cpu().numpy(), experts, idx.cpu().numpy())
    np.testing.assert_array_equal(sf.cpu().numpy(), sf_ref)
    p, pw, s, sw = oracle.grouped_quantize("nvfp4", bits, u32(ro), u32(so), every.cpu().numpy(), sf_ref, idx.cpu().numpy())
    n, m = min(len(p), packed.shape[0]), min(len(s), scales.numel())
    assert pw[:n].sum() > 0 and (ids >= 0).sum().item() == int(ro[-1])
    np.testing.assert_array_equal(packed.cpu().numpy()[:n][pw[:n]], p[:n][pw[:n]])
    np.testing.assert_array_equal(scales.cpu().numpy()[:m][sw[:m]], s[:m][sw[:m]])
    rows = pos.long()
    assert (idx[rows[:tokens - 10]] == torch.arange(tokens - 10, device="cuda")[:, None]).all() and (rows[tokens - 10:] == -1).all()


def test_graph_and_streams(bsq):
    z, bias = logits(100, 256, "f32", seed=10), biases(256, 0.1)
    ids, w = bsq.moe_route(z, 8, "sigmoid", bias, 8, 4)
    bsq.moe_rows(ids, 256)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        bsq.moe_route(z, 8, "sigmoid", bias, 8, 4, ids=ids, weights=w)
        rows = bsq.moe_rows(ids, 256)
    for seed in (11, 12):
        z.copy_(logits(100, 256, "f32", seed=seed))
        expect, ew = check(bsq, z, 8, "sigmoid", bias, 8, 4)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, expect) and torch.equal(w, ew)
        for a, b in zip(rows, ref.rows(ids.cpu().numpy(), 256)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
    got = bsq.moe_route(z, 8, "sigmoid", bias, 8, 4, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got[0], expect)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups", [(128, 8, 3), (96, 6, 2), (250, 10, 5), (512, 4, 2), (1000, 20, 3)])
def test_few_groups_of_many(bsq, scoring, experts, groups, top_groups):
    """Groups that fill at most half of the experts: values left in all, some and none of them, equal ones, and ones closer than FP32 tells apart."""
    rng = np.random.default_rng(experts)
    z = logits(9, experts, "f32", seed=experts)
    per = experts // groups
    z[1, 5:] = -np.inf                        # five left, all in the first groups
    z[2, :experts - 3] = -np.inf              # three left in the last group: the others are the first experts of all
    z[3] = -np.inf
    z[4, ::2] = -np.inf
    z[5] = 0.5                                # all equal
    z[6] = torch.from_numpy(np.repeat(rng.standard_normal(groups), per).astype(np.float32)).cuda()  # equal within a group
    z[7, per:] = -np.inf
    for bias in (None, biases(experts, 0.2)):
        for group_top in (1, 2):
            check(bsq, z, 8, scoring, bias, groups, top_groups, group_top)
    one = rng.standard_normal(experts).astype(np.float32)
    p = 1 / (1 + np.exp(-one.astype(np.float64))) if scoring == "sigmoid" else np.exp(one.astype(np.float64)) / np.exp(one.astype(np.float64)).sum()
    bias = (1.0 - p).astype(np.float32)
    bias[per * top_groups:] -= np.float32(0.25)  # the first groups stay, their values one apart by the bias's rounding
    check(bsq, torch.from_numpy(np.tile(one, (5, 1))).cuda(), 8, scoring, torch.from_numpy(bias).cuda(), groups, top_groups, 1)
