"""moe_layer with a finished routing against its 64-bit statement: the choices'
outputs, each as serving_reference.moe gives it for that expert alone, in
their weights."""
import numpy as np
import pytest

import serving_reference as ref
from test_gpu_moe_layer import FORMATS, Layer, bsq  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def expect(layer, xn, ids, weights):
    tokens, top_k = ids.shape
    y, tol = np.zeros((2, tokens, layer.hidden))
    for t in range(tokens):
        for e, w in zip(ids[t], weights[t]):
            if 0 <= e < layer.experts and w != 0:
                z = np.full((1, layer.experts), -np.inf, np.float32)
                z[0, e] = 0
                a, b = ref.moe(layer.fmt, xn[t:t + 1], z, *layer.w, 1, layer.x_sf, layer.h_sf, True)
                y[t] += w * a[0]
                tol[t] += abs(w) * b[0]      # a rounding of the sum to BF16 among it, for the sum of magnitudes
    return y, tol * (1 + 2.0 ** -20) + np.abs(y) * 2.0 ** -8 + 1e-30


def run(bsq, layer, ids, weights, x=None, **kw):  # noqa: F811
    xt, xn, _ = layer.inputs(ids.shape[0], 1)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    y = bsq.moe_layer(xt, None, *layer.args, layer.fmt, ids.shape[1], routing=(dev(ids, torch.int32), dev(weights, torch.float32)), **layer.kw, **kw)
    return y, xn


def check(bsq, layer, ids, weights, **kw):  # noqa: F811
    weights = weights.astype(np.float32)
    y, xn = run(bsq, layer, ids, weights, **kw)
    e, tol = expect(layer, xn, ids, weights)
    err = np.abs(y.double().cpu().numpy() - e)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance"
    return y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden,inter,experts,top_k,tokens", [(32, 128, 1, 1, 1), (96, 128, 5, 3, 2), (288, 256, 33, 4, 17), (544, 128, 40, 16, 64)])
def test_sizes_with_missing_and_repeated_experts(bsq, fmt, hidden, inter, experts, top_k, tokens):  # noqa: F811
    layer = Layer(bsq, fmt, hidden, inter, experts, seed=hidden)
    rng = np.random.default_rng(tokens)
    for lowest in (0, -2):                      # negative ids: no choice; experts come twice
        ids = rng.integers(lowest, experts, (tokens, top_k))
        weights = rng.standard_normal((tokens, top_k)) * 2
        weights[rng.random(weights.shape) < 0.1] = 0
        # one weight per expert and token, as the call adds them: the statement then has no cancellation that it has not
        for t in range(tokens):
            for k in range(top_k):
                first = list(ids[t]).index(ids[t, k])
                weights[t, k] = abs(weights[t, k]) if first != k else weights[t, k]
                weights[t, first] = abs(weights[t, first]) if first != k else weights[t, first]
        check(bsq, layer, ids, weights)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nothing_chosen_and_one_workspace(bsq, fmt):  # noqa: F811
    layer = Layer(bsq, fmt, 160, 128, 6, seed=2)
    ws = torch.zeros(bsq.moe_layer_workspace_bytes(fmt, 9, 160, 128, 6, 3), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    ids, weights = rng.permuted(np.tile(np.arange(6), (9, 1)), axis=1)[:, :3], rng.random((9, 3))
    full = check(bsq, layer, ids, weights, workspace=ws)
    y, _ = run(bsq, layer, np.full((9, 3), -1), np.full((9, 3), np.nan), workspace=ws)
    assert (y == 0).all()
    ids[4] = -1
    some = check(bsq, layer, ids, weights, workspace=ws)
    assert (some[4] == 0).all() and torch.equal(some[:4], full[:4]) and torch.equal(some[5:], full[5:])


def test_ids_past_the_last_are_reported(bsq):  # noqa: F811
    layer = Layer(bsq, "mxfp8", 64, 128, 4, seed=4)
    ids, weights = np.array([[0, 4], [3, 1]]), np.ones((2, 2))
    check(bsq, layer, ids, weights)
    assert bsq.device_error() == 4 and bsq.device_error() == 0


def test_with_moe_route(bsq):  # noqa: F811
    """Softmax over the logits inside the layer and by moe_route: the same experts, weights equal to FP32, so outputs that differ
    by a BF16 step at most where they differ."""
    layer = Layer(bsq, "nvfp4", 288, 256, 33, seed=5)
    x, _, z = layer.inputs(20, 6)
    z = torch.from_numpy(z).cuda()
    for renormalize in (True, False):
        inside = bsq.moe_layer(x, z, *layer.args, "nvfp4", 4, renormalize=renormalize, **layer.kw)
        routed = bsq.moe_layer(x, None, *layer.args, "nvfp4", 4, routing=bsq.moe_route(z, 4, renormalize=renormalize), **layer.kw)
        a, b = inside.float(), routed.float()
        # weights off by 2^-20 of themselves move the sum of the choices by 2^-20 of its parts, then one rounding to BF16
        assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 2.0 ** -16).all()
