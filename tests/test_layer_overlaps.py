"""Outputs that share bytes with what a call reads, or with another output, are
refused; views that lie between one another are not.  On the CPU: a call that
passes the checks ends where a device is looked for."""
import random

import pytest
import torch

P = 0x100000
OK, NULL, SHAPE, ALIGN, VALUE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def bsq():
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would run")
    from fp8_activation_quantization_bsq_gb300 import _build
    _build.build()
    import fp8_activation_quantization_bsq_gb300 as m
    return m


def passed(code):
    return code not in (OK, NULL, SHAPE, ALIGN, VALUE)


def rope(bsq, tokens, heads, kv_heads, dim, q, k, qo, ko, pos=P << 8, freq=P << 9, qw=P << 10, kw=P << 11, wd=0):
    """q, k, qo, ko: (address, token stride, head stride)."""
    return bsq.lib().bsq_qk_norm_rope(0, *q, *k, tokens, heads, kv_heads, dim, pos, freq, dim // 2, 0, qw, kw, wd, 1e-6, *qo, *ko, None)


@pytest.mark.parametrize("change,refused", [
    (dict(), False),                                                             # both in place, in one projection's output
    (dict(qo=(P + 128, 768, 64)), True),                                         # a head further
    (dict(qo=(P + 1536, 768, 64)), True),                                        # a token further
    (dict(ko=(P + 2 * 448, 768, 64)), True),                                     # into the queries
    (dict(qo=(P + 2 * 128, 768, 64)), True),                                     # into the keys too
    (dict(ko=(P + 2 * 640, 768, 64)), False),                                    # where the values are
    (dict(ko=(P + 2 * 576, 768, 64)), True),                                     # half there
    (dict(qo=(8 * P, 512, 64), ko=(8 * P + 2 * 448, 512, 64)), True),            # outputs into one another
    (dict(qo=(8 * P, 640, 64), ko=(8 * P + 2 * 512, 640, 64)), False),
    (dict(qo=(8 * P, 640, 64), ko=(8 * P + 2 * 504, 640, 64)), True),
    (dict(qo=(8 * P, 64, 64 * 20), ko=(8 * P + 2 * 64 * 160, 64, 64 * 20)), False),  # (heads, tokens, dim)
    (dict(qo=(8 * P, 64, 64 * 20), ko=(8 * P + 2 * 64 * 159, 64, 64 * 20)), True),
    (dict(qo=(8 * P, 2048, 256), ko=(8 * P + 2 * 64, 2048, 256)), False),        # keys between the queries
    (dict(qo=(8 * P, 2048, 256), ko=(8 * P + 2 * 32, 2048, 256)), True),
    (dict(pos=P + 64), True), (dict(freq=P + 1536), True), (dict(qw=P + 2 * 512), True), (dict(kw=P), True),
    (dict(pos=P + 2 * 640), False),                                              # in front of the values: 20 positions
    (dict(qw=P + 2 * 640 - 64), True), (dict(kw=P + 2 * 720, wd=2), True), (dict(kw=P + 2 * 640, wd=2), False)])
def test_rope_overlaps(bsq, change, refused):
    call = dict(tokens=20, heads=8, kv_heads=2, dim=64, q=(P, 768, 64), k=(P + 2 * 512, 768, 64), qo=(P, 768, 64), ko=(P + 2 * 512, 768, 64))
    got = rope(bsq, **{**call, **change})
    assert got == VALUE if refused else passed(got)


@pytest.mark.parametrize("qo,code", [((8 * P, 512, 64), None), ((8 * P, 448, 64), SHAPE), ((8 * P, 64, 64), SHAPE), ((8 * P, 64, 1280), None),
                                     ((8 * P, 64, 1216), SHAPE), ((8 * P, 128, 64), SHAPE), ((8 * P, 72, 1440), None), ((8 * P, 768, 128), SHAPE)])
def test_rope_rows_of_an_output_in_one_another(bsq, qo, code):
    got = rope(bsq, 20, 8, 2, 64, (P, 512, 64), (4 * P, 128, 64), qo, (16 * P, 128, 64))
    assert passed(got) if code is None else got == code


def test_rope_overlaps_by_counting_bytes(bsq):
    """Small calls of random strides and places against the sets of bytes themselves.  Where token or head strides differ a call may be
    refused that shares none."""
    rng = random.Random(1)
    dim, counts = 8, {True: 0, False: 0}
    for _ in range(20000):
        tokens, n = rng.randint(1, 4), (rng.randint(1, 4), rng.randint(1, 4))
        same = rng.random() < 0.7
        strides = (8 * rng.randint(0, 16), 8 * rng.randint(0, 16))
        place = lambda: (P + 16 * rng.randint(0, 100), *(strides if same else (8 * rng.randint(0, 16), 8 * rng.randint(0, 16))))  # noqa: E731
        ins = [place(), place()]
        outs = [ins[i] if rng.random() < 0.4 else place() for i in range(2)]
        rows = lambda v, heads: [v[0] + 2 * (t * v[1] + h * v[2]) for t in range(tokens) for h in range(heads)]  # noqa: E731
        of = lambda v, heads: {b for r in rows(v, heads) for b in range(r // 16, r // 16 + dim // 8)}  # noqa: E731  (all are multiples of 16 bytes)
        got = rope(bsq, tokens, *n, dim, *ins, *outs)
        if any(len(of(outs[i], n[i])) < tokens * n[i] * dim // 8 for i in range(2)):
            assert got in (SHAPE, VALUE)
            continue
        clash = bool(of(outs[0], n[0]) & of(outs[1], n[1]))
        for i in range(2):
            itself = rows(outs[i], n[i]) == rows(ins[i], n[i])
            clash |= not itself and bool(of(outs[i], n[i]) & of(ins[i], n[i]))
            clash |= bool(of(outs[i], n[i]) & of(ins[1 - i], n[1 - i]))
        if clash:
            assert got == VALUE, (tokens, n, ins, outs)
        elif same:
            assert passed(got), (tokens, n, ins, outs, got)
        else:
            assert passed(got) or got == VALUE
        counts[clash] += 1
    assert min(counts.values()) > 300


ROUTE = dict(dtype=2, z=P, ld=64, tokens=3, experts=64, top_k=4, sigmoid=0, bias=2 * P, groups=8, top_groups=2, group_top=2, renorm=1, scale=1.0,
             ids=3 * P, weights=4 * P, stream=None)


@pytest.mark.parametrize("change,refused", [
    (dict(), False), (dict(ids=P), True), (dict(weights=P + 3 * 256 - 4), True), (dict(weights=P + 3 * 256), False), (dict(ids=P - 48), False),
    (dict(ids=P - 44), True), (dict(ids=2 * P + 252), True), (dict(ids=2 * P + 256), False), (dict(weights=3 * P), True), (dict(weights=3 * P + 44), True),
    (dict(weights=3 * P + 48), False), (dict(ids=4 * P + 4), True), (dict(bias=None, ids=2 * P), False), (dict(dtype=0, ids=P + 384), False),
    (dict(dtype=0, ids=P + 380), True), (dict(ld=128, ids=P + 256), False), (dict(ld=128, ids=P + 468), True), (dict(tokens=1, ld=0, ids=P + 256), False)])
def test_route_overlaps(bsq, change, refused):
    got = bsq.lib().bsq_moe_route(*{**ROUTE, **change}.values())
    assert got == VALUE if refused else passed(got)


ROWS = dict(ids=P, tokens=3, top_k=2, experts=5, ro=2 * P, so=3 * P, idx=4 * P, pos=5 * P, stream=None)


@pytest.mark.parametrize("change,refused", [
    (dict(), False), (dict(ro=P), True), (dict(ro=P + 20), True), (dict(ro=P + 24), False), (dict(so=P - 20), True), (dict(so=P - 24), False),
    (dict(idx=P), True), (dict(pos=P), True), (dict(so=2 * P + 20), True), (dict(so=2 * P + 24), False), (dict(idx=2 * P + 4), True),
    (dict(pos=3 * P - 4), True), (dict(pos=4 * P + 20), True), (dict(pos=4 * P + 24), False), (dict(tokens=0, ids=2 * P), False),
    (dict(tokens=0, so=2 * P), True)])
def test_rows_overlaps(bsq, change, refused):
    got = bsq.lib().bsq_moe_rows(*{**ROWS, **change}.values())
    assert got == VALUE if refused else passed(got)


LINEAR = dict(fmt=0, dtype=0, x=P, tokens=3, cols=64, ld_x=64, w=2 * P, ws=3 * P, rows=100, sf=4 * P, add=None, ld_add=0, out_dtype=0, out=8 * P,
              ld_out=256, stream=None)


@pytest.mark.parametrize("change,refused", [
    (dict(add=8 * P + 512 - 200), False),                       # a bias between the rows of an output
    (dict(add=8 * P + 200), False), (dict(add=8 * P + 512 - 198), True), (dict(add=8 * P + 198), True), (dict(add=8 * P + 512), True),
    (dict(add=8 * P + 1024 + 200), False), (dict(add=8 * P + 200, ld_add=256), False), (dict(add=8 * P + 198, ld_add=256), True),
    (dict(add=8 * P + 200, ld_add=200), True), (dict(add=8 * P, ld_add=256), False), (dict(tokens=1, add=8 * P + 200, ld_add=7), False),
    (dict(x=8 * P + 208, ld_x=256), False), (dict(x=8 * P + 192, ld_x=256), True)])
def test_linear_overlaps(bsq, change, refused):
    got = bsq.lib().bsq_packed_linear(*{**LINEAR, **change}.values())
    assert got == VALUE if refused else passed(got)
