"""The polynomials of the attention with modified scores, read from the sources and replayed on the host.

exp2_fma (attn_ex_fwd.cu): 2^x on the FMA pipe; cap_scores (attn_ex.cuh) with the factors that cap_fn
(api_ex.cu) makes of the constants in mcs_internal.h: cap log2(e) tanh(scale s / cap). The steps run in float32 with
one rounding per fused multiply-add, against double precision. e = 2^-24 is half an fp32 step.
"""
import math
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "free_sparse_attention_pddp_b200", "csrc")
E = 2.0 ** -24
F = np.float32


def fma(a, b, c):
    a, b, c = (np.asarray(x, F).astype(np.float64) for x in (a, b, c))
    return (a * b + c).astype(F)


def round_down(x):
    y = x.astype(F)
    return np.where(y.astype(np.float64) > x, np.nextafter(y, F(-np.inf)), y).astype(F)


def exp2_coefficients():
    body = open(os.path.join(CSRC, "attn_ex_fwd.cu")).read()
    body = body[body.index("void exp2_fma("):]
    body = body[:body.index("\n}\n")]
    c = [F(x) for x in re.findall(r"f2_pack\(([0-9.]+)f, \1f\)", body)]
    assert c[0] == F(12582912.0) and len(c) == 7
    return c[1:]  # highest degree first


def exp2_fma(x):
    x = np.asarray(x, F)
    x = np.where(np.isnan(x), x, np.maximum(x, F(-127)))
    with np.errstate(invalid="ignore"):
        t = round_down(x.astype(np.float64) + 12582912.0)
        r = (x + (F(12582912.0) - t)).astype(F)
        c = exp2_coefficients()
        p = fma(c[0], r, c[1])
        for k in c[2:]:
            p = fma(p, r, k)
        n = ((t.view(np.uint32) << np.uint32(23)) + np.uint32(0x3f800000)).view(F)
        return (p * n).astype(F)


def test_exp2_error():
    """The polynomial 9.5e-8 on [0, 1]; its last step rounds by e, the one before by e / 2 and the others by less than e / 4
    together, the fraction by e / 2 times ln 2."""
    r = np.linspace(0, 1, 1_000_001)
    p = np.zeros_like(r)
    for c in exp2_coefficients():
        p = p * r + float(c)
    assert np.abs(p / np.exp2(r) - 1).max() < 9.5e-8
    x = np.concatenate([np.linspace(-126, 4, 1_000_001), -np.logspace(-12, 2, 10_001)]).astype(F)
    rel = np.abs(exp2_fma(x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1)
    assert rel.max() < 9.5e-8 + (1 + 0.5 + 0.25 + 0.35) * E


def test_exp2_ends():
    whole = np.arange(-126, 5).astype(F)
    assert np.array_equal(exp2_fma(whole), np.exp2(whole.astype(np.float64)).astype(F))
    assert np.all(exp2_fma(np.array([-126.5, -127, -1e5, -np.inf], F)) == 0)
    assert np.isnan(exp2_fma(np.array([np.nan, -np.nan], F))).all()


def tanh_constants():
    src = open(os.path.join(CSRC, "mcs_internal.h")).read()
    return [float(F(re.search(rf"kTanh{n} = (-?[0-9.]+)f", src).group(1))) for n in ("P0", "P1", "P2", "P3", "R0", "R1", "R2")]


def cap_fn(scale, cap):
    """The library's factors: pre, k, and the coefficients of both polynomials."""
    P0, P1, P2, P3, R0, R1, R2 = tanh_constants()
    ratio, cl = float(F(scale)) / float(F(cap)), float(F(cap)) * 1.4426950408889634074

    def coefficients(k):
        return [[c * cl * k ** (2 * i + 1) for i, c in enumerate(cs)] for cs in ((1.0, P0, P1, P2, P3), (1.0, R0, R1, R2))]

    pre = 1.0
    normal = all(2.0 ** -126 <= abs(c) < 2.0 ** 128 for c in coefficients(ratio)[0])
    if not normal or (0.625 / ratio) ** 2 >= 2.0 ** 128:
        pre = 2.0 ** (math.floor(math.log2(ratio)) + 1)
    a, b = coefficients(ratio / pre)
    assert all(2.0 ** -126 <= abs(c) < 2.0 ** 128 for c in a + b)
    return pre, ratio / pre, cl, [F(c) for c in a], [F(c) for c in b]


def poly_cap(x, coefficients):
    z = (x * x).astype(F)
    q = np.full_like(x, coefficients[-1])
    for c in coefficients[-2::-1]:
        q = fma(q, z, c)
    return (x * q).astype(F)


@pytest.mark.parametrize("scale,cap", [(0.125, 30.0), (128 ** -0.5, 50.0), (1.0, 5.0), (0.125, 0.5), (0.125, 1e5), (1e-4, 1000.0),
                                       (1e-12, 1e6), (1e12, 1e6), (1e12, 1e-6), (1.0, 1e20), (1e-12, 1e20)])
def test_cap_error(scale, cap):
    """Both polynomials are within 1.3e-7 of tanh where they are used; their factors, z, the steps and the last product
    round by e each, of which the steps before the last count at most half. Beyond, 2 / (1 + y) with y = 2^(2 |x| log2 e) is
    off by at most 0.35 of y's relative error (e of an argument of 1.8 or less where y matters, and e) and its own
    rounding, e, beside a value of 0.55 or more."""
    pre, k, cl, a, b = cap_fn(scale, cap)
    for coefficients, top in ((b, 0.4), (a, 0.625)):
        s = (np.linspace(-top, top, 200_000) / (k * pre) * (1 - 1e-6)).astype(F)
        want = cl * np.tanh(k * pre * s.astype(np.float64))
        got = poly_cap((s * F(pre)).astype(F), coefficients).astype(np.float64)
        assert np.abs(got / want - 1).max() < 1.3e-7 + 4.5 * E
    s = (np.linspace(0.625, 12, 200_000) / (k * pre)).astype(F)
    x = (s * F(pre)).astype(F)
    y = np.exp2((x * F(2 * k * 1.4426950408889634074)).astype(np.float64)).astype(F)
    r = (1 / (F(1) + y)).astype(F)
    got = fma(F(-2) * F(cl), r, F(cl))
    want = cl * np.tanh(k * pre * s.astype(np.float64))
    assert np.abs(got.astype(np.float64) / want - 1).max() < (0.35 * (1.8 + 1) + 1 + 1 + 1) / 0.55 * E
    # t^2 - 1 for the gradients: t rounds twice, which counts double in its square, and the sum once
    t = (got * F(1 / cl)).astype(F)
    slope = fma(t, t, F(-1)).astype(np.float64)
    assert np.abs(slope - ((got.astype(np.float64) / cl) ** 2 - 1)).max() < 5 * E
