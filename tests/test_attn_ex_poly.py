"""The polynomials of the attention with modified scores, read from the sources and replayed on the host.

exp2_fma (attn_ex_fwd.cu): 2^x on the FMA pipe. The steps run in float32 with one rounding per fused multiply-add,
against double precision. e = 2^-24 is half an fp32 step.
"""
import os
import re

import numpy as np

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
