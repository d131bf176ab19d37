"""The normal distribution function's tail as the feed-forward kernels form it (mhcm_ffn.cuh): its
polynomial, with the constants as they are rounded there, stays within what its comment says (no GPU
needed)."""
import os
import re

import numpy as np
import pytest

erfcx = pytest.importorskip("scipy.special").erfcx
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rms_backward_gb300", "csrc", "mhcm_ffn.cuh")


def _source():
    """(the factor of |g|, the coefficients from the highest, the two figures of the comment)"""
    text = open(HEADER).read()
    body = text[text.index("float normal_tail("):text.index("return 0.5f * e")]
    coefficients = [np.float32(v) for v in re.findall(r"(?:float p = |t, )(-?[\d.]+)f", body)]
    factor = np.float32(re.search(r"([\d.]+)f \* fabsf", body).group(1))
    figures = re.search(r"off by ([\d.e-]+) of it at most \(in FP32 arithmetic\s*(?://)?\s*([\d.e-]+)\)", text)
    assert len(coefficients) == 9 and factor in (np.float32("0.28284271"), np.float32(0.4 / 2 ** 0.5)), "as the source is read"
    return factor, coefficients, tuple(map(float, figures.groups()))


# |g| up to where exp(-g^2 / 2) is zero in FP32
G = np.linspace(0.0, 14.5, 2000001)


def test_polynomial_is_as_near_as_its_comment_says():
    factor, coefficients, (exact, _) = _source()
    t = 1.0 / (1.0 + float(factor) * G)
    p = np.zeros_like(t)
    for c in coefficients:
        p = p * t + float(c)
    assert abs(p * t / erfcx(G / 2 ** 0.5) - 1.0).max() <= exact


def test_polynomial_in_fp32_is_as_near_as_its_comment_says():
    """Each operation rounded to FP32 (the multiply-adds once, as formed in FP64)."""
    factor, coefficients, (_, single) = _source()
    g = G.astype(np.float32)
    t = np.float32(1) / (1.0 + np.float64(factor) * g).astype(np.float32)
    p = np.full_like(t, coefficients[0])
    for c in coefficients[1:]:
        p = (p.astype(np.float64) * t + np.float64(c)).astype(np.float32)
    assert abs((p * t).astype(np.float64) / erfcx(g.astype(np.float64) / 2 ** 0.5) - 1.0).max() <= single
