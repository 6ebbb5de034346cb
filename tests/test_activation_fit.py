"""The committed polynomial behind gelu's normal distribution against erfc (CPU)."""

import math
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_fp8_grouped_amd", "csrc",
                      "activation.h")


def test_normal_cdf_polynomial():
    """g(t) = e^(t^2/2) erfc(t / sqrt 2) / 2 within 5.8e-8 of itself for t in [0, 14], in exact arithmetic on the FP32
    coefficients (float64 adds less than 1e-13: t^2 / 2 roundings of the exponentials)."""
    with open(SOURCE) as f:
        body = f.read().split("float normal_cdf(float z)")[1].split("return z < 0.0f")[0]
    scale = float(np.float32(re.search(r"fmaf\(([\d.]+)f, t, 1\.0f\)", body)[1]))
    coefficients = [float(np.float32(c)) for c in re.findall(r"float p = (-?[\d.e-]+)f;", body)
                    + re.findall(r"p = fmaf\(p, u, (-?[\d.e-]+)f\)", body)]
    assert len(coefficients) == 9
    t = np.linspace(0.0, 14.0, 70001)
    p = np.polyval(coefficients, 1.0 / (1.0 + scale * t))
    g = np.array([math.exp(v * v / 2.0) * math.erfc(v / math.sqrt(2.0)) / 2.0 for v in t])
    assert np.abs(p / g - 1.0).max() <= 5.8e-8
