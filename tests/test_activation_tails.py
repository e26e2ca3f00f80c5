"""The activations where their value is a small part of x: the oracle's forms keep
relative accuracy there, and so does the erf-GELU polynomial of the dense layers'
epilogue, replayed in float32 from the source (csrc/wave_dense.cuh)."""
import math
import os
import re

import numpy as np
import pytest

from oracle import token as otok

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "block_causal_attention_wave_b200", "csrc", "wave_dense.cuh")


@pytest.mark.parametrize("x", [-0.5, -3.0, -5.5, -8.0, -12.0])
def test_oracle_keeps_the_tails(x):
    """Against the continued fraction of erfc, and against exp(-2u) alone, from
    which 1 / (1 + e^(2u)) differs by less than e^(-2u)."""
    z = -x / math.sqrt(2.0)
    frac = z
    for k in range(4000, 0, -1):
        frac = z + k / 2.0 / frac
    want = 0.5 * x * math.exp(-z * z) / math.sqrt(math.pi) / frac
    assert abs(otok.activation(x, "gelu_erf") / want - 1) < 1e-9
    u = math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
    assert abs(otok.activation(x, "gelu_tanh") / (x * math.exp(2 * u)) - 1) <= math.exp(2 * u) + 1e-12
    assert otok.activation(np.array([-1e4, 1e4]), "gelu_tanh").tolist() == [0.0, 1e4]
    assert otok.activation(np.array([-1e4, 1e4]), "gelu_erf").tolist() == [0.0, 1e4]


def test_erf_gelu_polynomial():
    text = open(SRC).read()
    body = text[text.index("if constexpr (ACT == WAVE_ACT_GELU_ERF)"):text.index("const float h = ")]
    first = re.search(r"float e = fmaf\(([-0-9.]+)f, t, ([-0-9.]+)f\)", body)
    coeffs = [np.float32(v) for v in first.groups()]
    coeffs += [np.float32(v) for v in re.findall(r"e = fmaf\(e, t, ([-0-9.]+)f\)", body)]
    slope = [np.float32(v) for v in re.search(r"fmaf\(([0-9.]+)f \* ([0-9.]+)f, fabsf\(x\), 1.f\)", body).groups()]
    x = np.linspace(0.0, 13.2, 200001).astype(np.float32)
    t = np.float32(1) / (slope[0] * slope[1] * x + np.float32(1))
    e = np.full_like(x, coeffs[0])
    for c in coeffs[1:]:
        e = e * t + c
    w = x * x * np.float32(-0.7213475204)
    got = (e * t).astype(np.float64) * np.exp2(w.astype(np.float64))
    want = np.array([math.erfc(v / math.sqrt(2.0)) for v in x.astype(np.float64)])
    # the exponent's two roundings: 2 * 2^-24 of at most 126, times ln 2, and the fit's 2^-20
    assert np.abs(got / want - 1).max() <= 2.0 ** -16
