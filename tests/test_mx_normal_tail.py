"""The polynomial of the normal distribution's tail, read from the kernels' source, against its definition in 64 bits."""
import os
import re

import numpy as np
import pytest

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
HEADER = os.path.join(os.path.dirname(fp4.__file__), "csrc", "mx_epilogue.h")


def test_the_fit_is_as_near_as_stated():
    from scipy.special import erfcx
    text = open(HEADER).read()
    body = text[text.index("normal_tail(float z"):]
    body = body[:body.index("return")]
    slope = [float(v) for v in re.search(r"1\.0f \+ \(([\d.]+)f \* ([\d.]+)f\)", body).groups()]
    signs, sizes = zip(*re.findall(r"p = (?:p \* t )?([-+] )?-?0\.5f \* ([\d.]+)f;", body))
    assert len(sizes) == 8 and body.count("-0.5f * ") == 2              # the first coefficient, and the exponential's
    coefficients = [float(v) * (-0.5 if s == "- " or not i else 0.5) for i, (s, v) in enumerate(zip(signs, sizes))]
    stated = float(re.search(r"weights: ([\d.]+e-7) off at most", text).group(1))
    z = np.linspace(0, 10.5 * np.sqrt(2), 400_001)
    want = erfcx(z / np.sqrt(2)) / 2                                      # the tail over exp(-z^2 / 2)
    for to in (np.float64, np.float32):                                  # as written, and as FP32 holds the constants
        t = 1 / (1 + float(to(to(slope[0]) * to(slope[1]))) * z)
        p = np.zeros_like(z)
        for c in coefficients:
            p = p * t + float(to(c))
        assert np.abs(p * t / want - 1).max() <= stated < 2 * 2.0 ** -23  # the oracle allows the fit two steps
