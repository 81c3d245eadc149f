"""The polynomial that stands for tanh near 0, as the kernels' header gives it."""

import os
import re

import numpy as np

import attention_distillation_kl_gb300 as skl


def test_the_polynomials_error():
    text = open(os.path.join(os.path.dirname(skl.__file__), "csrc", "mod_common.cuh")).read()
    body = re.search(r"constexpr float tanh_p\(int k\) \{(.*?)\}", text, re.S).group(1)
    p = [float(c) for c in re.findall(r"(-?\d+\.\d+)f", body)]
    most = float(re.search(r"constexpr float kTanhMax = ([0-9.]+)f", text).group(1))
    assert len(p) == 5 and most == 0.5
    u = np.linspace(0.0, most, 1_000_001)[1:]
    for coef in (p, [float(np.float32(c)) for c in p]):
        err = np.abs(u * np.polynomial.polynomial.polyval(u * u, coef) / np.tanh(u) - 1).max()
        # half of fp32's own rounding; the comment beside the constants says 2.9e-8
        assert err < 2.9e-8 < 2.0 ** -25
