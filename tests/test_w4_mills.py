"""The polynomial behind the normal distribution function (csrc/cq_w4.cuh): its coefficients
as the kernel has them, against erfc, on the CPU."""
import math
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "minimax_scale_search_b200", "csrc")


def test_ratio_of_mills():
    with open(os.path.join(CSRC, "cq_w4.cuh")) as f:
        body = f.read().split("float normal_distribution(float z")[1].split("return")[0]
    c = [np.float32(v) for v in re.findall(r"float m = ([-\d.]+)f|fmaf\(m, t, ([-\d.]+)f\)", body) for v in v if v]
    assert len(c) == 8
    z = np.linspace(0, 14, 28001)
    ratio = np.array([math.sqrt(math.pi / 2) * math.exp(v * v / 2) * math.erfc(v / math.sqrt(2)) for v in z])
    t = 1 / (1 + np.float64(np.float32(0.3)) * z)
    m = np.full_like(t, c[0])
    for k in c[1:]:
        m = m * t + np.float64(k)
    assert np.max(np.abs(m * t / ratio - 1)) < 2.1e-7
    # each step rounded to fp32, as the kernel has it (a step in fp64 is exact to 2^-53, then rounded once: an fma)
    z = z.astype(np.float32)
    t = np.float32(1) / (np.float32(1) + np.float32(0.3) * z)
    m = np.full_like(t, c[0])
    for k in c[1:]:
        m = (m.astype(np.float64) * t + np.float64(k)).astype(np.float32)
    ratio = np.array([math.sqrt(math.pi / 2) * math.exp(v * v / 2) * math.erfc(v / math.sqrt(2)) for v in z.astype(np.float64)])
    assert np.max(np.abs((m * t).astype(np.float64) / ratio - 1)) < 2.0 ** -22 + 2.0 ** -21
