"""The series of the scan's kernels for 1 - exp(u) near 0, evaluated on the
CPU with the constants that csrc/scan.cu holds, each step rounded as the
kernel's fused multiply-add and product round."""
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_state_linear_router_gb300",
                   "csrc", "scan.cu")


def _coefficients():
    """Those of bf16 and of float32 gates, from the highest power on."""
    text = open(SRC).read()
    body = text[text.index("one_minus_exp_near0(typename"):]
    body = body[:body.index("\n}")]
    low, high = body.split("return mul2(p, u);")[:2]
    number = r"splat\((-?[0-9.]+)f\)"
    return [np.float32(v) for v in re.findall(number, low)], [np.float32(v) for v in re.findall(number, high)]


@pytest.mark.parametrize("which,degree,exactly,rounded", [(0, 4, 1.05e-7, 1.9e-7), (1, 5, 3.2e-9, 1.0e-7)],
                         ids=["bf16", "float32"])
def test_relative_error(which, degree, exactly, rounded):
    """The bounds that the comment at the series states."""
    co = _coefficients()[which]
    assert len(co) == degree + 1
    u = -np.concatenate([np.linspace(1e-6, 0.5, 400001), 2.0 ** np.linspace(-100, -1, 100001)]).astype(np.float32)
    wide = u.astype(np.float64)
    want = -np.expm1(wide)
    exact, p = np.full_like(wide, co[0]), np.full_like(u, co[0])
    for c in co[1:]:
        exact = exact * wide + np.float64(c)
        p = (p.astype(np.float64) * wide + np.float64(c)).astype(np.float32)
    p = (p.astype(np.float64) * wide).astype(np.float32)
    assert np.abs(exact * wide / want - 1).max() < exactly
    assert np.abs(p / want - 1).max() < rounded
