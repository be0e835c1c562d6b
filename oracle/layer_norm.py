"""Layer norm with the residual stream -- TEST INFRASTRUCTURE (float64, numpy).

Only ``tests/`` may use this module; nothing on the CUDA side shares code with
it.  Per token, r' = x + residual and

    out = (r' - mean r') / sqrt(mean (r' - mean r')^2 + eps) * weight + bias

Parity status: pinned by ``tests/test_oracle_state_space.py`` against rows of
known moments, finite differences and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import to_f64


def _norm(r, eps):
    d = r - r.mean(1, keepdims=True)
    rstd = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return d * rstd, rstd


def forward(x, weight=None, bias=None, residual=None, eps=1e-5) -> dict:
    r = to_f64(x) if residual is None else to_f64(x) + to_f64(residual)
    hat, _ = _norm(r, eps)
    out = hat if weight is None else hat * to_f64(weight)
    return {"out": out if bias is None else out + to_f64(bias), "residual_out": r, "hat": hat}


def backward(r, weight, d_out, d_residual_out=None, eps=1e-5) -> dict:
    """At r, the residual stream behind the sum.  Returns dx, d_weight, d_bias."""
    r, dy = to_f64(r), to_f64(d_out)
    hat, rstd = _norm(r, eps)
    p = dy if weight is None else dy * to_f64(weight)
    dx = rstd * (p - p.mean(1, keepdims=True) - hat * (p * hat).mean(1, keepdims=True))
    return {"dx": dx if d_residual_out is None else dx + to_f64(d_residual_out), "d_weight": (dy * hat).sum(0),
            "d_bias": dy.sum(0)}
