"""Gated linear recurrence -- TEST INFRASTRUCTURE (float64, numpy).

Only ``tests/`` may use this module; nothing on the CUDA side shares code with
it.  Per sequence and channel, token by token, with a_t = exp(log_gate_t):

    h_t = a_t h_{t-1} + s(a_t) x_t
    s = 1 ("plain"), 1 - a ("complement") or sqrt(1 - a^2) ("unit")

and the gradients of L = sum(d_out * h) + sum(d_final * h_T) by the adjoint
recurrence dh_t = d_out_t + a_{t+1} dh_{t+1}.

Parity status: pinned by ``tests/test_oracle_scan.py`` against the unrolled
sum over earlier tokens, finite differences and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import to_f64


def input_scale(la, mode):
    """s(a) and its derivative in log_gate (zero where "unit" has none)."""
    if mode == "plain":
        return np.ones_like(la), np.zeros_like(la)
    if mode == "complement":
        return -np.expm1(la), -np.exp(la)
    s = np.sqrt(-np.expm1(2 * la))
    safe = np.where(s > 0, s, 1.0)
    return s, np.where(s > 0, -np.exp(2 * la) / safe, 0.0)


def forward(x, log_gate, cu_seqlens, mode, initial_state=None) -> dict:
    """x, log_gate [T, W]; returns out [T, W] (NaN in rows of no sequence),
    before [T, W] (the state ahead of each token) and final_state [S, W]."""
    x, la = to_f64(x), to_f64(log_gate)
    S, W = len(cu_seqlens) - 1, x.shape[1]
    out, before = np.full_like(x, np.nan), np.full_like(x, np.nan)
    final = np.zeros((S, W)) if initial_state is None else to_f64(initial_state).copy()
    a, (s, _) = np.exp(la), input_scale(la, mode)
    for b in range(S):
        h = final[b].copy()
        for t in range(cu_seqlens[b], cu_seqlens[b + 1]):
            before[t] = h
            h = a[t] * h + s[t] * x[t]
            out[t] = h
        final[b] = h
    return {"out": out, "before": before, "final_state": final}


def backward(x, log_gate, cu_seqlens, mode, d_out, initial_state=None, d_final_state=None) -> dict:
    """Returns dx, d_log_gate [T, W] (NaN in rows of no sequence), d_initial_state [S, W]."""
    f = forward(x, log_gate, cu_seqlens, mode, initial_state)
    x, la, dy = to_f64(x), to_f64(log_gate), to_f64(d_out)
    S, W = len(cu_seqlens) - 1, x.shape[1]
    dx, dla = np.full_like(x, np.nan), np.full_like(x, np.nan)
    d_init = np.zeros((S, W)) if d_final_state is None else to_f64(d_final_state).copy()
    a, (s, ds) = np.exp(la), input_scale(la, mode)
    for b in range(S):
        e = d_init[b].copy()
        for t in range(cu_seqlens[b + 1] - 1, cu_seqlens[b] - 1, -1):
            dh = dy[t] + e
            dx[t] = s[t] * dh
            dla[t] = dh * (a[t] * f["before"][t] + ds[t] * x[t])
            e = a[t] * dh
        d_init[b] = e
    return {"dx": dx, "d_log_gate": dla, "d_initial_state": d_init}
