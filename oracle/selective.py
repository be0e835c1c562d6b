"""Selective state space scan -- TEST INFRASTRUCTURE (float64, numpy).

Only ``tests/`` may use this module; nothing on the CUDA side shares code with
it.  Per sequence, channel c of group g and state n, token by token, with
D_t = softplus(delta_t + delta_bias):

    h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t B_t[g, n] x_t
    y_t = sum_n C_t[g, n] h_t[n] + skip x_t,  out_t = y_t silu(gate_t)

and the gradients of L = sum(d_out * out) + sum(d_final * final) by the adjoint
recurrence g_t = C_t dy_t + a_{t+1} g_{t+1}.

Parity status: pinned by ``tests/test_oracle_state_space.py`` against the
unrolled sum over earlier tokens, finite differences and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import to_f64
from .conv import silu


def softplus(u):
    """log(1 + exp(u)) and its derivative."""
    return np.logaddexp(u, 0.0), 1 / (1 + np.exp(-u))


def _inputs(x, delta, A, B, C, delta_bias, skip, gate):
    x, delta, A, B, C = (to_f64(v) for v in (x, delta, A, B, C))
    W = x.shape[1]
    bias = np.zeros(W) if delta_bias is None else to_f64(delta_bias)
    per = np.arange(W) // (W // B.shape[1])  # the group of a channel
    return (x, *softplus(delta + bias), A, B[:, per], C[:, per], np.zeros(W) if skip is None else to_f64(skip),
            None if gate is None else to_f64(gate))


def forward(x, delta, A, B, C, cu_seqlens, delta_bias=None, skip=None, gate=None, initial_state=None) -> dict:
    """x, delta, gate [T, W], A [W, N], B, C [T, G, N]; returns out, y [T, W]
    (NaN in rows of no sequence), before [T, W, N] (the state ahead of each
    token) and final_state [S, W, N]."""
    x, d, _, A, B, C, skip, z = _inputs(x, delta, A, B, C, delta_bias, skip, gate)
    S, (W, N) = len(cu_seqlens) - 1, A.shape
    y, before = np.full_like(x, np.nan), np.full(x.shape + (N,), np.nan)
    final = np.zeros((S, W, N)) if initial_state is None else to_f64(initial_state).copy()
    for q in range(S):
        h = final[q].copy()
        for t in range(cu_seqlens[q], cu_seqlens[q + 1]):
            before[t] = h
            h = np.exp(d[t][:, None] * A) * h + (d[t] * x[t])[:, None] * B[t]
            y[t] = (C[t] * h).sum(1) + skip * x[t]
        final[q] = h
    return {"out": y if z is None else y * silu(z)[0], "y": y, "before": before, "final_state": final}


def backward(x, delta, A, B, C, cu_seqlens, d_out, delta_bias=None, skip=None, gate=None, initial_state=None,
             d_final_state=None) -> dict:
    """Returns dx, d_delta, d_gate [T, W], d_B, d_C [T, G, N] (NaN in rows of no
    sequence), d_A, d_delta_bias, d_skip and d_initial_state."""
    f = forward(x, delta, A, B, C, cu_seqlens, delta_bias, skip, gate, initial_state)
    G = np.shape(B)[1]
    x, d, slope, A, B, C, skip, z = _inputs(x, delta, A, B, C, delta_bias, skip, gate)
    dy = to_f64(d_out)
    S, (W, N) = len(cu_seqlens) - 1, A.shape
    d_gate = None
    if z is not None:
        s, ds = silu(z)
        d_gate, dy = dy * f["y"] * ds, dy * s
    nan = np.full_like(x, np.nan)
    dx, dd = nan.copy(), nan.copy()
    dB, dC = np.full((len(x), G, N), np.nan), np.full((len(x), G, N), np.nan)
    dA, d_skip, d_bias = np.zeros_like(A), np.zeros(W), np.zeros(W)
    d_init = np.zeros((S, W, N)) if d_final_state is None else to_f64(d_final_state).copy()
    for q in range(S):
        e = d_init[q].copy()
        for t in range(cu_seqlens[q + 1] - 1, cu_seqlens[q] - 1, -1):
            a, h0 = np.exp(d[t][:, None] * A), f["before"][t]
            h = a * h0 + (d[t] * x[t])[:, None] * B[t]
            g = C[t] * dy[t][:, None] + e
            dC[t] = (dy[t][:, None] * h).reshape(G, W // G, N).sum(1)
            dB[t] = (g * (d[t] * x[t])[:, None]).reshape(G, W // G, N).sum(1)
            Bg = (B[t] * g).sum(1)
            dx[t] = skip * dy[t] + d[t] * Bg
            dd[t] = (x[t] * Bg + (A * g * a * h0).sum(1)) * slope[t]
            dA += d[t][:, None] * g * a * h0
            d_skip += dy[t] * x[t]
            d_bias += dd[t]
            e = a * g
        d_init[q] = e
    return {"dx": dx, "d_delta": dd, "d_gate": d_gate, "d_A": dA, "d_B": dB, "d_C": dC, "d_delta_bias": d_bias,
            "d_skip": d_skip, "d_initial_state": d_init}
