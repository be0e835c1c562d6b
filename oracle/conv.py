"""Short causal convolution -- TEST INFRASTRUCTURE (float64, numpy).

Only ``tests/`` may use this module; nothing on the CUDA side shares code with
it.  Per sequence and channel, with K taps and the rows before the sequence
from its state (K - 1 rows, the newest last):

    u_t = bias + sum_j weight[j] x_{t - (K - 1) + j},  out_t = act(u_t)

and the gradients of L = sum(d_out * out) + sum(d_final * final).

Parity status: pinned by ``tests/test_oracle_state_space.py`` against the
product with a banded matrix, finite differences and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import to_f64


def silu(u):
    """u sigmoid(u) and its derivative."""
    s = 1 / (1 + np.exp(-u))
    return u * s, s * (1 + u * (1 - s))


def act(u, kind):
    return silu(u) if kind == "silu" else (u, np.ones_like(u))


def forward(x, weight, cu_seqlens, bias=None, initial_state=None, kind="silu") -> dict:
    """x [T, W], weight [W, K]; returns out, pre (u) [T, W] (NaN in rows of no
    sequence), final_state [S, K - 1, W] and rows, each sequence's with its
    state in front."""
    x, w = to_f64(x), to_f64(weight)
    S, (W, K) = len(cu_seqlens) - 1, w.shape
    b = np.zeros(W) if bias is None else to_f64(bias)
    init = np.zeros((S, K - 1, W)) if initial_state is None else to_f64(initial_state)
    out, pre, final, rows = np.full_like(x, np.nan), np.full_like(x, np.nan), np.zeros((S, K - 1, W)), []
    for q in range(S):
        lo, hi = cu_seqlens[q], cu_seqlens[q + 1]
        r = np.concatenate([init[q], x[lo:hi]])
        for t in range(lo, hi):
            pre[t] = b + sum(w[:, j] * r[t - lo + j] for j in range(K))
        out[lo:hi] = act(pre[lo:hi], kind)[0]
        final[q] = r[hi - lo:]
        rows.append(r)
    return {"out": out, "pre": pre, "final_state": final, "rows": rows}


def backward(x, weight, cu_seqlens, d_out, bias=None, initial_state=None, d_final_state=None, kind="silu") -> dict:
    """Returns dx (NaN in rows of no sequence), d_weight, d_bias, d_initial_state."""
    f = forward(x, weight, cu_seqlens, bias, initial_state, kind)
    x, w, dy = to_f64(x), to_f64(weight), to_f64(d_out)
    S, (W, K) = len(cu_seqlens) - 1, w.shape
    d_fin = np.zeros((S, K - 1, W)) if d_final_state is None else to_f64(d_final_state)
    dx, dw, db, d_init = np.full_like(x, np.nan), np.zeros_like(w), np.zeros(W), np.zeros((S, K - 1, W))
    for q in range(S):
        lo, hi = cu_seqlens[q], cu_seqlens[q + 1]
        g = dy[lo:hi] * act(f["pre"][lo:hi], kind)[1]
        d_rows = np.zeros((K - 1 + hi - lo, W))
        d_rows[hi - lo:] += d_fin[q]
        for t in range(hi - lo):
            for j in range(K):
                d_rows[t + j] += w[:, j] * g[t]
                dw[:, j] += g[t] * f["rows"][q][t + j]
        db += g.sum(0)
        d_init[q], dx[lo:hi] = d_rows[:K - 1], d_rows[K - 1:]
    return {"dx": dx, "d_weight": dw, "d_bias": db, "d_initial_state": d_init}
