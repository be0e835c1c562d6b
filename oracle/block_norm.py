"""Norms before and after a block -- TEST INFRASTRUCTURE (float64, numpy).

Only ``tests/`` may use this module; nothing on the CUDA side shares code with
it.  With RMS_G(u; w) = w u / sqrt(mean of u^2 over each G columns + eps):

    r' = residual_scale r + branch_scale c act(z) RMS_group(o; w_after)
    x' = RMS_width(r'; w_before)

each part optional; the gradients by the chain rule, the norm before taken at
the residual_out it is given.

Parity status: pinned by ``tests/test_oracle_block_norm.py`` against closed
forms, finite differences and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import to_f64


def act(z, gate):
    """act(z) and its derivative."""
    if gate == "linear":
        return z, np.ones_like(z)
    sg = 1.0 / (1.0 + np.exp(-z))
    if gate == "sigmoid":
        return sg, sg * (1 - sg)
    return z * sg, sg + z * sg * (1 - sg)


def _hat(u, group, eps):
    """u / sqrt(mean of u^2 per group + eps), and that factor on every column."""
    v = u.reshape(u.shape[0], -1, group)
    f = 1.0 / np.sqrt((v * v).mean(axis=2, keepdims=True) + eps)
    return (v * f).reshape(u.shape), np.broadcast_to(f, v.shape).reshape(u.shape)


def _pull(d_hat, hat, factor, group):
    dot = (d_hat * hat).reshape(hat.shape[0], -1, group).mean(axis=2, keepdims=True)
    dot = np.broadcast_to(dot, (hat.shape[0], hat.shape[1] // group, group)).reshape(hat.shape)
    return factor * (d_hat - hat * dot)


def _opt(x):
    return None if x is None else to_f64(x)


def forward(o=None, *, z=None, r=None, w_after=None, channel=None, w_before=None, group=0, gate="none", eps=1e-6,
            residual_scale=1.0, branch_scale=1.0) -> dict:
    o, z, r, w_after, channel, w_before = (_opt(v) for v in (o, z, r, w_after, channel, w_before))
    out = 0.0
    if r is not None:
        out = out + residual_scale * r
    if o is not None:
        u = o
        if w_after is not None:
            u = _hat(o, group or o.shape[1], eps)[0] * w_after
        if z is not None:
            u = u * act(z, gate)[0]
        if channel is not None:
            u = u * channel
        out = out + branch_scale * u
    nxt = None if w_before is None else _hat(out, out.shape[1], eps)[0] * w_before
    return {"residual_out": out, "next_in": nxt}


def backward(d_residual_out=None, o=None, *, z=None, w_after=None, channel=None, w_before=None, residual_out=None,
             d_next_in=None, group=0, gate="none", eps=1e-6, residual_scale=1.0, branch_scale=1.0) -> dict:
    d, o, z, w_after, channel, w_before, at, dn = (
        _opt(v) for v in (d_residual_out, o, z, w_after, channel, w_before, residual_out, d_next_in))
    g = dict.fromkeys(("d_block_out", "d_gate", "d_residual", "d_w_after", "d_channel_scale", "d_w_before"))
    if dn is not None:
        hat, f = _hat(at, at.shape[1], eps)
        g["d_w_before"] = (dn * hat).sum(axis=0)
        pulled = _pull(dn * w_before, hat, f, at.shape[1])
        d = pulled if d is None else d + pulled
    g["d_residual"] = residual_scale * d
    if o is None:
        return g
    d = branch_scale * d
    group = group or o.shape[1]
    hat, f = _hat(o, group, eps) if w_after is not None else (o, None)
    wa = 1.0 if w_after is None else w_after
    ch = 1.0 if channel is None else channel
    av, da = (1.0, 0.0) if z is None else act(z, gate)
    if z is not None:
        g["d_gate"] = d * ch * wa * hat * da
    if w_after is not None:
        g["d_w_after"] = (d * ch * av * hat).sum(axis=0)
    if channel is not None:
        g["d_channel_scale"] = (d * av * wa * hat).sum(axis=0)
    d = d * ch * av * wa
    g["d_block_out"] = d if w_after is None else _pull(d, hat, f, group)
    return g
