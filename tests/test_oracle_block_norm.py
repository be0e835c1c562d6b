"""Pins of the block norms' oracle (``oracle/block_norm.py``), CPU only: unit
mean squares, closed forms of each optional part, finite differences for every
gradient, and planted mistakes in a copy of the source that each fail a pin."""
import inspect
import types

import numpy as np
import pytest

from oracle import block_norm as bn

SET = dict(eps=1e-3, residual_scale=0.7, branch_scale=1.3)


def _case(seed, T=3, W=8):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.normal(size=s)  # noqa: E731
    return {"o": n(T, W), "z": n(T, W), "r": n(T, W), "w_after": n(W), "channel": n(W), "w_before": n(W)}, rng


def check_forms(mod):
    c, _ = _case(1)
    w = np.ones(8)
    f = mod.forward(c["o"], w_after=w, group=4, eps=1e-300)
    np.testing.assert_allclose((f["residual_out"].reshape(3, 2, 4) ** 2).mean(axis=2), 1.0, rtol=1e-12)
    f = mod.forward(c["o"], w_after=w, eps=1e-300)
    np.testing.assert_allclose((f["residual_out"] ** 2).mean(axis=1), 1.0, rtol=1e-12)
    f = mod.forward(r=c["r"], w_before=c["w_before"], **SET)
    np.testing.assert_allclose(f["residual_out"], 0.7 * c["r"], rtol=1e-15)
    np.testing.assert_allclose(f["next_in"], c["w_before"] * 0.7 * c["r"] /
                               np.sqrt(0.49 * (c["r"] ** 2).mean(axis=1, keepdims=True) + 1e-3), rtol=1e-12)
    f = mod.forward(c["o"], z=c["z"], r=c["r"], channel=c["channel"], gate="silu", **SET)
    np.testing.assert_allclose(f["residual_out"], 0.7 * c["r"] + 1.3 * c["channel"] * c["o"] * c["z"] /
                               (1 + np.exp(-c["z"])), rtol=1e-12)
    f = mod.forward(np.zeros((2, 8)), w_after=w, **SET)  # an empty row stays zero
    np.testing.assert_array_equal(f["residual_out"], 0.0)


def check_differences(mod, gate, group):
    c, rng = _case(2)
    if gate == "none":
        c["z"] = None
    dr, dn = rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    kw = dict(group=group, gate=gate, **SET)

    def loss(**v):
        f = mod.forward(v["o"], z=v["z"], r=v["r"], w_after=v["w_after"], channel=v["channel"],
                        w_before=v["w_before"], **kw)
        return (dr * f["residual_out"]).sum() + (dn * f["next_in"]).sum()

    at = mod.forward(c["o"], z=c["z"], r=c["r"], w_after=c["w_after"], channel=c["channel"], **kw)["residual_out"]
    g = mod.backward(dr, c["o"], z=c["z"], w_after=c["w_after"], channel=c["channel"], w_before=c["w_before"],
                     residual_out=at, d_next_in=dn, **kw)
    for name, key in (("d_block_out", "o"), ("d_gate", "z"), ("d_residual", "r"), ("d_w_after", "w_after"),
                      ("d_channel_scale", "channel"), ("d_w_before", "w_before")):
        if c[key] is None:
            assert g[name] is None
            continue
        for k in np.ndindex(c[key].shape):
            h = 1e-5
            hi, lo = dict(c, **{key: c[key].copy()}), dict(c, **{key: c[key].copy()})
            hi[key][k] += h
            lo[key][k] -= h
            fd = (loss(**hi) - loss(**lo)) / (2 * h)
            # central differences: h^2 times a third derivative, and 1e-16 / h of rounding
            np.testing.assert_allclose(g[name][k], fd, rtol=1e-5, atol=1e-7, err_msg=f"{name} {k}")


def test_forms():
    check_forms(bn)


@pytest.mark.parametrize("gate", ["none", "silu", "sigmoid", "linear"])
@pytest.mark.parametrize("group", [0, 2, 4])
def test_gradients_by_differences(gate, group):
    check_differences(bn, gate, group)


MISTAKES = [
    (".mean(axis=2, keepdims=True) + eps)", ".sum(axis=2, keepdims=True) + eps)"),
    ("out = out + residual_scale * r", "out = out + r"),
    ("out = out + branch_scale * u", "out = out + u"),
    ("return z * sg, sg + z * sg * (1 - sg)", "return z * sg, sg"),
    ("factor * (d_hat - hat * dot)", "factor * d_hat"),
    ("g[\"d_w_after\"] = (d * ch * av * hat)", "g[\"d_w_after\"] = (d * av * hat)"),
    ("g[\"d_channel_scale\"] = (d * av * wa * hat)", "g[\"d_channel_scale\"] = (d * av * hat)"),
    ("d = branch_scale * d", "d = 1.0 * d"),
    ("g[\"d_residual\"] = residual_scale * d", "g[\"d_residual\"] = d"),
    ("_pull(dn * w_before, hat, f, at.shape[1])", "_pull(dn, hat, f, at.shape[1])"),
]


@pytest.mark.parametrize("old,new", MISTAKES)
def test_planted_mistakes_are_caught(old, new):
    src = inspect.getsource(bn)
    assert src.count(old) == 1
    mod = types.ModuleType("oracle.mutant")
    mod.__package__ = "oracle"
    exec(compile(src.replace(old, new), "mutant", "exec"), mod.__dict__)
    caught = 0
    for check, args in ((check_forms, ()), (check_differences, ("silu", 4)), (check_differences, ("none", 0))):
        try:
            check(mod, *args)
        except AssertionError:
            caught += 1
    assert caught
