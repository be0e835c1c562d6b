"""Pins of the gated linear recurrence's oracle (``oracle/scan.py``), CPU only:
the unrolled sum over earlier tokens, the special decays 1 and 0, splitting a
sequence at any token, finite differences for every gradient, and planted
mistakes in a copy of the source that each fail a pin."""
import inspect
import types

import numpy as np
import pytest

from oracle import scan as sc

MODES = ("plain", "complement", "unit")
LENS = [5, 0, 1, 7]


def _case(seed, W=3, lens=LENS):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return rng.normal(size=(T, W)), -np.abs(rng.normal(size=(T, W))) * 0.4, cu, rng.normal(size=(len(lens), W)), rng


def check_unrolled(mod, mode):
    x, la, cu, init, _ = _case(1)
    f = mod.forward(x, la, cu, mode, init)
    s = {"plain": np.ones_like(la), "complement": 1 - np.exp(la), "unit": np.sqrt(1 - np.exp(la) ** 2)}[mode]
    for b in range(len(LENS)):
        lo, hi = cu[b], cu[b + 1]
        for t in range(lo, hi):
            want = np.exp(la[lo:t + 1].sum(axis=0)) * init[b]
            for u in range(lo, t + 1):
                want = want + np.exp(la[u + 1:t + 1].sum(axis=0)) * s[u] * x[u]
            np.testing.assert_allclose(f["out"][t], want, rtol=1e-12, atol=1e-13)
        np.testing.assert_array_equal(f["final_state"][b], f["out"][hi - 1] if hi > lo else init[b])


def check_differences(mod, mode):
    x, la, cu, init, rng = _case(2)
    dy, df = rng.normal(size=x.shape), rng.normal(size=init.shape)

    def loss(x, la, init):
        f = mod.forward(x, la, cu, mode, init)
        return (dy * f["out"]).sum() + (df * f["final_state"]).sum()

    g = mod.backward(x, la, cu, mode, dy, init, df)
    for i, name in enumerate(("dx", "d_log_gate", "d_initial_state")):
        args = [x, la, init]
        for k in np.ndindex(args[i].shape):
            h = 1e-5
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[i][k] += h
            lo[i][k] -= h
            fd = (loss(*hi) - loss(*lo)) / (2 * h)
            # central differences: h^2 times a third derivative of a few units, and 1e-16 / h of rounding
            np.testing.assert_allclose(g[name][k], fd, rtol=1e-6, atol=1e-8, err_msg=f"{name} {k}")


@pytest.mark.parametrize("mode", MODES)
def test_unrolled_sum(mode):
    check_unrolled(sc, mode)


@pytest.mark.parametrize("mode", MODES)
def test_gradients_by_differences(mode):
    check_differences(sc, mode)


def test_special_decays():
    x, la, cu, init, _ = _case(3)
    keep = sc.forward(x, np.zeros_like(la), cu, "plain", init)["out"]
    np.testing.assert_allclose(keep[:5], init[0] + np.cumsum(x[:5], axis=0), rtol=1e-13)
    for mode in ("complement", "unit"):  # nothing enters a state that keeps everything
        f = sc.forward(x, np.zeros_like(la), cu, mode, init)
        np.testing.assert_array_equal(f["out"][:5], np.broadcast_to(init[0], (5, 3)))
        g = sc.backward(x, np.zeros_like(la), cu, mode, np.ones_like(x), init)
        assert np.all(np.isfinite(g["d_log_gate"]))
    empty = np.full_like(la, -np.inf)
    for mode in MODES:  # a state that keeps nothing is its input
        np.testing.assert_array_equal(sc.forward(x, empty, cu, mode, init)["out"], x)


def test_split_anywhere():
    x, la, _, init, _ = _case(4, lens=[9])
    whole = sc.forward(x, la, [0, 9], "unit", init[:1])
    for k in range(10):
        a = sc.forward(x[:k], la[:k], [0, k], "unit", init[:1])
        b = sc.forward(x[k:], la[k:], [0, 9 - k], "unit", a["final_state"])
        np.testing.assert_array_equal(np.concatenate([a["out"], b["out"]]), whole["out"])


MISTAKES = [
    ("h = a[t] * h + s[t] * x[t]", "h = a[t] * (h + s[t] * x[t])"),
    ("h = final[b].copy()", "h = 0 * final[b]"),
    ("np.sqrt(-np.expm1(2 * la))", "np.sqrt(-np.expm1(la))"),
    ("dh = dy[t] + e", "dh = dy[t] + a[t] * e"),
    ("a[t] * f[\"before\"][t]", "a[t] * f[\"out\"][t]"),
    ("-np.exp(2 * la) / safe", "np.exp(2 * la) / safe"),
    ("return -np.expm1(la), -np.exp(la)", "return -np.expm1(la), np.exp(la)"),
]


@pytest.mark.parametrize("old,new", MISTAKES)
def test_planted_mistakes_are_caught(old, new):
    src = inspect.getsource(sc)
    assert src.count(old) == 1
    mod = types.ModuleType("oracle.mutant")
    mod.__package__ = "oracle"
    exec(compile(src.replace(old, new), "mutant", "exec"), mod.__dict__)
    caught = 0
    for mode in MODES:
        for check in (check_unrolled, check_differences):
            try:
                check(mod, mode)
            except AssertionError:
                caught += 1
    assert caught
