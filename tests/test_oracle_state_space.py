"""Pins of the oracles of the short convolution, the selective scan and the
layer norm (``oracle/conv.py``, ``selective.py``, ``layer_norm.py``), CPU only:
independent closed forms, splits of a sequence at any token, finite differences
for every gradient, and planted mistakes in copies of the sources that each
fail a pin."""
import inspect
import types

import numpy as np
import pytest

from oracle import conv as cv
from oracle import layer_norm as ln
from oracle import selective as sl

LENS = [5, 0, 1, 7]
CU = np.concatenate([[0], np.cumsum(LENS)])
T, S = sum(LENS), len(LENS)


def differences(loss, args, grads, rtol=1e-6, atol=1e-8):
    """Central differences (h^2 times a third derivative of a few units, 1e-16 / h of rounding) of every argument."""
    for name, v in args.items():
        for k in np.ndindex(v.shape):
            hi, lo = ({n: a.copy() for n, a in args.items()} for _ in range(2))
            hi[name][k] += 1e-5
            lo[name][k] -= 1e-5
            np.testing.assert_allclose(grads[name][k], (loss(**hi) - loss(**lo)) / 2e-5, rtol=rtol, atol=atol,
                                       err_msg=f"{name} {k}")


# --- convolution ------------------------------------------------------------
def _conv(seed, K, W=3):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(T, W)), weight=r.normal(size=(W, K)), bias=r.normal(size=W),
                initial_state=r.normal(size=(S, K - 1, W))), r


def check_conv_banded(mod):
    for K in (2, 3, 4):
        a, _ = _conv(K, K)
        f = mod.forward(a["x"], a["weight"], CU, a["bias"], a["initial_state"], "none")
        for q in range(S):
            lo, n = CU[q], LENS[q]
            rows = np.concatenate([a["initial_state"][q], a["x"][lo:lo + n]])
            np.testing.assert_array_equal(f["final_state"][q], rows[len(rows) - (K - 1):])
            for c in range(3):
                band = np.zeros((n, n + K - 1))
                for t in range(n):
                    band[t, t:t + K] = a["weight"][c]
                np.testing.assert_allclose(f["out"][lo:lo + n, c], band @ rows[:, c] + a["bias"][c], rtol=1e-12, atol=1e-12)
        u = f["out"]
        silu = mod.forward(a["x"], a["weight"], CU, a["bias"], a["initial_state"], "silu")["out"]
        np.testing.assert_allclose(silu, u / (1 + np.exp(-u)), rtol=1e-12, atol=1e-13)


def check_conv_differences(mod):
    for K, kind in ((4, "silu"), (2, "none"), (3, "silu")):
        a, r = _conv(10 + K, K)
        dy, df = r.normal(size=a["x"].shape), r.normal(size=a["initial_state"].shape)

        def loss(x, weight, bias, initial_state):
            f = mod.forward(x, weight, CU, bias, initial_state, kind)
            return (dy * f["out"]).sum() + (df * f["final_state"]).sum()

        g = mod.backward(a["x"], a["weight"], CU, dy, a["bias"], a["initial_state"], df, kind)
        differences(loss, a, {"x": g["dx"], "weight": g["d_weight"], "bias": g["d_bias"],
                              "initial_state": g["d_initial_state"]})


def test_conv_is_a_banded_product():
    check_conv_banded(cv)


def test_conv_gradients_by_differences():
    check_conv_differences(cv)


def test_conv_split_anywhere():
    a, _ = _conv(3, 4)
    x = a["x"][:9]
    whole = cv.forward(x, a["weight"], [0, 9], a["bias"], a["initial_state"][:1])
    for k in range(10):
        p = cv.forward(x[:k], a["weight"], [0, k], a["bias"], a["initial_state"][:1])
        q = cv.forward(x[k:], a["weight"], [0, 9 - k], a["bias"], p["final_state"])
        np.testing.assert_array_equal(np.concatenate([p["out"], q["out"]]), whole["out"])
        np.testing.assert_array_equal(q["final_state"], whole["final_state"])


# --- selective scan ---------------------------------------------------------
W, N, G = 4, 3, 2


def _sel(seed):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(T, W)), delta=r.normal(size=(T, W)), A=-np.exp(r.normal(size=(W, N))),
                B=r.normal(size=(T, G, N)), C=r.normal(size=(T, G, N)), delta_bias=r.normal(size=W) - 1,
                skip=r.normal(size=W), gate=r.normal(size=(T, W)), initial_state=r.normal(size=(S, W, N))), r


def check_sel_unrolled(mod):
    a, _ = _sel(1)
    f = mod.forward(cu_seqlens=CU, **a)
    d = np.log1p(np.exp(a["delta"] + a["delta_bias"]))
    for q in range(S):
        for t in range(CU[q], CU[q + 1]):
            for c in range(W):
                g = c // (W // G)
                h = np.exp(d[CU[q]:t + 1, c].sum() * a["A"][c]) * a["initial_state"][q, c]
                for s in range(CU[q], t + 1):
                    h = h + np.exp(d[s + 1:t + 1, c].sum() * a["A"][c]) * d[s, c] * a["x"][s, c] * a["B"][s, g]
                z = a["gate"][t, c]
                y = (h @ a["C"][t, g] + a["skip"][c] * a["x"][t, c]) * z / (1 + np.exp(-z))
                np.testing.assert_allclose(f["out"][t, c], y, rtol=1e-11, atol=1e-12)
                if t + 1 == CU[q + 1]:
                    np.testing.assert_allclose(f["final_state"][q, c], h, rtol=1e-11, atol=1e-12)
        if LENS[q] == 0:
            np.testing.assert_array_equal(f["final_state"][q], a["initial_state"][q])


def check_sel_differences(mod):
    a, r = _sel(2)
    dy, df = r.normal(size=(T, W)), r.normal(size=(S, W, N))

    def loss(**k):
        f = mod.forward(cu_seqlens=CU, **k)
        return (dy * f["out"]).sum() + (df * f["final_state"]).sum()

    g = mod.backward(cu_seqlens=CU, d_out=dy, d_final_state=df, **a)
    differences(loss, a, {"x": g["dx"], **{k: g["d_" + k] for k in a if k != "x"}}, rtol=2e-6, atol=2e-8)


def test_selective_unrolled_sum():
    check_sel_unrolled(sl)


def test_selective_gradients_by_differences():
    check_sel_differences(sl)


def test_selective_split_anywhere():
    a, _ = _sel(3)
    w = {k: a[k] for k in ("A", "delta_bias", "skip")}
    t = {k: a[k][:9] for k in ("x", "delta", "B", "C", "gate")}
    whole = sl.forward(cu_seqlens=[0, 9], initial_state=a["initial_state"][:1], **t, **w)
    for k in range(10):
        p = sl.forward(cu_seqlens=[0, k], initial_state=a["initial_state"][:1], **{n: v[:k] for n, v in t.items()}, **w)
        q = sl.forward(cu_seqlens=[0, 9 - k], initial_state=p["final_state"], **{n: v[k:] for n, v in t.items()}, **w)
        np.testing.assert_array_equal(np.concatenate([p["out"], q["out"]]), whole["out"])


# --- layer norm -------------------------------------------------------------
def _norm(seed, W=5):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(4, W)) + 3, weight=r.normal(size=W), bias=r.normal(size=W), residual=r.normal(size=(4, W))), r


def check_norm_moments(mod):
    a, _ = _norm(1, 64)
    for eps in (1e-12, 0.5):
        f = mod.forward(a["x"], None, None, a["residual"], eps)
        r = a["x"] + a["residual"]
        np.testing.assert_array_equal(f["residual_out"], r)
        np.testing.assert_allclose(f["out"].mean(1), 0, atol=1e-13)
        np.testing.assert_allclose(f["out"].std(1) ** 2, r.var(1) / (r.var(1) + eps), rtol=1e-10)
        np.testing.assert_allclose((f["out"][:, 1:] - f["out"][:, :1]) * np.sqrt(r.var(1, keepdims=True) + eps),
                                   r[:, 1:] - r[:, :1], rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(mod.forward(a["x"], a["weight"], a["bias"], a["residual"], eps)["out"],
                                   f["out"] * a["weight"] + a["bias"], rtol=1e-12, atol=1e-13)


def check_norm_differences(mod):
    a, r = _norm(2)
    dy, dr = r.normal(size=a["x"].shape), r.normal(size=a["x"].shape)

    def loss(x, weight, bias, residual):
        f = mod.forward(x, weight, bias, residual, 0.3)
        return (dy * f["out"]).sum() + (dr * f["residual_out"]).sum()

    g = mod.backward(a["x"] + a["residual"], a["weight"], dy, dr, 0.3)
    differences(loss, a, {"x": g["dx"], "residual": g["dx"], "weight": g["d_weight"], "bias": g["d_bias"]})


def test_layer_norm_moments():
    check_norm_moments(ln)


def test_layer_norm_gradients_by_differences():
    check_norm_differences(ln)


MISTAKES = [
    (cv, (check_conv_banded, check_conv_differences), [
        ("r[t - lo + j]", "r[t - lo + K - 1 - j]"),
        ("final[q] = r[hi - lo:]", "final[q] = init[q]"),
        ("pre[t] = b + sum", "pre[t] = sum"),
        ("s * (1 + u * (1 - s))", "s * (1 + u * (1 + s))"),
        ("d_rows[hi - lo:] += d_fin[q]", "d_rows[:K - 1] += d_fin[q]"),
        ("dw[:, j] += g[t] * f[\"rows\"][q][t + j]", "dw[:, j] += g[t] * f[\"rows\"][q][t]"),
        ("db += g.sum(0)", "db += dy[lo:hi].sum(0)"),
    ]),
    (sl, (check_sel_unrolled, check_sel_differences), [
        ("* h + (d[t] * x[t])[:, None] * B[t]", "* (h + (d[t] * x[t])[:, None] * B[t])"),
        ("h = final[q].copy()", "h = 0 * final[q]"),
        ("np.arange(W) // (W // B.shape[1])", "np.arange(W) % B.shape[1]"),
        ("+ skip * x[t]", "+ skip"),
        ("g = C[t] * dy[t][:, None] + e", "g = C[t] * dy[t][:, None] + a * e"),
        ("dd[t] = (x[t] * Bg + (A * g * a * h0).sum(1)) * slope[t]", "dd[t] = (x[t] * Bg + (A * g * h).sum(1)) * slope[t]"),
        ("dA += d[t][:, None] * g * a * h0", "dA += d[t][:, None] * g * h0"),
        ("dx[t] = skip * dy[t] + d[t] * Bg", "dx[t] = skip + d[t] * Bg"),
        ("dC[t] = (dy[t][:, None] * h)", "dC[t] = (dy[t][:, None] * h0)"),
        ("d_gate, dy = dy * f[\"y\"] * ds, dy * s", "d_gate, dy = dy * f[\"out\"] * ds, dy * s"),
    ]),
    (ln, (check_norm_moments, check_norm_differences), [
        ("d = r - r.mean(1, keepdims=True)", "d = r"),
        ("(d * d).mean(1, keepdims=True) + eps", "(d * d).mean(1, keepdims=True)"),
        ("p - p.mean(1, keepdims=True) -", "p -"),
        ("(p * hat).mean(1, keepdims=True)", "(dy * hat).mean(1, keepdims=True)"),
        ("(dy * hat).sum(0)", "(p * hat).sum(0)"),
        ("dx + to_f64(d_residual_out)", "dx"),
    ]),
]


@pytest.mark.parametrize("mod,checks,old,new", [(m, c, o, n) for m, c, pairs in MISTAKES for o, n in pairs])
def test_planted_mistakes_are_caught(mod, checks, old, new):
    src = inspect.getsource(mod)
    assert src.count(old) == 1
    mutant = types.ModuleType("oracle.mutant")
    mutant.__package__ = "oracle"
    exec(compile(src.replace(old, new), "mutant", "exec"), mutant.__dict__)
    caught = 0
    for check in checks:
        try:
            check(mutant)
        except (AssertionError, ValueError):
            caught += 1
    assert caught
