"""Selective state space scan on the GPU against its float64 oracle (marked gpu).

Tolerances are element by element, from running error analysis
(tests/_bounds.py): the recurrence and its adjoint token by token with an
exponential and two products a step, sums over states, channels and tokens in
any order, and one rounding of the output to its type.  A state that a range
of tokens hands to the next is composed of the range's decay exp(A sum D) and
its own states: CUT adds a few such steps to every state."""
import numpy as np
import pytest

from oracle import selective as oracle
from tests._bounds import R, ROUND, EX2, close, silu, silu_slope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CUT = 4 * (EX2 + 8 * ROUND)


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _half(dtype):
    return torch.finfo(_dt(dtype)).eps / 2


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lens, W, N, G, dtype, seed, gate=True, skip=True, bias=True, states=True, tail=0, extra=0, step=-3.0):
    """Inputs on the GPU; `tail` rows behind the last sequence, `extra` columns between rows; softplus(step): usual steps."""
    g = torch.Generator().manual_seed(seed)
    T, S = sum(lens) + tail, len(lens)

    def n(rows, cols, mean=0.0):
        return (torch.randn(rows, cols + extra, generator=g) + mean).to(_dt(dtype)).cuda()[:, :cols]

    f = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    c = {"x": n(T, W), "delta": n(T, W, 0.0 if bias else step), "B": n(T, G * N).unflatten(1, (G, N)),
         "C": n(T, G * N).unflatten(1, (G, N)), "A": -torch.exp(f(W, N)), "bias": f(W) + step if bias else None,
         "skip": f(W) if skip else None, "gate": n(T, W) if gate else None, "n": sum(lens),
         "cu": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda(),
         "init": f(S, W, N) if states else None, "d_final": f(S, W, N) if states else None}
    c["d_out"] = torch.randn(T, W, generator=g).to(_dt(dtype)).cuda()
    return c


def cfg_of(b, c, dtype):
    W, N = c["A"].shape
    return b.make_selective_config(W, N, c["B"].shape[1], dtype)


def run(b, c, dtype, **kw):
    cfg = cfg_of(b, c, dtype)
    args = (c["x"], c["delta"], c["A"], c["B"], c["C"], c["cu"])
    parts = dict(delta_bias=c["bias"], skip=c["skip"], gate=c["gate"], initial_state=c["init"])
    f = b.selective_forward(cfg, *args, want_checkpoints=True, **parts, **kw)
    g = b.selective_backward(cfg, *args, f["checkpoints"], c["d_out"], d_final_state=c["d_final"], **parts)
    torch.cuda.synchronize()
    return f, g


def _stack(items):
    return R(np.stack([i.v for i in items]), np.stack([i.e for i in items]))


def bounds(c):
    """Every output as a value and its bound, over the tokens of sequences."""
    n, cu = c["n"], c["cu"].cpu().numpy()
    x, delta, B, C, dy = (_f64(c[k])[:n] for k in ("x", "delta", "B", "C", "d_out"))
    A, bias, skip, init, d_fin = (_f64(c[k]) for k in ("A", "bias", "skip", "init", "d_final"))
    (W, N), S, G = A.shape, len(cu) - 1, B.shape[1]
    per = np.arange(W) // (W // G)
    u = R(delta) + (0.0 if bias is None else bias)
    d = u.softplus()
    dx_ = d * x
    z = None if c["gate"] is None else R(_f64(c["gate"])[:n])
    dY = R(dy) if z is None else R(dy) * silu(z)
    col = lambda r: R(r.v[..., None], r.e[..., None])  # noqa: E731
    out = {"final": [], "d_init": []}
    per_t = {k: [None] * n for k in ("y", "Bg", "Aw", "dA", "dB", "dC")}
    for q in range(S):
        h = R(init[q] if init is not None else np.zeros((W, N)))
        before, decay, now = {}, {}, {}
        for t in range(cu[q], cu[q + 1]):
            before[t] = h
            decay[t] = (col(d[t]) * A).exp()
            h = decay[t] * h + col(dx_[t]) * B[t][per]
            h = R(h.v, h.e + CUT * np.abs(h.v) / 64)
            now[t] = h
            y = (h * C[t][per]).sum(1)
            per_t["y"][t] = y if skip is None else y + R(skip) * x[t]
        out["final"].append(R(h.v, h.e + CUT * np.abs(h.v)))
        e = R(d_fin[q] if d_fin is not None else np.zeros((W, N)))
        for t in range(cu[q + 1] - 1, cu[q] - 1, -1):
            g = col(dY[t]) * C[t][per] + e
            g = R(g.v, g.e + CUT * np.abs(g.v) / 64)
            w = g * (decay[t] * before[t])
            # the state behind the decay may be formed as now - D B x: one more rounding of both
            w = R(w.v, w.e + 4 * ROUND * np.abs(g.v) * (np.abs(now[t].v) + np.abs(col(dx_[t]).v * B[t][per])))
            per_t["Bg"][t] = (g * B[t][per]).sum(1)
            per_t["Aw"][t] = (w * A).sum(1)
            per_t["dA"][t] = w * col(d[t])
            for k, v in (("dB", g * col(dx_[t])), ("dC", now[t] * col(dY[t]))):
                per_t[k][t] = R(v.v.reshape(G, W // G, N), v.e.reshape(G, W // G, N)).sum(1)
            e = decay[t] * g
        out["d_init"].append(R(e.v, e.e + CUT * np.abs(e.v)))
    if not n:
        return out
    p = {k: _stack(v) for k, v in per_t.items()}
    out["out"] = p["y"] if z is None else p["y"] * silu(z)
    out["d_gate"] = None if z is None else R(dy) * p["y"] * silu_slope(z)
    out["d_B"], out["d_C"], out["d_A"] = p["dB"], p["dC"], p["dA"].sum(0)
    out["dx"] = d * p["Bg"]
    out["d_skip"] = None
    if skip is not None:
        out["dx"] = out["dx"] + dY * skip
        out["d_skip"] = (dY * x).sum(0)
    out["d_delta"] = (p["Bg"] * x + p["Aw"]) * u.sigmoid()
    out["d_delta_bias"] = None if bias is None else out["d_delta"].sum(0)
    return out


def check(c, dtype, f, g):
    n, cu, half, f32 = c["n"], c["cu"].cpu().numpy(), _half(dtype), 2.0 ** -24
    bd = bounds(c)
    kw = {k: _f64(c[v]) for k, v in (("delta_bias", "bias"), ("skip", "skip"), ("initial_state", "init"))}
    a = [_f64(c[k])[:n] for k in ("x", "delta")] + [_f64(c["A"])] + [_f64(c[k])[:n] for k in ("B", "C")]
    z = None if c["gate"] is None else _f64(c["gate"])[:n]
    o = oracle.forward(*a, cu, gate=z, **kw)
    want = oracle.backward(*a, cu, _f64(c["d_out"])[:n], gate=z, d_final_state=_f64(c["d_final"]), **kw)
    want.update(out=o["out"])
    if n:
        for k in ("out", "dx", "d_delta", "d_gate", "d_B", "d_C"):
            got = (f if k == "out" else g)[k]
            if bd[k] is None:
                assert got is None
                continue
            np.testing.assert_allclose(bd[k].v, want[k], rtol=1e-9, atol=1e-9)
            close(_f64(got)[:n], bd[k], half, k)
        for k in ("d_A", "d_skip", "d_delta_bias"):
            if bd[k] is None:
                assert g[k] is None
                continue
            np.testing.assert_allclose(bd[k].v, want[k], rtol=1e-9, atol=1e-9)
            close(_f64(g[k]), bd[k], f32, k)
    for q in range(len(cu) - 1):
        np.testing.assert_allclose(bd["final"][q].v, o["final_state"][q], rtol=1e-9, atol=1e-9)
        close(_f64(f["final_state"][q]), bd["final"][q], f32, "final_state")
        np.testing.assert_allclose(bd["d_init"][q].v, want["d_initial_state"][q], rtol=1e-9, atol=1e-9)
        close(_f64(g["d_initial_state"][q]), bd["d_init"][q], f32, "d_initial_state")


SHAPES = [  # lengths, width, states, groups
    ([1], 8, 8, 1), ([1], 16, 16, 2), ([2, 1], 24, 32, 1), ([3], 8, 64, 1), ([17], 64, 16, 1),
    ([5, 0, 0, 1, 16, 2, 0], 72, 16, 1), ([40], 136, 16, 1), ([33, 0, 15, 1, 16, 32], 64, 16, 4), ([70], 40, 64, 1),
    ([31, 50], 48, 32, 2), ([100, 3], 200, 8, 1), ([129], 264, 16, 1), ([64, 65, 63], 144, 16, 3), ([0, 0, 7], 24, 8, 3),
    ([1] * 40, 24, 16, 1), ([300], 32, 16, 1), ([0], 16, 16, 1), ([260, 270], 16, 16, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,W,N,G", SHAPES)
def test_matches_oracle(b, dtype, lens, W, N, G):
    c = make(lens, W, N, G, dtype, seed=len(lens) + W + N, extra=8 if W % 3 else 0)
    f, g = run(b, c, dtype)
    check(c, dtype, f, g)


@pytest.mark.parametrize("kw", [dict(gate=False), dict(skip=False), dict(bias=False), dict(states=False),
                                dict(gate=False, skip=False, bias=False, states=False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_optional_parts(b, kw, dtype):
    c = make([20, 0, 37], 72, 16, 1, dtype, 5, **kw)
    f, g = run(b, c, dtype)
    check(c, dtype, f, g)


@pytest.mark.parametrize("step", [-12.0, -8.0, 1.0, 30.0])
def test_steps_of_every_size(b, step):
    """Steps from 6e-6 (a state that keeps all) to 30 (one that keeps nothing)."""
    for dtype in ("bf16", "f32"):
        c = make([50, 33], 40, 16, 1, dtype, 6, step=step)
        f, g = run(b, c, dtype)
        check(c, dtype, f, g)


def test_long_sequence_cut_into_ranges(b):
    """Few channels and many tokens: the token axis is cut, in the middle of sequences and at their edges."""
    for lens in ([1500], [700, 0, 801, 1, 200], [3, 1400, 5]):
        c = make(lens, 16, 16, 1, "bf16", len(lens))
        f, g = run(b, c, "bf16")
        check(c, "bf16", f, g)
    c = make([1500], 8, 8, 1, "f32", 9)
    f, g = run(b, c, "f32")
    check(c, "f32", f, g)


def test_rows_behind_the_last_sequence_stay(b):
    c = make([5, 40], 64, 16, 2, "bf16", 3, tail=50)
    for k in ("x", "delta", "B", "C", "gate", "d_out"):
        c[k][45:] = float("nan")
    cfg, P = cfg_of(b, c, "bf16"), lambda t: None if t is None else t.data_ptr()
    out = torch.full_like(c["d_out"], 7.0)
    f, _ = run(b, c, "bf16", out=out)
    assert bool((out[45:] == 7).all())
    T, W, N, G = 95, 64, 16, 2
    t = {k: torch.full_like(c["d_out"], 7.0) for k in ("dx", "dd", "dz")}
    t.update({k: torch.full((T, G, N), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("dB", "dC")})
    w = {"db": torch.empty(W, device="cuda"), "dA": torch.empty(W, N, device="cuda"), "dk": torch.empty(W, device="cuda"),
         "di": torch.empty(2, W, N, device="cuda")}
    n = b.sse_selective_backward_workspace_size(cfg, T, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert b.sse_selective_backward(
        cfg, P(c["x"]), c["x"].stride(0), P(c["delta"]), c["delta"].stride(0), P(c["bias"]), P(c["A"]), P(c["B"]),
        c["B"].stride(0), P(c["C"]), c["C"].stride(0), P(c["skip"]), P(c["gate"]), c["gate"].stride(0), P(c["cu"]), 2, T,
        P(c["init"]), P(f["checkpoints"]), P(c["d_out"]), P(c["d_final"]), P(t["dx"]), P(t["dd"]), P(w["db"]), P(w["dA"]),
        P(t["dB"]), P(t["dC"]), P(w["dk"]), P(t["dz"]), P(w["di"]), P(ws), n, None) == b.SSE_OK
    torch.cuda.synchronize()
    assert all(bool((v[45:] == 7).all()) for v in t.values())
    g = {"dx": t["dx"], "d_delta": t["dd"], "d_gate": t["dz"], "d_B": t["dB"], "d_C": t["dC"], "d_A": w["dA"],
         "d_skip": w["dk"], "d_delta_bias": w["db"], "d_initial_state": w["di"]}
    check(c, "bf16", {"out": out, "final_state": f["final_state"]}, g)


def test_nan_stays_in_its_sequence_and_channel(b):
    c = make([30, 30, 30], 64, 16, 1, "bf16", 9)
    c["x"][40, 5] = float("nan")
    f, g = run(b, c, "bf16")
    want = torch.zeros(90, 64, dtype=torch.bool)
    want[40:60, 5] = True
    assert torch.equal(f["out"].isnan().cpu(), want)
    assert torch.equal(f["final_state"].isnan().any(2).nonzero().cpu(), torch.tensor([[1, 5]]))
    # d_B, d_C sum over channels: from the token on, within the sequence
    assert torch.equal(g["d_C"].isnan().any(2).any(1).nonzero().flatten().cpu(), torch.arange(40, 60))
    assert torch.equal(g["d_B"].isnan().any(2).any(1).nonzero().flatten().cpu(), torch.tensor([40]))
    for k in ("dx", "d_delta", "d_gate"):
        bad = g[k].isnan().cpu()
        assert not bad[:40].any() and not bad[60:].any() and not bad[:, :5].any() and not bad[:, 6:].any(), k
    assert torch.equal(g["d_A"].isnan().any(1).nonzero().flatten().cpu(), torch.tensor([5]))


def test_infinite_gradient_stays_in_its_sequence(b):
    c = make([30, 30, 30], 64, 16, 1, "bf16", 9)
    c["d_final"][1, 7, 3] = float("inf")
    _, g = run(b, c, "bf16")
    bad = ~g["dx"].isfinite().cpu()
    assert bad.any() and not bad[:30].any() and not bad[60:].any() and not bad[:, :7].any() and not bad[:, 8:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,N,G", [(1, 8, 8, 1), (3, 136, 16, 1), (256, 2048, 16, 1), (2, 48, 64, 2), (5, 72, 32, 3)])
def test_step_matches_oracle(b, dtype, B, W, N, G):
    c = make([1] * B, W, N, G, dtype, W + N, extra=8)
    state = c["init"].clone()
    out = b.selective_step(cfg_of(b, c, dtype), state, c["x"], c["delta"], c["A"], c["B"], c["C"], delta_bias=c["bias"],
                           skip=c["skip"], gate=c["gate"])["out"]
    if B > 8:  # the first and last streams
        keep = [0, 1, B - 1]
        c = {k: v[keep] if torch.is_tensor(v) and k in ("x", "delta", "B", "C", "gate", "init", "d_final", "d_out") else v
             for k, v in c.items()}
        c["cu"], c["n"], out, state = torch.arange(4, dtype=torch.int32), 3, out[keep], state[keep]
    bd = bounds(c)
    close(_f64(out), bd["out"], _half(dtype), "out")
    close(_f64(state), _stack(bd["final"]), 2.0 ** -24, "state")


def test_steps_follow_a_forward(b):
    """Prompt, then tokens one at a time: the whole sequence's oracle."""
    c = make([60], 72, 16, 1, "f32", 4)
    cfg = cfg_of(b, c, "f32")
    p = dict(delta_bias=c["bias"], skip=c["skip"])
    cut = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    f = b.selective_forward(cfg, c["x"][:50], c["delta"][:50], c["A"], c["B"][:50], c["C"][:50], cut, gate=c["gate"][:50],
                            initial_state=c["init"], **p)
    outs, state = [f["out"]], f["final_state"]
    for t in range(50, 60):
        s = slice(t, t + 1)
        outs.append(b.selective_step(cfg, state, c["x"][s], c["delta"][s], c["A"], c["B"][s], c["C"][s], gate=c["gate"][s],
                                     **p)["out"])
    bd = bounds(c)
    close(_f64(torch.cat(outs)), bd["out"], 2.0 ** -24, "out")
    close(_f64(state[0]), bd["final"][0], 2.0 ** -24, "state")


def test_checkpoints_are_the_states(b):
    """Row i of the checkpoints is the state before token 16 i, within a sequence."""
    c = make([100], 24, 16, 1, "f32", 2)
    f, _ = run(b, c, "f32")
    for i in (1, 2, 5):
        sub = {**c, "n": 16 * i, "cu": torch.tensor([0, 16 * i], dtype=torch.int32)}
        close(_f64(f["checkpoints"][i]), bounds(sub)["final"][0], 2.0 ** -24, "checkpoint")


def test_no_tokens(b):
    c = make([0, 0], 16, 16, 1, "bf16", 1)
    f, g = run(b, c, "bf16")
    assert torch.equal(f["final_state"], c["init"]) and torch.equal(g["d_initial_state"], c["d_final"])
    assert not g["d_A"].any() and not g["d_skip"].any() and not g["d_delta_bias"].any()
    c = make([], 16, 16, 1, "bf16", 1)
    _, g = run(b, c, "bf16")
    assert not g["d_A"].any() and not g["d_skip"].any()


def test_row_offsets_past_32_bits(b):
    """The last rows of tensors of more than 2^32 elements are the rows of a short call, within two float32 forms' distance."""
    W, T = 8192, (1 << 19) + 100
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    delta = torch.full((T, W), -3.0, dtype=torch.bfloat16, device="cuda")
    x[-90:] = torch.randn(90, W, generator=gen, device="cuda").bfloat16()
    B, C = (torch.randn(T, 1, 8, generator=gen, device="cuda").bfloat16() for _ in range(2))
    A = -torch.rand(W, 8, generator=gen, device="cuda") - 0.5
    cfg = b.make_selective_config(W, 8)
    cu, short = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T - 90, T], [0, 90]))
    f = b.selective_forward(cfg, x, delta, A, B, C, cu, want_checkpoints=True)
    s = slice(T - 90, T)
    e = b.selective_forward(cfg, x[s], delta[s], A, B[s], C[s], short, want_checkpoints=True)
    torch.testing.assert_close(f["out"][s], e["out"], rtol=2.0 ** -7, atol=1e-5)
    assert not f["out"][:-90].any()
    torch.testing.assert_close(f["final_state"][1], e["final_state"][0], rtol=1e-4, atol=1e-5)
    g = b.selective_backward(cfg, x, delta, A, B, C, cu, f["checkpoints"], x, want_d_initial_state=False)
    h = b.selective_backward(cfg, x[s], delta[s], A, B[s], C[s], short, e["checkpoints"], x[s], want_d_initial_state=False)
    torch.testing.assert_close(g["dx"][s], h["dx"], rtol=2.0 ** -7, atol=1e-4)
    torch.testing.assert_close(g["d_B"][s], h["d_B"], rtol=2.0 ** -7, atol=1e-3)
    torch.testing.assert_close(g["d_A"], h["d_A"], rtol=1e-4, atol=1e-4)


def test_graph_stream_and_repeat(b):
    """Calls repeat bit for bit, on another stream and replayed from two graphs at the same time."""
    c = make([33, 0, 290], 136, 16, 1, "bf16", 8)
    f, g = run(b, c, "bf16")
    want = [f["out"], f["final_state"], *g.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f, g = run(b, c, "bf16")
    for a, e in zip([f["out"], f["final_state"], *g.values()], want):
        assert torch.equal(a, e)
    cfg = cfg_of(b, c, "bf16")
    args = (c["x"], c["delta"], c["A"], c["B"], c["C"], c["cu"])
    parts = dict(delta_bias=c["bias"], skip=c["skip"], gate=c["gate"], initial_state=c["init"])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = b.selective_forward(cfg, *args, want_checkpoints=True, **parts)
            g = b.selective_backward(cfg, *args, f["checkpoints"], c["d_out"], d_final_state=c["d_final"], **parts)
        graphs.append((graph, [f["out"], f["final_state"], *g.values()]))
    torch.cuda.synchronize()
    for graph, _ in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for a, e in zip(got, want):
            assert torch.equal(a, e)


def test_helpers_refuse(b):
    c = make([6], 64, 16, 1, "bf16", 1)
    cfg = cfg_of(b, c, "bf16")
    v = {k: c[k] for k in ("x", "delta", "A", "B", "C")}
    st, ck = torch.zeros(6, 64, 16, device="cuda"), torch.zeros(1, 64, 16, device="cuda")

    def fwd(cu=c["cu"], **kw):
        a = {**v, **{k: kw.pop(k) for k in list(kw) if k in v}}
        return lambda: b.selective_forward(cfg, *a.values(), cu, **kw)

    calls = [fwd(**{k: None}) for k in v] + [
        fwd(cu=None), fwd(cu=c["cu"].long()), fwd(x=c["x"].float()), fwd(A=c["A"].bfloat16()), fwd(A=c["A"][:, :8]),
        fwd(B=c["B"][:5]), fwd(B=c["B"][..., :8]), fwd(delta=c["delta"][:, :32]), fwd(x=c["x"].cpu()), fwd(gate=c["gate"][:5]),
        fwd(skip=c["skip"][:8]), fwd(delta_bias=c["bias"].bfloat16()), fwd(initial_state=c["init"][:, :8]),
        fwd(initial_state=c["init"], final_state=c["init"]), fwd(out=c["x"][:3]), fwd(checkpoints=ck[:0]),
        fwd(workspace=torch.empty(16, device="cuda")),
        lambda: b.selective_backward(cfg, *v.values(), c["cu"], None, c["d_out"]),
        lambda: b.selective_backward(cfg, *v.values(), c["cu"], ck, None),
        lambda: b.selective_backward(cfg, *v.values(), c["cu"], ck[:0], c["d_out"]),
        lambda: b.selective_backward(cfg, *v.values(), c["cu"], ck, c["d_out"][:5]),
        lambda: b.selective_step(cfg, None, *v.values()), lambda: b.selective_step(cfg, st[:5], *v.values()),
        lambda: b.selective_step(cfg, st.bfloat16(), *v.values())]
    for call in calls:
        with pytest.raises(b.SSEError) as e:
            call()
        assert e.value.status == b.SSE_ERR_INVALID_ARG
    with pytest.raises(b.SSEError) as e:
        b.selective_backward(cfg, *v.values(), c["cu"], ck, c["d_out"],
                             workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == b.SSE_ERR_WORKSPACE
