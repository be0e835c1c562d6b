"""Gated linear recurrence on the GPU against its float64 oracle (marked gpu).

Tolerances are element by element and come from the arithmetic: one rounding
of the output to its type (at most half a step, finfo.eps / 2 of the value)
plus the float32 error of the recurrence.  Each step multiplies what it
carries by a decay that is at most 2^-21 off (exponential and product) and
rounds the sum (2^-24), the input factor is at most 2^-21 off: a term that has
gone through n steps is at most (n + 2) 2^-20 of itself off.  _spread sums
(n + 2) |term| over the terms.  Below float32's smallest normal value, 2^-126,
a decay or a product may be lost altogether: with the other factors below 2^16
(inputs and states of a few units, sums over a few thousand tokens) that is at
most 2^-110 of any output.
"""
import numpy as np
import pytest

from oracle import scan as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D = 2.0 ** -20
LEAST = 2.0 ** -110
MODES = ("plain", "complement", "unit")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _half(dtype):
    return torch.finfo(_dt(dtype)).eps / 2


def _f64(t):
    return t.detach().double().cpu().numpy()


def make(lens, width, dtype, seed, states=True, tau=4.0, tail=0, extra=0):
    """Inputs on the GPU; `tail` rows behind the last sequence, `extra` columns between rows."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    buf = n(T, 2 * width + extra)
    buf[:, width:2 * width] = torch.nn.functional.logsigmoid(buf[:, width:2 * width]) / tau
    buf = buf.to(_dt(dtype)).cuda()
    x, la = buf[:, :width], buf[:, width:2 * width]
    if not extra:
        x, la = x.contiguous(), la.contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    S = len(lens)
    c = {"x": x, "la": la, "cu": cu, "d_out": n(T, width).to(_dt(dtype)).cuda(), "T": sum(lens)}
    c["init"] = n(S, width).cuda() if states else None
    c["d_final"] = n(S, width).cuda() if states else None
    return c


def _spread(a, term, cu, first):
    """Sum of (n + 2) |term| of the terms in each state, and their sum of |term|; a, term [T, W], first [S, W]."""
    m, e = np.zeros_like(a), np.zeros_like(a)
    mf, ef = np.abs(first).copy(), 2 * np.abs(first)
    for b in range(len(cu) - 1):
        mm, ee = mf[b].copy(), ef[b].copy()
        for t in range(cu[b], cu[b + 1]):
            ee = a[t] * (ee + mm) + 2 * np.abs(term[t])
            mm = a[t] * mm + np.abs(term[t])
            m[t], e[t] = mm, ee
        mf[b], ef[b] = mm, ee
    return m, e, ef


def _close(got, want, tol, name):
    bad = ~(np.abs(got - want) <= tol + LEAST)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}, tolerance {tol[bad][0]}")


def run(c, mode, dtype, **kw):
    from sparse_state_linear_router_gb300 import binding
    cfg = binding.make_scan_config(c["x"].shape[-1], mode, dtype)
    f = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=c["init"], want_checkpoints=True, **kw)
    b = binding.scan_backward(cfg, c["x"], c["la"], c["cu"], f["checkpoints"], c["d_out"], initial_state=c["init"],
                              d_final_state=c["d_final"])
    torch.cuda.synchronize()
    return f, b


def check(c, mode, dtype, f, b):
    n, cu = c["T"], c["cu"].cpu().numpy()
    x, la, dy = (_f64(c[k])[:n] for k in ("x", "la", "d_out"))
    S, W = len(cu) - 1, x.shape[1]
    init = np.zeros((S, W)) if c["init"] is None else _f64(c["init"])
    d_fin = np.zeros((S, W)) if c["d_final"] is None else _f64(c["d_final"])
    want = oracle.forward(x, la, cu, mode, init)
    s, ds = oracle.input_scale(la, mode)
    a, h = np.exp(la), _half(dtype)
    _, e, ef = _spread(a, s * x, cu, init)
    _close(_f64(f["out"])[:n], want["out"], h * np.abs(want["out"]) + D * e, "out")
    _close(_f64(f["final_state"]), want["final_state"], 2.0 ** -24 * np.abs(want["final_state"]) + D * ef, "final")
    grad = oracle.backward(x, la, cu, mode, dy, init, d_fin)
    # the adjoint runs the same recurrence backwards with the decay of the token behind
    flip = slice(None, None, -1)
    rcu = [n - v for v in cu[::-1]]
    behind = np.zeros_like(a)
    behind[:-1] = a[1:]
    last = np.array([v - 1 for v, u in zip(cu[1:], cu[:-1]) if v > u], dtype=int)
    full = np.array([v > u for v, u in zip(cu[1:], cu[:-1])], dtype=bool)
    behind[last] = 0
    seed = np.abs(dy)
    seed[last] += np.abs(d_fin[full])
    md, ed, _ = _spread(behind[flip], seed[flip], rcu, np.zeros((S, W)))
    md, ed = md[flip], ed[flip]
    _close(_f64(b["dx"])[:n], grad["dx"], h * np.abs(grad["dx"]) + D * s * (ed + md), "dx")
    first = np.array([u for v, u in zip(cu[1:], cu[:-1]) if v > u], dtype=int)
    mb, eb = np.zeros_like(a), np.zeros_like(a)
    mh, eh, _ = _spread(a, s * x, cu, init)
    mb[1:], eb[1:] = mh[:-1], eh[:-1]
    mb[first], eb[first] = np.abs(init[full]), 0
    mag = a * mb + np.abs(ds * x)
    tol = h * np.abs(grad["d_log_gate"]) + D * (ed * mag + md * (a * eb + 4 * mag))
    _close(_f64(b["d_log_gate"])[:n], grad["d_log_gate"], tol, "d_log_gate")
    tol = np.abs(d_fin) * D
    tol[full] = D * a[first] * (ed + md)[first]
    _close(_f64(b["d_initial_state"]), grad["d_initial_state"], tol + 2.0 ** -24 * np.abs(grad["d_initial_state"]),
           "d_init")


LENGTHS = [
    [1],
    [63], [64], [65],
    [130, 0, 1, 257, 0, 0, 64],
    [1] * 40 + [0, 3, 5, 8, 0],
    [128, 128, 128],
    [2500],
    [700, 9, 1800, 0, 33],
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "-".join(map(str, v[:5])))
def test_against_the_oracle(lens, dtype, mode):
    c = make(lens, 72, dtype, seed=len(lens) + lens[0], states=lens[0] != 64)
    check(c, mode, dtype, *run(c, mode, dtype))


@pytest.mark.parametrize("width,dtype", [(4, "f32"), (8, "bf16"), (60, "f32"), (136, "bf16"), (1000, "f32"),
                                         (2048, "bf16")])
def test_widths(width, dtype):
    c = make([300, 77], width, dtype, seed=width)
    check(c, "unit", dtype, *run(c, "unit", dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slow_and_strong_decays(dtype):
    for tau in (2000.0, 0.02):  # decays of almost 1 over 3000 tokens, and of exp(-40)
        c = make([3000, 40], 16, dtype, seed=5, tau=tau)
        check(c, "complement", dtype, *run(c, "complement", dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_strides_and_heads(dtype):
    c = make([150, 90], 64, dtype, seed=6, extra=24)
    f, b = run(c, "unit", dtype)
    check(c, "unit", dtype, f, b)
    heads = dict(c, x=c["x"].unflatten(1, (4, 16)), la=c["la"].unflatten(1, (4, 16)))
    from sparse_state_linear_router_gb300 import binding
    cfg = binding.make_scan_config(64, "unit", dtype)
    g = binding.scan_forward(cfg, heads["x"], heads["la"], c["cu"], initial_state=c["init"])
    assert g["out"].shape == (240, 4, 16)
    assert torch.equal(g["out"].flatten(1), f["out"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_batch_keeps_the_rows_behind(dtype):
    c = make([70, 0, 41], 40, dtype, seed=7, tail=37)
    c["x"][111:] = float("nan")
    c["la"][111:] = float("nan")
    c["d_out"][111:] = float("nan")
    out = torch.full((148, 40), 7.0, dtype=_dt(dtype), device="cuda")
    f, b = run(c, "unit", dtype, out=out)
    check(c, "unit", dtype, f, b)
    assert bool((f["out"][111:] == 7).all())


def test_gradient_rows_behind_the_last_sequence_stay(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    c = make([70, 41], 40, dtype, seed=8, tail=60)
    f, _ = run(c, "plain", dtype)
    cfg = binding.make_scan_config(40, "plain", dtype)
    dx, dg = (torch.full((171, 40), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = binding.sse_scan_backward(cfg, c["x"].data_ptr(), 40, c["la"].data_ptr(), 40, c["cu"].data_ptr(), 2, 171,
                                   c["init"].data_ptr(), f["checkpoints"].data_ptr(), c["d_out"].data_ptr(), None,
                                   dx.data_ptr(), dg.data_ptr(), None, binding._stream())
    torch.cuda.synchronize()
    assert st == binding.SSE_OK
    assert bool((dx[111:] == 5).all()) and bool((dg[111:] == 5).all())
    assert not bool((dx[:111] == 5).all())


@pytest.mark.parametrize("mode", MODES)
def test_emptied_and_kept_states(mode, dtype="f32"):
    """Log-gates of -infinity (the state is emptied) and of 0 (it is kept)."""
    c = make([200, 90], 24, dtype, seed=9)
    c["la"][5:200:17] = float("-inf")
    c["la"][3:200:11] = 0.0
    check(c, mode, dtype, *run(c, mode, dtype))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bad_value_stays_in_its_sequence_and_channel(dtype, bad):
    lens = [300, 50, 0, 1, 400]
    c = make(lens, 64, dtype, seed=10)
    ref, ref_b = run(c, "plain", dtype)
    c["x"][320, 3] = bad   # 20 tokens into the second sequence
    got, got_b = run(c, "plain", dtype)
    same = torch.ones(751, 64, dtype=torch.bool, device="cuda")
    same[320:350, 3] = False
    assert torch.equal(got["out"][same], ref["out"][same])
    assert not bool(torch.isfinite(got["out"][320:350, 3]).any())
    fin = torch.ones(5, 64, dtype=torch.bool, device="cuda")
    fin[1, 3] = False
    assert torch.equal(got["final_state"][fin], ref["final_state"][fin])
    assert torch.equal(got_b["dx"], ref_b["dx"])          # the adjoint does not meet x here
    same[320, 3] = True                                    # its own gate's gradient uses the state before it
    assert torch.equal(got_b["d_log_gate"][same], ref_b["d_log_gate"][same])
    # and a bad gradient stays among the earlier tokens of its sequence and channel
    c["x"][320, 3] = 1.0
    ref, ref_b = run(c, "plain", dtype)
    c["d_out"][330, 5] = bad
    _, got_b = run(c, "plain", dtype)
    same = torch.ones(751, 64, dtype=torch.bool, device="cuda")
    same[300:331, 5] = False
    assert torch.equal(got_b["dx"][same], ref_b["dx"][same])
    assert torch.equal(got_b["d_log_gate"][same], ref_b["d_log_gate"][same])
    assert not bool(torch.isfinite(got_b["dx"][300:331, 5]).any())


def test_final_state_may_be_the_initial_state(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    for lens in ([900, 0, 5, 700], [1] * 30 + [0, 2], [3000]):
        c = make(lens, 200, dtype, seed=11)
        ref, _ = run(c, "unit", dtype)
        state = c["init"].clone()
        cfg = binding.make_scan_config(200, "unit", dtype)
        got = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=state, final_state=state)
        torch.cuda.synchronize()
        assert torch.equal(got["out"], ref["out"]) and torch.equal(state, ref["final_state"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(dtype):
    from sparse_state_linear_router_gb300 import binding
    cfg = binding.make_scan_config(16, "plain", dtype)
    x = torch.empty(0, 16, dtype=_dt(dtype), device="cuda")
    init = torch.randn(3, 16, device="cuda")
    f = binding.scan_forward(cfg, x, x, torch.zeros(4, dtype=torch.int32, device="cuda"), initial_state=init,
                             want_checkpoints=True)
    b = binding.scan_backward(cfg, x, x, torch.zeros(4, dtype=torch.int32, device="cuda"), f["checkpoints"], x,
                              initial_state=init, d_final_state=init)
    assert f["out"].shape == (0, 16) and torch.equal(f["final_state"], init)
    assert torch.equal(b["d_initial_state"], init)
    f = binding.scan_forward(cfg, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert f["final_state"].shape == (0, 16)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_continue_a_forward(dtype, mode):
    from sparse_state_linear_router_gb300 import binding
    B, W, n = 5, 72, 6
    c = make([n] * B, W, dtype, seed=12, extra=8)
    cfg = binding.make_scan_config(W, mode, dtype)
    state = c["init"].clone()
    cu = c["cu"].long()
    want = oracle.forward(_f64(c["x"]), _f64(c["la"]), c["cu"].cpu().numpy(), mode, _f64(c["init"]))
    s, _ = oracle.input_scale(_f64(c["la"]), mode)
    _, e, ef = _spread(np.exp(_f64(c["la"])), s * _f64(c["x"]), c["cu"].cpu().numpy(), _f64(c["init"]))
    for t in range(n):
        rows = (cu[:-1] + t)
        out = binding.scan_step(cfg, state, c["x"][rows], c["la"][rows])["out"]
        r = rows.cpu().numpy()
        _close(_f64(out), want["out"][r], _half(dtype) * np.abs(want["out"][r]) + D * e[r], f"token {t}")
    _close(_f64(state), want["final_state"], D * ef, "state")
    # a row slice of a wider tensor, every n-th row: the stride is taken as it is
    state = c["init"].clone()
    a = binding.scan_step(cfg, state, c["x"][::n], c["la"][::n])["out"]
    assert torch.equal(a, binding.scan_step(cfg, c["init"].clone(), c["x"][::n].contiguous(),
                                            c["la"][::n].contiguous())["out"])
    empty = torch.empty(0, W, dtype=_dt(dtype), device="cuda")
    assert binding.scan_step(cfg, torch.empty(0, W, device="cuda"), empty, empty)["out"].shape == (0, W)


@pytest.mark.parametrize("mode", MODES)
def test_gradients_by_differences(mode):
    """A step along a direction changes the loss by the gradients' product with it (float32 kernels)."""
    lens, W = [40, 25], 16
    c = make(lens, W, "f32", seed=13)
    f, b = run(c, mode, "f32")
    g = torch.Generator().manual_seed(1)
    eps = 2.0 ** -6
    dirs = {k: torch.randn(c[k].shape, generator=g).cuda() for k in ("x", "la", "init")}
    dirs["la"] *= c["la"].abs().clamp(max=1) * 0.5   # keeps the log-gates negative

    def loss(sign):
        d = dict(c, **{k: c[k] + sign * eps * dirs[k] for k in dirs})
        r, _ = run(d, mode, "f32")
        return float((d["d_out"].double() * r["out"].double()).sum() +
                     (d["d_final"].double() * r["final_state"].double()).sum())

    fd = (loss(1) - loss(-1)) / (2 * eps)
    by = {"x": "dx", "la": "d_log_gate", "init": "d_initial_state"}
    terms = [float((b[by[k]].double() * dirs[k].double()).sum()) for k in dirs]
    size = sum(float((b[by[k]].double() * dirs[k].double()).abs().sum()) for k in dirs)
    # eps^2 / 6 times a third derivative (of products of a few such factors), and the losses' rounding over 2 eps
    assert abs(fd - sum(terms)) < 4 * eps * eps * size + 2.0 ** -20 * size / eps


def _guarded(shape, dtype):
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((8192 + n,), 0x5A, dtype=torch.uint8, device="cuda")
    return raw[4096:4096 + n].view(dtype).view(*shape), raw


def test_writes_only_its_outputs_and_repeats_itself(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    lens, W = [300, 0, 1, 517], 136
    c = make(lens, W, dtype, seed=14)
    ref, ref_b = run(c, "unit", dtype)
    out, r0 = _guarded((818, W), torch.bfloat16)
    fin, r1 = _guarded((4, W), torch.float32)
    ck, r2 = _guarded((13, W), torch.float32)
    cfg = binding.make_scan_config(W, "unit", dtype)
    got = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=c["init"], out=out, final_state=fin,
                               checkpoints=ck)
    b = binding.scan_backward(cfg, c["x"], c["la"], c["cu"], got["checkpoints"], c["d_out"], initial_state=c["init"],
                              d_final_state=c["d_final"])
    torch.cuda.synchronize()
    for raw in (r0, r1, r2):
        assert bool((raw[:4096] == 0x5A).all()) and bool((raw[-4096:] == 0x5A).all())
    assert torch.equal(out, ref["out"]) and torch.equal(fin, ref["final_state"]) and torch.equal(ck, ref["checkpoints"])
    for k in b:
        assert torch.equal(b[k], ref_b[k])


def test_many_sequences_and_long_axis(dtype="bf16"):
    """700 ragged sequences, and one of 30000 tokens: sampled channels against the oracle."""
    rng = np.random.default_rng(3)
    for lens in (rng.integers(0, 40, 700).tolist(), [30000], [20000, 3, 4000]):
        c = make(lens, 256, dtype, seed=15)
        f, b = run(c, "unit", dtype)
        pick = [0, 63, 64, 200, 255]
        sub = {k: (c[k][:, pick] if k in ("x", "la", "d_out", "init", "d_final") else c[k]) for k in c}
        check(sub, "unit", dtype, {k: f[k][:, pick] for k in ("out", "final_state")},
              {k: b[k][:, pick] for k in b})


def test_wide_rows(dtype="bf16"):
    """More channel groups than the GPU holds at once."""
    c = make([520, 70], 24000, dtype, seed=16)
    f, b = run(c, "complement", dtype)
    pick = [0, 1, 7777, 12345, 23999]
    sub = {k: (c[k][:, pick] if k in ("x", "la", "d_out", "init", "d_final") else c[k]) for k in c}
    check(sub, "complement", dtype, {k: f[k][:, pick] for k in ("out", "final_state")}, {k: b[k][:, pick] for k in b})


def _pick(c, f, b, cols):
    sub = {k: (c[k][:, cols] if k in ("x", "la", "d_out", "init", "d_final") else c[k]) for k in c}
    return sub, {k: f[k][:, cols] for k in ("out", "final_state")}, {k: b[k][:, cols] for k in b}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype,width", [("bf16", 2048), ("f32", 1024)])
def test_enough_columns_to_fill_the_gpu(dtype, width, mode):
    """Widths whose clusters fill the GPU (the form that keeps rows in registers, for the costly input factors): ragged
    lengths with several starts and ends in one tile, emptied and kept states, the final state over the initial one."""
    lens = [2600, 0, 5, 700, 1, 1, 130, 9, 3, 250]
    c = make(lens, width, dtype, seed=18)
    c["la"][7::41, 3] = float("-inf")
    c["la"][5::37, 5] = 0.0
    c["la"][4000:, 64:128] = -3.0   # a column whose log-gates leave [-1/2, 0] in its last tiles only
    f, b = run(c, mode, dtype)
    cols = [0, 3, 5, 31, 32, 63, 64, 100, 500, width - 1]
    sub, sub_f, sub_b = _pick(c, f, b, cols)
    check(sub, mode, dtype, sub_f, sub_b)
    from sparse_state_linear_router_gb300 import binding
    state = c["init"].clone()
    cfg = binding.make_scan_config(width, mode, dtype)
    got = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=state, final_state=state)
    torch.cuda.synchronize()
    assert torch.equal(got["out"], f["out"]) and torch.equal(state, f["final_state"])
    c["x"][2605 + 350, 70] = float("nan")   # in the sequence of 700
    bad, bad_b = run(c, mode, dtype)
    same = torch.ones(sum(lens), width, dtype=torch.bool, device="cuda")
    same[2955:3305, 70] = False
    assert torch.equal(bad["out"][same], f["out"][same])
    assert not bool(torch.isfinite(bad["out"][2955:3305, 70]).any())
    same[2955, 70] = False
    assert torch.equal(bad_b["d_log_gate"][same], b["d_log_gate"][same])
    assert torch.equal(bad_b["dx"], b["dx"])


def test_calls_side_by_side(dtype="bf16"):
    """Different calls in flight on several streams at once: nothing is shared."""
    from sparse_state_linear_router_gb300 import binding
    sets = [make([900 + 100 * i, 7, 0, 333], 256 * (i + 1), dtype, seed=30 + i) for i in range(4)]
    want = [run(c, "unit", dtype) for c in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got = []
        for c, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                cfg = binding.make_scan_config(c["x"].shape[1], "unit", dtype)
                f = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=c["init"], want_checkpoints=True)
                b = binding.scan_backward(cfg, c["x"], c["la"], c["cu"], f["checkpoints"], c["d_out"],
                                          initial_state=c["init"], d_final_state=c["d_final"])
                got.append((f, b))
        torch.cuda.synchronize()
    for (f, b), (wf, wb) in zip(got, want):
        assert torch.equal(f["out"], wf["out"]) and torch.equal(f["final_state"], wf["final_state"])
        for k in b:
            assert torch.equal(b[k], wb[k])


def test_graph_replays_on_new_inputs_and_other_streams(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    W, lens = 320, [800, 3, 0, 211]
    sets = [make(lens, W, dtype, seed=s) for s in (21, 22)]
    want = [run(c, "unit", dtype) for c in sets]
    buf = {k: sets[0][k].clone() for k in ("x", "la", "d_out", "init", "d_final")}
    cfg, cu = binding.make_scan_config(W, "unit", dtype), sets[0]["cu"]

    def call():
        f = binding.scan_forward(cfg, buf["x"], buf["la"], cu, initial_state=buf["init"], want_checkpoints=True)
        b = binding.scan_backward(cfg, buf["x"], buf["la"], cu, f["checkpoints"], buf["d_out"],
                                  initial_state=buf["init"], d_final_state=buf["d_final"])
        return f, b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f, b = call()
        for t in (f["out"], b["dx"]):
            t.record_stream(side)
    side.synchronize()
    assert torch.equal(f["out"], want[0][0]["out"]) and torch.equal(b["dx"], want[0][1]["dx"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f, b = call()
    for c, (wf, wb) in zip(sets + sets[::-1], want + want[::-1]):
        for k in buf:
            buf[k].copy_(c[k])
        g.replay()
        torch.cuda.synchronize()
        for k in ("out", "final_state"):
            assert torch.equal(f[k], wf[k])
        for k in b:
            assert torch.equal(b[k], wb[k])


def test_helpers_refuse(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    c = make([30, 20], 64, dtype, seed=17)
    cfg = binding.make_scan_config(64, "plain", dtype)

    def refused(fn, *a, **kw):
        with pytest.raises(binding.SSEError) as e:
            fn(*a, **kw)
        assert e.value.status in (binding.SSE_ERR_INVALID_ARG, binding.SSE_ERR_UNSUPPORTED)

    fwd, x, la, cu = binding.scan_forward, c["x"], c["la"], c["cu"]
    refused(fwd, cfg, x.float(), la, cu)
    refused(fwd, cfg, x.cpu(), la, cu)
    refused(fwd, cfg, x, la[:-1], cu)
    refused(fwd, cfg, x, la.t().contiguous().t(), cu)            # columns of a row not packed
    refused(fwd, cfg, x, la[:1].expand(50, 64), cu)              # one row for all tokens
    refused(fwd, cfg, x, la, cu.long())
    refused(fwd, cfg, x, la, cu.cpu())
    refused(fwd, cfg, x, la, cu, initial_state=c["init"].bfloat16())
    refused(fwd, cfg, x, la, cu, initial_state=c["init"][:1])
    refused(fwd, cfg, x, la, cu, out=torch.empty(50, 128, dtype=torch.bfloat16, device="cuda")[:, :64])
    refused(fwd, binding.make_scan_config(60, "plain", dtype), x[:, :60], la[:, :60], cu)  # 120-byte rows
    odd = torch.empty(50, 66, dtype=torch.bfloat16, device="cuda")[:, :64]                 # 132-byte row stride
    refused(fwd, cfg, odd, la, cu)
    refused(binding.scan_backward, cfg, x, la, cu, None, c["d_out"])
    refused(binding.scan_backward, cfg, x, la, cu, torch.empty(2, 64, device="cuda"), c["d_out"])
    refused(binding.scan_step, cfg, c["init"], x, la)
    refused(binding.scan_step, cfg, None, x, la)


EVEN = [
    ([512] * 8, 0),                                          # every CTA has a sequence of its own
    ([500, 0, 520, 512, 480, 0, 508, 530, 505, 515, 0], 37),  # nearly so, with empty ones and rows behind
    ([512] * 4 + [2048], 0),                                 # the first clusters' CTAs alone, the last ones together
    ([64] * 61 + [130], 0),                                  # many to a CTA, edges inside tiles
]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype,width", [("bf16", 2048), ("f32", 1024)])
@pytest.mark.parametrize("lens,tail", EVEN, ids=["even", "nearly", "half", "many"])
def test_even_sequences_beside_uneven_ones(lens, tail, dtype, width, mode):
    """Sequences that fall evenly into the parts of a cluster's CTAs (which then exchange nothing), next to some that
    do not; the final states over the initial ones."""
    c = make(lens, width, dtype, seed=23, tail=tail)
    f, b = run(c, mode, dtype)
    sub, sub_f, sub_b = _pick(c, f, b, [0, 1, 31, 63, 64, 129, 700, width - 1])
    check(sub, mode, dtype, sub_f, sub_b)
    from sparse_state_linear_router_gb300 import binding
    state = c["init"].clone()
    cfg = binding.make_scan_config(width, mode, dtype)
    got = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=state, final_state=state)
    torch.cuda.synchronize()
    n = sum(lens)
    assert torch.equal(got["out"][:n], f["out"][:n]) and torch.equal(state, f["final_state"])
