"""Short causal convolution on the GPU against its float64 oracle (marked gpu).

Tolerances are element by element, from running error analysis (tests/_bounds.py):
K products and sums per token, the activation's own error, sums over the tokens
for the weights, and one rounding of the output to its type."""
import numpy as np
import pytest

from oracle import conv as oracle
from tests._bounds import R, close, silu, silu_slope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def make(lens, W, K, dtype, seed, states=True, bias=True, tail=0, extra=0):
    """Inputs on the GPU; `tail` rows behind the last sequence, `extra` columns between rows."""
    g = torch.Generator().manual_seed(seed)
    T, S = sum(lens) + tail, len(lens)
    n = lambda *s: torch.randn(*s, generator=g).to(_dt(dtype)).cuda()  # noqa: E731
    x = n(T, W + extra)[:, :W]
    return {"x": x, "w": torch.randn(W, K, generator=g).cuda(), "bias": torch.randn(W, generator=g).cuda() if bias else None,
            "cu": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda(), "d_out": n(T, W),
            "init": n(S, K - 1, W) if states else None, "d_final": n(S, K - 1, W) if states else None, "n": sum(lens)}


def run(b, c, act, dtype, **kw):
    cfg = b.make_conv_config(c["x"].shape[1], c["w"].shape[1], act, dtype)
    f = b.conv_forward(cfg, c["x"], c["w"], c["cu"], bias=c["bias"], initial_state=c["init"], **kw)
    g = b.conv_backward(cfg, c["x"], c["w"], c["cu"], c["d_out"], bias=c["bias"], initial_state=c["init"],
                        d_final_state=c["d_final"])
    torch.cuda.synchronize()
    return f, g


def check(c, act, dtype, f, g):
    n, cu, half = c["n"], c["cu"].cpu().numpy(), _half(dtype)
    x, w, bias, init, d_fin, dy = (_f64(c[k]) for k in ("x", "w", "bias", "init", "d_final", "d_out"))
    x, dy, K = x[:n], dy[:n], w.shape[1]
    o = oracle.forward(x, w, cu, bias, init, act)
    want = oracle.backward(x, w, cu, dy, bias, init, d_fin, act)
    S, W = len(cu) - 1, w.shape[0]
    outs, dxs, dinits, dws, dbs = [], [], [], [], []
    for q in range(S):
        r, m = o["rows"][q], cu[q + 1] - cu[q]
        taps = np.stack([r[j:j + m] for j in range(K)])  # [K, m, W]
        u = (R(taps) * w.T[:, None, :]).sum(0, K + 1)
        u = u + (np.zeros(W) if bias is None else bias)
        outs.append(silu(u) if act == "silu" else u)
        gr = R(dy[cu[q]:cu[q + 1]])
        if act == "silu":
            gr = gr * silu_slope(u)
        d = R(np.zeros((K - 1 + m, W)))
        for j in range(K):
            p = gr * w[:, j]
            d = d + R(np.pad(p.v, ((j, K - 1 - j), (0, 0))), np.pad(p.e, ((j, K - 1 - j), (0, 0))))
        fin = np.zeros((K - 1 + m, W))
        if d_fin is not None:
            fin[m:] = d_fin[q]
        d = d + fin
        dinits.append(d[:K - 1])
        dxs.append(d[K - 1:])
        dws.append(gr * R(taps))
        dbs.append(gr)
    cat = lambda v, ax=0: R(np.concatenate([i.v for i in v], ax), np.concatenate([i.e for i in v], ax))  # noqa: E731
    pairs = [("out", cat(outs), f["out"][:n], half), ("dx", cat(dxs), g["dx"][:n], half),
             ("d_weight", R(cat(dws, 1).sum(1).v.T, cat(dws, 1).sum(1).e.T), g["d_weight"], 2.0 ** -24)]
    if bias is not None:
        pairs.append(("d_bias", cat(dbs).sum(0), g["d_bias"], 2.0 ** -24))
    else:
        assert g["d_bias"] is None
    for q in range(S):
        pairs.append((f"d_initial_state[{q}]", dinits[q], g["d_initial_state"][q], half))
    for name, bound, got, h in pairs:
        key = name.split("[")[0]
        ref = o["out"] if name == "out" else want[key][int(name[:-1].split("[")[1])] if "[" in name else want[key]
        # the analysis' own values are the oracle's
        np.testing.assert_allclose(bound.v, ref, rtol=1e-9, atol=1e-9)
        close(_f64(got), R(ref, bound.e), h, name)
    assert torch.equal(f["final_state"].cpu(), torch.from_numpy(o["final_state"]).to(f["final_state"].dtype))


SHAPES = [
    ([1], 8, 4), ([2], 16, 4), ([3, 1, 2], 64, 4), ([5, 0, 0, 1, 4, 2, 0], 136, 3), ([40], 128, 2), ([97, 0, 61, 1, 33], 264, 4),
    ([0, 0, 7], 40, 4), ([300], 72, 3), ([8, 8, 8, 8, 31, 32, 33], 520, 4), ([1] * 20, 24, 4), ([2] * 33, 24, 4), ([0], 8, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("lens,W,K", SHAPES)
def test_matches_oracle(b, dtype, act, lens, W, K):
    c = make(lens, W, K, dtype, seed=len(lens) + W + K, extra=8 if W % 3 else 0)
    f, g = run(b, c, act, dtype)
    check(c, act, dtype, f, g)


@pytest.mark.parametrize("states,bias", [(False, True), (True, False), (False, False)])
def test_optional_parts(b, states, bias):
    c = make([9, 0, 70, 2], 72, 4, "bf16", 5, states=states, bias=bias)
    f, g = run(b, c, "silu", "bf16")
    check(c, "silu", "bf16", f, g)


@pytest.mark.parametrize("W", [8, 2048, 4160])
def test_many_tokens(b, W):
    """Runs of every length that the choice makes, sequences cut inside and at the runs' edges."""
    lens = [1, 64, 63, 65, 0, 128, 2, 800, 31, 3] if W > 8 else [700, 1, 0, 2300, 64, 999]
    c = make(lens, W, 4, "bf16", W)
    f, g = run(b, c, "silu", "bf16")
    check(c, "silu", "bf16", f, g)


def test_rows_behind_the_last_sequence_stay(b):
    c = make([5, 40], 64, 4, "bf16", 3, tail=50)
    cfg = b.make_conv_config(64)
    out = torch.full_like(c["d_out"], 7.0)
    for k in ("x", "d_out"):
        c[k][45:] = float("nan")
    f = b.conv_forward(cfg, c["x"], c["w"], c["cu"], bias=c["bias"], initial_state=c["init"], out=out)
    assert bool((out[45:] == 7).all()) and not out[:45].isnan().any()
    g = b.conv_backward(cfg, c["x"], c["w"], c["cu"], c["d_out"], bias=c["bias"], initial_state=c["init"],
                        d_final_state=c["d_final"])
    g["dx"][45:] = 0
    assert all(not v.isnan().any() for v in g.values())
    c["x"], c["d_out"] = c["x"][:45], c["d_out"][:45]
    check(c, "silu", "bf16", {"out": out, "final_state": f["final_state"]}, g)


def test_backward_leaves_the_rows_behind(b):
    """dx rows behind the last sequence through the C call, into a buffer with marks."""
    c = make([5, 40], 64, 4, "bf16", 3, tail=50)
    cfg, P = b.make_conv_config(64), torch.Tensor.data_ptr
    dx, dw = torch.full_like(c["d_out"], 7.0), torch.empty(64, 4, device="cuda")
    n = b.sse_conv_backward_workspace_size(cfg, 95)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert b.sse_conv_backward(cfg, P(c["x"]), c["x"].stride(0), P(c["w"]), P(c["bias"]), P(c["cu"]), 2, 95, None,
                               P(c["d_out"]), None, P(dx), P(dw), None, None, P(ws), n, None) == b.SSE_OK
    torch.cuda.synchronize()
    assert bool((dx[45:] == 7).all()) and not bool((dx[:45] == 7).all())


def test_nan_stays_in_reach(b):
    """A NaN reaches the K tokens that read it, in its own sequence and channel."""
    c = make([30, 30], 64, 4, "bf16", 9)
    c["x"][28, 5] = float("nan")
    f, g = run(b, c, "silu", "bf16")
    want = torch.zeros(60, 64, dtype=torch.bool)
    want[28:30, 5] = True
    assert torch.equal(f["out"].isnan().cpu(), want)
    assert torch.equal(f["final_state"].isnan().nonzero().cpu(), torch.tensor([[0, 1, 5]]))
    bad = g["dx"].isnan().cpu()
    assert bool(bad[28, 5]) and not bad[30:].any() and not bad[:, :5].any() and not bad[:25].any()
    assert torch.equal(g["d_weight"].isnan().any(1).nonzero().flatten().cpu(), torch.tensor([5]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,K", [(1, 8, 4), (3, 136, 3), (256, 2048, 4), (5, 4160, 2)])
def test_step_continues_a_forward(b, dtype, B, W, K):
    """Steps from a state give the rows and states of one forward, bit for bit."""
    g = torch.Generator().manual_seed(W)
    x = torch.randn(B, 7, W, generator=g).to(_dt(dtype)).cuda()
    w, bias = torch.randn(W, K, generator=g).cuda(), torch.randn(W, generator=g).cuda()
    cfg = b.make_conv_config(W, K, "silu", dtype)
    cu = torch.arange(0, 7 * B + 1, 7, dtype=torch.int32, device="cuda")
    f = b.conv_forward(cfg, x.reshape(7 * B, W), w, cu, bias=bias)
    state = torch.zeros(B, K - 1, W, dtype=_dt(dtype), device="cuda")
    for t in range(7):
        out = b.conv_step(cfg, state, x[:, t], w, bias=bias)["out"]
        assert torch.equal(out, f["out"].view(B, 7, W)[:, t])
    assert torch.equal(state, f["final_state"])


def test_split_is_bitwise(b):
    """A sequence in two calls, the second from the first's state."""
    c = make([150], 72, 4, "bf16", 4)
    cfg = b.make_conv_config(72)
    whole = b.conv_forward(cfg, c["x"], c["w"], c["cu"], bias=c["bias"], initial_state=c["init"])
    for k in (0, 1, 2, 3, 64, 149, 150):
        cut = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
        p = b.conv_forward(cfg, c["x"][:k], c["w"], cut(k), bias=c["bias"], initial_state=c["init"])
        q = b.conv_forward(cfg, c["x"][k:], c["w"], cut(150 - k), bias=c["bias"], initial_state=p["final_state"])
        assert torch.equal(torch.cat([p["out"], q["out"]]), whole["out"])
        assert torch.equal(q["final_state"], whole["final_state"])


def test_no_tokens(b):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    w, cu = torch.ones(64, 4, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    init = torch.randn(2, 3, 64, device="cuda").bfloat16()
    cfg = b.make_conv_config(64)
    f = b.conv_forward(cfg, x, w, cu, initial_state=init)
    assert torch.equal(f["final_state"], init)
    g = b.conv_backward(cfg, x, w, cu, x, bias=w[:, 0].contiguous(), initial_state=init, d_final_state=2 * init)
    assert torch.equal(g["d_initial_state"], 2 * init) and not g["d_weight"].any() and not g["d_bias"].any()
    g = b.conv_backward(cfg, x, w, cu[:1], x, initial_state=init[:0])
    assert not g["d_weight"].any()


def test_row_offsets_past_32_bits(b):
    """The last rows of a tensor of more than 2^32 elements are the rows of a short call."""
    W, T = 8192, (1 << 19) + 100
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-90:] = torch.randn(90, W, generator=g, device="cuda").bfloat16()
    w = torch.randn(W, 4, generator=g, device="cuda")
    cu = torch.tensor([0, T - 90, T], dtype=torch.int32, device="cuda")
    cfg = b.make_conv_config(W)
    out = b.conv_forward(cfg, x, w, cu)["out"]
    short = b.conv_forward(cfg, x[-90:], w, torch.tensor([0, 90], dtype=torch.int32, device="cuda"))["out"]
    assert torch.equal(out[-90:], short)
    dx = b.conv_backward(cfg, x, w, cu, x, want_d_initial_state=False)["dx"]
    short = b.conv_backward(cfg, x[-90:], w, torch.tensor([0, 90], dtype=torch.int32, device="cuda"),
                            x[-90:], want_d_initial_state=False)["dx"]
    assert torch.equal(dx[-90:], short)


def test_graph_stream_and_repeat(b):
    """Calls repeat bit for bit, on another stream and replayed from two graphs at the same time."""
    c = make([33, 0, 90], 136, 4, "bf16", 8)
    f, g = run(b, c, "silu", "bf16")
    want = [f["out"], f["final_state"], *g.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f, g = run(b, c, "silu", "bf16")
    for a, e in zip([f["out"], f["final_state"], *g.values()], want):
        assert torch.equal(a, e)
    cfg = b.make_conv_config(136)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = b.conv_forward(cfg, c["x"], c["w"], c["cu"], bias=c["bias"], initial_state=c["init"])
            g = b.conv_backward(cfg, c["x"], c["w"], c["cu"], c["d_out"], bias=c["bias"], initial_state=c["init"],
                                d_final_state=c["d_final"])
        graphs.append((graph, [f["out"], f["final_state"], *g.values()]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for (graph, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for a, e in zip(got, want):
            assert torch.equal(a, e)


def test_helpers_refuse(b):
    c = make([6], 64, 4, "bf16", 1)
    cfg = b.make_conv_config(64)
    x, w, cu, d = c["x"], c["w"], c["cu"], c["d_out"]
    st = torch.zeros(6, 3, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: b.conv_forward(cfg, None, w, cu), lambda: b.conv_forward(cfg, x, None, cu),
                 lambda: b.conv_forward(cfg, x, w[:, :3], cu), lambda: b.conv_forward(cfg, x, w.bfloat16(), cu),
                 lambda: b.conv_forward(cfg, x.float(), w, cu), lambda: b.conv_forward(cfg, x, w, cu.long()),
                 lambda: b.conv_forward(cfg, x, w, None), lambda: b.conv_forward(cfg, x.cpu(), w, cu),
                 lambda: b.conv_forward(cfg, x, w, cu, initial_state=c["init"].float()),
                 lambda: b.conv_forward(cfg, x, w, cu, initial_state=c["init"][:, :2]),
                 lambda: b.conv_forward(cfg, x, w, cu, initial_state=c["init"], final_state=c["init"]),
                 lambda: b.conv_forward(cfg, x[:, ::2], w, cu), lambda: b.conv_forward(cfg, x, w, cu, out=x[:3]),
                 lambda: b.conv_backward(cfg, x, w, cu, None), lambda: b.conv_backward(cfg, x, w, cu, d[:5]),
                 lambda: b.conv_backward(cfg, x, w, cu, d, workspace=torch.empty(16, device="cuda")),
                 lambda: b.conv_step(cfg, None, x, w), lambda: b.conv_step(cfg, st[:5], x, w),
                 lambda: b.conv_step(cfg, st.float(), x, w), lambda: b.conv_step(cfg, st, x, None)):
        with pytest.raises(b.SSEError) as e:
            call()
        assert e.value.status == b.SSE_ERR_INVALID_ARG
    with pytest.raises(b.SSEError) as e:
        b.conv_backward(cfg, x, w, cu, d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == b.SSE_ERR_WORKSPACE
