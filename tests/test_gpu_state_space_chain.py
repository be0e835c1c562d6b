"""The operators of a selective state space block as a model uses them, one
after another (marked gpu): the layer norm with the residual stream, the
projection to the mixer's input and its gate, the short convolution, the
projection to steps, B and C, the selective scan, the projection back and the
next layer norm.  Each stage is checked against its float64 oracle on the values
it was given; the whole run is replayed as one CUDA graph; the gradients run
back through all of it; a prompt is continued token by token."""
import numpy as np
import pytest

from oracle import conv as conv_oracle
from oracle import layer_norm as norm_oracle
from oracle import selective as scan_oracle
from tests._helpers import max_abs_rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, W, N, K, RANK = 128, 256, 16, 4, 16   # model width, channels, states, taps, rank of the steps
LENS = [150, 0, 61, 1]
TOL = 2e-2                               # the bf16 tolerance of the other layers' runs (tests/_helpers.py)


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


def _np(t):
    return t.detach().double().cpu().numpy()


def _setup(seed, T=sum(LENS)):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    f = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).cuda()  # noqa: E731
    return {"x": n(T, D), "r": n(T, D, std=2.0), "w1": f(D, std=0.1, mean=1), "b1": f(D, std=0.1), "w2": f(D, std=0.1, mean=1),
            "w_in": n(2 * W, D, std=D ** -0.5), "w_conv": f(W, K, std=0.5), "b_conv": f(W, std=0.1),
            "w_x": n(RANK + 2 * N, W, std=W ** -0.5), "w_dt": n(W, RANK, std=RANK ** -0.5), "dt_bias": f(W) - 3,
            "A": -torch.exp(f(W, N, std=0.5)), "skip": f(W), "w_out": n(D, W, std=W ** -0.5)}


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def _block(b, p, cu, states=(None, None)):
    ln, cv, sc = b.make_layer_norm_config(D), b.make_conv_config(W, K), b.make_selective_config(W, N)
    s = {"ln": b.layer_norm(ln, p["x"], p["w1"], p["b1"], residual=p["r"])}
    s["xz"] = s["ln"]["out"] @ p["w_in"].t()
    s["conv"] = b.conv_forward(cv, s["xz"][:, :W], p["w_conv"], cu, bias=p["b_conv"], initial_state=states[0])
    s["dbc"] = s["conv"]["out"] @ p["w_x"].t()
    s["delta"] = s["dbc"][:, :RANK] @ p["w_dt"].t()
    s["args"] = (s["conv"]["out"], s["delta"], p["A"], s["dbc"][:, RANK:RANK + N].unflatten(1, (1, N)),
                 s["dbc"][:, RANK + N:].unflatten(1, (1, N)), cu)
    s["kw"] = dict(delta_bias=p["dt_bias"], skip=p["skip"], gate=s["xz"][:, W:], initial_state=states[1])
    s["scan"] = b.selective_forward(sc, *s["args"], want_checkpoints=True, **s["kw"])
    s["back"] = s["scan"]["out"] @ p["w_out"].t()
    s["next"] = b.layer_norm(ln, s["back"], p["w2"], residual=s["ln"]["residual_out"])
    return s


def test_block(b):
    cu, p = _cu(LENS), _setup(1)
    s = _block(b, p, cu)
    torch.cuda.synchronize()
    n, hcu = {k: _np(v) for k, v in p.items()}, cu.cpu().numpy()
    want = norm_oracle.forward(n["x"], n["w1"], n["b1"], n["r"])
    assert max_abs_rel(_np(s["ln"]["out"]), want["out"]) < TOL
    assert max_abs_rel(_np(s["ln"]["residual_out"]), want["residual_out"]) < TOL
    xz = _np(s["xz"])
    want = conv_oracle.forward(xz[:, :W], n["w_conv"], hcu, n["b_conv"])
    assert max_abs_rel(_np(s["conv"]["out"]), want["out"]) < TOL
    args = [_np(v) for v in s["args"][:5]]
    want = scan_oracle.forward(*args, hcu, n["dt_bias"], n["skip"], xz[:, W:])
    assert max_abs_rel(_np(s["scan"]["out"]), want["out"]) < TOL
    assert max_abs_rel(_np(s["scan"]["final_state"]), want["final_state"]) < TOL
    want = norm_oracle.forward(_np(s["back"]), n["w2"], None, _np(s["ln"]["residual_out"]))
    assert max_abs_rel(_np(s["next"]["out"]), want["out"]) < TOL
    assert max_abs_rel(_np(s["next"]["residual_out"]), want["residual_out"]) < TOL


def _gradients(b, p, s, d_next, cu):
    ln, cv, sc = b.make_layer_norm_config(D), b.make_conv_config(W, K), b.make_selective_config(W, N)
    g = {"next": b.layer_norm_backward(ln, s["next"]["residual_out"], p["w2"], d_next)}
    g["d_scan"] = g["next"]["dx"] @ p["w_out"]
    g["scan"] = b.selective_backward(sc, *s["args"], s["scan"]["checkpoints"], g["d_scan"], **s["kw"])
    d_dbc = torch.cat([g["scan"]["d_delta"] @ p["w_dt"], g["scan"]["d_B"].flatten(1), g["scan"]["d_C"].flatten(1)], 1)
    g["d_conv"] = g["scan"]["dx"] + d_dbc @ p["w_x"]
    g["conv"] = b.conv_backward(cv, s["xz"][:, :W], p["w_conv"], cu, g["d_conv"], bias=p["b_conv"])
    g["d_ln"] = torch.cat([g["conv"]["dx"], g["scan"]["d_gate"]], 1) @ p["w_in"]
    g["ln"] = b.layer_norm_backward(ln, s["ln"]["residual_out"], p["w1"], g["d_ln"], d_residual_out=g["next"]["dx"])
    return g


def test_gradients(b):
    cu, p = _cu(LENS), _setup(2)
    s = _block(b, p, cu)
    d_next = torch.randn(sum(LENS), D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    g = _gradients(b, p, s, d_next, cu)
    torch.cuda.synchronize()
    n, hcu, xz = {k: _np(v) for k, v in p.items()}, cu.cpu().numpy(), _np(s["xz"])
    want = norm_oracle.backward(_np(s["next"]["residual_out"]), n["w2"], _np(d_next))
    for k in ("dx", "d_weight", "d_bias"):
        assert max_abs_rel(_np(g["next"][k]), want[k]) < TOL, k
    args = [_np(v) for v in s["args"][:5]]
    want = scan_oracle.backward(*args, hcu, _np(g["d_scan"]), n["dt_bias"], n["skip"], xz[:, W:])
    for k, v in g["scan"].items():
        assert max_abs_rel(_np(v), want[k]) < TOL, k
    want = conv_oracle.backward(xz[:, :W], n["w_conv"], hcu, _np(g["d_conv"]), n["b_conv"])
    for k, v in g["conv"].items():
        assert max_abs_rel(_np(v), want[k]) < TOL, k
    want = norm_oracle.backward(_np(s["ln"]["residual_out"]), n["w1"], _np(g["d_ln"]), _np(g["next"]["dx"]))
    for k in ("dx", "d_weight", "d_bias"):
        assert max_abs_rel(_np(g["ln"][k]), want[k]) < TOL, k


def test_training_step_replays_as_one_graph(b):
    cu, p, q = _cu(LENS), _setup(4), _setup(5)
    d_next = torch.randn(sum(LENS), D, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()

    def step(v):
        s = _block(b, v, cu)
        g = _gradients(b, v, s, d_next, cu)
        return {"out": s["next"]["out"], "dx": g["ln"]["dx"], **{"scan_" + k: t for k, t in g["scan"].items()},
                **{"conv_" + k: t for k, t in g["conv"].items()}}

    want = []
    for v in (p, q):
        want.append({k: t.clone() for k, t in step(v).items()})
        torch.cuda.synchronize()
    buf = {k: v.clone() for k, v in p.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for v, w in ((q, want[1]), (p, want[0])):
        for k in buf:
            buf[k].copy_(v[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in w:
            assert torch.equal(got[k], w[k]), k


def test_prompt_then_tokens(b):
    """A prompt of 70 tokens, then five tokens through the steps: the block over 75 tokens, stage by stage."""
    p = _setup(7, 75)
    whole = _block(b, p, _cu([75]))
    head = _block(b, {**p, "x": p["x"][:70], "r": p["r"][:70]}, _cu([70]))
    conv_state, state = head["conv"]["final_state"], head["scan"]["final_state"]
    cv, sc = b.make_conv_config(W, K), b.make_selective_config(W, N)
    for t in range(70, 75):
        xz = whole["xz"][t:t + 1]
        c = b.conv_step(cv, conv_state, xz[:, :W], p["w_conv"], bias=p["b_conv"])["out"]
        assert torch.equal(c, whole["conv"]["out"][t:t + 1])
        delta, B, C = (v[t:t + 1] for v in (whole["args"][1], whole["args"][3], whole["args"][4]))
        o = b.selective_step(sc, state, c, delta, p["A"], B, C, delta_bias=p["dt_bias"], skip=p["skip"], gate=xz[:, W:])["out"]
        assert max_abs_rel(_np(o), _np(whole["scan"]["out"][t:t + 1])) < TOL
    assert torch.equal(conv_state, whole["conv"]["final_state"])
    assert max_abs_rel(_np(state), _np(whole["scan"]["final_state"])) < 1e-4
