"""The operators as a layer uses them, one after another (marked gpu): norm
before the block, the front end's projections, the mixer (sse_forward or the
scan on the front end's v and log-gate), the per-head norm with its gate and
the residual stream, the next norm before; each stage checked against its
float64 oracle on the values it was given, and the whole run replayed as one
CUDA graph.  The gradients run back through the norms and the scan."""
import numpy as np
import pytest

import oracle
from oracle import block_norm as norm_oracle
from oracle import scan as scan_oracle
from tests._helpers import max_abs_rel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

H, C, N, D = 2, 64, 8, 128           # heads, key = value width, partitions, hidden = H * C
LENS = [150, 0, 61, 1]
TOL = 2e-2                           # the layer's bf16 tolerance (tests/_helpers.py)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _setup(seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(LENS)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    p = {"r": n(T, D, std=2.0), "z": n(T, D)}
    p.update({k: n(H * C, D, std=D ** -0.5) for k in ("w_q", "w_k", "w_v", "w_g")})
    p["w_e"] = n(H * N, D, std=D ** -0.5)
    p.update({k: (torch.randn(D, generator=g) * 0.1 + 1).cuda() for k in ("before", "after", "next")})
    return p


def _layer(p, cu, mixer):
    from sparse_state_linear_router_gb300 import binding as b
    cfg = b.make_config(H, C, C, N, 2)
    pre = b.block_norm(b.make_norm_config(D), residual=p["r"], w_before=p["before"], want_residual_out=False)["next_in"]
    fe = b.front_end(cfg, pre, p["w_q"], p["w_k"], p["w_v"], p["w_g"], p["w_e"])
    s = {"pre": pre, "fe": fe}
    if mixer == "sse":
        s["mix"] = b.forward(cfg, fe["q"], fe["k"], fe["v"], fe["log_gate"], fe["logits"], cu)["out"]
    else:
        s["scan"] = b.scan_forward(b.make_scan_config(D, "unit"), fe["v"], fe["log_gate"], cu, want_checkpoints=True)
        s["mix"] = s["scan"]["out"]
    s["post"] = b.block_norm(b.make_norm_config(D, group=C, gate="silu", residual_scale=0.9), s["mix"], gate=p["z"],
                             residual=p["r"], w_after=p["after"], w_before=p["next"])
    return s


@pytest.mark.parametrize("mixer", ["sse", "scan"])
def test_layer(mixer):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    p = _setup(1)
    s = _layer(p, cu, mixer)
    torch.cuda.synchronize()
    n = {k: _np(v) for k, v in p.items()}
    want = norm_oracle.forward(r=n["r"], w_before=n["before"])["next_in"]
    assert max_abs_rel(_np(s["pre"]), want) < TOL
    fe = {k: _np(v) for k, v in s["fe"].items() if k in ("q", "k", "v", "log_gate", "logits")}
    hcu = cu.cpu().numpy()
    if mixer == "sse":
        want = oracle.forward(*(fe[k].astype(np.float32) for k in ("q", "k", "v", "log_gate", "logits")), hcu,
                              top_k=2, use_shared=1)["out"].reshape(-1, D)
    else:
        want = scan_oracle.forward(fe["v"].reshape(-1, D), fe["log_gate"].reshape(-1, D), hcu, "unit")["out"]
    assert max_abs_rel(_np(s["mix"]).reshape(-1, D), want) < TOL
    want = norm_oracle.forward(_np(s["mix"]).reshape(-1, D), z=n["z"], r=n["r"], w_after=n["after"],
                               w_before=n["next"], group=C, gate="silu", residual_scale=0.9)
    assert max_abs_rel(_np(s["post"]["residual_out"]), want["residual_out"]) < TOL
    assert max_abs_rel(_np(s["post"]["next_in"]), want["next_in"]) < TOL


@pytest.mark.parametrize("mixer", ["sse", "scan"])
def test_layer_replays_as_one_graph(mixer):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    p, q = _setup(2), _setup(3)
    want = []
    for v in (p, q):
        s = _layer(v, cu, mixer)
        torch.cuda.synchronize()
        want.append({k: t.clone() for k, t in s["post"].items()})
    buf = {k: v.clone() for k, v in p.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = _layer(buf, cu, mixer)
    for v, w in ((q, want[1]), (p, want[0])):
        for k in buf:
            buf[k].copy_(v[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in w:
            assert torch.equal(s["post"][k], w[k])


def test_gradients_through_norm_and_scan():
    """Back from the next block's input through the norms and the scan to the front end's v and log-gate."""
    from sparse_state_linear_router_gb300 import binding as b
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32).cuda()
    p = _setup(4)
    s = _layer(p, cu, "scan")
    T = p["r"].shape[0]
    g = torch.Generator().manual_seed(5)
    d_next = torch.randn(T, D, generator=g).bfloat16().cuda()
    gn = b.block_norm_backward(b.make_norm_config(D, group=C, gate="silu", residual_scale=0.9), None, s["mix"],
                               gate=p["z"], w_after=p["after"], w_before=p["next"],
                               residual_out=s["post"]["residual_out"], d_next_in=d_next)
    gs = b.scan_backward(b.make_scan_config(D, "unit"), s["fe"]["v"], s["fe"]["log_gate"], cu,
                         s["scan"]["checkpoints"], gn["d_block_out"])
    torch.cuda.synchronize()
    assert gs["dx"].shape == s["fe"]["v"].shape
    n = {k: _np(v) for k, v in p.items()}
    wn = norm_oracle.backward(None, _np(s["mix"]).reshape(-1, D), z=n["z"], w_after=n["after"], w_before=n["next"],
                              residual_out=_np(s["post"]["residual_out"]), d_next_in=_np(d_next), group=C, gate="silu",
                              residual_scale=0.9)
    for k in ("d_gate", "d_residual", "d_w_after", "d_w_before"):
        assert max_abs_rel(_np(gn[k]), wn[k]) < TOL
    assert max_abs_rel(_np(gn["d_block_out"]).reshape(-1, D), wn["d_block_out"]) < TOL
    ws = scan_oracle.backward(_np(s["fe"]["v"]).reshape(-1, D), _np(s["fe"]["log_gate"]).reshape(-1, D),
                              cu.cpu().numpy(), "unit", _np(gn["d_block_out"]).reshape(-1, D))
    assert max_abs_rel(_np(gs["dx"]).reshape(-1, D), ws["dx"]) < TOL
    assert max_abs_rel(_np(gs["d_log_gate"]).reshape(-1, D), ws["d_log_gate"]) < TOL
