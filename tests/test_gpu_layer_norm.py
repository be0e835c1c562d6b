"""Layer norm on the GPU against its float64 oracle (marked gpu).

Tolerances are element by element, from running error analysis (tests/_bounds.py):
sums over the row in any order, a reciprocal root 2^-22 off, and one rounding of
the output to its type."""
import numpy as np
import pytest

from oracle import layer_norm as oracle
from tests._bounds import R, ROUND, close

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-5


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


def make(T, W, dtype, seed, mean=1.0, extra=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(_dt(dtype)).cuda()  # noqa: E731
    v = lambda std, mean: (torch.randn(W, generator=g) * std + mean).cuda()  # noqa: E731
    return {"x": n(T, W + extra, std=2.0, mean=mean)[:, :W], "r": n(T, W + extra, std=0.7)[:, :W], "w": v(0.3, 1.0),
            "b": v(0.3, 0.0), "d_out": n(T, W), "d_r": n(T, W)}


def _terms(W):
    # a thread's 32 elements one after the other (16 float32), five shuffles, up to 32 warps' sums
    return 32 + 5 + 32


def _moments(r, W):
    """d = r - mean, and rstd, as bounds.  The mean's error goes into every d."""
    n = _terms(W)
    mean = r.sum(1, n) * (1.0 / W)
    d = r - R(mean.v[:, None], mean.e[:, None])
    # the squares about a mean that is off by e are off by W e^2 in sum: second order, in the products' bounds
    var = (d * d).sum(1, n) * (1.0 / W) + EPS
    rstd = 1 / np.sqrt(var.v)
    return d, R(rstd[:, None], (rstd * (0.5 * var.e / var.v * 1.01 + 4 * ROUND))[:, None])


def check(c, dtype, f, g, residual, weight=True, bias=True, d_res=True):
    half = _half(dtype)
    x, r, w, bb, dy, dr = (_f64(c[k]) for k in ("x", "r", "w", "b", "d_out", "d_r"))
    T, W = x.shape
    o = oracle.forward(x, w if weight else None, bb if bias else None, r if residual else None, EPS)
    s = R(x) + r if residual else R(x)
    d, rstd = _moments(s, W)
    out = d * rstd
    if weight:
        out = out * w
    if bias:
        out = out + bb
    np.testing.assert_allclose(out.v, o["out"], rtol=1e-9, atol=1e-9)
    close(_f64(f["out"]), out, half, "out")
    if residual:
        close(_f64(f["residual_out"]), s, half, "residual_out")
    # backward at the stored stream
    at = _f64(f["residual_out"]) if residual else x
    want = oracle.backward(at, w if weight else None, dy, dr if d_res else None, EPS)
    d, rstd = _moments(R(at), W)
    p = R(dy) * w if weight else R(dy)
    n = _terms(W)
    mp, mx = p.sum(1, n) * (1.0 / W), (p * d).sum(1, n) * (1.0 / W)
    col = lambda v: R(v.v[:, None], v.e[:, None])  # noqa: E731
    dx = (p - col(mp) - d * (col(mx) * rstd * rstd)) * rstd
    if d_res:
        dx = dx + dr
    np.testing.assert_allclose(dx.v, want["dx"], rtol=1e-8, atol=1e-8)
    close(_f64(g["dx"]), dx, half, "dx")
    close(_f64(g["d_weight"]), (R(dy) * (d * rstd)).sum(0), 2.0 ** -24, "d_weight")
    close(_f64(g["d_bias"]), R(dy).sum(0), 2.0 ** -24, "d_bias")


def run(b, c, dtype, residual, weight=True, bias=True, d_res=True):
    cfg = b.make_layer_norm_config(c["x"].shape[1], EPS, dtype)
    f = b.layer_norm(cfg, c["x"], c["w"] if weight else None, c["b"] if bias else None, residual=c["r"] if residual else None)
    g = b.layer_norm_backward(cfg, f["residual_out"] if residual else c["x"], c["w"] if weight else None, c["d_out"],
                              d_residual_out=c["d_r"] if d_res else None)
    torch.cuda.synchronize()
    return f, g


# one warp and many, words per thread of every kind, rows that fill no warp
WIDTHS = {"bf16": [8, 16, 264, 512, 520, 768, 1024, 1032, 2048, 2304, 4096, 8192, 8200, 16384],
          "f32": [4, 12, 128, 132, 260, 512, 516, 1000, 2048, 4096, 4100, 8192]}


@pytest.mark.parametrize("dtype,W", [(d, w) for d in WIDTHS for w in WIDTHS[d]])
@pytest.mark.parametrize("residual", [False, True])
def test_matches_oracle(b, dtype, W, residual):
    c = make(11, W, dtype, W, extra=8 if W % 3 else 0)
    f, g = run(b, c, dtype, residual)
    check(c, dtype, f, g, residual)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 700, 4097])
def test_many_rows(b, T):
    for W in (64, 520):
        c = make(T, W, "bf16", T)
        f, g = run(b, c, "bf16", True)
        check(c, "bf16", f, g, True)


@pytest.mark.parametrize("weight,bias,d_res", [(False, False, True), (True, False, False), (False, True, False)])
def test_optional_parts(b, weight, bias, d_res):
    c = make(9, 520, "bf16", 3)
    f, g = run(b, c, "bf16", False, weight, bias, d_res)
    assert f["residual_out"] is None
    check(c, "bf16", f, g, False, weight, bias, d_res)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_from_zero(b, dtype):
    """A mean of a thousand deviations: the squares are about the mean, not the difference of two sums."""
    c = make(7, 2048, dtype, 2, mean=2000.0)
    f, g = run(b, c, dtype, False)
    check(c, dtype, f, g, False)


def test_constant_rows(b):
    """Variance zero: out is the bias, the gradient finite."""
    x = torch.full((5, 1024), 3.0, dtype=torch.bfloat16, device="cuda")
    c = make(5, 1024, "bf16", 1)
    cfg = b.make_layer_norm_config(1024, EPS)
    out = b.layer_norm(cfg, x, c["w"], c["b"])["out"]
    assert torch.equal(out, c["b"].bfloat16().expand(5, -1))
    g = b.layer_norm_backward(cfg, x, c["w"], c["d_out"])
    assert bool(g["dx"].isfinite().all()) and not g["d_weight"].any()


def test_nan_stays_in_its_row(b):
    c = make(40, 520, "bf16", 1)
    c["x"][17, 3] = float("nan")
    f, g = run(b, c, "bf16", True)
    assert torch.equal(f["out"].isnan().any(1).nonzero().flatten().cpu(), torch.tensor([17]))
    assert torch.equal(g["dx"].isnan().any(1).nonzero().flatten().cpu(), torch.tensor([17]))


def test_in_place_residual_stream(b):
    c = make(300, 520, "bf16", 6)
    cfg = b.make_layer_norm_config(520, EPS)
    want = b.layer_norm(cfg, c["x"], c["w"], c["b"], residual=c["r"])
    for which in ("x", "r"):
        a = {k: c[k].clone() for k in ("x", "r")}
        got = b.layer_norm(cfg, a["x"], c["w"], c["b"], residual=a["r"], residual_out=a[which])
        assert torch.equal(got["out"], want["out"]) and torch.equal(a[which], want["residual_out"])


def test_no_tokens(b):
    cfg = b.make_layer_norm_config(64, EPS)
    x, w = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    assert b.layer_norm(cfg, x, w, w, residual=x)["out"].shape == (0, 64)
    g = b.layer_norm_backward(cfg, x, w, x)
    assert not g["d_weight"].any() and not g["d_bias"].any()


def test_row_offsets_past_32_bits(b):
    W, T = 8192, (1 << 19) + 100
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-90:] = torch.randn(90, W, generator=g, device="cuda").bfloat16()
    cfg = b.make_layer_norm_config(W, EPS)
    w = torch.randn(W, generator=g, device="cuda")
    out = b.layer_norm(cfg, x, w, residual=x)["out"]
    assert torch.equal(out[-90:], b.layer_norm(cfg, x[-90:], w, residual=x[-90:])["out"])
    del out
    dx = b.layer_norm_backward(cfg, x, w, x)["dx"]
    assert torch.equal(dx[-90:], b.layer_norm_backward(cfg, x[-90:], w, x[-90:])["dx"])


def test_graph_stream_and_repeat(b):
    c = make(301, 2304, "bf16", 8)
    f, g = run(b, c, "bf16", True)
    want = [f["out"], f["residual_out"], *g.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f, g = run(b, c, "bf16", True)
    for a, e in zip([f["out"], f["residual_out"], *g.values()], want):
        assert torch.equal(a, e)
    cfg = b.make_layer_norm_config(2304, EPS)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = b.layer_norm(cfg, c["x"], c["w"], c["b"], residual=c["r"])
            g = b.layer_norm_backward(cfg, f["residual_out"], c["w"], c["d_out"], d_residual_out=c["d_r"])
        graphs.append((graph, [f["out"], f["residual_out"], *g.values()]))
    torch.cuda.synchronize()
    for graph, _ in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for a, e in zip(got, want):
            assert torch.equal(a, e)


def test_helpers_refuse(b):
    c = make(6, 64, "bf16", 1)
    cfg, x, w, d = b.make_layer_norm_config(64), c["x"], c["w"], c["d_out"]
    wide = torch.zeros(6, 72, dtype=torch.bfloat16, device="cuda")[:, :64]
    for call in (lambda: b.layer_norm(cfg, None, w), lambda: b.layer_norm(cfg, x.float(), w),
                 lambda: b.layer_norm(cfg, x, w.bfloat16()), lambda: b.layer_norm(cfg, x, w[:32]),
                 lambda: b.layer_norm(cfg, x, w, residual=x[:5]), lambda: b.layer_norm(cfg, x.cpu(), w),
                 lambda: b.layer_norm(cfg, x, w, out=wide), lambda: b.layer_norm(cfg, x[:, :32], w),
                 lambda: b.layer_norm_backward(cfg, x, w, None), lambda: b.layer_norm_backward(cfg, x, w, d[:5]),
                 lambda: b.layer_norm_backward(cfg, x, w, wide),
                 lambda: b.layer_norm_backward(cfg, x, w, d, workspace=torch.empty(16, device="cuda"))):
        with pytest.raises(b.SSEError) as e:
            call()
        assert e.value.status == b.SSE_ERR_INVALID_ARG


def test_long_sums_of_the_weights_gradients(b):
    """Column sums over 2^19 equal rows, of which a team of threads has some 3450: float32 additions in one chain would all be
    off in the same direction."""
    T, W = 1 << 19, 8192
    c = make(1, W, "bf16", 12)
    x, d_out = (c[k].expand(T, -1).contiguous() for k in ("x", "d_out"))
    g = b.layer_norm_backward(b.make_layer_norm_config(W, EPS), x, c["w"], d_out)
    d, rstd = _moments(R(_f64(c["x"])), W)
    chain = 256 + T // 152 // 256 + 8 + 64  # rows of a part, parts, teams in 32 runs, runs
    for k, one in (("d_weight", R(_f64(c["d_out"])) * (d * rstd)), ("d_bias", R(_f64(c["d_out"])))):
        want, tol = T * one.v[0], T * (one.e[0] + chain * ROUND * np.abs(one.v[0]))
        off = np.abs(_f64(g[k]) - want)
        assert (off <= tol).all(), (k, (off / np.abs(want)).max(), (tol / np.abs(want)).max())
