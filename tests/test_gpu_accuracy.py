"""Float32 accuracy of the scan and the block norms against float64 where
approximate instructions, or the order of a sum, could lose it (marked gpu).
u = 2^-24 is half a step of float32 next to 1; rsqrt.approx is at most
2^-22.9 off."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
ROOT = 2.0 ** -22.9


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


def _f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("each", [False, True], ids=["one", "many"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slope_of_the_unit_input_factor(b, dtype, each):
    """s = sqrt(1 - a^2) and its slope -a^2 / s for log-gates between 0 and -2^-32, read off from a token with x = 1
    and d_out = 1 that no other token reaches: d_log_gate is the slope, dx is s.

    There a and a^2 round to 1 and 1 - a^2 to -2 log_gate without an error, so what is left is one root in the slope
    (2^-22.9) and in s, which may be formed from the reciprocal root, another product (u).  With a token in every
    sequence a comes from the exponential: at most 2^-22 + u off (ex2.approx and a product), twice that and u in a^2,
    and the series for 1 - a^2 at most 1e-7.  2^-30 covers 1 - a^2 against 1 and the second order."""
    T, W = 96, 4096
    g = torch.Generator().manual_seed(3)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    la = -(2.0 ** (torch.rand(T, W, generator=g) * -90 - 32))      # from 2^-122 to 2^-32
    la = la.to(dt).cuda()
    if each:
        cu, at = torch.arange(T + 1), None
        x = d = torch.ones(T, W)
    else:
        cu, at = torch.tensor([0, T]), torch.randint(16, T - 16, (W,), generator=g)   # no first or last rows
        x = d = torch.zeros(T, W).scatter_(0, at[None], 1.0)
    cu, x, d = cu.int().cuda(), x.to(dt).cuda(), d.to(dt).cuda()
    cfg = b.make_scan_config(W, "unit", dtype)
    f = b.scan_forward(cfg, x, la, cu, want_checkpoints=True)
    r = b.scan_backward(cfg, x, la, cu, f["checkpoints"], d)
    torch.cuda.synchronize()
    l64 = _f64(la)
    s = np.sqrt(-np.expm1(2 * l64))
    slope = -np.exp(2 * l64) / s
    got_slope, got_s = _f64(r["d_log_gate"]), _f64(r["dx"])
    if not each:
        pick = at.numpy(), np.arange(W)
        s, slope, got_slope, got_s = (v[pick] for v in (s, slope, got_slope, got_s))
    half = 0.0 if dtype == "f32" else torch.finfo(dt).eps / 2
    slack = 2.0 ** -30 + half
    gate = 2 * (2.0 ** -22 + U) + U if each else 0.0
    series = 0.5e-7 if each else 0.0
    worst = np.abs(got_slope / slope - 1).max()
    assert worst <= ROOT + gate + series + 2 * U * each + slack, worst
    worst = np.abs(got_s / s - 1).max()
    assert worst <= ROOT + U + series + slack, worst


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_float32_gates(b, gate):
    """act(z) and act'(z) of float32 gates from -86 to 30.

    sigma = 1 / (1 + exp(-z)): exp at most 2 units in the last place off (4 u), the sum rounded (u), the reciprocal
    one unit off (2 u): 7 u.  act: one product more, and those with the block's output of 1 are exact.  act' = sigma
    (1 - sigma) or sigma (1 + z (1 - sigma)): 1 - sigma is off by 7 u sigma + u, z times that and its own rounding in
    the sum, and one more product."""
    W, T = 1024, 32
    z = torch.linspace(-86, 30, T * W).reshape(T, W).cuda()
    one = torch.ones(T, W, device="cuda")
    cfg = b.make_norm_config(W, gate=gate, dtype="f32")
    f = b.block_norm(cfg, one, gate=z)["residual_out"]
    r = b.block_norm_backward(cfg, one, one, gate=z)
    torch.cuda.synchronize()
    z = _f64(z)
    sg = 1 / (1 + np.exp(-z))
    rest = 1 / (1 + np.exp(z))              # 1 - sigma
    act = z * sg if gate == "silu" else sg
    for got in (_f64(f), _f64(r["d_block_out"])):
        bad = np.abs(got - act) > 8.5 * U * np.abs(act)
        assert not bad.any(), (bad.sum(), z[bad][0], got[bad][0], act[bad][0])
    inner = 1 + z * rest if gate == "silu" else rest
    off = (np.abs(z) if gate == "silu" else 1.0) * (7 * U * sg + U)
    tol = sg * (off + 9 * U * np.abs(inner) + U)
    bad = np.abs(_f64(r["d_gate"]) - sg * inner) > 1.01 * tol
    assert not bad.any(), (bad.sum(), z[bad][0])


@pytest.mark.parametrize("group", [4096, 2048, 1360])
def test_sums_of_wide_groups(b, group):
    """Norms over float32 groups whose first 16-byte word outweighs every other so far that a sum over the words one
    by one would lose each of them: they are a little under half a step of the first.  The tolerance is that of a
    mean of at most a few hundred serially added terms, 2^-17, its root (half) and u for each product."""
    T, W = 3, group * 2
    o = torch.full((T, W), (0.9 * 2.0 ** -24) ** 0.5)
    o[:, ::group], o[:, 1::group], o[:, 2::group], o[:, 3::group] = 1.0, 1.0, 1.0, 1.0   # sum 4, half a step 2^-22
    o = o.cuda()
    w = torch.ones(W, device="cuda")
    cfg = b.make_norm_config(W, group=group, eps=1e-12, dtype="f32")
    f = b.block_norm(cfg, o, w_after=w)["residual_out"]
    d = torch.ones(T, W, device="cuda")
    r = b.block_norm_backward(cfg, d, o, w_after=w)
    torch.cuda.synchronize()
    v = _f64(o).reshape(T, 2, group)
    rstd = 1 / np.sqrt((v * v).mean(axis=2, keepdims=True) + 1e-12)
    hat = v * rstd
    want = hat.reshape(T, W)
    assert (np.abs(_f64(f) / want - 1) <= 2.0 ** -18 + ROOT + 4 * U).all()
    dot = hat.mean(axis=2, keepdims=True)
    back = (rstd * (1 - hat * dot)).reshape(T, W)
    size = (rstd * (1 + np.abs(hat * dot))).reshape(T, W)
    assert (np.abs(_f64(r["d_block_out"]) - back) <= (2.0 ** -16 + 8 * U) * size).all()
