"""Block norms on the GPU against their float64 oracle (marked gpu).

Tolerances are element by element and come from the arithmetic: one rounding
of the output to its type (at most half a step, finfo.eps / 2 of the value)
plus the float32 error of the terms it is the sum of.  A mean of squares of at
most a few hundred serially added terms is 2^-17 off at most, its inverse root
half of that; a sigmoid of |z| < 8 at most 2^-20; every other operation rounds
by 2^-24: R = 2^-16 of the sum of the terms' sizes covers them.  Column sums
add at most a few hundred terms in a row: another 2^-16.  Below float32's
smallest normal value, 2^-126, a gate may be lost altogether: with the other
factors (1 / sqrt(eps) = 2^8.3, the rest a few units) that is at most 2^-110 of
any output.
"""
import numpy as np
import pytest

from oracle import block_norm as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

R = 2.0 ** -16
LEAST = 2.0 ** -110
SET = dict(eps=1e-5, residual_scale=0.8, branch_scale=1.25)


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


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, want, tol, name):
    bad = ~(np.abs(got - want) <= tol + LEAST)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}, tolerance {np.broadcast_to(tol, bad.shape)[bad][0]}")


def make(T, W, dtype, seed, parts="ozracb", extra=0):
    """parts: o block_out, z gate, r residual, a w_after, c channel_scale, b w_before; `extra` columns between rows."""
    g = torch.Generator().manual_seed(seed)

    def rows(std=1.0):
        t = (torch.randn(T, W + extra, generator=g) * std).to(_dt(dtype)).cuda()
        return t[:, :W] if extra else t

    vec = lambda m: (torch.randn(W, generator=g) * 0.3 + m).cuda()  # noqa: E731
    c = {"o": rows(), "z": rows(1.5), "r": rows(2.0), "a": vec(1.0), "c": vec(0.5), "b": vec(1.0)}
    c = {k: (v if k in parts else None) for k, v in c.items()}
    c["at"], c["dr"] = rows(2.0), rows().contiguous()
    c["dn"] = rows().contiguous() if "b" in parts else None
    return c


def config(W, dtype, group, gate):
    from sparse_state_linear_router_gb300 import binding
    return binding.make_norm_config(W, group=group, gate=gate, dtype=dtype, **SET)


def run(c, cfg, **kw):
    from sparse_state_linear_router_gb300 import binding
    f = binding.block_norm(cfg, c["o"], gate=c["z"], residual=c["r"], w_after=c["a"], channel_scale=c["c"],
                           w_before=c["b"], **kw)
    g = binding.block_norm_backward(cfg, c["dr"], c["o"], gate=c["z"], w_after=c["a"], channel_scale=c["c"],
                                    w_before=c["b"], residual_out=c["at"] if c["b"] is not None else None,
                                    d_next_in=c["dn"])
    torch.cuda.synchronize()
    return f, g


def check(c, group, gate, dtype, f, g):
    n = {k: _np(v) for k, v in c.items()}
    W, h, abs_ = n["dr"].shape[1], _half(dtype), np.abs
    o, z, r = n["o"], n["z"], n["r"]
    kw = dict(group=group, gate=gate, **SET)
    want = oracle.forward(o, z=z, r=r, w_after=n["a"], channel=n["c"], w_before=n["b"], **kw)
    res = want["residual_out"]
    size = 0.0
    if r is not None:
        size = size + abs_(SET["residual_scale"] * r)
    if o is not None:
        size = size + abs_(oracle.forward(o, z=z, w_after=n["a"], channel=n["c"], **kw)["residual_out"])
    _close(_np(f["residual_out"]), res, h * abs_(res) + R * size, "residual_out")
    if n["b"] is not None:
        _, rstd = oracle._hat(res, W, SET["eps"])
        _close(_np(f["next_in"]), want["next_in"], h * abs_(want["next_in"]) +
               R * abs_(n["b"]) * rstd * (size + abs_(res)), "next_in")
    grad = oracle.backward(n["dr"], o, z=z, w_after=n["a"], channel=n["c"], w_before=n["b"],
                           residual_out=n["at"] if n["b"] is not None else None, d_next_in=n["dn"], **kw)
    # sizes of the terms, by the same rules with absolute values
    d = abs_(n["dr"])
    if n["b"] is not None:
        hat, rstd = oracle._hat(n["at"], W, SET["eps"])
        t = abs_(n["dn"] * n["b"])
        d = d + rstd * (t + abs_(hat) * (t * abs_(hat)).mean(axis=1, keepdims=True))
        _close(_np(g["d_w_before"]), grad["d_w_before"], 2 * R * abs_(n["dn"] * hat).sum(axis=0), "d_w_before")
    _close(_np(g["d_residual"]), grad["d_residual"], h * abs_(grad["d_residual"]) +
           R * SET["residual_scale"] * d, "d_residual")
    if o is None:
        assert g["d_block_out"] is None and g["d_gate"] is None
        return
    d = SET["branch_scale"] * d
    hat, rstd = oracle._hat(o, group or W, SET["eps"]) if n["a"] is not None else (o, 1.0)
    wa = 1.0 if n["a"] is None else abs_(n["a"])
    ch = 1.0 if n["c"] is None else abs_(n["c"])
    av, da = (1.0, 0.0) if z is None else (abs_(v) for v in oracle.act(z, gate))
    if z is not None:
        # silu' is a sum of two terms of size up to 1 + |z|
        tol = R * d * ch * wa * abs_(hat) * (da + (1 + abs_(z) if gate == "silu" else 1.0) * 0.25)
        _close(_np(g["d_gate"]), grad["d_gate"], h * abs_(grad["d_gate"]) + tol, "d_gate")
    if n["a"] is not None:
        _close(_np(g["d_w_after"]), grad["d_w_after"], 2 * R * (d * ch * av * abs_(hat)).sum(axis=0), "d_w_after")
    if n["c"] is not None:
        _close(_np(g["d_channel_scale"]), grad["d_channel_scale"], 2 * R * (d * av * wa * abs_(hat)).sum(axis=0),
               "d_channel_scale")
    d = d * ch * av * wa
    if n["a"] is not None:
        m = (d * abs_(hat)).reshape(len(d), -1, group or W).mean(axis=2, keepdims=True)
        m = np.broadcast_to(m, (len(d), W // (group or W), group or W)).reshape(d.shape)
        d = rstd * (d + abs_(hat) * m)
    _close(_np(g["d_block_out"]), grad["d_block_out"], h * abs_(grad["d_block_out"]) + R * d, "d_block_out")


SHAPES = [  # tokens, width, group, dtype
    (1, 8, 0, "bf16"), (3, 4, 0, "f32"), (1, 2048, 128, "bf16"), (5, 2304, 0, "bf16"), (77, 256, 64, "bf16"),
    (33, 1000, 0, "f32"), (33, 1000, 40, "f32"), (65, 960, 96, "bf16"), (9, 1536, 768, "bf16"), (200, 72, 8, "bf16"),
    (200, 64, 16, "f32"), (130, 512, 256, "f32"), (7, 4096, 256, "bf16"), (3, 8192, 0, "bf16"), (2, 8200, 8, "bf16"),
    (3, 16384, 128, "bf16"), (2, 16384, 0, "bf16"), (3, 8192, 2048, "f32"), (2, 4100, 0, "f32"), (1500, 264, 0, "bf16"),
    (3001, 128, 32, "f32"),
]


@pytest.mark.parametrize("T,W,group,dtype", SHAPES)
def test_against_the_oracle(T, W, group, dtype):
    c = make(T, W, dtype, seed=T + W)
    check(c, group, "silu", dtype, *run(c, config(W, dtype, group, "silu")))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "silu", "sigmoid", "linear"])
@pytest.mark.parametrize("parts", ["o", "r", "rb", "oa", "or", "oac", "ob", "oab", "ocrb", "oarb", "oacrb"])
def test_every_part_is_optional(parts, gate, dtype):
    if gate != "none":
        if "o" not in parts:
            pytest.skip("no gate without a block")
        parts += "z"
    for T, W, group in ((19, 320, 64), (6, 1104, 0)):
        c = make(T, W, dtype, seed=len(parts), parts=parts)
        check(c, group, gate, dtype, *run(c, config(W, dtype, group, gate)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_strides_and_heads(dtype):
    from sparse_state_linear_router_gb300 import binding
    c = make(45, 256, dtype, seed=3, extra=40)
    cfg = config(256, dtype, 64, "silu")
    f, g = run(c, cfg)
    check(c, 64, "silu", dtype, f, g)
    h = lambda t: t.unflatten(1, (4, 64))  # noqa: E731
    f3 = binding.block_norm(cfg, h(c["o"]), gate=h(c["z"]), residual=c["r"], w_after=c["a"], channel_scale=c["c"],
                            w_before=c["b"])
    assert torch.equal(f3["residual_out"], f["residual_out"]) and torch.equal(f3["next_in"], f["next_in"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_rows_and_large_values(dtype):
    """Rows of zeros have mean square 0: rstd is 1 / sqrt(eps), everything stays finite."""
    c = make(12, 192, dtype, seed=4)
    for k in ("o", "r", "at"):
        c[k][::3] = 0
    c["o"][1] *= 1e6
    c["z"][2] = -200.0     # a closed gate: exp(200) is infinite, the gate 0
    c["z"][5] = 200.0
    c["z"][8] = 0.0
    f, g = run(c, config(192, dtype, 64, "sigmoid"))
    check(c, 64, "sigmoid", dtype, f, g)
    f, g = run(c, config(192, dtype, 0, "silu"))
    for t in list(f.values()) + list(g.values()):
        assert bool(torch.isfinite(t).all())
    assert bool((f["next_in"][0] == 0).all())


def test_a_bad_value_stays_in_its_row_and_group(dtype="bf16"):
    c = make(40, 256, dtype, seed=5)
    cfg = config(256, dtype, 64, "silu")
    ref, ref_g = run(c, cfg)
    c["o"][7, 70] = float("nan")
    got, got_g = run(c, cfg)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[7] = False
    for k in ref:
        assert torch.equal(got[k][rows], ref[k][rows])
    cols = torch.ones(256, dtype=torch.bool, device="cuda")
    cols[64:128] = False
    assert torch.equal(got["residual_out"][7][cols], ref["residual_out"][7][cols])
    assert not bool(torch.isfinite(got["residual_out"][7, 64:128]).any())
    assert not bool(torch.isfinite(got["next_in"][7]).any())
    for k in ("d_block_out", "d_gate", "d_residual"):
        assert torch.equal(got_g[k][rows], ref_g[k][rows])
    assert torch.equal(got_g["d_w_after"][cols], ref_g["d_w_after"][cols])


def test_residual_stream_in_place(dtype="bf16"):
    from sparse_state_linear_router_gb300 import binding
    c = make(700, 264, dtype, seed=6)
    cfg = config(264, dtype, 0, "silu")
    ref, _ = run(c, cfg)
    stream = c["r"].clone()
    got = binding.block_norm(cfg, c["o"], gate=c["z"], residual=stream, w_after=c["a"], channel_scale=c["c"],
                             w_before=c["b"], residual_out=stream)
    torch.cuda.synchronize()
    assert torch.equal(stream, ref["residual_out"]) and torch.equal(got["next_in"], ref["next_in"])
    only = binding.block_norm(cfg, c["o"], gate=c["z"], residual=c["r"], w_after=c["a"], channel_scale=c["c"],
                              w_before=c["b"], want_residual_out=False)
    assert only["residual_out"] is None and torch.equal(only["next_in"], ref["next_in"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(dtype):
    from sparse_state_linear_router_gb300 import binding
    c = make(0, 64, dtype, seed=7)
    cfg = config(64, dtype, 0, "silu")
    f, g = run(c, cfg)
    assert f["next_in"].shape == (0, 64) and g["d_block_out"].shape == (0, 64)
    for k in ("d_w_after", "d_channel_scale", "d_w_before"):
        assert bool((g[k] == 0).all())


def test_gradients_by_differences():
    """A step along a direction changes the loss by the gradients' product with it (float32 kernels)."""
    from sparse_state_linear_router_gb300 import binding
    T, W, group = 12, 96, 32
    c = make(T, W, "f32", seed=8)
    cfg = config(W, "f32", group, "silu")
    f, _ = run(c, cfg)
    g = binding.block_norm_backward(cfg, c["dr"], c["o"], gate=c["z"], w_after=c["a"], channel_scale=c["c"],
                                    w_before=c["b"], residual_out=f["residual_out"], d_next_in=c["dn"])
    gen = torch.Generator().manual_seed(2)
    names = {"o": "d_block_out", "z": "d_gate", "r": "d_residual", "a": "d_w_after", "c": "d_channel_scale",
             "b": "d_w_before"}
    dirs = {k: torch.randn(c[k].shape, generator=gen).cuda() for k in names}
    eps = 2.0 ** -8

    def loss(sign):
        r, _ = run(dict(c, **{k: c[k] + sign * eps * dirs[k] for k in names}), cfg)
        return float((c["dr"].double() * r["residual_out"].double()).sum() +
                     (c["dn"].double() * r["next_in"].double()).sum())

    fd = (loss(1) - loss(-1)) / (2 * eps)
    products = [g[v].double() * dirs[k].double() for k, v in names.items()]
    total, size = sum(float(p.sum()) for p in products), sum(float(p.abs().sum()) for p in products)
    # eps^2 / 6 times a third derivative (of products of a few such factors), and the losses' rounding over 2 eps
    assert abs(fd - total) < 8 * eps * eps * size + 2.0 ** -20 * size / eps


def _guarded(shape, dtype):
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((8192 + n,), 0x5A, dtype=torch.uint8, device="cuda")
    return raw[4096:4096 + n].view(dtype).view(*shape), raw


def test_writes_only_its_outputs_and_repeats_itself():
    from sparse_state_linear_router_gb300 import binding
    T, W = 501, 2056
    c = make(T, W, "bf16", seed=9)
    cfg = config(W, "bf16", 8, "silu")
    ref, ref_g = run(c, cfg)
    out, r0 = _guarded((T, W), torch.bfloat16)
    nxt, r1 = _guarded((T, W), torch.bfloat16)
    got, _ = run(c, cfg, residual_out=out, next_in=nxt)
    assert torch.equal(out, ref["residual_out"]) and torch.equal(nxt, ref["next_in"])
    n = binding.sse_block_norm_backward_workspace_size(cfg, T)
    for fill in (0, 0xFF):
        ws, r2 = _guarded((n,), torch.uint8)
        ws.fill_(fill)
        g = binding.block_norm_backward(cfg, c["dr"], c["o"], gate=c["z"], w_after=c["a"], channel_scale=c["c"],
                                        w_before=c["b"], residual_out=c["at"], d_next_in=c["dn"], workspace=ws)
        torch.cuda.synchronize()
        for k in g:
            assert torch.equal(g[k], ref_g[k])
        for raw in (r0, r1, r2):
            assert bool((raw[:4096] == 0x5A).all()) and bool((raw[-4096:] == 0x5A).all())


def test_many_rows():
    """More rows than the persistent grid holds at once, and gradients that start from the row behind alone."""
    from sparse_state_linear_router_gb300 import binding
    c = make(9001, 136, "bf16", seed=10)
    cfg = config(136, "bf16", 136, "linear")
    f, g = run(c, cfg)
    check(c, 136, "linear", "bf16", f, g)
    zero = binding.block_norm_backward(cfg, torch.zeros_like(c["dr"]), c["o"], gate=c["z"], w_after=c["a"],
                                       channel_scale=c["c"], w_before=c["b"], residual_out=c["at"], d_next_in=c["dn"])
    none = binding.block_norm_backward(cfg, None, c["o"], gate=c["z"], w_after=c["a"], channel_scale=c["c"],
                                       w_before=c["b"], residual_out=c["at"], d_next_in=c["dn"])
    for k in zero:
        assert torch.equal(zero[k], none[k])


def test_calls_side_by_side():
    """Different calls in flight on several streams at once, each with its own workspace: nothing is shared."""
    sets = [make(700 + 50 * i, 256 * (i + 1), "bf16", seed=20 + i) for i in range(4)]
    cfgs = [config(256 * (i + 1), "bf16", 64, "silu") for i in range(4)]
    want = [run(c, cfg) for c, cfg in zip(sets, cfgs)]
    streams = [torch.cuda.Stream() for _ in sets]
    from sparse_state_linear_router_gb300 import binding
    got = []
    for c, cfg, st in zip(sets, cfgs, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            f = binding.block_norm(cfg, c["o"], gate=c["z"], residual=c["r"], w_after=c["a"], channel_scale=c["c"],
                                   w_before=c["b"])
            g = binding.block_norm_backward(cfg, c["dr"], c["o"], gate=c["z"], w_after=c["a"], channel_scale=c["c"],
                                            w_before=c["b"], residual_out=c["at"], d_next_in=c["dn"])
            got.append((f, g))
    torch.cuda.synchronize()
    for (f, g), (wf, wg) in zip(got, want):
        for a, b in ((f, wf), (g, wg)):
            for k in a:
                assert torch.equal(a[k], b[k])


def test_graph_replays_on_new_inputs_and_other_streams():
    from sparse_state_linear_router_gb300 import binding
    T, W = 333, 512
    sets = [make(T, W, "bf16", seed=s) for s in (11, 12)]
    cfg = config(W, "bf16", 128, "silu")
    want = [run(c, cfg) for c in sets]
    buf = {k: v.clone() for k, v in sets[0].items()}

    def call():
        f = binding.block_norm(cfg, buf["o"], gate=buf["z"], residual=buf["r"], w_after=buf["a"],
                               channel_scale=buf["c"], w_before=buf["b"])
        g = binding.block_norm_backward(cfg, buf["dr"], buf["o"], gate=buf["z"], w_after=buf["a"],
                                        channel_scale=buf["c"], w_before=buf["b"], residual_out=buf["at"],
                                        d_next_in=buf["dn"])
        return f, g

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f, g = call()
    side.synchronize()
    assert torch.equal(f["next_in"], want[0][0]["next_in"]) and torch.equal(g["d_w_after"], want[0][1]["d_w_after"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, g = call()
    for c, (wf, wg) in zip(sets + sets[::-1], want + want[::-1]):
        for k in buf:
            buf[k].copy_(c[k])
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in ((f, wf), (g, wg)):
            for k in got:
                assert torch.equal(got[k], ref[k])


def test_helpers_refuse():
    from sparse_state_linear_router_gb300 import binding
    c = make(20, 64, "bf16", seed=13)
    cfg = config(64, "bf16", 0, "silu")

    def refused(fn, *a, **kw):
        with pytest.raises(binding.SSEError) as e:
            fn(*a, **kw)
        assert e.value.status in (binding.SSE_ERR_INVALID_ARG, binding.SSE_ERR_UNSUPPORTED)

    f = binding.block_norm
    refused(f, cfg, c["o"])                                     # the config's gate is missing
    refused(f, cfg, c["o"], gate=c["z"].float())
    refused(f, cfg, c["o"], gate=c["z"][:19])
    refused(f, cfg, c["o"], gate=c["z"][:, :1].expand(20, 64))  # one gate per row
    refused(f, cfg, c["o"], gate=c["z"][:1].expand(20, 64))     # one row for all tokens
    refused(f, cfg, c["o"], gate=c["z"].cpu())
    refused(f, cfg, c["o"], gate=c["z"], w_after=c["a"].bfloat16())
    refused(f, cfg, c["o"], gate=c["z"], w_after=c["a"][:32])
    refused(f, cfg, c["o"], gate=c["z"], want_residual_out=False)  # nothing to write
    wide = torch.empty(20, 128, dtype=torch.bfloat16, device="cuda")
    refused(f, cfg, c["o"], gate=c["z"], residual_out=wide[:, :64])
    refused(f, cfg, c["o"], gate=c["z"], residual=wide[:, :64], residual_out=wide[:, :64])
    bw = binding.block_norm_backward
    refused(bw, cfg, None, c["o"], gate=c["z"])
    refused(bw, cfg, c["dr"], c["o"], gate=c["z"], w_before=c["b"])
    refused(bw, cfg, c["dr"][:1].expand(20, 64), c["o"], gate=c["z"])
    with pytest.raises(binding.SSEError):
        bw(cfg, c["dr"], c["o"], gate=c["z"], w_after=c["a"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
