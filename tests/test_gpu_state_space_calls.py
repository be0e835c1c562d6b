"""The calls of the short convolution, the selective scan and the layer norm
that a program makes beside the ordinary ones (marked gpu): from several host
threads at once, with workspaces of the caller, at the largest widths, with
many short sequences, and with infinite steps."""
import threading

import numpy as np
import pytest

from oracle import selective as scan_oracle
from tests import test_gpu_conv as conv
from tests.test_gpu_selective import check, make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


def _n(*s, seed=0, dtype=torch.bfloat16):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def test_from_several_threads(b):
    """Calls of one kernel with different sizes from host threads at the same time, each on its own stream: as alone."""
    def conv(W):
        x, w, cu = _n(40, W, seed=W), _n(W, 4, seed=1, dtype=torch.float32), torch.tensor([0, 40], dtype=torch.int32).cuda()
        cfg = b.make_conv_config(W)
        return lambda: b.conv_backward(cfg, x, w, cu, x)

    def norm(W, dtype):
        x, w = _n(9, W, seed=W, dtype=dtype), _n(W, seed=1, dtype=torch.float32)
        cfg = b.make_layer_norm_config(W, dtype="bf16" if dtype is torch.bfloat16 else "f32")
        return lambda: b.layer_norm_backward(cfg, x, w, x)

    def scan(W, N):
        c = make([70, 3], W, N, 1, "f32", W)
        return lambda: {k: v for d in run(b, c, "f32") for k, v in d.items() if k != "checkpoints"}

    calls = [conv(64), conv(520), norm(8192, torch.bfloat16), norm(16384, torch.bfloat16), scan(64, 64), scan(96, 16)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, wrong = [[] for _ in calls], []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(60):
                    got[i] = calls[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
    for g, w in zip(got, want):
        for k in w:
            assert w[k] is None and g[k] is None or torch.equal(g[k], w[k]), k


def test_workspaces_of_the_caller(b):
    """A workspace with NaN in it, of exactly the size that is asked for, gives the same as one of the call's own."""
    c = make([300, 0, 45], 72, 16, 1, "bf16", 1)
    cfg = b.make_selective_config(72, 16)
    args = (c["x"], c["delta"], c["A"], c["B"], c["C"], c["cu"])
    kw = dict(delta_bias=c["bias"], skip=c["skip"], gate=c["gate"], initial_state=c["init"])
    f, g = run(b, c, "bf16")
    nan = lambda n: torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)  # noqa: E731
    n = b.sse_selective_forward_workspace_size(cfg, 345, 3)
    assert n > 0
    f2 = b.selective_forward(cfg, *args, want_checkpoints=True, workspace=nan(n), **kw)
    assert torch.equal(f2["out"], f["out"]) and torch.equal(f2["final_state"], f["final_state"])
    with pytest.raises(b.SSEError) as e:
        b.selective_forward(cfg, *args, workspace=nan(n)[:n - 256], **kw)
    assert e.value.status == b.SSE_ERR_WORKSPACE
    n = b.sse_selective_backward_workspace_size(cfg, 345, 3)
    g2 = b.selective_backward(cfg, *args, f["checkpoints"], c["d_out"], d_final_state=c["d_final"], workspace=nan(n), **kw)
    for k in g:
        assert torch.equal(g2[k], g[k]), k
    x, w = c["x"].contiguous(), _n(72, 4, seed=2, dtype=torch.float32)
    cfg = b.make_conv_config(72)
    want = b.conv_backward(cfg, x, w, c["cu"], c["d_out"])
    got = b.conv_backward(cfg, x, w, c["cu"], c["d_out"], workspace=nan(b.sse_conv_backward_workspace_size(cfg, 345)))
    assert all(want[k] is None or torch.equal(want[k], got[k]) for k in want)
    cfg = b.make_layer_norm_config(72)
    want = b.layer_norm_backward(cfg, x, c["skip"], c["d_out"])
    got = b.layer_norm_backward(cfg, x, c["skip"], c["d_out"], workspace=nan(b.sse_layer_norm_backward_workspace_size(cfg, 345)))
    assert all(torch.equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("W,G", [(65536, 1), (65536, 8), (4096, 512)])
def test_largest_widths_and_many_groups(b, W, G):
    c = make([3, 2], W, 8, G, "bf16", 3)
    f, g = run(b, c, "bf16")
    check(c, "bf16", f, g)


def test_many_short_sequences(b):
    lens = [(7 * i) % 4 for i in range(400)]  # 0 to 3 tokens
    c = make(lens, 24, 16, 1, "bf16", 4)
    f, g = run(b, c, "bf16")
    check(c, "bf16", f, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_steps(b, dtype):
    """A step of softplus(-infinity) = 0 leaves the state as it is and lets nothing in, and its gradients are finite."""
    c = make([40], 40, 16, 1, dtype, 5)
    c["delta"][17], c["delta"][23, 3] = -float("inf"), -float("inf")
    f, g = run(b, c, dtype)
    far = dict(c, delta=c["delta"].clone())
    far["delta"][torch.isinf(far["delta"])] = -300.0  # exp(-300) is 0 in float32, too
    f2, g2 = run(b, far, dtype)
    assert torch.equal(f["out"], f2["out"]) and torch.equal(f["final_state"], f2["final_state"])
    for k in g:
        assert bool(g[k].isfinite().all()) and torch.equal(g[k], g2[k]), k
    check(far, dtype, f, g)
    # an infinite step forgets the state: decay 0; its own input is infinite unless x is 0
    c["delta"][17], c["delta"][23, 3], c["x"][17] = float("inf"), 0.0, 0.0
    out = run(b, c, dtype)[0]["out"]
    assert bool(out[17:].isnan().all())  # infinity times zero


def test_conv_keeps_infinities_in_reach(b):
    x = _n(30, 64, seed=6)
    x[10, 7] = float("inf")
    w, cu = torch.ones(64, 4, device="cuda"), torch.tensor([0, 12, 30], dtype=torch.int32).cuda()
    out = b.conv_forward(b.make_conv_config(64, act="none"), x, w, cu)["out"]
    assert torch.equal(torch.isinf(out).nonzero().cpu(), torch.tensor([[10, 7], [11, 7]]))


def test_gradients_against_differences(b):
    """The selective scan's gradients against central differences of the float64 forward, in a few directions."""
    c = make([25, 0, 18], 16, 8, 2, "f32", 7)
    _, g = run(b, c, "f32")
    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    v = {"x": n(c["x"]), "delta": n(c["delta"]), "A": n(c["A"]), "B": n(c["B"]), "C": n(c["C"]), "delta_bias": n(c["bias"]),
         "skip": n(c["skip"]), "gate": n(c["gate"]), "initial_state": n(c["init"])}
    cu = c["cu"].cpu().numpy()
    r = np.random.default_rng(1)

    def loss(a):
        f = scan_oracle.forward(cu_seqlens=cu, **a)
        return (f["out"] * n(c["d_out"])).sum() + (f["final_state"] * n(c["d_final"])).sum()

    for k in v:
        got = n(g["dx" if k == "x" else "d_" + k])
        for _ in range(3):
            d = r.normal(size=v[k].shape)
            h = 1e-6
            fd = (loss({**v, k: v[k] + h * d}) - loss({**v, k: v[k] - h * d})) / (2 * h)
            # float32 sums of some hundred terms; differences: h^2 of a third derivative and 1e-16 / h of rounding
            assert abs((got * d).sum() - fd) < 1e-4 * np.abs(got * d).sum(), k


def test_zero_gradients_are_zero(b):
    c = make([50], 40, 16, 1, "bf16", 8)
    c["d_out"].zero_()
    c["d_final"] = None
    _, g = run(b, c, "bf16")
    assert all(not v.any() for v in g.values())


@pytest.mark.parametrize("lens", [[8300], [5000, 0, 3450, 2]])
def test_more_than_32_ranges(b, lens):
    """Sequences over more ranges than a warp has lanes: the lookups go round."""
    c = make(lens, 8, 8, 1, "f32", 9)
    cfg = b.make_selective_config(8, 8, dtype="f32")
    assert b.sse_selective_forward_workspace_size(cfg, sum(lens), len(lens)) > 100 * 4 * 8 * 9  # a hundred ranges and more
    f, g = run(b, c, "f32")
    check(c, "f32", f, g)


@pytest.mark.parametrize("lens,tail", [([66] * 16, 0), ([70, 62] * 8, 0), ([71, 61] * 8, 0), ([60] * 16, 0), ([0, 132] + [66] * 14, 0),
                                       ([80] * 16, 300), ([64] * 15 + [84], 7), ([128, 127, 129], 0)])
def test_even_and_uneven_sequences(b, lens, tail):
    """Sequences that make enough warps have a range each where they are even (every start within a sixteenth of its place);
    the others are cut.  Nothing that the workspaces held matters."""
    W = 2048 if len(lens) > 3 else 16384
    c = make(lens, W, 8, 1, "bf16", 6, tail=tail)
    f, g = run(b, c, "bf16")
    check(c, "bf16", f, g)
    cfg, T, S = b.make_selective_config(W, 8), sum(lens) + tail, len(lens)
    nan = lambda n: torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # noqa: E731
    args = (c["x"], c["delta"], c["A"], c["B"], c["C"], c["cu"])
    parts = dict(delta_bias=c["bias"], skip=c["skip"], gate=c["gate"], initial_state=c["init"])
    f2 = b.selective_forward(cfg, *args, want_checkpoints=True, workspace=nan(b.sse_selective_forward_workspace_size(cfg, T, S)), **parts)
    g2 = b.selective_backward(cfg, *args, f2["checkpoints"], c["d_out"], d_final_state=c["d_final"],
                              workspace=nan(b.sse_selective_backward_workspace_size(cfg, T, S)), **parts)
    n = sum(lens)
    assert torch.equal(f["out"][:n], f2["out"][:n]) and torch.equal(f["final_state"], f2["final_state"])
    assert all(torch.equal(g[k][:n], g2[k][:n]) for k in ("dx", "d_delta", "d_gate", "d_B", "d_C"))
    assert all(torch.equal(g[k], g2[k]) for k in ("d_A", "d_skip", "d_delta_bias", "d_initial_state"))


EMPTY = [[5] + [0] * 300 + [7] + [0] * 90 + [40, 3], [0] * 70 + [2], [1] + [0] * 33, [0] * 129]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", EMPTY)
def test_many_empty_sequences(b, dtype, lens):
    """Empty sequences by the hundred, in a row, at both ends, alone: their states go through."""
    for W, K in ((40, 4), (136, 2)):
        c = conv.make(lens, W, K, dtype, 11)
        f, g = conv.run(b, c, "silu", dtype)
        if sum(lens):
            conv.check(c, "silu", dtype, f, g)
        empty = [q for q, n in enumerate(lens) if n == 0]
        assert torch.equal(f["final_state"][empty], c["init"][empty]) and torch.equal(g["d_initial_state"][empty], c["d_final"][empty])
    for N in (8, 64):
        c = make(lens, 24, N, 1, dtype, 12)
        f, g = run(b, c, dtype)
        if sum(lens):
            check(c, dtype, f, g)
        assert torch.equal(f["final_state"][empty], c["init"][empty]) and torch.equal(g["d_initial_state"][empty], c["d_final"][empty])
    c = make(lens, 24, 16, 1, dtype, 13, states=False)
    f, g = run(b, c, dtype)
    assert not f["final_state"][empty].any() and not g["d_initial_state"][empty].any()
