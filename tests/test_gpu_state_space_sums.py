"""What the sums and the ranges of the selective scan promise beyond ordinary
values (marked gpu): the gradient of A beside rows of no token, even sequences
that have a range each, long float32 sums, and states handed on between ranges with
every number of states."""
import numpy as np
import pytest

from oracle import selective as oracle
from tests._bounds import ROUND
from tests.test_gpu_selective import bounds, cfg_of, check, make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,N", [("bf16", 8), ("bf16", 16), ("f32", 16), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("lens", [[21], [16], [30, 0, 25], [9, 7, 40]])
def test_the_gradient_of_A_does_not_see_the_last_input(b, value, dtype, N, lens):
    """A sequence's last input is in no state that d_A reads: whatever it is, d_A is the same."""
    c = make(lens, 40, N, 1, dtype, 3)
    _, g = run(b, c, dtype)
    last = [int(n) - 1 for n in np.cumsum(lens) if n]
    c["x"][last, 5] = value
    _, bad = run(b, c, dtype)
    assert not bad["d_skip"][5].isfinite()
    assert torch.equal(bad["d_A"], g["d_A"])


def test_an_infinite_gradient_of_a_first_token(b):
    """d_A of a sequence that begins a range in the middle of a tile: infinite where the first token's gradient is (the
    state before it is not zero), never a NaN from the rows in front of it."""
    lens = [200, 203, 190, 205]
    c = make(lens, 8, 8, 1, "f32", 5, gate=False)
    assert b.sse_selective_forward_workspace_size(cfg_of(b, c, "f32"), sum(lens), len(lens)) > 0
    _, fine = run(b, c, "f32")
    for t in (200, 403, 593):
        d = dict(c, d_out=c["d_out"].clone())
        d["d_out"][t, 3] = float("inf")
        _, g = run(b, d, "f32")
        assert bool(torch.isinf(g["d_A"][3]).all())
        keep = [i for i in range(8) if i != 3]
        assert torch.equal(g["d_A"][keep], fine["d_A"][keep])


@pytest.mark.parametrize("lens", [[70, 62] * 8, [67, 65] * 8, [69, 63, 66] * 6, [66] * 16, [80] * 16])
def test_even_sequences_have_a_range_each(b, lens):
    """Nothing is handed on between ranges: where the workspaces keep the states and the sums of steps of ranges they stay as
    they were, and every sequence gives bit for bit what it gives in a call of its own (one range)."""
    W, N, S = 2048, 8, len(lens)
    c = make(lens, W, N, 1, "f32", 6)
    cfg, args = cfg_of(b, c, "f32"), (c["x"], c["delta"], c["A"], c["B"], c["C"], c["cu"])
    kw = dict(delta_bias=c["bias"], skip=c["skip"], gate=c["gate"], initial_state=c["init"])
    marked = lambda n: torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # noqa: E731
    room = marked(b.sse_selective_forward_workspace_size(cfg, sum(lens), S))
    handed = 4 * S * W * (N + 1)  # a row of states and a step for each of at least S ranges
    assert room.numel() >= handed
    f = b.selective_forward(cfg, *args, want_checkpoints=True, workspace=room, **kw)
    assert bool((room == 0xFF).all())
    room = marked(b.sse_selective_backward_workspace_size(cfg, sum(lens), S))
    g = b.selective_backward(cfg, *args, f["checkpoints"], c["d_out"], d_final_state=c["d_final"], workspace=room, **kw)
    assert bool((room[-handed:] == 0xFF).all()) and not bool((room[:-handed] == 0xFF).all())
    cu = np.concatenate([[0], np.cumsum(lens)])
    for q in range(len(lens)):
        s = slice(cu[q], cu[q + 1])
        one = {k: v[s] if k in ("x", "delta", "B", "C", "gate", "d_out") else v for k, v in c.items()}
        one.update(cu=torch.tensor([0, lens[q]], dtype=torch.int32, device="cuda"), init=c["init"][q:q + 1],
                   d_final=c["d_final"][q:q + 1], n=lens[q])
        assert b.sse_selective_forward_workspace_size(cfg_of(b, one, "f32"), lens[q], 1) == 0
        f1, g1 = run(b, one, "f32")
        assert torch.equal(f["out"][s], f1["out"]) and torch.equal(f["final_state"][q], f1["final_state"][0]), q
        assert torch.equal(g["dx"][s], g1["dx"]) and torch.equal(g["d_delta"][s], g1["d_delta"]), q
        assert torch.equal(g["d_initial_state"][q], g1["d_initial_state"][0]), q


def test_long_sums_of_the_weights_gradients(b):
    """d_A, d_skip and d_delta_bias over 131072 tokens in one range: the same inputs at every token, so that the float32
    additions of one long chain would all be off in the same direction."""
    T, N, per, G = 1 << 17, 8, 8, 610
    W = per * G
    r = torch.Generator().manual_seed(3)
    row = {k: torch.rand(n, generator=r) + 0.5 for k, n in (("x", per), ("delta", per), ("B", N), ("C", N), ("d_out", per))}
    row = {k: v.bfloat16() for k, v in row.items()}
    A, bias, skip = -torch.rand(per, N, generator=r) - 1, torch.rand(per, generator=r), torch.rand(per, generator=r)
    wide = lambda k, n: row[k].repeat(G).cuda().expand(n, -1).contiguous()  # noqa: E731
    v = {k: wide(k, T) for k in ("x", "delta", "d_out")}
    B, C = (wide(k, T).unflatten(1, (G, N)) for k in ("B", "C"))
    cfg, cu = b.make_selective_config(W, N, G), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    args = (v["x"], v["delta"], A.repeat(G, 1).cuda(), B, C, cu)
    kw = dict(delta_bias=bias.repeat(G).cuda(), skip=skip.repeat(G).cuda())
    ck = b.selective_forward(cfg, *args, want_checkpoints=True, want_final_state=False, **kw)["checkpoints"]
    g = b.selective_backward(cfg, *args, ck, v["d_out"], want_d_initial_state=False, **kw)
    torch.cuda.synchronize()

    # Decays of at most exp(-0.9): behind 100 tokens every token gives the same terms (to 1e-39), which 300 tokens and 301 show.
    n64 = lambda t: t.double().numpy()  # noqa: E731

    def some(n):
        e = lambda k: np.tile(n64(row[k]), (n, 1))  # noqa: E731
        return oracle.backward(e("x"), e("delta"), n64(A), e("B")[:, None], e("C")[:, None], [0, n], e("d_out"), n64(bias), n64(skip))

    few, more = some(300), some(301)
    # The error of one token's terms: that of 60 tokens' sum, a factor of 60 above at most what 60 additions add to it.
    small = {k: row[k].expand(60, -1) for k in ("x", "delta", "d_out")}
    small.update({k: row[k].expand(60, -1).unflatten(1, (1, N)) for k in ("B", "C")})
    small.update(A=A, bias=bias, skip=skip, gate=None, init=None, d_final=None, n=60, cu=torch.tensor([0, 60], dtype=torch.int32))
    bd = bounds(small)
    chain = 2 * 64 + T // 1024 + 64  # halves of a tile in 1024 tokens, the parts, and what is within a half and behind them
    for k in ("d_A", "d_skip", "d_delta_bias"):
        want = few[k] + (T - 300) * (more[k] - few[k])
        off = np.abs(n64(g[k].cpu()).reshape(G, *want.shape) - want).max(0)
        tol = (np.abs(bd[k].e / bd[k].v) + chain * ROUND) * np.abs(want)
        assert (off <= tol).all(), (k, (off / np.abs(want)).max(), (tol / np.abs(want)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,G", [(32, 1), (32, 3), (64, 1), (64, 2), (8, 3)])
@pytest.mark.parametrize("lens", [[300], [140, 0, 170, 3], [5, 331]])
def test_states_handed_on(b, dtype, N, G, lens):
    """Sequences over several ranges with every number of states and groups."""
    c = make(lens, 24 * G, N, G, dtype, N + len(lens))
    cfg = cfg_of(b, c, dtype)
    assert b.sse_selective_forward_workspace_size(cfg, sum(lens), len(lens)) >= 4 * 4 * 24 * G * N  # four ranges
    f, g = run(b, c, dtype)
    check(c, dtype, f, g)
