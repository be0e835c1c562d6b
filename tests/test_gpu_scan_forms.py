"""The scan's forward in the form that one to three long bf16 sequences take
with a costly input factor at 1536 to 2432 channels: clusters of 7 or 8 CTAs
that exchange their runs and hold their rows in registers between the passes
(marked gpu).  Tolerances are those of tests/test_gpu_scan.py."""
import ctypes

import numpy as np
import pytest

from oracle import scan as oracle
from tests.test_gpu_scan import D, MODES, _close, _f64, _pick, _spread, check, make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()


# width, lengths, rows behind the last sequence: one sequence; two; several starts and ends inside a worker's 16 rows,
# or an empty sequence there
HELD = [(2048, [5000], 0), (2368, [5000], 0), (2048, [3000, 1900], 50), (2048, [2900, 7, 1100], 0),
        (2048, [2897, 0, 2103], 0)]
IDS = ["one", "wide", "two", "short", "empty"]
COLS = [0, 1, 3, 5, 31, 62, 63, 64, 100, 129, 700, 2047]


def _form(width, mode, dtype, tokens, seqs):
    from sparse_state_linear_router_gb300 import binding
    query = binding.load().sse_debug_scan_form
    csize, ranges = ctypes.c_int32(), ctypes.c_int32()
    cfg = binding.make_scan_config(width, mode, dtype)
    return query(ctypes.byref(cfg), tokens, seqs, ctypes.byref(csize), ctypes.byref(ranges)), csize.value, ranges.value


@pytest.mark.parametrize("mode", ["complement", "unit"])
@pytest.mark.parametrize("width,lens,tail", HELD, ids=IDS)
def test_held_rows_in_exchanging_clusters(width, lens, tail, mode):
    """Values and gradients, emptied and kept states, a column whose gates leave [-1/2, 0] late; the final state over
    the initial one; a NaN stays in its sequence and channel."""
    from sparse_state_linear_router_gb300 import binding
    n = sum(lens)
    form, csize, ranges = _form(width, mode, "bf16", n + tail, len(lens))
    assert (form, ranges) == (2, 1) and csize >= 7   # a new rule for the choice needs new cases here
    c = make(lens, width, "bf16", seed=41, tail=tail)
    c["la"][7:n:41, 3] = float("-inf")
    c["la"][5:n:37, 5] = 0.0
    c["la"][4000:, 64:128] = -3.0
    f, b = run(c, mode, "bf16")
    check(*(lambda s, sf, sb: (s, mode, "bf16", sf, sb))(*_pick(c, f, b, COLS)))
    # the states that the backward starts from: before every 64th token but a sequence's first
    sub, _, _ = _pick(c, f, b, COLS)
    cu, init, la = c["cu"].cpu().numpy(), _f64(sub["init"]), _f64(sub["la"])[:n]
    x = _f64(sub["x"])[:n]
    before = oracle.forward(x, la, cu, mode, init)["before"]
    _, e, _ = _spread(np.exp(la), oracle.input_scale(la, mode)[0] * x, cu, init)
    rows = np.array([t for t in range(64, n, 64) if t not in set(cu.tolist())])
    _close(_f64(f["checkpoints"][:, COLS])[rows // 64], before[rows], D * e[rows - 1], "checkpoints")
    state = c["init"].clone()
    cfg = binding.make_scan_config(width, mode, "bf16")
    again = binding.scan_forward(cfg, c["x"], c["la"], c["cu"], initial_state=state, final_state=state)
    torch.cuda.synchronize()
    assert torch.equal(again["out"][:n], f["out"][:n]) and torch.equal(state, f["final_state"])
    # a NaN 50 tokens into the first sequence
    c["x"][50, 70] = float("nan")
    bad, _ = run(c, mode, "bf16")
    same = torch.ones(n, width, dtype=torch.bool, device="cuda")
    same[50:lens[0], 70] = False
    assert torch.equal(bad["out"][:n][same], f["out"][:n][same])
    assert not bool(torch.isfinite(bad["out"][50:lens[0], 70]).any())
    same = torch.ones(len(lens), width, dtype=torch.bool, device="cuda")
    same[0, 70] = False
    assert torch.equal(bad["final_state"][same], f["final_state"][same])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width,lens", [(64, [300, 50, 0, 1, 400]), (2048, [300, 2600, 0, 400])], ids=["few", "many"])
def test_a_nan_gate_stays_in_its_sequence_and_channel(width, lens, dtype, mode):
    """From its token on in the states, up to its token in the adjoint; all else stays within the tolerances (not bit
    for bit: a tile with a gate that is none takes the general form of 1 - a)."""
    c = make(lens, width, dtype, seed=43)
    ref, ref_b = run(c, mode, dtype)
    cols = [0, 2, 3, 4, 63, width - 1]
    s0, s1 = lens[0], lens[0] + lens[1]
    at = s0 + 20
    bits, nans = (torch.int32, (0x7fc00000, -0x400000)) if dtype == "f32" else (torch.int16, (0x7fc0, -0x40))
    for value in nans:  # of either sign
        bad = dict(c, la=c["la"].clone())
        bad["la"].view(bits)[at, 3] = value
        assert bool(torch.isnan(bad["la"][at, 3]))
        f, b = run(bad, mode, dtype)
        for t in (f["out"][at:s1, 3], b["dx"][s0:at, 3], b["d_log_gate"][at:s1, 3], f["final_state"][1, 3],
                  b["d_initial_state"][1, 3]):
            assert not bool(torch.isfinite(t).any())
        # with that sequence and channel as they were, everything else is right
        f, b = {k: v.clone() for k, v in f.items()}, {k: v.clone() for k, v in b.items()}
        for got, want in ((f["out"], ref["out"]), (b["dx"], ref_b["dx"]), (b["d_log_gate"], ref_b["d_log_gate"])):
            got[s0:s1, 3] = want[s0:s1, 3]
        f["final_state"][1, 3], b["d_initial_state"][1, 3] = ref["final_state"][1, 3], ref_b["d_initial_state"][1, 3]
        sub, sub_f, sub_b = _pick(c, f, b, cols)
        check(sub, mode, dtype, sub_f, sub_b)
