"""What the sums and the ranges of the selective scan promise beyond ordinary
values (marked gpu): the gradient of A beside rows of no token."""
import numpy as np
import pytest

from tests.test_gpu_selective import cfg_of, make, run

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
