"""The host side of the scan's and the block norms' calls (marked gpu)."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_state_linear_router_gb300 import binding
    binding.load()
    return binding


def test_norms_of_several_sizes_from_several_threads(b):
    """Calls of one kernel with different amounts of shared memory, from host threads at the same time (the library
    is thread-safe, and ctypes gives up the interpreter's lock during a call): each is launched and right."""
    T, W, calls = 3, 4096, 1500
    g = torch.Generator().manual_seed(1)
    o, r, dr, dn = ((torch.randn(T, W, generator=g)).bfloat16().cuda() for _ in range(4))
    w = (torch.randn(W, generator=g) * 0.1 + 1).cuda()
    cfg = b.make_norm_config(W)
    n = b.sse_block_norm_backward_workspace_size(cfg, T)
    P = torch.Tensor.data_ptr

    def between(out):
        return b.sse_block_norm(cfg, T, P(o), W, None, W, P(r), W, P(w), None, P(w), P(out[0]), P(out[1]), None)

    def before(out):
        return b.sse_block_norm(cfg, T, None, W, None, W, P(r), W, None, None, P(w), None, P(out[1]), None)

    def between_backward(out):
        return b.sse_block_norm_backward(cfg, T, P(o), W, None, W, P(r), W, P(w), None, P(w), P(dr), P(dn), P(out[0]),
                                         None, P(out[1]), None, None, None, P(out[2]), n, None)

    def before_backward(out):
        return b.sse_block_norm_backward(cfg, T, None, W, None, W, P(r), W, None, None, P(w), None, P(dn), None, None,
                                         P(out[1]), None, None, None, P(out[2]), n, None)

    def outputs():
        return [torch.zeros(T, W, dtype=torch.bfloat16, device="cuda") for _ in range(2)] + [
            torch.zeros(n, dtype=torch.uint8, device="cuda")]

    for pair in ((between, before), (between_backward, before_backward)):
        want, got, status = [outputs() for _ in pair], [outputs() for _ in pair], [set() for _ in pair]
        for call, out in zip(pair, want):
            assert call(out) == b.SSE_OK
        torch.cuda.synchronize()
        start = threading.Barrier(len(pair))

        def work(call, out, seen):
            start.wait()
            for _ in range(calls):
                seen.add(call(out))

        threads = [threading.Thread(target=work, args=a) for a in zip(pair, got, status)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert status == [{b.SSE_OK}] * len(pair)
        for a, e in zip(got, want):
            assert torch.equal(a[0], e[0]) and torch.equal(a[1], e[1])


def test_missing_tensors_are_refused(b):
    T, W = 6, 64
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    check, cfg = torch.zeros(1, W, device="cuda"), b.make_scan_config(W)
    state = torch.zeros(T, W, device="cuda")
    for call in (lambda: b.scan_forward(cfg, None, x, cu), lambda: b.scan_forward(cfg, x, None, cu),
                 lambda: b.scan_forward(cfg, x, x, None), lambda: b.scan_backward(cfg, x, None, cu, check, x),
                 lambda: b.scan_backward(cfg, x, x, None, check, x), lambda: b.scan_backward(cfg, x, x, cu, check, None),
                 lambda: b.scan_backward(cfg, x, x, cu, None, x), lambda: b.scan_step(cfg, state, x, None),
                 lambda: b.scan_step(cfg, None, x, x)):
        with pytest.raises(b.SSEError) as e:
            call()
        assert e.value.status == b.SSE_ERR_INVALID_ARG
