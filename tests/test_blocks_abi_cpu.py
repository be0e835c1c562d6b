"""CPU-only checks of the scan's and the block norms' entry points: bad
arguments are refused on the host before any launch."""
import ctypes

import pytest

FAKE = 1 << 20  # aligned non-null "device" address; never dereferenced


@pytest.fixture(scope="module")
def b():
    from sparse_state_linear_router_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def _scan(b, cfg=None, T=16, S=1, x=FAKE, xs=64, gs=64, cu=FAKE, out=FAKE, init=None, ck=None):
    return b.sse_scan_forward(cfg or b.make_scan_config(64), x, xs, FAKE, gs, cu, S, T, init, None, out, ck, None)


def test_scan_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    assert _scan(b, b.make_scan_config(0)) == I
    assert _scan(b, b.make_scan_config(64, dtype=5)) == I
    assert _scan(b, b.make_scan_config(64, 3)) == I
    assert _scan(b, b.make_scan_config(60), xs=64) == U
    assert _scan(b, b.make_scan_config(62, dtype="f32")) == U
    assert _scan(b, b.make_scan_config((1 << 16) + 8), xs=1 << 17, gs=1 << 17) == U
    assert _scan(b, T=-1) == I
    assert _scan(b, S=-1) == I
    assert _scan(b, S=0, T=4) == I
    assert _scan(b, T=1 << 30) == U
    assert _scan(b, S=1 << 30) == U
    assert _scan(b, x=None) == I
    assert _scan(b, out=None) == I
    assert _scan(b, cu=None) == I
    assert _scan(b, x=FAKE + 8) == I
    assert _scan(b, init=FAKE + 4) == I
    assert _scan(b, ck=FAKE + 4) == I
    assert _scan(b, xs=56) == I          # rows overlap
    assert _scan(b, gs=68) == I          # 136-byte rows
    assert _scan(b, gs=1 << 41) == I
    assert _scan(b, S=0, T=0) == b.SSE_OK
    assert b.load().sse_scan_forward(None, FAKE, 64, FAKE, 64, FAKE, 1, 16, None, None, FAKE, None, None) == I


def test_scan_backward_and_step_refuse(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED

    def back(cfg=b.make_scan_config(64), T=16, S=1, ck=FAKE, d_out=FAKE, dx=FAKE, dg=FAKE, d_init=None, xs=64):
        return b.sse_scan_backward(cfg, FAKE, xs, FAKE, 64, FAKE, S, T, None, ck, d_out, None, dx, dg, d_init, None)

    assert back(ck=None) == I and back(d_out=None) == I and back(dx=None) == I and back(dg=None) == I
    assert back(d_init=FAKE + 4) == I and back(xs=8) == I and back(T=1 << 40) == U
    assert back(S=0, T=0) == b.SSE_OK

    def step(cfg=b.make_scan_config(64), B=4, state=FAKE, out=FAKE, xs=64):
        return b.sse_scan_step(cfg, FAKE, xs, FAKE, 64, B, state, out, None)

    assert step(state=None) == I and step(out=None) == I and step(B=-1) == I and step(xs=32) == I
    assert step(b.make_scan_config(12)) == U
    assert step(B=0) == b.SSE_OK


def test_checkpoint_rows(b):
    assert [b.sse_scan_checkpoint_rows(n) for n in (0, 1, 64, 65, 1000)] == [0, 1, 1, 2, 16]
    assert b.sse_scan_checkpoint_rows(-1) == 0 and b.sse_scan_checkpoint_rows(1 << 31) == 0
    assert b.SCAN_CHECKPOINT == 64


def _norm(b, cfg, T=16, o=FAKE, os=64, z=None, zs=64, r=FAKE, rs=64, wa=None, ch=None, wb=FAKE, ro=FAKE + 4096,
          nx=FAKE + 8192):
    return b.sse_block_norm(cfg, T, o, os, z, zs, r, rs, wa, ch, wb, ro, nx, None)


def test_norm_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    mk = b.make_norm_config
    assert _norm(b, mk(0)) == I
    assert _norm(b, mk(64, group=-8)) == I
    assert _norm(b, mk(64, group=24)) == I            # does not divide the row
    assert _norm(b, mk(64, group=4)) == U             # 8-byte groups
    assert _norm(b, mk(60)) == U
    assert _norm(b, mk(16392), os=16392, rs=16392) == U
    assert _norm(b, mk(8196, dtype="f32"), os=8196, rs=8196) == U
    assert _norm(b, mk(64, gate=4)) == I
    assert _norm(b, mk(64, dtype=3)) == I
    for eps in (0.0, -1.0, 1e-40, float("nan"), float("inf")):
        assert _norm(b, mk(64, eps=eps)) == I
    assert _norm(b, mk(64, residual_scale=float("nan"))) == I
    assert _norm(b, mk(64, branch_scale=float("inf"))) == I
    assert _norm(b, mk(64), T=-1) == I
    assert _norm(b, mk(64), T=1 << 31) == U
    assert _norm(b, mk(64), o=None, r=None) == I
    assert _norm(b, mk(64), o=None, wa=FAKE) == I     # a norm after nothing
    assert _norm(b, mk(64), z=FAKE) == I              # a gate the config does not name
    assert _norm(b, mk(64, gate="silu")) == I         # a named gate that is missing
    assert _norm(b, mk(64), wb=None) == I             # next_in without its weight
    assert _norm(b, mk(64), nx=None) == I
    assert _norm(b, mk(64), wb=None, nx=None, ro=None) == I
    assert _norm(b, mk(64), os=56) == I
    assert _norm(b, mk(64), rs=68) == I
    assert _norm(b, mk(64), o=FAKE + 2) == I
    assert _norm(b, mk(64), r=FAKE, ro=FAKE, rs=128) == I  # in place with gaps between rows
    assert _norm(b, mk(64), T=0) == b.SSE_OK


def test_norm_backward_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    mk = b.make_norm_config

    def back(cfg=mk(64), T=16, o=FAKE, z=None, at=FAKE, wa=FAKE, ch=None, wb=FAKE, dr=FAKE, dn=FAKE, do=FAKE, dz=None,
             dwa=FAKE, dch=None, dwb=FAKE, ws=FAKE, n=1 << 40):
        return b.sse_block_norm_backward(cfg, T, o, 64, z, 64, at, 64, wa, ch, wb, dr, dn, do, dz, FAKE, dwa, dch, dwb,
                                         ws, n, None)

    assert back(do=None) == I and back(o=None) == I
    assert back(mk(64, gate="silu")) == I and back(mk(64, gate="silu"), z=FAKE) == I
    assert back(dn=None) == I and back(at=None) == I and back(wb=None) == I
    assert back(wb=None, dn=None, at=None, dwb=None, dr=None) == I
    assert back(wa=None) == I and back(dch=FAKE) == I
    assert back(dr=FAKE + 8) == I
    assert back(mk(64, group=4)) == U
    assert back(ws=None) == b.SSE_ERR_WORKSPACE and back(ws=FAKE + 16) == b.SSE_ERR_WORKSPACE
    assert back(n=255) == b.SSE_ERR_WORKSPACE
    small, large = (b.sse_block_norm_backward_workspace_size(mk(64), n) for n in (1, 100000))
    assert 256 <= small <= large and large % 256 == 0
    assert b.sse_block_norm_backward_workspace_size(mk(60), 10) == 0


def test_config_structs_match_the_header(b):
    assert ctypes.sizeof(b.sse_scan_config_t) == 12 and ctypes.sizeof(b.sse_norm_config_t) == 28


def test_helpers_refuse_tensors_on_the_host(b):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: b.scan_forward(b.make_scan_config(64), x, x, torch.zeros(2, dtype=torch.int32)),
                 lambda: b.scan_step(b.make_scan_config(64), torch.zeros(4, 64), x, x),
                 lambda: b.block_norm(b.make_norm_config(64), x),
                 lambda: b.block_norm(b.make_norm_config(64)),
                 lambda: b.block_norm_backward(b.make_norm_config(64), x, x)):
        with pytest.raises(b.SSEError) as e:
            call()
        assert e.value.status == b.SSE_ERR_INVALID_ARG
