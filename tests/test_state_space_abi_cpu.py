"""CPU-only checks of the entry points of the short convolution, the selective
scan and the layer norm: bad arguments are refused on the host before any
launch."""
import ctypes

import pytest

FAKE = 1 << 20  # aligned non-null "device" address; never dereferenced
ROOM = 1 << 40


@pytest.fixture(scope="module")
def b():
    from sparse_state_linear_router_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def test_conv_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    mk = b.make_conv_config

    def fwd(cfg=mk(64), T=16, S=1, x=FAKE, xs=64, w=FAKE, bias=None, cu=FAKE, init=None, fin=None, out=FAKE):
        return b.sse_conv_forward(cfg, x, xs, w, bias, cu, S, T, init, fin, out, None)

    assert fwd(mk(0)) == I and fwd(mk(64, 0)) == I and fwd(mk(64, dtype=5)) == I and fwd(mk(64, act=7)) == I
    assert fwd(mk(64, 1)) == U and fwd(mk(64, 5)) == U and fwd(mk(64, act="sigmoid")) == U
    assert fwd(mk(60)) == U and fwd(mk(62, dtype="f32")) == U and fwd(mk((1 << 16) + 8), xs=1 << 17) == U
    assert fwd(T=-1) == I and fwd(S=-1) == I and fwd(S=0, T=4) == I and fwd(T=1 << 30) == U and fwd(S=1 << 30) == U
    assert fwd(x=None) == I and fwd(w=None) == I and fwd(out=None) == I and fwd(cu=None) == I
    assert fwd(x=FAKE + 8) == I and fwd(w=FAKE + 4) == I and fwd(bias=FAKE + 8) == I and fwd(init=FAKE + 2) == I
    assert fwd(xs=56) == I and fwd(xs=68) == I and fwd(xs=1 << 41) == I
    assert fwd(init=FAKE, fin=FAKE) == I                     # in place is refused
    assert fwd(S=0, T=0) == b.SSE_OK
    assert b.load().sse_conv_forward(None, FAKE, 64, FAKE, None, FAKE, 1, 16, None, None, FAKE, None) == I

    def back(cfg=mk(64), T=16, S=1, w=FAKE, d_out=FAKE, dx=FAKE, dw=FAKE, db=None, di=None, ws=FAKE, n=ROOM, xs=64):
        return b.sse_conv_backward(cfg, FAKE, xs, w, None, FAKE, S, T, None, d_out, None, dx, dw, db, di, ws, n, None)

    assert back(w=None) == I and back(d_out=None) == I and back(dx=None) == I and back(dw=None) == I and back(xs=8) == I
    assert back(db=FAKE + 4) == I and back(di=FAKE + 8) == I and back(mk(64, 9)) == U
    assert back(ws=None) == b.SSE_ERR_WORKSPACE and back(ws=FAKE + 16) == b.SSE_ERR_WORKSPACE
    assert back(n=64) == b.SSE_ERR_WORKSPACE
    assert b.sse_conv_backward_workspace_size(mk(64), 1000) >= 4 * 5 * 64
    assert b.sse_conv_backward_workspace_size(mk(64, 9), 1000) == 0

    def step(cfg=mk(64), B=4, state=FAKE, out=FAKE, xs=64, w=FAKE):
        return b.sse_conv_step(cfg, FAKE, xs, w, None, B, state, out, None)

    assert step(state=None) == I and step(out=None) == I and step(w=None) == I and step(B=-1) == I and step(xs=32) == I
    assert step(mk(12)) == U and step(state=FAKE + 8) == I and step(B=0) == b.SSE_OK


def test_selective_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    mk = b.make_selective_config

    def fwd(cfg=mk(64), T=16, S=1, x=FAKE, xs=64, d=FAKE, ds=64, bias=None, A=FAKE, B=FAKE, bs=16, C=FAKE, cs=16, skip=None,
            z=None, zs=64, cu=FAKE, init=None, fin=None, out=FAKE, ck=None, ws=FAKE, n=ROOM):
        return b.sse_selective_forward(cfg, x, xs, d, ds, bias, A, B, bs, C, cs, skip, z, zs, cu, S, T, init, fin, out, ck,
                                       ws, n, None)

    assert fwd(mk(0)) == I and fwd(mk(64, 0)) == I and fwd(mk(64, 16, 0)) == I and fwd(mk(64, 16, 3)) == I
    assert fwd(mk(64, dtype=5)) == I and fwd(mk(64, 12)) == U and fwd(mk(64, 128)) == U and fwd(mk(64, 4)) == U
    assert fwd(mk(60)) == U and fwd(mk(64, 16, 16), bs=256, cs=256) == U    # four channels a group: no 16-byte word
    assert fwd(mk((1 << 16) + 8), xs=1 << 17, ds=1 << 17) == U
    assert fwd(T=-1) == I and fwd(S=-1) == I and fwd(S=0, T=4) == I and fwd(T=1 << 30) == U and fwd(S=1 << 30) == U
    for k in ("x", "d", "A", "B", "C", "out", "cu"):
        assert fwd(**{k: None}) == I
    for k in ("x", "d", "A", "B", "C", "out", "bias", "skip", "z", "init", "fin", "ck"):
        assert fwd(**{k: FAKE + 4}) == I
    assert fwd(xs=56) == I and fwd(ds=68) == I and fwd(bs=8) == I and fwd(cs=20) == I and fwd(z=FAKE, zs=32) == I
    assert fwd(init=FAKE, fin=FAKE) == I
    assert fwd(S=0, T=0) == b.SSE_OK
    assert b.sse_selective_forward_workspace_size(mk(64, 12), 100, 1) == 0
    big = b.sse_selective_forward_workspace_size(mk(64), 1 << 20, 1)
    assert fwd(T=1 << 20, ws=None) == b.SSE_ERR_WORKSPACE if big else True

    def back(cfg=mk(64), T=16, S=1, z=None, skip=None, ck=FAKE, d_out=FAKE, dx=FAKE, dd=FAKE, db=None, dA=FAKE, dB=FAKE,
             dC=FAKE, dk=None, dz=None, di=None, ws=FAKE, n=ROOM):
        return b.sse_selective_backward(cfg, FAKE, 64, FAKE, 64, None, FAKE, FAKE, 16, FAKE, 16, skip, z, 64, FAKE, S, T, None,
                                        ck, d_out, None, dx, dd, db, dA, dB, dC, dk, dz, di, ws, n, None)

    for k in ("ck", "d_out", "dx", "dd", "dA", "dB", "dC"):
        assert back(**{k: None}) == I and back(**{k: FAKE + 4}) == I
    for k in ("db", "di"):
        assert back(**{k: FAKE + 4}) == I
    assert back(z=FAKE) == I and back(dz=FAKE) == I and back(dk=FAKE) == I
    assert back(ws=None) == b.SSE_ERR_WORKSPACE and back(ws=FAKE + 16) == b.SSE_ERR_WORKSPACE and back(n=1) == b.SSE_ERR_WORKSPACE

    def step(cfg=mk(64), B=4, state=FAKE, out=FAKE, bs=16, d=FAKE):
        return b.sse_selective_step(cfg, FAKE, 64, d, 64, None, FAKE, FAKE, bs, FAKE, 16, None, None, 64, B, state, out, None)

    assert step(state=None) == I and step(out=None) == I and step(d=None) == I and step(B=-1) == I and step(bs=8) == I
    assert step(mk(12)) == U and step(state=FAKE + 8) == I and step(B=0) == b.SSE_OK


def test_selective_checkpoint_rows(b):
    assert [b.sse_selective_checkpoint_rows(n) for n in (0, 1, 16, 17, 1000)] == [0, 1, 1, 2, 63]
    assert b.sse_selective_checkpoint_rows(-1) == 0 and b.sse_selective_checkpoint_rows(1 << 31) == 0
    assert b.SELECTIVE_CHECKPOINT == 16


def test_layer_norm_refuses(b):
    I, U = b.SSE_ERR_INVALID_ARG, b.SSE_ERR_UNSUPPORTED
    mk = b.make_layer_norm_config

    def fwd(cfg=mk(64), T=16, x=FAKE, xs=64, r=None, rs=64, w=FAKE, bias=None, ro=None, out=FAKE + 8192):
        return b.sse_layer_norm(cfg, T, x, xs, r, rs, w, bias, ro, out, None)

    assert fwd(mk(0)) == I and fwd(mk(64, eps=0)) == I and fwd(mk(64, eps=-1)) == I and fwd(mk(64, eps=float("nan"))) == I
    assert fwd(mk(64, eps=float("inf"))) == I and fwd(mk(64, eps=1e-40)) == I and fwd(mk(64, dtype=9)) == I
    assert fwd(mk(60)) == U and fwd(mk(16392), xs=16392) == U and fwd(mk(8196, dtype="f32"), xs=8196) == U
    assert fwd(T=-1) == I and fwd(T=1 << 31) == U and fwd(x=None) == I and fwd(out=None) == I
    assert fwd(xs=56) == I and fwd(r=FAKE, rs=60) == I
    for k in ("x", "w", "bias", "ro", "out", "r"):
        assert fwd(**{k: FAKE + 4}) == I
    assert fwd(ro=FAKE, xs=72) == I and fwd(r=FAKE + 4096, rs=72, ro=FAKE + 4096) == I   # in place with a stride
    assert fwd(T=0, x=None, out=None) == b.SSE_OK
    assert b.load().sse_layer_norm(None, 16, FAKE, 64, None, 64, FAKE, None, None, FAKE, None) == I

    def back(cfg=mk(64), T=16, x=FAKE, xs=64, d_out=FAKE, dr=None, dx=FAKE, dw=FAKE, db=None, ws=FAKE, n=ROOM):
        return b.sse_layer_norm_backward(cfg, T, x, xs, FAKE, d_out, dr, dx, dw, db, ws, n, None)

    assert back(x=None) == I and back(d_out=None) == I and back(dx=None) == I and back(xs=8) == I
    for k in ("x", "d_out", "dr", "dx", "dw", "db"):
        assert back(**{k: FAKE + 4}) == I
    assert back(ws=None) == b.SSE_ERR_WORKSPACE and back(ws=FAKE + 8) == b.SSE_ERR_WORKSPACE and back(n=8) == b.SSE_ERR_WORKSPACE
    assert b.sse_layer_norm_backward_workspace_size(mk(60), 16) == 0


def test_configs_have_the_headers_layout(b):
    assert ctypes.sizeof(b.sse_conv_config_t) == 16 and ctypes.sizeof(b.sse_selective_config_t) == 16
    assert ctypes.sizeof(b.sse_layer_norm_config_t) == 12


def test_weights_are_asked_for_without_tokens(b):
    """The kernels that pass states of empty sequences on read the weights: none is refused on the host, tokens or not."""
    I, cv, sc = b.SSE_ERR_INVALID_ARG, b.make_conv_config(64), b.make_selective_config(64)
    for T, S in ((0, 1), (0, 3), (16, 1)):
        assert b.sse_conv_forward(cv, FAKE, 64, None, None, FAKE, S, T, FAKE, None, FAKE, None) == I
        assert b.sse_conv_backward(cv, FAKE, 64, None, None, FAKE, S, T, FAKE, FAKE, None, FAKE, FAKE, None, None, FAKE, ROOM, None) == I
        inputs = (FAKE, 64, FAKE, 64, None, None, FAKE, 16, FAKE, 16, None, None, 64, FAKE, S, T, FAKE)
        assert b.sse_selective_forward(sc, *inputs, None, FAKE, None, FAKE, ROOM, None) == I
        assert b.sse_selective_backward(sc, *inputs, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, None, FAKE,
                                        ROOM, None) == I
    # the gradients' kernel runs without sequences, too: d_A is zeroed
    inputs = (FAKE, 64, FAKE, 64, None, None, FAKE, 16, FAKE, 16, None, None, 64, FAKE, 0, 0, None)
    assert b.sse_selective_backward(sc, *inputs, None, None, None, None, None, None, FAKE, None, None, None, None, None, FAKE,
                                    ROOM, None) == I


def test_selective_forward_asks_for_its_workspace(b):
    """A missing, misaligned or short workspace of the forward is refused; a million tokens of 64 channels need one."""
    cfg, W = b.make_selective_config(64), b.SSE_ERR_WORKSPACE
    size = b.sse_selective_forward_workspace_size(cfg, 1 << 20, 1)
    assert size > 0

    def fwd(ws, n):
        return b.sse_selective_forward(cfg, FAKE, 64, FAKE, 64, None, FAKE, FAKE, 16, FAKE, 16, None, None, 64, FAKE, 1, 1 << 20,
                                       None, None, FAKE, None, ws, n, None)

    assert fwd(None, 0) == W and fwd(None, size) == W
    assert fwd(FAKE + 16, ROOM) == W and fwd(FAKE + 128, ROOM) == W
    assert fwd(FAKE, size - 256) == W and fwd(FAKE, 0) == W
