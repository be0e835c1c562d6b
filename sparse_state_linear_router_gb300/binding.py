"""Thin ctypes binding of libsse (include/sse.h).

The functions named like the C entry points (``sse_route``, ``sse_forward``,
``sse_decode_step``, ...) take raw integers (device pointers, sizes, a CUDA
stream handle) and only marshal arguments.  The ``route`` / ``forward`` /
``decode_step`` helpers take torch tensors, allocate outputs and the
workspace with torch (device memory plumbing only) and call the C entry
points on the current torch stream.  The ``scan_*`` and ``block_norm*`` helpers
also check the tensors' shapes, types, strides and device (SSEError with
SSE_ERR_INVALID_ARG) and run on the tensors' device, whichever is current.  Every step of the layer runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback: if libsse.so is
missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsse.so")

(SSE_OK, SSE_ERR_INVALID_ARG, SSE_ERR_UNSUPPORTED, SSE_ERR_WORKSPACE, SSE_ERR_CUDA, SSE_ERR_DEVICE,
 SSE_ERR_DEVICE_TIMEOUT) = range(7)
# device-status bits (sse_read_device_status)
SSE_DEVICE_TIMEOUT, SSE_DEVICE_RECOMPUTED = 2, 4
SSE_F32, SSE_BF16 = 0, 1
SSE_ALGO_AUTO, SSE_ALGO_CHUNKED, SSE_ALGO_RECURRENT, SSE_ALGO_MASKED = 0, 1, 2, 3
_ALGOS = {"auto": SSE_ALGO_AUTO, "chunked": SSE_ALGO_CHUNKED, "recurrent": SSE_ALGO_RECURRENT,
          "masked": SSE_ALGO_MASKED}

# Every extern "C" symbol that include/sse.h declares.
EXPORTED = ("sse_abi_version", "sse_status_string", "sse_route_workspace_size", "sse_route",
            "sse_route_noalloc", "sse_forward_workspace_size", "sse_forward", "sse_forward_timed", "sse_decode_step",
            "sse_front_end_workspace_size", "sse_front_end", "sse_read_device_status",
            "sse_get_last_device_error", "sse_backward_workspace_size", "sse_backward",
            "sse_delta_forward_workspace_size", "sse_delta_forward", "sse_delta_decode_step",
            "sse_scan_checkpoint_rows", "sse_scan_forward", "sse_scan_backward", "sse_scan_step",
            "sse_block_norm", "sse_block_norm_backward_workspace_size", "sse_block_norm_backward")

SSE_INPUT_PLAIN, SSE_INPUT_COMPLEMENT, SSE_INPUT_UNIT = 0, 1, 2
_INPUT_SCALES = {"plain": SSE_INPUT_PLAIN, "complement": SSE_INPUT_COMPLEMENT, "unit": SSE_INPUT_UNIT}
SSE_GATE_NONE, SSE_GATE_SILU, SSE_GATE_SIGMOID, SSE_GATE_LINEAR = 0, 1, 2, 3
_GATES = {"none": SSE_GATE_NONE, "silu": SSE_GATE_SILU, "sigmoid": SSE_GATE_SIGMOID, "linear": SSE_GATE_LINEAR}
SCAN_CHECKPOINT = 64  # packed tokens between two of the scan's stored states


class sse_config_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("key_dim", ctypes.c_int32),
                ("value_dim", ctypes.c_int32), ("num_partitions", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("use_shared", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("algo", ctypes.c_int32)]


class sse_scan_config_t(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("input_scale", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class sse_norm_config_t(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("group", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class SSEError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {sse_status_string(status)} (status {status})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libsse.so.  Raises when the library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libsse.so not found at {path}; build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(sse_config_t)
    lib.sse_abi_version.restype = i32
    lib.sse_abi_version.argtypes = []
    lib.sse_status_string.restype = ctypes.c_char_p
    lib.sse_status_string.argtypes = [ctypes.c_int]
    lib.sse_route_workspace_size.restype = sz
    lib.sse_route_workspace_size.argtypes = [cfgp, i64, i32]
    lib.sse_route.restype = ctypes.c_int
    lib.sse_route.argtypes = [cfgp, P, P, i32, i64, P, P, P, P, P, sz, P]
    lib.sse_route_noalloc.restype = ctypes.c_int
    lib.sse_route_noalloc.argtypes = [cfgp, P, P, i32, i64, P, P, P, P, P]
    lib.sse_forward_workspace_size.restype = sz
    lib.sse_forward_workspace_size.argtypes = [cfgp, i64, i32]
    lib.sse_forward.restype = ctypes.c_int
    lib.sse_forward.argtypes = [cfgp, P, P, P, P, P, P, P, P, i32, i64, P, P, P, P, P, P, sz, P]
    lib.sse_forward_timed.restype = ctypes.c_int
    lib.sse_forward_timed.argtypes = [cfgp, P, P, P, P, P, P, P, P, i32, i64, P, P, P, P, P, P, sz, P,
                                      P, ctypes.POINTER(i32)]
    lib.sse_decode_step.restype = ctypes.c_int
    lib.sse_decode_step.argtypes = [cfgp, P, P, P, P, P, P, P, i32, P, P, P, P, P]
    lib.sse_front_end_workspace_size.restype = sz
    lib.sse_front_end_workspace_size.argtypes = [cfgp, i32, i64]
    lib.sse_front_end.restype = ctypes.c_int
    lib.sse_front_end.argtypes = [cfgp, i32, i64, P, P, P, P, P, P, P, P, P, P, ctypes.c_float,
                                  P, P, P, P, P, P, P, P, sz, P]
    lib.sse_read_device_status.restype = ctypes.c_int
    lib.sse_read_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int32), P]
    lib.sse_get_last_device_error.restype = ctypes.c_int
    lib.sse_get_last_device_error.argtypes = [P, P]
    lib.sse_backward_workspace_size.restype = sz
    lib.sse_backward_workspace_size.argtypes = [cfgp, i64, i32]
    lib.sse_backward.restype = ctypes.c_int
    lib.sse_backward.argtypes = [cfgp, P, P, P, P, P, P, P, P, i32, i64, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.sse_delta_forward_workspace_size.restype = sz
    lib.sse_delta_forward_workspace_size.argtypes = [cfgp, i64, i32]
    lib.sse_delta_forward.restype = ctypes.c_int
    lib.sse_delta_forward.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, i32, i64, P, P, P, P, P, P, sz, P]
    lib.sse_delta_decode_step.restype = ctypes.c_int
    lib.sse_delta_decode_step.argtypes = [cfgp, P, P, P, P, P, P, P, P, i32, P, P, P, P, P]
    scanp, normp = ctypes.POINTER(sse_scan_config_t), ctypes.POINTER(sse_norm_config_t)
    lib.sse_scan_checkpoint_rows.restype = i64
    lib.sse_scan_checkpoint_rows.argtypes = [i64]
    lib.sse_scan_forward.restype = ctypes.c_int
    lib.sse_scan_forward.argtypes = [scanp, P, i64, P, i64, P, i32, i64, P, P, P, P, P]
    lib.sse_scan_backward.restype = ctypes.c_int
    lib.sse_scan_backward.argtypes = [scanp, P, i64, P, i64, P, i32, i64, P, P, P, P, P, P, P, P]
    lib.sse_scan_step.restype = ctypes.c_int
    lib.sse_scan_step.argtypes = [scanp, P, i64, P, i64, i32, P, P, P]
    lib.sse_block_norm.restype = ctypes.c_int
    lib.sse_block_norm.argtypes = [normp, i64, P, i64, P, i64, P, i64, P, P, P, P, P, P]
    lib.sse_block_norm_backward_workspace_size.restype = sz
    lib.sse_block_norm_backward_workspace_size.argtypes = [normp, i64]
    lib.sse_block_norm_backward.restype = ctypes.c_int
    lib.sse_block_norm_backward.argtypes = [normp, i64, P, i64, P, i64, P, i64, P, P, P, P, P, P, P, P, P, P, P, P,
                                            sz, P]
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# Raw C entry points (integers in, status out)
# ---------------------------------------------------------------------------
def sse_abi_version() -> int:
    return load().sse_abi_version()


def sse_status_string(status: int) -> str:
    return load().sse_status_string(status).decode()


def sse_route_workspace_size(cfg: sse_config_t, total_tokens: int, num_seqs: int) -> int:
    return load().sse_route_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs)


def sse_forward_workspace_size(cfg: sse_config_t, total_tokens: int, num_seqs: int) -> int:
    return load().sse_forward_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs)


def sse_route(cfg, logits, cu_seqlens, num_seqs, total_tokens, topk_idx, topk_w, seg_off, perm,
              workspace, workspace_bytes, stream) -> int:
    return load().sse_route(ctypes.byref(cfg), logits, cu_seqlens, num_seqs, total_tokens, topk_idx,
                            topk_w, seg_off, perm, workspace, workspace_bytes, stream)


def sse_forward(cfg, q, k, v, log_gate, logits, q_shared, k_shared, cu_seqlens, num_seqs,
                total_tokens, initial_state, final_state, out, topk_idx, topk_w, workspace,
                workspace_bytes, stream) -> int:
    return load().sse_forward(ctypes.byref(cfg), q, k, v, log_gate, logits, q_shared, k_shared,
                              cu_seqlens, num_seqs, total_tokens, initial_state, final_state, out,
                              topk_idx, topk_w, workspace, workspace_bytes, stream)


def sse_forward_timed(cfg, q, k, v, log_gate, logits, q_shared, k_shared, cu_seqlens, num_seqs,
                      total_tokens, initial_state, final_state, out, topk_idx, topk_w, workspace,
                      workspace_bytes, stream, stage_events=None):
    """Returns (status, kernels launched).  stage_events: 4 raw cudaEvent_t handles or None."""
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * 4)(*stage_events)
    n = ctypes.c_int32(0)
    st = load().sse_forward_timed(ctypes.byref(cfg), q, k, v, log_gate, logits, q_shared, k_shared,
                                  cu_seqlens, num_seqs, total_tokens, initial_state, final_state, out,
                                  topk_idx, topk_w, workspace, workspace_bytes, stream, ev,
                                  ctypes.byref(n))
    return st, n.value


def sse_decode_step(cfg, q, k, v, log_gate, logits, q_shared, k_shared, batch, state, out,
                    topk_idx, topk_w, stream) -> int:
    return load().sse_decode_step(ctypes.byref(cfg), q, k, v, log_gate, logits, q_shared, k_shared,
                                  batch, state, out, topk_idx, topk_w, stream)


def sse_front_end_workspace_size(cfg: sse_config_t, hidden: int, total_tokens: int) -> int:
    return int(load().sse_front_end_workspace_size(ctypes.byref(cfg), hidden, total_tokens))


def sse_front_end(cfg, hidden, total_tokens, x, w_q, w_k, w_v, w_g, w_e, a_q, b_q, a_k, b_k,
                  gate_inv_tau, q, k, v, log_gate, logits, q_shared, k_shared, workspace,
                  workspace_bytes, stream) -> int:
    return load().sse_front_end(ctypes.byref(cfg), hidden, total_tokens, x, w_q, w_k, w_v, w_g, w_e,
                                a_q, b_q, a_k, b_k, float(gate_inv_tau), q, k, v, log_gate, logits,
                                q_shared, k_shared, workspace, workspace_bytes, stream)


def sse_read_device_status(workspace, stream):
    flags = ctypes.c_int32(0)
    st = load().sse_read_device_status(workspace, ctypes.byref(flags), stream)
    return st, flags.value


def sse_get_last_device_error(workspace, stream) -> int:
    return load().sse_get_last_device_error(workspace, stream)


def sse_backward_workspace_size(cfg: sse_config_t, total_tokens: int, num_seqs: int) -> int:
    return load().sse_backward_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs)


def sse_backward(cfg, q, k, v, log_gate, logits, q_shared, k_shared, cu_seqlens, num_seqs, total_tokens,
                 initial_state, d_out, d_final_state, dq, dk, dv, d_log_gate, d_logits, dq_shared, dk_shared,
                 d_initial_state, workspace, workspace_bytes, stream) -> int:
    return load().sse_backward(ctypes.byref(cfg), q, k, v, log_gate, logits, q_shared, k_shared, cu_seqlens,
                               num_seqs, total_tokens, initial_state, d_out, d_final_state, dq, dk, dv, d_log_gate,
                               d_logits, dq_shared, dk_shared, d_initial_state, workspace, workspace_bytes, stream)


def sse_scan_checkpoint_rows(total_tokens: int) -> int:
    return load().sse_scan_checkpoint_rows(total_tokens)


def sse_scan_forward(cfg, x, x_stride, log_gate, gate_stride, cu_seqlens, num_seqs, total_tokens, initial_state,
                     final_state, out, checkpoints, stream) -> int:
    return load().sse_scan_forward(ctypes.byref(cfg), x, x_stride, log_gate, gate_stride, cu_seqlens, num_seqs,
                                   total_tokens, initial_state, final_state, out, checkpoints, stream)


def sse_scan_backward(cfg, x, x_stride, log_gate, gate_stride, cu_seqlens, num_seqs, total_tokens, initial_state,
                      checkpoints, d_out, d_final_state, dx, d_log_gate, d_initial_state, stream) -> int:
    return load().sse_scan_backward(ctypes.byref(cfg), x, x_stride, log_gate, gate_stride, cu_seqlens, num_seqs,
                                    total_tokens, initial_state, checkpoints, d_out, d_final_state, dx, d_log_gate,
                                    d_initial_state, stream)


def sse_scan_step(cfg, x, x_stride, log_gate, gate_stride, batch, state, out, stream) -> int:
    return load().sse_scan_step(ctypes.byref(cfg), x, x_stride, log_gate, gate_stride, batch, state, out, stream)


def sse_block_norm(cfg, total_tokens, block_out, block_stride, gate, gate_stride, residual, residual_stride, w_after,
                   channel_scale, w_before, residual_out, next_in, stream) -> int:
    return load().sse_block_norm(ctypes.byref(cfg), total_tokens, block_out, block_stride, gate, gate_stride,
                                 residual, residual_stride, w_after, channel_scale, w_before, residual_out, next_in,
                                 stream)


def sse_block_norm_backward_workspace_size(cfg: sse_norm_config_t, total_tokens: int) -> int:
    return load().sse_block_norm_backward_workspace_size(ctypes.byref(cfg), total_tokens)


def sse_block_norm_backward(cfg, total_tokens, block_out, block_stride, gate, gate_stride, residual_out,
                            residual_stride, w_after, channel_scale, w_before, d_residual_out, d_next_in, d_block_out,
                            d_gate, d_residual, d_w_after, d_channel_scale, d_w_before, workspace, workspace_bytes,
                            stream) -> int:
    return load().sse_block_norm_backward(ctypes.byref(cfg), total_tokens, block_out, block_stride, gate, gate_stride,
                                          residual_out, residual_stride, w_after, channel_scale, w_before,
                                          d_residual_out, d_next_in, d_block_out, d_gate, d_residual, d_w_after,
                                          d_channel_scale, d_w_before, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# torch-tensor helpers (allocation of outputs/workspace + marshalling)
# ---------------------------------------------------------------------------
def make_config(num_heads, key_dim, value_dim, num_partitions, top_k, use_shared=1, scale=1.0,
                dtype="bf16", algo="auto") -> sse_config_t:
    dt = {"bf16": SSE_BF16, "f32": SSE_F32}[dtype] if isinstance(dtype, str) else dtype
    return sse_config_t(num_heads, key_dim, value_dim, num_partitions, top_k, int(use_shared),
                        float(scale), dt, _ALGOS[algo] if isinstance(algo, str) else int(algo))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(status: int, what: str):
    if status != SSE_OK:
        raise SSEError(status, what)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _token_dtype(cfg):
    torch = _torch()
    return torch.bfloat16 if cfg.dtype == SSE_BF16 else torch.float32


def route(cfg, logits, cu_seqlens, group: bool = True, workspace=None):
    """Returns dict(topk_idx [T,H,k] int32, topk_w [T,H,k] f32, seg_off, perm)."""
    import torch
    T = logits.shape[0]
    S = cu_seqlens.numel() - 1
    H, k, N = cfg.num_heads, cfg.top_k, cfg.num_partitions
    dev = logits.device
    idx = torch.empty((T, H, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, H, k), dtype=torch.float32, device=dev)
    seg_off = torch.empty(S * H * N + 1, dtype=torch.int32, device=dev) if group else None
    perm = torch.empty(max(1, H * k * T), dtype=torch.int32, device=dev) if group else None
    nbytes = sse_route_workspace_size(cfg, T, S)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _check(sse_route(cfg, _ptr(logits), _ptr(cu_seqlens), S, T, _ptr(idx), _ptr(w), _ptr(seg_off),
                     _ptr(perm), _ptr(workspace), workspace.numel(), _stream()), "sse_route")
    return {"topk_idx": idx, "topk_w": w, "seg_off": seg_off,
            "perm": None if perm is None else perm[:H * k * T]}


def forward_workspace(cfg, total_tokens: int, num_seqs: int, device="cuda"):
    import torch
    n = sse_forward_workspace_size(cfg, total_tokens, num_seqs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def forward(cfg, q, k, v, log_gate, logits, cu_seqlens, *, q_shared=None, k_shared=None,
            initial_state=None, want_final_state=True, out=None, final_state=None,
            want_routing=False, workspace=None):
    """SSE forward on device tensors; returns dict(out, final_state, topk_idx, topk_w)."""
    import torch
    T = q.shape[0]
    S = cu_seqlens.numel() - 1
    H, d, c = cfg.num_heads, cfg.value_dim, cfg.key_dim
    P = cfg.num_partitions + cfg.use_shared
    dev = q.device
    if out is None:
        out = torch.empty((T, H, d), dtype=_token_dtype(cfg), device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((S, H, P, c, d), dtype=torch.float32, device=dev)
    idx = w = None
    if want_routing:
        idx = torch.empty((T, H, cfg.top_k), dtype=torch.int32, device=dev)
        w = torch.empty((T, H, cfg.top_k), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = forward_workspace(cfg, T, S, dev)
    _check(sse_forward(cfg, _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(logits), _ptr(q_shared),
                       _ptr(k_shared), _ptr(cu_seqlens), S, T, _ptr(initial_state), _ptr(final_state),
                       _ptr(out), _ptr(idx), _ptr(w), _ptr(workspace), workspace.numel(), _stream()),
           "sse_forward")
    return {"out": out, "final_state": final_state, "topk_idx": idx, "topk_w": w,
            "workspace": workspace}


def decode_step(cfg, state, q, k, v, log_gate, logits, *, q_shared=None, k_shared=None, out=None,
                want_routing=False):
    """One decode step; ``state`` [B,H,P,c,d] float32 is updated in place."""
    import torch
    B = q.shape[0]
    H, d = cfg.num_heads, cfg.value_dim
    dev = q.device
    if out is None:
        out = torch.empty((B, H, d), dtype=_token_dtype(cfg), device=dev)
    idx = w = None
    if want_routing:
        idx = torch.empty((B, H, cfg.top_k), dtype=torch.int32, device=dev)
        w = torch.empty((B, H, cfg.top_k), dtype=torch.float32, device=dev)
    _check(sse_decode_step(cfg, _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(logits),
                           _ptr(q_shared), _ptr(k_shared), B, _ptr(state), _ptr(out), _ptr(idx),
                           _ptr(w), _stream()), "sse_decode_step")
    return {"out": out, "topk_idx": idx, "topk_w": w}


def backward(cfg, q, k, v, log_gate, logits, cu_seqlens, d_out, *, q_shared=None, k_shared=None,
             initial_state=None, d_final_state=None, want_d_initial_state=True, workspace=None):
    """Gradients of <d_out, out> + <d_final_state, final_state> on device
    tensors; returns dict(dq, dk, dv, dg, dlogits, dq_shared, dk_shared,
    d_initial_state, workspace)."""
    import torch
    T = q.shape[0]
    S = cu_seqlens.numel() - 1
    H, c, d, N = cfg.num_heads, cfg.key_dim, cfg.value_dim, cfg.num_partitions
    P = N + cfg.use_shared
    dev = q.device
    dt = _token_dtype(cfg)
    e = lambda w: torch.empty((T, H, w), dtype=dt, device=dev)  # noqa: E731
    out = {"dq": e(c), "dk": e(c), "dv": e(d), "dg": e(c), "dlogits": e(N),
           "dq_shared": e(c) if q_shared is not None else None,
           "dk_shared": e(c) if k_shared is not None else None,
           "d_initial_state": (torch.empty((S, H, P, c, d), dtype=torch.float32, device=dev)
                               if want_d_initial_state else None)}
    if workspace is None:
        workspace = torch.empty(max(sse_backward_workspace_size(cfg, T, S), 256), dtype=torch.uint8, device=dev)
    _check(sse_backward(cfg, _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(logits), _ptr(q_shared),
                        _ptr(k_shared), _ptr(cu_seqlens), S, T, _ptr(initial_state), _ptr(d_out),
                        _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                        _ptr(out["dlogits"]), _ptr(out["dq_shared"]), _ptr(out["dk_shared"]),
                        _ptr(out["d_initial_state"]), _ptr(workspace), workspace.numel(), _stream()),
           "sse_backward")
    return dict(out, workspace=workspace)


def delta_forward(cfg, q, k, v, log_alpha, beta, logits, cu_seqlens, *, q_shared=None, k_shared=None,
                  initial_state=None, want_final_state=True, want_routing=False, workspace=None):
    """SSE on the gated delta rule (sse_delta_forward) on device tensors;
    returns dict(out, final_state, topk_idx, topk_w, workspace)."""
    import torch
    T = q.shape[0]
    S = cu_seqlens.numel() - 1
    H, d, c = cfg.num_heads, cfg.value_dim, cfg.key_dim
    P = cfg.num_partitions + cfg.use_shared
    dev = q.device
    out = torch.empty((T, H, d), dtype=_token_dtype(cfg), device=dev)
    fin = torch.empty((S, H, P, c, d), dtype=torch.float32, device=dev) if want_final_state else None
    idx = w = None
    if want_routing:
        idx = torch.empty((T, H, cfg.top_k), dtype=torch.int32, device=dev)
        w = torch.empty((T, H, cfg.top_k), dtype=torch.float32, device=dev)
    if workspace is None:
        n = load().sse_delta_forward_workspace_size(ctypes.byref(cfg), T, S)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    _check(load().sse_delta_forward(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                    _ptr(logits), _ptr(q_shared), _ptr(k_shared), _ptr(cu_seqlens), S, T,
                                    _ptr(initial_state), _ptr(fin), _ptr(out), _ptr(idx), _ptr(w), _ptr(workspace),
                                    workspace.numel(), _stream()), "sse_delta_forward")
    return {"out": out, "final_state": fin, "topk_idx": idx, "topk_w": w, "workspace": workspace}


def delta_decode_step(cfg, state, q, k, v, log_alpha, beta, logits, *, q_shared=None, k_shared=None,
                      want_routing=False):
    """One delta-rule decode step; ``state`` [B,H,P,c,d] float32 is updated in place."""
    import torch
    B = q.shape[0]
    H, d = cfg.num_heads, cfg.value_dim
    dev = q.device
    out = torch.empty((B, H, d), dtype=_token_dtype(cfg), device=dev)
    idx = w = None
    if want_routing:
        idx = torch.empty((B, H, cfg.top_k), dtype=torch.int32, device=dev)
        w = torch.empty((B, H, cfg.top_k), dtype=torch.float32, device=dev)
    _check(load().sse_delta_decode_step(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                        _ptr(logits), _ptr(q_shared), _ptr(k_shared), B, _ptr(state), _ptr(out),
                                        _ptr(idx), _ptr(w), _stream()), "sse_delta_decode_step")
    return {"out": out, "topk_idx": idx, "topk_w": w}


def front_end(cfg, x, w_q, w_k, w_v, w_g, w_e, *, a_q=None, b_q=None, a_k=None, b_k=None,
              gate_inv_tau=1.0 / 16.0, outs=None, workspace=None):
    """Projections from the hidden states x [T, D] (bf16 device tensors);
    returns dict(q, k, v, log_gate, logits, q_shared, k_shared, workspace)."""
    import torch
    T, D = x.shape
    H, c, d, N = cfg.num_heads, cfg.key_dim, cfg.value_dim, cfg.num_partitions
    dev = x.device
    lora = a_q is not None
    if outs is None:
        e = lambda w: torch.empty((T, H, w), dtype=torch.bfloat16, device=dev)  # noqa: E731
        outs = {"q": e(c), "k": e(c), "v": e(d), "log_gate": e(c), "logits": e(N),
                "q_shared": e(c) if lora else None, "k_shared": e(c) if lora else None}
    if workspace is None:
        workspace = torch.empty(max(sse_front_end_workspace_size(cfg, D, T), 256), dtype=torch.uint8,
                                device=dev)
    _check(sse_front_end(cfg, D, T, _ptr(x), _ptr(w_q), _ptr(w_k), _ptr(w_v), _ptr(w_g), _ptr(w_e),
                         _ptr(a_q), _ptr(b_q), _ptr(a_k), _ptr(b_k), gate_inv_tau, _ptr(outs["q"]),
                         _ptr(outs["k"]), _ptr(outs["v"]), _ptr(outs["log_gate"]), _ptr(outs["logits"]),
                         _ptr(outs["q_shared"]), _ptr(outs["k_shared"]), _ptr(workspace), workspace.numel(),
                         _stream()), "sse_front_end")
    return dict(outs, workspace=workspace)


# ---------------------------------------------------------------------------
# Gated linear recurrence and block norms: helpers that check their tensors
# ---------------------------------------------------------------------------
def make_scan_config(width, input_scale="plain", dtype="bf16") -> sse_scan_config_t:
    return sse_scan_config_t(width, _INPUT_SCALES[input_scale] if isinstance(input_scale, str) else int(input_scale),
                             {"bf16": SSE_BF16, "f32": SSE_F32}[dtype] if isinstance(dtype, str) else dtype)


def make_norm_config(width, group=0, gate="none", eps=1e-6, residual_scale=1.0, branch_scale=1.0,
                     dtype="bf16") -> sse_norm_config_t:
    return sse_norm_config_t(width, group, _GATES[gate] if isinstance(gate, str) else int(gate), float(eps),
                             float(residual_scale), float(branch_scale),
                             {"bf16": SSE_BF16, "f32": SSE_F32}[dtype] if isinstance(dtype, str) else dtype)


def _refuse(what: str, why: str):
    raise SSEError(SSE_ERR_INVALID_ARG, f"{what}: {why}")


def _refuse_tokens(what, name, t, rows, width, dtype, device):
    if t.dtype != dtype or t.device != device:
        _refuse(what, f"{name} is {t.dtype} on {t.device}, not {dtype} on {device}")
    _refuse(what, f"{name} has shape {tuple(t.shape)}, not [{rows}, {width}] or [{rows}, heads, {width} / heads]")


def _rows(what, name, t, rows, width, dtype, device):
    """(pointer, row stride) of a token tensor [rows, width] or [rows, heads, width / heads] whose rows are packed."""
    if t is None:
        return None, width
    if t.dtype is not dtype or t.device != device or t.shape != (rows, width) and (
            t.dim() < 2 or t.shape[0] != rows or t.numel() != rows * width):
        _refuse_tokens(what, name, t, rows, width, dtype, device)
    if t.is_contiguous():
        return t.data_ptr(), width
    stride = t.stride()
    inner = 1
    for n, s in zip(t.shape[:0:-1], stride[:0:-1]):
        if n != 1 and s != inner:
            _refuse(what, f"{name} has strides {stride}: the columns of a row are not packed")
        inner *= n
    if rows <= 1:
        return t.data_ptr(), width
    if stride[0] < width:
        _refuse(what, f"{name} has row stride {stride[0]}, below its width {width}")
    return t.data_ptr(), stride[0]


def _packed(what, name, t, rows, width, dtype, device):
    """Pointer of a contiguous token tensor."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.shape != (rows, width) and (
            t.dim() < 2 or t.shape[0] != rows or t.numel() != rows * width):
        _refuse_tokens(what, name, t, rows, width, dtype, device)
    if not t.is_contiguous():
        _refuse(what, f"{name} is not contiguous")
    return t.data_ptr()


def _floats(what, name, t, shape, device):
    """Pointer of a contiguous float32 tensor."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not _torch().float32 or t.device != device or not t.is_contiguous():
        _refuse(what, f"{name} is not a contiguous float32 {list(shape)} on {device}")
    return t.data_ptr()


def _on_device(what, device, call, *args):
    """One C call on the tensors' device and its current stream, whichever device is current."""
    # The device and the stream as numbers: torch.cuda's own functions put objects around them, 1.2 us of a
    # 10 us step on the host of a GB300.
    torch, index = _torch(), device.index
    if index == torch._C._cuda_getDevice():
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != SSE_OK:
        raise SSEError(status, what)


def _first(what, t):
    """Rows, device and type check of the tensor that the others are compared with."""
    if t is None or not t.is_cuda or t.dim() < 2:
        _refuse(what, "a [tokens, width] CUDA tensor is required")
    return t.shape[0], t.device


def _sequences(what, cu_seqlens, device):
    if (cu_seqlens is None or cu_seqlens.dtype is not _torch().int32 or cu_seqlens.device != device or
            cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous()):
        _refuse(what, f"cu_seqlens is not a contiguous int32 [sequences + 1] on {device}")
    return cu_seqlens.numel() - 1


def _like(t):
    """A packed tensor of t's shape and type."""
    torch = _torch()
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def scan_forward(cfg, x, log_gate, cu_seqlens, *, initial_state=None, want_final_state=True, want_checkpoints=False,
                 out=None, final_state=None, checkpoints=None):
    """The gated linear recurrence (sse_scan_forward) over packed sequences;
    x, log_gate [T, width] or [T, H, width / H].  Returns dict(out,
    final_state, checkpoints); checkpoints are what scan_backward reads."""
    torch, what = _torch(), "sse_scan_forward"
    T, dev = _first(what, x)
    S, W, dt = _sequences(what, cu_seqlens, dev), cfg.width, _token_dtype(cfg)
    px, sx = _rows(what, "x", x, T, W, dt, dev)
    pg, sg = _rows(what, "log_gate", log_gate, T, W, dt, dev)
    pi = _floats(what, "initial_state", initial_state, (S, W), dev)
    po, pf, pc = (_packed(what, "out", out, T, W, dt, dev), _floats(what, "final_state", final_state, (S, W), dev),
                  _floats(what, "checkpoints", checkpoints, (-(-T // SCAN_CHECKPOINT), W), dev))
    if out is None:
        out = _like(x)
        po = out.data_ptr()
    if final_state is None and want_final_state:
        final_state = torch.empty((S, W), dtype=torch.float32, device=dev)
        pf = final_state.data_ptr()
    if checkpoints is None and want_checkpoints:
        checkpoints = torch.empty((-(-T // SCAN_CHECKPOINT), W), dtype=torch.float32, device=dev)
        pc = checkpoints.data_ptr()
    _on_device(what, dev, load().sse_scan_forward, ctypes.byref(cfg), px, sx, pg, sg, cu_seqlens.data_ptr(), S, T, pi,
               pf, po, pc)
    return {"out": out, "final_state": final_state, "checkpoints": checkpoints}


def scan_backward(cfg, x, log_gate, cu_seqlens, checkpoints, d_out, *, initial_state=None, d_final_state=None,
                  want_d_initial_state=True):
    """Gradients of <d_out, out> + <d_final_state, final_state> of scan_forward
    (sse_scan_backward); returns dict(dx, d_log_gate, d_initial_state)."""
    torch, what = _torch(), "sse_scan_backward"
    T, dev = _first(what, x)
    S, W, dt = _sequences(what, cu_seqlens, dev), cfg.width, _token_dtype(cfg)
    px, sx = _rows(what, "x", x, T, W, dt, dev)
    pg, sg = _rows(what, "log_gate", log_gate, T, W, dt, dev)
    pd = _packed(what, "d_out", d_out, T, W, dt, dev)
    if log_gate is None:
        _refuse(what, "log_gate is None")
    if checkpoints is None:
        _refuse(what, "checkpoints is None: scan_forward(..., want_checkpoints=True) returns them")
    pc = _floats(what, "checkpoints", checkpoints, (-(-T // SCAN_CHECKPOINT), W), dev)
    dx, dg = _like(x), _like(log_gate)
    d_init = torch.empty((S, W), dtype=torch.float32, device=dev) if want_d_initial_state else None
    _on_device(what, dev, load().sse_scan_backward, ctypes.byref(cfg), px, sx, pg, sg, cu_seqlens.data_ptr(), S, T,
               _floats(what, "initial_state", initial_state, (S, W), dev), pc, pd,
               _floats(what, "d_final_state", d_final_state, (S, W), dev), dx.data_ptr(), dg.data_ptr(), _ptr(d_init))
    return {"dx": dx, "d_log_gate": dg, "d_initial_state": d_init}


def scan_step(cfg, state, x, log_gate, *, out=None):
    """One token of each sequence (sse_scan_step): x, log_gate [B, width];
    ``state`` [B, width] float32 is updated in place.  Returns dict(out)."""
    what = "sse_scan_step"
    B, dev = _first(what, x)
    W, dt = cfg.width, _token_dtype(cfg)
    px, sx = _rows(what, "x", x, B, W, dt, dev)
    pg, sg = _rows(what, "log_gate", log_gate, B, W, dt, dev)
    if state is None:
        _refuse(what, "state is None")
    ps = _floats(what, "state", state, (B, W), dev)
    if out is None:
        out = _like(x)
        po = out.data_ptr()
    else:
        po = _packed(what, "out", out, B, W, dt, dev)
    _on_device(what, dev, load().sse_scan_step, ctypes.byref(cfg), px, sx, pg, sg, B, ps, po)
    return {"out": out}


def block_norm(cfg, block_out=None, *, gate=None, residual=None, w_after=None, channel_scale=None, w_before=None,
               residual_out=None, next_in=None, want_residual_out=True):
    """The norms before and after a block with its gate and the residual
    stream (sse_block_norm); token tensors [T, width] or [T, H, width / H].
    Returns dict(residual_out, next_in); next_in is None without w_before."""
    what = "sse_block_norm"
    like = residual if residual is not None else block_out
    T, dev = _first(what, like)
    W, dt = cfg.width, _token_dtype(cfg)
    po, so = _rows(what, "block_out", block_out, T, W, dt, dev)
    pz, sz = _rows(what, "gate", gate, T, W, dt, dev)
    pr, sr = _rows(what, "residual", residual, T, W, dt, dev)
    wa = _floats(what, "w_after", w_after, (W,), dev)
    wc = _floats(what, "channel_scale", channel_scale, (W,), dev)
    wb = _floats(what, "w_before", w_before, (W,), dev)
    pt, pn = (_packed(what, "residual_out", residual_out, T, W, dt, dev),
              _packed(what, "next_in", next_in, T, W, dt, dev))
    if residual_out is None and want_residual_out:
        residual_out = _like(like)
        pt = residual_out.data_ptr()
    if next_in is None and w_before is not None:
        next_in = _like(like)
        pn = next_in.data_ptr()
    _on_device(what, dev, load().sse_block_norm, ctypes.byref(cfg), T, po, so, pz, sz, pr, sr, wa, wc, wb, pt, pn)
    return {"residual_out": residual_out, "next_in": next_in}


def block_norm_backward(cfg, d_residual_out, block_out=None, *, gate=None, w_after=None, channel_scale=None,
                        w_before=None, residual_out=None, d_next_in=None, want_d_residual=True, workspace=None):
    """Gradients of <d_residual_out, residual_out> + <d_next_in, next_in> of
    block_norm (sse_block_norm_backward); residual_out is the forward's.
    Returns dict(d_block_out, d_gate, d_residual, d_w_after, d_channel_scale,
    d_w_before), None where the part is absent."""
    torch, what = _torch(), "sse_block_norm_backward"
    first = d_residual_out if d_residual_out is not None else d_next_in
    T, dev = _first(what, first)
    W, dt = cfg.width, _token_dtype(cfg)
    po, so = _rows(what, "block_out", block_out, T, W, dt, dev)
    pz, sz = _rows(what, "gate", gate, T, W, dt, dev)
    pr, sr = _rows(what, "residual_out", residual_out, T, W, dt, dev)
    pd = _packed(what, "d_residual_out", d_residual_out, T, W, dt, dev)
    pn = _packed(what, "d_next_in", d_next_in, T, W, dt, dev)
    wa = _floats(what, "w_after", w_after, (W,), dev)
    wc = _floats(what, "channel_scale", channel_scale, (W,), dev)
    wb = _floats(what, "w_before", w_before, (W,), dev)
    g = {"d_block_out": None if block_out is None else _like(block_out), "d_gate": None if gate is None else _like(gate),
         "d_residual": _like(first) if want_d_residual else None,
         "d_w_after": None if w_after is None else _like(w_after),
         "d_channel_scale": None if channel_scale is None else _like(channel_scale),
         "d_w_before": None if w_before is None else _like(w_before)}
    if workspace is None:
        n = load().sse_block_norm_backward_workspace_size(ctypes.byref(cfg), T)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    elif workspace.dtype is not torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        _refuse(what, f"workspace is not a contiguous uint8 tensor on {dev}")
    _on_device(what, dev, load().sse_block_norm_backward, ctypes.byref(cfg), T, po, so, pz, sz, pr, sr, wa, wc, wb, pd,
               pn, *map(_ptr, g.values()), workspace.data_ptr(), workspace.numel())
    return g


def to_device(arr, device="cuda"):
    """numpy storage array (float32, or bf16 bits in uint16) -> torch tensor."""
    import numpy as np
    import torch
    if arr.dtype == np.uint16:
        return torch.from_numpy(arr.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(np.ascontiguousarray(arr)).to(device)
