"""ctypes binding of libkda (include/kda.h).

Argument marshalling only: the raw functions carry the C names and take
integer device pointers; the torch helpers below turn tensors into those
pointers and the current CUDA stream.  Every step of the computation runs in
libkda's kernels.  There is no fallback: if ``libkda.so`` is missing or the
device is unsupported, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(PKG, "libkda.so")

KDA_OK = 0
KDA_DTYPE_F32 = 0
KDA_DTYPE_BF16 = 1
KDA_CONV_SILU, KDA_CONV_L2NORM, KDA_CONV_HEAD_MAJOR = 1, 2, 4
KDA_PATH_AUTO, KDA_PATH_SIMT16, KDA_PATH_TC32 = 0, 1, 2
STATUS_NAMES = ["KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_SHAPE", "KDA_ERR_DTYPE", "KDA_ERR_ALIGNMENT",
                "KDA_ERR_ALIAS", "KDA_ERR_WORKSPACE", "KDA_ERR_CUDA", "KDA_ERR_TIMEOUT",
                "KDA_ERR_UNSUPPORTED", "KDA_ERR_DEVICE"]
EXPORTED = ["kda_chunk_fwd_plan", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd", "kda_recurrent_step",
            "kda_status_string", "kda_get_device_status", "kda_version", "kda_chunk_fwd_noalloc",
            "kda_noalloc_scratch_bytes", "kda_chunk_fwd_ckpt", "kda_chunk_fwd_gated", "kda_output_gate",
            "kda_kcp_compose", "kda_spec_replay_verify", "kda_debug_set_wait_limit", "kda_debug_inject_stall",
            "kda_chunk_fwd_outgate", "kda_chunk_transition", "kda_spec_replay_verify_fused", "kda_block_map",
            "kda_short_conv", "kda_short_conv_step", "kda_ssm_scan", "kda_ssm_scan_workspace_size", "kda_ssm_step"]


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s%s" % (kda_status_string(status), (" (" + what + ")") if what else ""))


class kda_plan_t(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("chunk_size", ctypes.c_int), ("segments", ctypes.c_int),
                ("launches", ctypes.c_int), ("workspace", ctypes.c_size_t), ("segment_tokens", ctypes.c_int)]


_lib = None
_lock = threading.Lock()


def load_library():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(SO):
                raise RuntimeError("libkda.so is not built (run gated_delta_rule_117_b200.build.build())")
            lib = ctypes.CDLL(SO)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.kda_chunk_fwd_plan.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(kda_plan_t)]
            lib.kda_chunk_fwd_plan.restype = i
            lib.kda_chunk_fwd_workspace_size.argtypes = [i] * 7
            lib.kda_chunk_fwd_workspace_size.restype = sz
            lib.kda_chunk_fwd.argtypes = [vp] * 8 + [i] * 7 + [f, vp, sz, vp]
            lib.kda_chunk_fwd.restype = i
            lib.kda_chunk_fwd_ckpt.argtypes = [vp] * 9 + [i] * 8 + [f, vp, sz, vp]
            lib.kda_chunk_fwd_ckpt.restype = i
            lib.kda_chunk_fwd_gated.argtypes = [vp] * 5 + [f] + [vp] * 4 + [i] * 7 + [f, vp, sz, vp]
            lib.kda_chunk_fwd_gated.restype = i
            lib.kda_chunk_fwd_outgate.argtypes = [vp] * 8 + [f, vp, vp] + [i] * 7 + [f, vp, sz, vp]
            lib.kda_chunk_fwd_outgate.restype = i
            lib.kda_chunk_transition.argtypes = [vp] * 6 + [i] * 6 + [vp]
            lib.kda_chunk_transition.restype = i
            lib.kda_output_gate.argtypes = [vp, vp, vp, f, vp] + [i] * 5 + [vp]
            lib.kda_output_gate.restype = i
            lib.kda_kcp_compose.argtypes = [vp] * 4 + [i] * 5 + [vp]
            lib.kda_kcp_compose.restype = i
            lib.kda_spec_replay_verify_fused.argtypes = [vp] * 5 + [f] + [vp] * 4 + [f] + [vp] * 2 + [i] * 6 + [f, vp]
            lib.kda_spec_replay_verify_fused.restype = i
            lib.kda_spec_replay_verify.argtypes = [vp] * 8 + [i] * 6 + [f, vp]
            lib.kda_spec_replay_verify.restype = i
            lib.kda_recurrent_step.argtypes = [vp] * 7 + [i] * 5 + [f, vp]
            lib.kda_recurrent_step.restype = i
            lib.kda_status_string.argtypes = [i]
            lib.kda_status_string.restype = ctypes.c_char_p
            lib.kda_get_device_status.argtypes = [vp]
            lib.kda_get_device_status.restype = i
            lib.kda_debug_set_wait_limit.argtypes = [ctypes.c_ulonglong]
            lib.kda_debug_set_wait_limit.restype = i
            lib.kda_debug_inject_stall.argtypes = [i]
            lib.kda_debug_inject_stall.restype = i
            lib.kda_version.argtypes = []
            lib.kda_version.restype = i
            lib.kda_chunk_fwd_noalloc.argtypes = [vp] * 8 + [i] * 7 + [f, vp]
            lib.kda_chunk_fwd_noalloc.restype = i
            lib.kda_noalloc_scratch_bytes.argtypes = []
            lib.kda_noalloc_scratch_bytes.restype = sz
            ll = ctypes.c_longlong
            lib.kda_block_map.argtypes = [vp, vp, vp, i, vp, i, i, vp, vp, vp, i, i, vp]
            lib.kda_block_map.restype = i
            lib.kda_short_conv.argtypes = [vp, ll, vp, vp, vp, i, vp, vp, vp, vp, ll] + [i] * 7 + [f, vp]
            lib.kda_short_conv.restype = i
            lib.kda_short_conv_step.argtypes = [vp, ll, vp, vp, vp, i, vp, vp, ll] + [i] * 6 + [f, vp]
            lib.kda_short_conv_step.restype = i
            lib.kda_ssm_scan.argtypes = ([vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, i, vp, i, vp, vp, vp, vp, i, vp, i, i,
                                          vp, ll] + [i] * 7 + [vp, sz, vp])
            lib.kda_ssm_scan.restype = i
            lib.kda_ssm_scan_workspace_size.argtypes = [i] * 7
            lib.kda_ssm_scan_workspace_size.restype = sz
            lib.kda_ssm_step.argtypes = [vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, i, vp, i, vp, vp, ll] + [i] * 6 + [vp]
            lib.kda_ssm_step.restype = i
            _lib = lib
    return _lib


# ---- raw C-ABI calls (integer pointers) ------------------------------------

def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return load_library().kda_version()


def kda_chunk_fwd_plan(B, H, T, dk, dv, dtype, chunk_size=0):
    p = kda_plan_t()
    st = load_library().kda_chunk_fwd_plan(B, H, T, dk, dv, dtype, chunk_size, ctypes.byref(p))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_plan")
    return dict(path=p.path, chunk_size=p.chunk_size, segments=p.segments, launches=p.launches,
                workspace=p.workspace, segment_tokens=p.segment_tokens)


def kda_chunk_fwd_workspace_size(B, H, T, dk, dv, dtype, chunk_size=0) -> int:
    return load_library().kda_chunk_fwd_workspace_size(B, H, T, dk, dv, dtype, chunk_size)


def kda_chunk_fwd(q, k, v, g, beta, h0, o, h_T, B, H, T, dk, dv, dtype, chunk_size, scale,
                  workspace, workspace_bytes, stream) -> int:
    """Returns the raw kda_status_t."""
    return load_library().kda_chunk_fwd(q, k, v, g, beta, h0, o, h_T, B, H, T, dk, dv, dtype, chunk_size,
                                        scale, workspace, workspace_bytes, stream)


def kda_chunk_fwd_ckpt(q, k, v, g, beta, h0, o, h_T, ckpt, ckpt_interval, B, H, T, dk, dv, dtype, chunk_size,
                       scale, workspace, workspace_bytes, stream) -> int:
    """kda_chunk_fwd that also writes state checkpoints every ckpt_interval tokens.
    Returns the raw kda_status_t."""
    return load_library().kda_chunk_fwd_ckpt(q, k, v, g, beta, h0, o, h_T, ckpt, ckpt_interval, B, H, T, dk, dv,
                                             dtype, chunk_size, scale, workspace, workspace_bytes, stream)


def kda_chunk_fwd_gated(q, k, v, z, A_log, g_min, beta, h0, o, h_T, B, H, T, dk, dv, dtype, chunk_size, scale,
                        workspace, workspace_bytes, stream) -> int:
    """kda_chunk_fwd with the Eq. 5 decay gate fused into the loads (takes the
    logits z and log-scales A_log instead of g).  Returns the raw kda_status_t."""
    return load_library().kda_chunk_fwd_gated(q, k, v, z, A_log, g_min, beta, h0, o, h_T, B, H, T, dk, dv, dtype,
                                              chunk_size, scale, workspace, workspace_bytes, stream)


def kda_chunk_fwd_outgate(q, k, v, g, beta, h0, gate, rms_weight, eps, y, h_T, B, H, T, dk, dv, dtype, chunk_size,
                          scale, workspace, workspace_bytes, stream) -> int:
    """kda_chunk_fwd with the Eq. 6 output edge fused into the epilogue: writes
    y = Sigmoid(gate) * RMSNorm_w(o) instead of o.  Returns the raw kda_status_t."""
    return load_library().kda_chunk_fwd_outgate(q, k, v, g, beta, h0, gate, rms_weight, eps, y, h_T, B, H, T, dk, dv,
                                                dtype, chunk_size, scale, workspace, workspace_bytes, stream)


def kda_chunk_transition(k, v, g, beta, St, M, B, H, T, dk, dv, dtype, stream) -> int:
    """Segment transition (S~, M) of every chain (Eq. 17).  Returns the raw kda_status_t."""
    return load_library().kda_chunk_transition(k, v, g, beta, St, M, B, H, T, dk, dv, dtype, stream)


def kda_output_gate(o, gate, rms_weight, eps, y, B, H, T, dv, dtype, stream) -> int:
    """Eq. 6 output edge: y = Sigmoid(gate) * RMSNorm(o).  Returns the raw kda_status_t."""
    return load_library().kda_output_gate(o, gate, rms_weight, eps, y, B, H, T, dv, dtype, stream)


def kda_kcp_compose(M, St, h0, S_in, R, B, H, dk, dv, stream) -> int:
    """Cross-device KCP prefix: S_in from the gathered (M_r, S~_r) of the R earlier segments."""
    return load_library().kda_kcp_compose(M, St, h0, S_in, R, B, H, dk, dv, stream)


def kda_spec_replay_verify(q, k, v, g, beta, S, o, n_replay, B, H, W, dk, dv, dtype, scale, stream) -> int:
    """Speculative-decode replay and verify over a W-token window.  Returns the raw kda_status_t."""
    return load_library().kda_spec_replay_verify(q, k, v, g, beta, S, o, n_replay, B, H, W, dk, dv, dtype, scale,
                                                 stream)


def kda_spec_replay_verify_fused(q, k, v, z, A_log, g_min, beta, S, gate, rms_weight, eps, y, n_replay, B, H, W, dk,
                                 dv, dtype, scale, stream) -> int:
    """The replay loop with the Eq. 5 gate (z, A_log) and the Eq. 6 edge (gate,
    rms_weight -> y) folded in.  Returns the raw kda_status_t."""
    return load_library().kda_spec_replay_verify_fused(q, k, v, z, A_log, g_min, beta, S, gate, rms_weight, eps, y,
                                                       n_replay, B, H, W, dk, dv, dtype, scale, stream)


def kda_chunk_fwd_noalloc(q, k, v, g, beta, h0, o, h_T, B, H, T, dk, dv, dtype, chunk_size, scale, stream) -> int:
    """kda_chunk_fwd with libkda's own fixed scratch array (no workspace argument).
    For callers that cannot allocate device memory.  Returns the raw kda_status_t."""
    return load_library().kda_chunk_fwd_noalloc(q, k, v, g, beta, h0, o, h_T, B, H, T, dk, dv, dtype, chunk_size,
                                                scale, stream)


def kda_noalloc_scratch_bytes() -> int:
    return load_library().kda_noalloc_scratch_bytes()


def kda_recurrent_step(q, k, v, g, beta, S, o, B, H, dk, dv, dtype, scale, stream) -> int:
    return load_library().kda_recurrent_step(q, k, v, g, beta, S, o, B, H, dk, dv, dtype, scale, stream)


def kda_block_map(length, ctx, free_pages, n_free, block_table, table_stride, page_size, cu, token_slots, pages_used, R,
                  rows, stream) -> int:
    """Block tables and token slots from request lengths.  Returns the raw kda_status_t."""
    return load_library().kda_block_map(length, ctx, free_pages, n_free, block_table, table_stride, page_size, cu,
                                        token_slots, pages_used, R, rows, stream)


def kda_short_conv(x, x_stride, w, bias, state, n_slots, slots, ctx, cu, y, y_stride, R, rows, C, K, head_dim, dtype,
                   flags, eps, stream) -> int:
    """Short causal convolution of packed prompts.  Returns the raw kda_status_t."""
    return load_library().kda_short_conv(x, x_stride, w, bias, state, n_slots, slots, ctx, cu, y, y_stride, R, rows, C, K,
                                         head_dim, dtype, flags, eps, stream)


def kda_short_conv_step(x, x_stride, w, bias, state, n_slots, slots, y, y_stride, R, C, K, head_dim, dtype, flags, eps,
                        stream) -> int:
    """Short causal convolution of single tokens.  Returns the raw kda_status_t."""
    return load_library().kda_short_conv_step(x, x_stride, w, bias, state, n_slots, slots, y, y_stride, R, C, K, head_dim,
                                              dtype, flags, eps, stream)


def kda_ssm_scan(x, x_stride, dt, dt_stride, A, B, b_stride, C, c_stride, D, dt_bias, softplus, state, n_slots, slots,
                 ctx, cu, block_table, table_stride, pages, n_pages, page_size, y, y_stride, R, rows, H, G, N, P, dtype,
                 workspace, workspace_bytes, stream) -> int:
    """Selective state space scan of packed prompts.  Returns the raw kda_status_t."""
    return load_library().kda_ssm_scan(x, x_stride, dt, dt_stride, A, B, b_stride, C, c_stride, D, dt_bias, softplus,
                                       state, n_slots, slots, ctx, cu, block_table, table_stride, pages, n_pages,
                                       page_size, y, y_stride, R, rows, H, G, N, P, dtype, workspace, workspace_bytes,
                                       stream)


def kda_ssm_scan_workspace_size(R, rows, H, G, N, P, dtype) -> int:
    return load_library().kda_ssm_scan_workspace_size(R, rows, H, G, N, P, dtype)


def kda_ssm_step(x, x_stride, dt, dt_stride, A, B, b_stride, C, c_stride, D, dt_bias, softplus, state, n_slots, slots, y,
                 y_stride, R, H, G, N, P, dtype, stream) -> int:
    """Selective state space step of single tokens.  Returns the raw kda_status_t."""
    return load_library().kda_ssm_step(x, x_stride, dt, dt_stride, A, B, b_stride, C, c_stride, D, dt_bias, softplus,
                                       state, n_slots, slots, y, y_stride, R, H, G, N, P, dtype, stream)


def kda_get_device_status(stream=None) -> int:
    return load_library().kda_get_device_status(stream)


def kda_debug_set_wait_limit(ns: int) -> int:
    return load_library().kda_debug_set_wait_limit(int(ns))


def kda_debug_inject_stall(on: bool) -> int:
    return load_library().kda_debug_inject_stall(1 if on else 0)


# ---- torch helpers ---------------------------------------------------------

def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError("q/k/v/g/beta must be bf16 or fp32, got %s" % t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkda takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libkda takes contiguous tensors")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def chunk_fwd(q, k, v, g, beta, h0=None, *, o=None, h_T=None, scale=0.0, chunk_size=0,
              output_final_state=True, workspace=None, stream=None, ckpt_interval=0, ckpt=None):
    """Prefill over [B, H, T, d] tensors (see kda_chunk_fwd in include/kda.h).

    Allocates o / h_T / workspace with torch when not given.  Returns (o, h_T),
    or (o, h_T, ckpt) when ckpt_interval > 0 (kda_chunk_fwd_ckpt: ckpt is
    [B, H, T // ckpt_interval, dk, dv] fp32, the state at every multiple of
    ckpt_interval tokens).
    """
    import torch
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_T is None and output_final_state:
        h_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    ws = kda_chunk_fwd_workspace_size(B, H, T, dk, dv, dt, chunk_size)
    if ws == (1 << 64) - 1:
        raise KdaError(2, "kda_chunk_fwd_workspace_size")
    if ws > 0 and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if ckpt_interval:
        if ckpt is None:
            ckpt = torch.empty(B, H, T // ckpt_interval, dk, dv, dtype=torch.float32, device=q.device)
        st = kda_chunk_fwd_ckpt(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(h_T),
                                _ptr(ckpt), ckpt_interval, B, H, T, dk, dv, dt, chunk_size, float(scale),
                                _ptr(workspace), wbytes, _stream(stream))
        if st != KDA_OK:
            raise KdaError(st, "kda_chunk_fwd_ckpt")
        return o, h_T, ckpt
    st = kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(h_T),
                       B, H, T, dk, dv, dt, chunk_size, float(scale), _ptr(workspace), wbytes, _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd")
    return o, h_T


def chunk_transition(k, v, g, beta, *, out=None, stream=None):
    """(S~, M) of every chain's segment: S~ [B, H, dk, dv] and M [B, H, dk, dk]
    fp32 (kda_chunk_transition).  `out`, if given, is one fp32 buffer of
    B*H*(dk*dk + dk*dv) elements that receives M then S~ (so a rank can
    publish both with one collective); the returned tensors are views of it."""
    import torch
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    n = B * H
    if out is None:
        out = torch.empty(n * (dk * dk + dk * dv), dtype=torch.float32, device=k.device)
    m = out[:n * dk * dk].view(B, H, dk, dk)
    st = out[n * dk * dk:n * (dk * dk + dk * dv)].view(B, H, dk, dv)
    code = kda_chunk_transition(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(st), _ptr(m), B, H, T, dk, dv,
                                _dtype_code(k), _stream(stream))
    if code != KDA_OK:
        raise KdaError(code, "kda_chunk_transition")
    return st, m


def chunk_fwd_outgate(q, k, v, g, beta, gate, rms_weight, h0=None, *, eps=1e-6, y=None, h_T=None, scale=0.0,
                      chunk_size=0, output_final_state=True, workspace=None, stream=None):
    """Prefill with the fused Eq. 6 output edge: gate [B, H, T, dv] (dtype of q),
    rms_weight [H, dv] fp32.  Allocates y / h_T / workspace when not given.
    Returns (y, h_T)."""
    import torch
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if y is None:
        y = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_T is None and output_final_state:
        h_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    ws = kda_chunk_fwd_workspace_size(B, H, T, dk, dv, dt, chunk_size)
    if ws == (1 << 64) - 1:
        raise KdaError(2, "kda_chunk_fwd_workspace_size")
    if ws > 0 and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = kda_chunk_fwd_outgate(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(gate), _ptr(rms_weight),
                               float(eps), _ptr(y), _ptr(h_T), B, H, T, dk, dv, dt, chunk_size, float(scale),
                               _ptr(workspace), wbytes, _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_outgate")
    return y, h_T


def chunk_fwd_gated(q, k, v, z, A_log, beta, h0=None, *, g_min=-5.0, o=None, h_T=None, scale=0.0, chunk_size=0,
                    output_final_state=True, workspace=None, stream=None):
    """Prefill with the fused Eq. 5 gate: z [B, H, T, dk] (dtype of q), A_log
    [H, dk] fp32.  Allocates o / h_T / workspace when not given.  Returns (o, h_T)."""
    import torch
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    if h_T is None and output_final_state:
        h_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    ws = kda_chunk_fwd_workspace_size(B, H, T, dk, dv, dt, chunk_size)
    if ws == (1 << 64) - 1:
        raise KdaError(2, "kda_chunk_fwd_workspace_size")
    if ws > 0 and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = kda_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), float(g_min), _ptr(beta), _ptr(h0),
                             _ptr(o), _ptr(h_T), B, H, T, dk, dv, dt, chunk_size, float(scale), _ptr(workspace),
                             wbytes, _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_gated")
    return o, h_T


def output_gate(o, gate, rms_weight, eps=1e-6, *, y=None, stream=None):
    """Eq. 6 output edge over [B, H, T, dv] tensors; rms_weight [H, dv] fp32.  Returns y."""
    import torch
    B, H, T, dv = o.shape
    if y is None:
        y = torch.empty_like(o)
    st = kda_output_gate(_ptr(o), _ptr(gate), _ptr(rms_weight), float(eps), _ptr(y), B, H, T, dv, _dtype_code(o),
                         _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_output_gate")
    return y


def spec_replay_verify(q, k, v, g, beta, S, n_replay, *, o=None, scale=0.0, stream=None):
    """Window of W tokens per sequence ([B, H, W, d]): replay the first
    n_replay[b] (accepted, committed to S in place), verify the rest (o).
    n_replay: [B] int32 CUDA tensor.  Returns o."""
    import torch
    B, H, W, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.zeros(B, H, W, dv, dtype=q.dtype, device=q.device)
    st = kda_spec_replay_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o), _ptr(n_replay),
                                B, H, W, dk, dv, _dtype_code(q), float(scale), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_spec_replay_verify")
    return o


def recurrent_step(q, k, v, g, beta, S, *, o=None, scale=0.0, stream=None):
    """One decode step over [B, H, d] tensors; S [B, H, dk, dv] fp32 updated in place.  Returns o."""
    import torch
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    st = kda_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o), B, H, dk, dv,
                            _dtype_code(q), float(scale), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_recurrent_step")
    return o


def spec_replay_verify_fused(q, k, v, z, A_log, beta, S, gate, rms_weight, n_replay, *, g_min=-5.0, eps=1e-6, y=None,
                             scale=0.0, stream=None):
    """spec_replay_verify with the Eq. 5 gate on the inputs (z [B, H, W, dk],
    A_log [H, dk] fp32) and the Eq. 6 edge on the verified outputs (gate
    [B, H, W, dv], rms_weight [H, dv] fp32).  Returns y (zeros for replayed tokens)."""
    import torch
    B, H, W, dk = q.shape
    dv = v.shape[-1]
    if y is None:
        y = torch.zeros(B, H, W, dv, dtype=q.dtype, device=q.device)
    st = kda_spec_replay_verify_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), float(g_min), _ptr(beta),
                                      _ptr(S), _ptr(gate), _ptr(rms_weight), float(eps), _ptr(y), _ptr(n_replay), B, H,
                                      W, dk, dv, _dtype_code(q), float(scale), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_spec_replay_verify_fused")
    return y


# ---- packed requests (kda_block_map, kda_short_conv*, kda_ssm_*) ---------------
#
# Token-major arguments may be row-strided views (the columns of a wider
# projection, or of the convolution's output): only the elements of a row have
# to be dense.  Integer arguments (cu, ctx, slots, lengths, tables) are int32
# tensors on the same device and are not read on the host.

# The checks below run on every call of a few microseconds, so each helper tests
# what a right call has in one expression of attribute reads, and only then, to
# name what is wrong, goes through the checks that raise.

def _on(x, *tensors):
    """Every tensor on x's CUDA device."""
    d = x.get_device()
    if d < 0:
        raise ValueError("libkda takes CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors of a call must be on one CUDA device (got %s and %s)" % (x.device, t.device))


def _typed(dtype, names, *tensors):
    for name, t in zip(names.split(), tensors):
        if t is not None and t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, str(dtype).replace("torch.", ""), t.dtype))


def _shaped(name, t, shape):
    if t is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _dense(names, *tensors):
    for name, t in zip(names.split(), tensors):
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


_INT_MAX = (1 << 31) - 1


def _too_large():
    raise ValueError("sizes must be below 2^31")  # (ctypes would cut them to 32 bits without a word)


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(name, t, lead, width):
    """Row stride of token-major `t`: `lead` leading dimensions of rows over dense rows of `width` elements."""
    if t.is_contiguous():
        return width
    shape, stride = t.shape, t.stride()
    want = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and stride[i] != want:
            raise ValueError("%s: the elements of a row must be dense" % name)
        want *= shape[i]
    if lead == 1:
        return stride[0] if shape[0] > 1 else want
    n0, n1 = shape[0], shape[1]
    if n0 > 1 and n1 > 1 and stride[0] != n1 * stride[1]:
        raise ValueError("%s: rows must have one stride" % name)
    return want if n0 * n1 <= 1 else stride[1] if n1 > 1 else stride[0]


_torch = _device = _raw_stream = None


def _init():
    global _torch, _device, _raw_stream
    import torch
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
    _torch = torch
    return torch


def _launch(fn, what, i, stream, args):
    """Call `fn` of the library on the stream (its last argument; None: the current one) with device i current."""
    stream = _raw_stream(i) if stream is None else getattr(stream, "cuda_stream", stream)
    if i == _device():
        code = fn(*args, stream)
    else:
        with _torch.cuda.device(i):
            code = fn(*args, stream)
    if code != KDA_OK:
        raise KdaError(code, what)


def _good_slots(t, R, d, i32):
    """Whether t is a vector of R int32 on device d (or None)."""
    return t is None or (t.dtype is i32 and t.shape == (R,) and t.get_device() == d and t.is_contiguous())


def _good_vector(t, n, d, dtype):
    """The same for a parameter vector."""
    return t is None or (t.dtype is dtype and t.shape == (n,) and t.get_device() == d and t.is_contiguous())


def _pool_entries(t, d, dtype, *entry):
    """Entries of a pool [n, *entry] on device d (0 without one), or -1 if t is not one."""
    if t is None:
        return 0
    shape = t.shape
    good = (len(shape) == len(entry) + 1 and shape == (shape[0], *entry) and t.dtype is dtype and t.get_device() == d and
            t.is_contiguous())
    return shape[0] if good else -1


def _bad_requests(slots, ctx, cu, R):
    i32 = _torch.int32
    _typed(i32, "slots ctx cu", slots, ctx, cu)
    _dense("slots ctx cu", slots, ctx, cu)
    _shaped("slots", slots, (R,))
    _shaped("ctx", ctx, (R,))
    raise ValueError("slots and ctx must be [R], cu [R + 1] int32 on the device of the call")


def _requests(x, lead, slots, ctx, cu, d):
    """(R, rows) of a packed call, after the checks of its integer arguments."""
    i32 = _torch.int32
    shape = x.shape
    if lead == 2:
        if cu is not None:
            raise ValueError("cu goes with [rows, ...] tensors")
        R = shape[0]
        rows = R * shape[1]
    else:
        rows = shape[0]
        R = 1 if cu is None else cu.numel() - 1
        if R < 0:
            raise ValueError("cu must hold R + 1 offsets")
    if not (_good_slots(slots, R, d, i32) and _good_slots(ctx, R, d, i32) and _good_slots(cu, R + 1, d, i32)):
        _on(x, slots, ctx, cu)
        _bad_requests(slots, ctx, cu, R)
    return R, rows


def block_map(lens, ctx, free_pages, block_table, page_size, rows, *, cu=None, token_slots=None, pages_used=None,
              stream=None):
    """Sequence offsets, block table and token slots from request lengths, on the
    device (kda_block_map).  lens, ctx (or None): [R] int32; free_pages: [n]
    int32; block_table: [R, blocks] int32, updated in place; rows: the most new
    tokens that the call may hold.  Returns (cu [R + 1] int32, token_slots [rows]
    int64, pages_used [1] int32)."""
    torch = _torch or _init()
    i32, R, n_free, d = torch.int32, lens.numel(), free_pages.numel(), lens.get_device()
    shape = block_table.shape
    if not (d >= 0 and _good_slots(lens, R, d, i32) and _good_slots(ctx, R, d, i32) and
            _good_slots(free_pages, n_free, d, i32) and block_table.dtype is i32 and len(shape) == 2 and shape[0] == R and
            block_table.get_device() == d and block_table.is_contiguous()):
        _typed(i32, "lens ctx free_pages block_table", lens, ctx, free_pages, block_table)
        _dense("lens ctx free_pages block_table", lens, ctx, free_pages, block_table)
        _on(lens, ctx, free_pages, block_table)
        _shaped("ctx", ctx, (R,))
        raise ValueError("lens and ctx must be [R], free_pages [n], block_table [R, blocks]")
    if (R | rows | n_free | shape[1]) > _INT_MAX or page_size > _INT_MAX:
        _too_large()
    given = cu is not None or token_slots is not None or pages_used is not None
    if cu is None:
        cu = _fresh(stream, d, lens.new_empty, R + 1)
    if token_slots is None:
        token_slots = _fresh(stream, d, lens.new_empty, rows, dtype=torch.int64)
    if pages_used is None:
        pages_used = _fresh(stream, d, lens.new_empty, 1)
    if given:
        _shaped("cu", cu, (R + 1,))
        _shaped("token_slots", token_slots, (rows,))
        _shaped("pages_used", pages_used, (1,))
        _typed(i32, "cu pages_used", cu, pages_used)
        _typed(torch.int64, "token_slots", token_slots)
        _dense("cu token_slots pages_used", cu, token_slots, pages_used)
        _on(lens, cu, token_slots, pages_used)
    _launch(load_library().kda_block_map, "kda_block_map", d, stream,
            (lens.data_ptr(), _at(ctx), free_pages.data_ptr(), n_free, block_table.data_ptr(), shape[1], page_size,
             cu.data_ptr(), token_slots.data_ptr(), pages_used.data_ptr(), R, rows))
    return cu, token_slots, pages_used


def _on_stream(stream, d):
    """A context whose allocations belong to the stream that will use them (`stream`: a torch stream or, of device d,
    a handle)."""
    return _torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else _torch.cuda.ExternalStream(stream, device=d))


def _fresh(stream, d, make, *args, **kw):
    """make(*args, **kw): a tensor on device d that belongs to the call's stream (None: the current one)."""
    if stream is None:
        return make(*args, **kw)
    with _on_stream(stream, d):
        return make(*args, **kw)


def _output(x, y, lead, width, stream):
    """(y, its row stride) for a token-major output like x."""
    if y is None:
        return _fresh(stream, x.get_device(), _torch.empty_like, x, memory_format=_torch.contiguous_format), width
    _typed(x.dtype, "y", y)
    _shaped("y", y, x.shape)
    _on(x, y)
    return y, _rows("y", y, lead, width)


def _conv_weights(x, w, bias, state, C, d):
    """(taps, entries of the pool), after the checks of weights and pool."""
    t, shape = x.dtype, w.shape
    K = shape[1] if len(shape) == 2 else 0
    n = _pool_entries(state, d, t, K - 1, C)
    if not (d >= 0 and K > 0 and n >= 0 and w.dtype is t and shape[0] == C and w.get_device() == d and w.is_contiguous() and
            _good_vector(bias, C, d, t)):
        _typed(t, "w bias state", w, bias, state)
        _dense("w bias state", w, bias, state)
        _on(x, w, bias, state)
        raise ValueError("w must be [C, K], bias [C], state [n_slots, K - 1, C]")
    return K, n


def short_conv(x, w, bias=None, *, state=None, slots=None, ctx=None, cu=None, silu=True, head_dim=0, l2norm=False,
               head_major=False, eps=1e-6, y=None, stream=None):
    """Short causal convolution of prompts with Swish and the L2 norm of each
    head (kda_short_conv).  x: [rows, C] with offsets cu [R + 1] int32 (None: one
    sequence), or [B, T, C]; w: [C, K]; bias: [C]; state: pool [n_slots, K - 1, C],
    updated in place; slots, ctx: [R] int32.  Returns y like x, or with
    head_major [B, C // head_dim, T, head_dim], which chunk_fwd reads."""
    torch = _torch or _init()
    code = _dtype_code(x)
    lead = x.dim() - 1
    if lead not in (1, 2):
        raise ValueError("x must be [rows, C] or [B, T, C]")
    C, d = x.shape[lead], x.get_device()
    K, n_slots = _conv_weights(x, w, bias, state, C, d)
    R, rows = _requests(x, lead, slots, ctx, cu, d)
    if (R | rows | C | n_slots) > _INT_MAX or head_dim > _INT_MAX:
        _too_large()
    if not head_major:
        y, ys = _output(x, y, lead, C, stream)
    else:
        if head_dim <= 0 or C % head_dim:
            raise ValueError("head_major needs a head_dim that divides C")
        shape, ys = (R, C // head_dim, rows // max(R, 1), head_dim), C
        if y is None:
            y = _fresh(stream, d, torch.empty, shape, dtype=x.dtype, device=x.device)
        else:
            _typed(x.dtype, "y", y)
            _shaped("y", y, shape)
            _dense("y", y)
            _on(x, y)
    flags = (KDA_CONV_SILU if silu else 0) | (KDA_CONV_L2NORM if l2norm else 0) | (KDA_CONV_HEAD_MAJOR if head_major else 0)
    _launch(load_library().kda_short_conv, "kda_short_conv", d, stream,
            (x.data_ptr(), _rows("x", x, lead, C), w.data_ptr(), _at(bias), _at(state), n_slots,
             _at(slots), _at(ctx), _at(cu), y.data_ptr(), ys, R, rows, C, K, head_dim, code, flags, eps))
    return y


def short_conv_step(x, w, state, bias=None, *, slots=None, silu=True, head_dim=0, l2norm=False, eps=1e-6, y=None,
                    stream=None):
    """short_conv for one new token of each of R sequences: x [R, C]; state: pool
    [n_slots, K - 1, C], shifted in place.  Returns y [R, C]."""
    torch = _torch or _init()
    code = _dtype_code(x)
    if x.dim() != 2:
        raise ValueError("x must be [R, C]")
    R, C = x.shape
    d = x.get_device()
    K, n_slots = _conv_weights(x, w, bias, state, C, d)
    if not _good_slots(slots, R, d, torch.int32):
        _on(x, slots)
        _bad_requests(slots, None, None, R)
    if (R | C | n_slots) > _INT_MAX or head_dim > _INT_MAX:
        _too_large()
    y, ys = _output(x, y, 1, C, stream)
    flags = (KDA_CONV_SILU if silu else 0) | (KDA_CONV_L2NORM if l2norm else 0)
    _launch(load_library().kda_short_conv_step, "kda_short_conv_step", d, stream,
            (x.data_ptr(), _rows("x", x, 1, C), w.data_ptr(), _at(bias), _at(state), n_slots, _at(slots),
             y.data_ptr(), ys, R, C, K, head_dim, code, flags, eps))
    return y


def _ssm_args(x, dt, A, B, C, D, dt_bias, state, lead, d):
    """(H, G, N, P, entries of the pool, row strides) after the checks of shapes, types and layouts."""
    f32, t = _torch.float32, x.dtype
    shape, bshape = x.shape, B.shape
    H, P, G, N = shape[lead], shape[lead + 1], bshape[lead], bshape[lead + 1]
    rows = shape[:lead]
    n = _pool_entries(state, d, f32, H, N, P)
    if not (d >= 0 and n >= 0 and dt.dtype is t and B.dtype is t and C.dtype is t and dt.shape == (*rows, H) and
            bshape == (*rows, G, N) and C.shape == bshape and dt.get_device() == d and B.get_device() == d and
            C.get_device() == d and _good_vector(A, H, d, f32) and _good_vector(D, H, d, f32) and
            _good_vector(dt_bias, H, d, f32)):
        _typed(t, "dt B C", dt, B, C)
        _typed(f32, "A D dt_bias state", A, D, dt_bias, state)
        _dense("A D dt_bias state", A, D, dt_bias, state)
        _on(x, dt, A, B, C, D, dt_bias, state)
        _shaped("dt", dt, shape[:-1])
        _shaped("B", B, shape[:-2] + bshape[-2:])
        _shaped("C", C, bshape)
        raise ValueError("A, D and dt_bias must be [H], state [n_slots, H, N, P]")
    return (H, G, N, P, n, _rows("x", x, lead, H * P), _rows("dt", dt, lead, H), _rows("B", B, lead, G * N),
            _rows("C", C, lead, G * N))


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, *, softplus=True, state=None, slots=None, ctx=None, cu=None,
             block_table=None, pages=None, page_size=0, y=None, workspace=None, stream=None):
    """Selective state space scan of prompts (kda_ssm_scan): S_t = exp(d A) S + d B x^T,
    y = S^T C + D x with d = softplus(dt + dt_bias).  x: [rows, H, P] with offsets
    cu [R + 1] int32 (None: one sequence), or [B, T, H, P]; dt [.., H]; B, C
    [.., G, N]; A, D, dt_bias [H] fp32; state: pool [n_slots, H, N, P] fp32,
    updated in place; slots, ctx [R] int32.  page_size > 0: the state at every
    multiple of it goes to pages [n_pages, H, N, P] through block_table
    [R, blocks] int32.  Returns y like x."""
    torch = _torch or _init()
    code = _dtype_code(x)
    lead = x.dim() - 2
    if lead not in (1, 2) or B.dim() != lead + 2:
        raise ValueError("x must be [rows, H, P] or [B, T, H, P], B and C [.., G, N]")
    d = x.get_device()
    H, G, N, P, n_slots, xs, ds, bs, cs = _ssm_args(x, dt, A, B, C, D, dt_bias, state, lead, d)
    R, rows = _requests(x, lead, slots, ctx, cu, d)
    width = n_pages = 0
    if page_size:
        if block_table is None or pages is None:
            raise ValueError("page_size needs block_table and pages")
        _typed(torch.int32, "block_table", block_table)
        _typed(torch.float32, "pages", pages)
        _dense("block_table pages", block_table, pages)
        _on(x, block_table, pages)
        if block_table.dim() != 2 or block_table.size(0) != R:
            raise ValueError("block_table must be [R, blocks]")
        n_pages, width = pages.size(0), block_table.size(1)
        _shaped("pages", pages, (n_pages, H, N, P))
    else:
        block_table = pages = None
    if (R | rows | n_slots | n_pages | width | H) > _INT_MAX or page_size > _INT_MAX:
        _too_large()
    y, ys = _output(x, y, lead, H * P, stream)
    lib = load_library()
    ws = lib.kda_ssm_scan_workspace_size(R, rows, H, G, N, P, code)
    if ws == (1 << 64) - 1:
        raise KdaError(2, "kda_ssm_scan_workspace_size")
    wbytes = 0
    if ws > 0 and workspace is None:
        # (it is given back when this returns, maybe before the stream is done with it)
        workspace = _fresh(stream, d, torch.empty, ws, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        _dense("workspace", workspace)
        _on(x, workspace)
        wbytes = workspace.numel() * workspace.element_size()
    _launch(lib.kda_ssm_scan, "kda_ssm_scan", d, stream,
            (x.data_ptr(), xs, dt.data_ptr(), ds, A.data_ptr(), B.data_ptr(), bs, C.data_ptr(), cs, _at(D), _at(dt_bias),
             1 if softplus else 0, _at(state), n_slots, _at(slots), _at(ctx), _at(cu),
             _at(block_table), width, _at(pages), n_pages, page_size, y.data_ptr(), ys, R, rows, H, G, N, P, code,
             _at(workspace), wbytes))
    return y


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, softplus=True, slots=None, y=None, stream=None):
    """ssm_scan for one new token of each of R sequences: x [R, H, P], dt [R, H],
    B, C [R, G, N]; state: pool [n_slots, H, N, P] fp32, updated in place.  Returns y [R, H, P]."""
    torch = _torch or _init()
    code = _dtype_code(x)
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [R, H, P], B and C [R, G, N]")
    R, d = x.shape[0], x.get_device()
    H, G, N, P, n_slots, xs, ds, bs, cs = _ssm_args(x, dt, A, B, C, D, dt_bias, state, 1, d)
    if not _good_slots(slots, R, d, torch.int32):
        _on(x, slots)
        _bad_requests(slots, None, None, R)
    if (R | n_slots | H) > _INT_MAX:
        _too_large()
    y, ys = _output(x, y, 1, H * P, stream)
    _launch(load_library().kda_ssm_step, "kda_ssm_step", d, stream,
            (x.data_ptr(), xs, dt.data_ptr(), ds, A.data_ptr(), B.data_ptr(), bs, C.data_ptr(), cs, _at(D), _at(dt_bias),
             1 if softplus else 0, _at(state), n_slots, _at(slots), y.data_ptr(), ys, R, H, G, N, P, code))
    return y
