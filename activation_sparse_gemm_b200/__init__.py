"""RT-Lynx activation-sparse linear layer for NVIDIA B200 (sm_100a).

Python binding of ``librtlynx.so`` (argument marshalling only; every step of
the layer runs in the library's CUDA kernels).  The C ABI is declared in
``include/rtlynx.h``; the functions below carry the same names and take
device pointers as ints, or torch tensors (their ``data_ptr()``), and a CUDA
stream handle (int) or a ``torch.cuda.Stream``.

    Y = S(X) W^T + X (L_A L_B)^T        mode = MODE_SPARSE
    Y = X W^T                           mode = MODE_DENSE_SKIP
    H = GELU(up(X)), Y = down(H)        rtlynx_mlp_block (two such layers)
    Y = down(act(gate(X)) * up(X))      rtlynx_gated_mlp_block
    R(p) x,  R(p) (w x / rms(x))        rtlynx_rope, rtlynx_qk_norm_rope (query and key heads)

(RT-Lynx summary page, four-step pipeline paragraph, steps 1-3.)

The library is built in-tree with ``python -m activation_sparse_gemm_b200.build``.
There is no fallback: if the library is missing every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
import sysconfig

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "librtlynx.so")

MODE_SPARSE = 0
MODE_DENSE_SKIP = 1

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_OOM = 4
ERR_DEVICE_TIMEOUT = 5

ACT_SILU, ACT_GELU = 0, 1                     # rtlynx_act
BF16, FP16, FP32 = 0, 1, 2                    # rtlynx_dtype
ROPE_INTERLEAVED, ROPE_HALF = 0, 1            # rtlynx_rope_pairing
POS_INT32, POS_INT64, POS_FP32 = 0, 1, 2      # rtlynx_pos_type
MAX_AXES = 4

# Every symbol include/rtlynx.h declares.
ABI_SYMBOLS = (
    "rtlynx_linear", "rtlynx_workspace_size", "rtlynx_linear_ws", "rtlynx_linear_ws_events",
    "rtlynx_workspace_layout",
    "rtlynx_sparsify_debug", "rtlynx_linear_host", "rtlynx_mlp_block", "rtlynx_linear_noalloc",
    "rtlynx_kernel_launches", "rtlynx_schedule_info",
    "rtlynx_quantize_weight_fp8", "rtlynx_linear_fp8", "rtlynx_linear_fp8_events", "rtlynx_sparsify_fp8_debug",
    "rtlynx_gated_mlp_block", "rtlynx_gated_mlp_block_workspace_size", "rtlynx_gated_mlp_backward_workspace_size", "rtlynx_gated_mlp_backward",
    "rtlynx_rope", "rtlynx_rope_backward", "rtlynx_qk_norm_rope", "rtlynx_qk_norm_rope_workspace_size",
    "rtlynx_qk_norm_rope_backward",
    "rtlynx_wait_selftest", "rtlynx_stream_status", "rtlynx_status_string", "rtlynx_release",
)

NOALLOC_MAX_BYTES = 32 << 20

_lib = None


class RtlynxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {rtlynx_status_string(status)} (status {status})")


class WsLayout(ctypes.Structure):
    _fields_ = [("M_pad", ctypes.c_int64), ("Kc_pad", ctypes.c_int64), ("k_chunks", ctypes.c_int64),
                ("R_pad", ctypes.c_int64), ("vals", ctypes.c_size_t), ("meta", ctypes.c_size_t),
                ("s", ctypes.c_size_t), ("T", ctypes.c_size_t), ("total", ctypes.c_size_t)]


class Schedule(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "prologue_ctas", "prologue_tiles", "prologue_max_segs", "row_blocks", "k_tiles_per_block",
        "gemm_pairs", "gemm_tiles", "tail_full", "tail_split", "tail_units", "k_stages", "lora_stages",
        "small_path")]


class HeadsView(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("heads", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("axis_dim", ctypes.c_int32 * MAX_AXES), ("pairing", ctypes.c_int32),
                ("pos_type", ctypes.c_int32), ("theta", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


def torch_lib_path(torch_version: str) -> str:
    """The host code of the torch-level calls, one file for each torch and Python that it was compiled against."""
    return os.path.join(_PKG, "_lib", f"rtlynx_torch-{torch_version}-{sysconfig.get_config_var('SOABI')}.so")


def lib() -> ctypes.CDLL:
    """Loads librtlynx.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m activation_sparse_gemm_b200.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.rtlynx_linear.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i, p]
        L.rtlynx_linear.restype = i
        L.rtlynx_workspace_size.argtypes = [i64, i64, i64, i64, i]
        L.rtlynx_workspace_size.restype = ctypes.c_size_t
        L.rtlynx_linear_ws.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i, p, ctypes.c_size_t, p]
        L.rtlynx_linear_ws.restype = i
        L.rtlynx_linear_ws_events.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i, p, ctypes.c_size_t, p, p, p,
                                               p]
        L.rtlynx_linear_ws_events.restype = i
        L.rtlynx_workspace_layout.argtypes = [i64, i64, i64, i64, ctypes.POINTER(WsLayout)]
        L.rtlynx_workspace_layout.restype = i
        L.rtlynx_sparsify_debug.argtypes = [p, p, i64, i64, i64, p, p, p, p, p]
        L.rtlynx_sparsify_debug.restype = i
        L.rtlynx_linear_host.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i, p, p, p]
        L.rtlynx_linear_host.restype = i
        L.rtlynx_mlp_block.argtypes = [p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, i, i, p]
        L.rtlynx_mlp_block.restype = i
        L.rtlynx_linear_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i, p, p]
        L.rtlynx_linear_noalloc.restype = i
        L.rtlynx_quantize_weight_fp8.argtypes = [p, p, p, p, p, i64, i64, i64, p]
        L.rtlynx_quantize_weight_fp8.restype = i
        L.rtlynx_linear_fp8.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, p]
        L.rtlynx_linear_fp8.restype = i
        L.rtlynx_linear_fp8_events.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, p, p, p, p]
        L.rtlynx_linear_fp8_events.restype = i
        L.rtlynx_sparsify_fp8_debug.argtypes = [p, i64, i64, p, p, p, p]
        L.rtlynx_sparsify_fp8_debug.restype = i
        L.rtlynx_kernel_launches.argtypes = [i64, i64, i64, i64, i]
        L.rtlynx_kernel_launches.restype = i
        L.rtlynx_schedule_info.argtypes = [i64, i64, i64, i64, i, ctypes.POINTER(Schedule)]
        L.rtlynx_schedule_info.restype = i
        L.rtlynx_gated_mlp_block.argtypes = [p] * 11 + [i64, i64, i64, i64, i, i, p, ctypes.c_size_t, p]
        L.rtlynx_gated_mlp_block.restype = i
        L.rtlynx_gated_mlp_block_workspace_size.argtypes = [i64, i64, i64, i]
        L.rtlynx_gated_mlp_block_workspace_size.restype = ctypes.c_size_t
        L.rtlynx_gated_mlp_backward_workspace_size.argtypes = [i64, i64, i64]
        L.rtlynx_gated_mlp_backward_workspace_size.restype = ctypes.c_size_t
        L.rtlynx_gated_mlp_backward.argtypes = [p] * 13 + [i64, i64, i64, i, p, ctypes.c_size_t, p]
        L.rtlynx_gated_mlp_backward.restype = i
        hv, spec, f = ctypes.POINTER(HeadsView), ctypes.POINTER(RopeSpec), ctypes.c_float
        L.rtlynx_rope.argtypes = [hv, hv, hv, hv, i64, i64, i64, i, spec, p, i64, i64, i64, p]
        L.rtlynx_rope.restype = i
        L.rtlynx_rope_backward.argtypes = L.rtlynx_rope.argtypes
        L.rtlynx_rope_backward.restype = i
        L.rtlynx_qk_norm_rope.argtypes = [hv, hv, p, p, hv, hv, i64, i64, i64, i, f, spec, p, i64, i64, i64, p]
        L.rtlynx_qk_norm_rope.restype = i
        L.rtlynx_qk_norm_rope_workspace_size.argtypes = [i64]
        L.rtlynx_qk_norm_rope_workspace_size.restype = ctypes.c_size_t
        L.rtlynx_qk_norm_rope_backward.argtypes = [hv, hv, hv, hv, p, p, hv, hv, p, p, i64, i64, i64, i, f, spec, p,
                                                   i64, i64, i64, p, ctypes.c_size_t, p]
        L.rtlynx_qk_norm_rope_backward.restype = i
        L.rtlynx_wait_selftest.argtypes = [i64, p]
        L.rtlynx_wait_selftest.restype = i
        L.rtlynx_stream_status.argtypes = [p]
        L.rtlynx_stream_status.restype = i
        L.rtlynx_status_string.argtypes = [i]
        L.rtlynx_status_string.restype = ctypes.c_char_p
        L.rtlynx_release.argtypes = []
        L.rtlynx_release.restype = None
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(s):
    if s is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(status: int, what: str) -> int:
    if status != OK:
        raise RtlynxError(status, what)
    return status


# ------------------------------------------------------------------ the ABI, one to one
def rtlynx_linear(X, W, L_A, L_B, Y, M, D_in, D_out, R, mode, stream=None) -> int:
    return _check(lib().rtlynx_linear(_ptr(X), _ptr(W), _ptr(L_A), _ptr(L_B), _ptr(Y), M, D_in, D_out, R,
                                      mode, _stream(stream)), "rtlynx_linear")


def rtlynx_mlp_block(X, W_up, LA_up, LB_up, W_down, LA_down, LB_down, H, Y, M, D, D_ff, R, mode_up=MODE_SPARSE,
                     mode_down=MODE_SPARSE, stream=None) -> int:
    """H = GELU(layer_up(X)) [M, D_ff], Y = layer_down(H) [M, D]; see include/rtlynx.h."""
    return _check(lib().rtlynx_mlp_block(_ptr(X), _ptr(W_up), _ptr(LA_up), _ptr(LB_up), _ptr(W_down), _ptr(LA_down),
                                         _ptr(LB_down), _ptr(H), _ptr(Y), M, D, D_ff, R, mode_up, mode_down,
                                         _stream(stream)), "rtlynx_mlp_block")


def rtlynx_workspace_size(M, D_in, D_out, R, mode) -> int:
    return int(lib().rtlynx_workspace_size(M, D_in, D_out, R, mode))


def rtlynx_linear_ws(X, W, L_A, L_B, Y, M, D_in, D_out, R, mode, workspace, ws_bytes, stream=None) -> int:
    return _check(lib().rtlynx_linear_ws(_ptr(X), _ptr(W), _ptr(L_A), _ptr(L_B), _ptr(Y), M, D_in, D_out, R,
                                         mode, _ptr(workspace), ws_bytes, _stream(stream)), "rtlynx_linear_ws")


def _event(ev):
    if ev is None or isinstance(ev, int):
        return ev
    return int(ev.cuda_event)


def rtlynx_linear_ws_events(X, W, L_A, L_B, Y, M, D_in, D_out, R, mode, workspace, ws_bytes, ev_start, ev_mid,
                            ev_end, stream=None) -> int:
    """Events may be raw cudaEvent_t ints or torch.cuda.Event objects that were recorded once already."""
    return _check(lib().rtlynx_linear_ws_events(_ptr(X), _ptr(W), _ptr(L_A), _ptr(L_B), _ptr(Y), M, D_in, D_out,
                                                R, mode, _ptr(workspace), ws_bytes, _event(ev_start),
                                                _event(ev_mid), _event(ev_end), _stream(stream)),
                  "rtlynx_linear_ws_events")


def rtlynx_workspace_layout(M, D_in, D_out, R) -> WsLayout:
    out = WsLayout()
    _check(lib().rtlynx_workspace_layout(M, D_in, D_out, R, ctypes.byref(out)), "rtlynx_workspace_layout")
    return out


def rtlynx_sparsify_debug(X, L_B, M, D_in, R, vals, meta, s, T, stream=None) -> int:
    return _check(lib().rtlynx_sparsify_debug(_ptr(X), _ptr(L_B), M, D_in, R, _ptr(vals), _ptr(meta), _ptr(s),
                                              _ptr(T), _stream(stream)), "rtlynx_sparsify_debug")


def rtlynx_linear_host(X_host, W, L_A, L_B, Y_host, M, D_in, D_out, R, mode, X_dev, Y_dev, stream=None) -> int:
    return _check(lib().rtlynx_linear_host(_ptr(X_host), _ptr(W), _ptr(L_A), _ptr(L_B), _ptr(Y_host), M, D_in,
                                           D_out, R, mode, _ptr(X_dev), _ptr(Y_dev), _stream(stream)),
                  "rtlynx_linear_host")


def rtlynx_linear_noalloc(X, W, L_A, L_B, Y, M, D_in, D_out, R, mode, dev_status=None, stream=None) -> int:
    """rtlynx_linear without any device allocation: for callers that cannot call
    cudaMalloc (their memory belongs to another pool, or the call sits on a path
    that must not synchronize).  The workspace is a static device array of
    NOALLOC_MAX_BYTES shared by all calls on a device; calls that overlap on the
    GPU race on it.  dev_status: optional device int32 that receives the
    device-side timeout code; without it a timeout goes to the library's error
    word, which rtlynx_stream_status reports."""
    return _check(lib().rtlynx_linear_noalloc(_ptr(X), _ptr(W), _ptr(L_A), _ptr(L_B), _ptr(Y), M, D_in, D_out, R,
                                              mode, _ptr(dev_status), _stream(stream)), "rtlynx_linear_noalloc")


def rtlynx_quantize_weight_fp8(W, L_A, W8, qw, L_A8, D_out, D_in, R, stream=None) -> int:
    return _check(lib().rtlynx_quantize_weight_fp8(_ptr(W), _ptr(L_A), _ptr(W8), _ptr(qw), _ptr(L_A8), D_out, D_in,
                                                   R, _stream(stream)), "rtlynx_quantize_weight_fp8")


def rtlynx_linear_fp8(X, W8, qw, L_A8, L_B, Y, M, D_in, D_out, R, stream=None) -> int:
    return _check(lib().rtlynx_linear_fp8(_ptr(X), _ptr(W8), _ptr(qw), _ptr(L_A8), _ptr(L_B), _ptr(Y), M, D_in,
                                          D_out, R, _stream(stream)), "rtlynx_linear_fp8")


def rtlynx_linear_fp8_events(X, W8, qw, L_A8, L_B, Y, M, D_in, D_out, R, ev_start, ev_mid, ev_end,
                             stream=None) -> int:
    """Events are torch.cuda.Event objects (or raw handles), any may be None."""
    def h(e):
        return None if e is None else (e if isinstance(e, int) else int(e.cuda_event))
    return _check(lib().rtlynx_linear_fp8_events(_ptr(X), _ptr(W8), _ptr(qw), _ptr(L_A8), _ptr(L_B), _ptr(Y), M,
                                                 D_in, D_out, R, h(ev_start), h(ev_mid), h(ev_end),
                                                 _stream(stream)), "rtlynx_linear_fp8_events")


def rtlynx_sparsify_fp8_debug(X, M, D_in, codes, meta, qx, stream=None) -> int:
    return _check(lib().rtlynx_sparsify_fp8_debug(_ptr(X), M, D_in, _ptr(codes), _ptr(meta), _ptr(qx),
                                                  _stream(stream)), "rtlynx_sparsify_fp8_debug")


def rtlynx_gated_mlp_block_workspace_size(M, D, D_ff, mode_down=MODE_DENSE_SKIP) -> int:
    return int(lib().rtlynx_gated_mlp_block_workspace_size(M, D, D_ff, mode_down))


def rtlynx_gated_mlp_block(X, W_gate, W_up, W_down, LA_down, LB_down, G, U, low, H, Y, M, D, D_ff, R, act, mode_down,
                           workspace, ws_bytes, stream=None) -> int:
    """H = act(X W_gate^T) * (X W_up^T) [M, D_ff], Y = layer_down(H) [M, D]; see include/rtlynx.h."""
    return _check(lib().rtlynx_gated_mlp_block(_ptr(X), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(LA_down),
                                               _ptr(LB_down), _ptr(G), _ptr(U), _ptr(low), _ptr(H), _ptr(Y), M, D, D_ff,
                                               R, act, mode_down, _ptr(workspace), ws_bytes, _stream(stream)),
                  "rtlynx_gated_mlp_block")


def rtlynx_gated_mlp_backward_workspace_size(M, D, D_ff) -> int:
    return int(lib().rtlynx_gated_mlp_backward_workspace_size(M, D, D_ff))


def rtlynx_gated_mlp_backward(dY, X, W_gate, W_up, W_down, G, U, low, H, dX, dW_gate, dW_up, dW_down, M, D, D_ff, act,
                              workspace, ws_bytes, stream=None) -> int:
    return _check(lib().rtlynx_gated_mlp_backward(_ptr(dY), _ptr(X), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(G),
                                                  _ptr(U), _ptr(low), _ptr(H), _ptr(dX), _ptr(dW_gate), _ptr(dW_up),
                                                  _ptr(dW_down), M, D, D_ff, act, _ptr(workspace), ws_bytes,
                                                  _stream(stream)), "rtlynx_gated_mlp_backward")


def rtlynx_rope(q, k, q_out, k_out, B, S, D_head, dtype, spec, positions, pos_strides, stream=None) -> int:
    """q, k, q_out, k_out: HeadsView (k and k_out may be None); spec: RopeSpec; pos_strides: (batch, token, axis)."""
    return _check(lib().rtlynx_rope(q, k, q_out, k_out, B, S, D_head, dtype, spec, _ptr(positions), *pos_strides,
                                    _stream(stream)), "rtlynx_rope")


def rtlynx_rope_backward(dq_out, dk_out, dq, dk, B, S, D_head, dtype, spec, positions, pos_strides,
                         stream=None) -> int:
    return _check(lib().rtlynx_rope_backward(dq_out, dk_out, dq, dk, B, S, D_head, dtype, spec, _ptr(positions),
                                             *pos_strides, _stream(stream)), "rtlynx_rope_backward")


def rtlynx_qk_norm_rope(q, k, w_q, w_k, q_out, k_out, B, S, D_head, dtype, eps, spec, positions, pos_strides,
                        stream=None) -> int:
    return _check(lib().rtlynx_qk_norm_rope(q, k, _ptr(w_q), _ptr(w_k), q_out, k_out, B, S, D_head, dtype, eps, spec,
                                            _ptr(positions), *pos_strides, _stream(stream)), "rtlynx_qk_norm_rope")


def rtlynx_qk_norm_rope_workspace_size(D_head) -> int:
    return int(lib().rtlynx_qk_norm_rope_workspace_size(D_head))


def rtlynx_qk_norm_rope_backward(dq_out, dk_out, q, k, w_q, w_k, dq, dk, dw_q, dw_k, B, S, D_head, dtype, eps, spec,
                                 positions, pos_strides, workspace, ws_bytes, stream=None) -> int:
    return _check(lib().rtlynx_qk_norm_rope_backward(dq_out, dk_out, q, k, _ptr(w_q), _ptr(w_k), dq, dk, _ptr(dw_q),
                                                     _ptr(dw_k), B, S, D_head, dtype, eps, spec, _ptr(positions),
                                                     *pos_strides, _ptr(workspace), ws_bytes, _stream(stream)),
                  "rtlynx_qk_norm_rope_backward")


def rtlynx_kernel_launches(M, D_in, D_out, R, mode) -> int:
    return int(lib().rtlynx_kernel_launches(M, D_in, D_out, R, mode))


def rtlynx_schedule_info(M, D_in, D_out, R, num_sms) -> Schedule:
    """The work split of a sparse-mode call on a GPU with num_sms SMs (host only)."""
    out = Schedule()
    _check(lib().rtlynx_schedule_info(M, D_in, D_out, R, num_sms, ctypes.byref(out)), "rtlynx_schedule_info")
    return out


def rtlynx_wait_selftest(limit_ns, stream=None) -> int:
    return _check(lib().rtlynx_wait_selftest(int(limit_ns), _stream(stream)), "rtlynx_wait_selftest")


def rtlynx_stream_status(stream=None) -> int:
    return int(lib().rtlynx_stream_status(_stream(stream)))


def rtlynx_status_string(status: int) -> str:
    try:
        return lib().rtlynx_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def rtlynx_release() -> None:
    lib().rtlynx_release()


# ------------------------------------------------------------------ torch convenience (marshalling only)
def linear(X, W, L_A=None, L_B=None, mode: int = MODE_SPARSE, out=None, stream=None):
    """Y for torch bf16 CUDA tensors X [M,D_in], W [D_out,D_in], L_A [D_out,R], L_B [R,D_in]."""
    import torch
    M, D_in = X.shape
    D_out = W.shape[0]
    R = 0 if (L_A is None or L_B is None or mode == MODE_DENSE_SKIP) else L_B.shape[0]
    for t in (X, W, L_A, L_B):
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous()):
            raise ValueError("inputs must be contiguous bf16 CUDA tensors")
    Y = out if out is not None else torch.empty((M, D_out), dtype=torch.bfloat16, device=X.device)
    rtlynx_linear(X, W, L_A if R else None, L_B if R else None, Y, M, D_in, D_out, R, mode, stream)
    return Y


# The operators around the linear layers.  Checks, outputs and the call itself are compiled (csrc/torch_calls.cpp):
# a call on a few tokens is as long as its host part.  They record nothing for autograd: an output carries no history,
# whatever its inputs require, and gradients come from the _backward calls.
_calls = None
_HERE = contextlib.nullcontext()


def _torch_calls():
    global _calls
    if _calls is None:
        import torch  # the extension needs its libraries in the process
        path = torch_lib_path(torch.__version__)
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m activation_sparse_gemm_b200.build`")
        spec = importlib.util.spec_from_file_location("rtlynx_torch", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        L = lib()
        module.bind({name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in ABI_SYMBOLS})
        _calls = module
    return _calls


def _on(tensor, stream):
    """The context in which a call on `tensor` runs on `stream` (a torch stream or a handle): outputs and workspaces
    then come from that stream's pool, so that memory is never handed on while in use."""
    import torch
    if isinstance(stream, int):
        # handle 0, the default stream, is to torch a request for a stream of its pool
        stream = (torch.cuda.ExternalStream(stream, device=tensor.device) if stream
                  else torch.cuda.default_stream(tensor.device))
    elif stream.device != tensor.device:
        raise ValueError(f"stream of {stream.device}, tensors on {tensor.device}")
    return torch.cuda.stream(stream)


class Rope:
    """A rotation by position, to keep and pass to rope() and qk_norm_rope().

    axes      channels of each axis, e.g. (44, 42, 42) for time, height and width of a head of 128, (128,) for text;
              channels past their sum pass through
    theta     base of the frequencies theta^(-2 j / axis)
    pairing   ROPE_INTERLEAVED (channels 2 i, 2 i + 1) or ROPE_HALF (channels i, i + sum(axes) / 2)
    inv_freq  the frequencies themselves, sum(axes) / 2 numbers in pair order, instead of theta
    """

    def __init__(self, axes, theta=10000.0, pairing=ROPE_INTERLEAVED, inv_freq=None):
        self.axes = tuple(int(a) for a in axes)
        if not 1 <= len(self.axes) <= MAX_AXES:
            raise ValueError(f"one to {MAX_AXES} axes, got {len(self.axes)}")
        if any(a < 2 or a % 2 for a in self.axes):
            raise ValueError(f"every axis has an even number of channels, got {self.axes}")
        pairs = sum(self.axes) // 2
        if inv_freq is None:
            theta = float(theta)
            if not 0.0 < theta < float("inf"):
                raise ValueError(f"theta is positive and finite, got {theta}")
            values = [theta ** (-2.0 * j / n) for n in self.axes for j in range(n // 2)]
        else:
            values = [float(v) for v in inv_freq]
            if len(values) != pairs:
                raise ValueError(f"inv_freq has {len(values)} values, the axes {pairs} pairs")
        self._lay_out(int(pairing), values)

    def _lay_out(self, pairing, values):
        # the calls read the frequencies from here, so no call has to raise theta to 64 powers
        self._freq = (ctypes.c_double * len(values))(*values)
        dims = (ctypes.c_int32 * MAX_AXES)(*self.axes)
        freq = ctypes.cast(self._freq, ctypes.POINTER(ctypes.c_double))
        self.specs = (RopeSpec * 3)(*(RopeSpec(len(self.axes), dims, pairing, t, 0.0, freq)
                                      for t in (POS_INT32, POS_INT64, POS_FP32)))
        self._at = ctypes.addressof(self.specs)

    # A copy, or what another process unpickles, has a layout of its own: addresses do not travel.
    def __getstate__(self):
        state = {name: value for name, value in self.__dict__.items() if name not in ("_freq", "specs", "_at")}
        return state, self.specs[0].pairing, list(self._freq)

    def __setstate__(self, state):
        self.__dict__.update(state[0])
        self._lay_out(*state[1:])


def rope(q, k, positions, rope, out=None, stream=None):
    """(R q, R k) for q [B, S, Hq, D] and k [B, S, Hk, D] (or [S, H, D], or k None), any strides.

    positions [S, axes] or [B, S, axes] (int32, int64, float32), rope a Rope; out=(q, k) works in place."""
    with _HERE if stream is None else _on(q, stream):
        return _torch_calls().rope(False, q, k, positions, rope._at, len(rope.axes), out)


def rope_backward(dq_out, dk_out, positions, rope, out=None, stream=None):
    """Gradients of rope()'s inputs from those of its outputs; out=(dq_out, dk_out) works in place."""
    with _HERE if stream is None else _on(dq_out, stream):
        return _torch_calls().rope(True, dq_out, dk_out, positions, rope._at, len(rope.axes), out)


def qk_norm_rope(q, k, w_q, w_k, positions, rope, eps=1e-6, out=None, stream=None):
    """rope() of the heads' RMS norms: (R (w_q q / rms q), R (w_k k / rms k)); w_q, w_k [D] in q's type, or None."""
    with _HERE if stream is None else _on(q, stream):
        return _torch_calls().qk_norm_rope(q, k, w_q, w_k, positions, rope._at, len(rope.axes), eps, out)


def qk_norm_rope_backward(dq_out, dk_out, q, k, w_q, w_k, positions, rope, eps=1e-6, out=None, weight_grads=True,
                          stream=None):
    """(dq, dk, dw_q, dw_k) of qk_norm_rope(); dw_q, dw_k are float32 [D], None without weight_grads or a weight.

    out=(dq_out, dk_out) or out=(q, k) works in place."""
    with _HERE if stream is None else _on(q, stream):
        return _torch_calls().qk_norm_rope_backward(dq_out, dk_out, q, k, w_q, w_k, positions, rope._at,
                                                    len(rope.axes), eps, out, weight_grads)


def gated_mlp(X, W_gate, W_up, W_down, act=ACT_SILU, L_A=None, L_B=None, mode_down=None, save=False, out=None,
              stream=None):
    """Y [M, D] of the gated feed-forward block, for contiguous bf16 CUDA tensors X [M, D], W_gate and W_up [D_ff, D],
    W_down [D, D_ff].

    mode_down  None or MODE_DENSE_SKIP: Y = H W_down^T.  MODE_SPARSE: the activation-sparse layer, with the LoRA pair
               L_A [D, R], L_B [R, D_ff] where both are given (MODE_DENSE_SKIP leaves a pair out, as linear() does;
               None refuses one).

    With save=True the result is (Y, saved), saved = (G, U, low, H) for gated_mlp_backward
    (low: the bits of G and U below bf16's, as int16; see include/rtlynx.h)."""
    with _HERE if stream is None else _on(X, stream):
        return _torch_calls().gated_mlp(X, W_gate, W_up, W_down, act, L_A, L_B, mode_down, save, out)


def gated_mlp_backward(dY, X, W_gate, W_up, W_down, saved, act=ACT_SILU, needs=(True, True, True, True), stream=None):
    """(dX, dW_gate, dW_up, dW_down) of gated_mlp with a dense down-projection, from dY [M, D] and its `saved`.

    needs: which of the four to compute; the others are None."""
    with _HERE if stream is None else _on(X, stream):
        return _torch_calls().gated_mlp_backward(dY, X, W_gate, W_up, W_down, saved, act, [bool(n) for n in needs])
