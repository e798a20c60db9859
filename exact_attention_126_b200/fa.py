"""Python binding of libfa.so: the C entry points of include/fa.h under the same names.

Only argument marshalling happens here: shapes, dtypes and devices are read off torch
tensors, their data pointers and the current CUDA stream are passed to the C ABI, and a
non-OK status is raised as ``FAError``. Every step of the computation runs in the
library's kernels; if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libfa.so")

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_MISALIGNED",
    4: "FA_ERR_WORKSPACE", 5: "FA_ERR_CUDA", 6: "FA_ERR_TIMEOUT",
}

#: every symbol include/fa.h declares
EXPORTED = ("fa_fwd", "fa_fwd_ex", "fa_fwd_fp8", "fa_bwd_workspace_bytes",
            "fa_bwd_workspace_bytes_ex", "fa_bwd", "fa_bwd_ex",
            "fa_fwd_alibi", "fa_bwd_alibi", "fa_bwd_preprocess", "fa_bwd_dkdv", "fa_bwd_dq",
            "fa_bwd_fused", "fa_bwd_dq_convert", "fa_bwd_noalloc", "fa_fwd_score",
            "fa_bwd_score", "fa_qk_norm_rope_fwd",
            "fa_qk_norm_rope_workspace_bytes", "fa_qk_norm_rope_bwd", "fa_status_string",
            "fa_debug_status", "fa_debug_set_fault", "fa_version")

#: fa_options_t.flags: the fused backward (head_dim 64; dQ by fp32 reductions)
FA_BWD_FUSED = 1


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().fa_status_string(status).decode() if _LIB is not None else STATUS_NAMES.get(status)
        super().__init__("%s returned %s" % (where, msg))


class fa_window_t(ctypes.Structure):
    _fields_ = [("left", ctypes.c_int), ("right", ctypes.c_int)]


class fa_options_t(ctypes.Structure):
    """Optional inputs and outputs of the _ex entry points (include/fa.h)."""
    _fields_ = [("alibi_slopes", ctypes.c_void_p), ("key_padding", ctypes.c_void_p),
                ("o_low", ctypes.c_void_p), ("dropout_p", ctypes.c_float),
                ("flags", ctypes.c_uint), ("dropout_seed", ctypes.c_ulonglong),
                ("dropout_offset", ctypes.c_ulonglong), ("seq_lengths", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("total_tokens", ctypes.c_int)]


class fa_score_t(ctypes.Structure):
    """Changes to the scores of fa_fwd_score and fa_bwd_score (include/fa.h)."""
    _fields_ = [("prefix_lengths", ctypes.c_void_p), ("softcap", ctypes.c_float)]


class fa_heads_t(ctypes.Structure):
    """Rows of queries, keys or values with their strides (include/fa.h)."""
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("batch_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong)]


class fa_norm_rope_t(ctypes.Structure):
    """Parameters of fa_qk_norm_rope_fwd and _bwd (include/fa.h)."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("seq_lengths", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("norm", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("axes", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("total_tokens", ctypes.c_int),
                ("fill_uncovered", ctypes.c_int)]


def options(alibi_slopes=None, key_padding=None, o_low=None, dropout_p=0.0, dropout_seed=0,
            dropout_offset=0, fused=False, seq_lengths=None, cu_seqlens=None, total_tokens=0):
    """An fa_options_t holding the device pointers of the given tensors (None = absent), the
    dropout parameters (probability, 64-bit seed, 32-bit offset), the backward's flags, the
    real lengths of a variable-length batch (B int32 on the device), or the cumulative
    lengths (B + 1 int32 on the device) and token count of a packed batch."""
    return fa_options_t(_ptr(alibi_slopes), _ptr(key_padding), _ptr(o_low), float(dropout_p),
                        FA_BWD_FUSED if fused else 0,
                        int(dropout_seed) & 0xFFFFFFFFFFFFFFFF, int(dropout_offset),
                        _ptr(seq_lengths), _ptr(cu_seqlens), int(total_tokens))


_LIB = None


def _lib() -> ctypes.CDLL:
    """The loaded library (built in-tree by ``build.build()``); raises if it is absent."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError("libfa.so is not built (run exact_attention_126_b200.build.build());"
                               " there is no fallback path")
        lib = ctypes.CDLL(LIBRARY)
        vp, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        W = fa_window_t
        OP = ctypes.POINTER(fa_options_t)
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, F, I, W, vp]
        lib.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP, vp]
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, F, F, F, vp, vp, I, I, I, I, F, I, W, vp]
        lib.fa_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP,
                                  vp, ctypes.c_size_t, vp]
        lib.fa_bwd_workspace_bytes.argtypes = [I, I, I, I]
        lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_bwd_workspace_bytes_ex.argtypes = [I, I, I, I, OP]
        lib.fa_bwd_workspace_bytes_ex.restype = ctypes.c_size_t
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, vp,
                               ctypes.c_size_t, vp]
        lib.fa_fwd_alibi.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, F, I, W, vp, vp]
        lib.fa_bwd_alibi.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, vp,
                                     vp, ctypes.c_size_t, vp]
        lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, vp, I, I, I, I, OP, vp]
        lib.fa_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP, vp]
        lib.fa_bwd_dq.argtypes = [vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP, vp]
        lib.fa_bwd_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP, vp]
        lib.fa_bwd_dq_convert.argtypes = [vp, vp, I, I, I, I, F, vp]
        lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W,
                                       vp]
        SP = ctypes.POINTER(fa_score_t)
        lib.fa_fwd_score.argtypes = [vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP, SP, vp]
        lib.fa_bwd_score.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, I, I, I, I, F, I, W, OP,
                                     SP, vp, ctypes.c_size_t, vp]
        HP, NP = ctypes.POINTER(fa_heads_t), ctypes.POINTER(fa_norm_rope_t)
        lib.fa_qk_norm_rope_fwd.argtypes = [HP, HP, HP, HP, HP, HP, I, I, I, NP, vp]
        lib.fa_qk_norm_rope_bwd.argtypes = [HP, HP, HP, HP, HP, HP, HP, HP, vp, vp, I, I, I, NP,
                                            vp, ctypes.c_size_t, vp]
        lib.fa_qk_norm_rope_workspace_bytes.argtypes = [I]
        lib.fa_qk_norm_rope_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_status_string.argtypes = [I]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_debug_status.argtypes = [vp]
        lib.fa_debug_set_fault.argtypes = [I]
        lib.fa_version.argtypes = []
        for name in ("fa_fwd", "fa_fwd_ex", "fa_fwd_fp8", "fa_bwd", "fa_bwd_ex", "fa_fwd_alibi",
                     "fa_bwd_alibi", "fa_bwd_preprocess", "fa_bwd_fused", "fa_bwd_dq_convert",
                     "fa_bwd_dkdv", "fa_bwd_dq", "fa_bwd_noalloc", "fa_fwd_score", "fa_bwd_score",
                     "fa_qk_norm_rope_fwd", "fa_qk_norm_rope_bwd", "fa_debug_status", "fa_debug_set_fault",
                     "fa_version"):
            getattr(lib, name).restype = I
        _LIB = lib
    return _LIB


def library() -> ctypes.CDLL:
    return _lib()


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # (the raw handle: building a torch.cuda.Stream costs several microseconds per call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _shape(q: torch.Tensor, dims=None):
    """(B, H, N, d) of a (batch, heads, seq_len, head_dim) tensor, or `dims` as given (a
    packed batch's (total, heads, head_dim) tensors do not carry B and N)."""
    if dims is not None:
        return tuple(map(int, dims))
    if q.dim() != 4:
        raise ValueError("expected a (batch, heads, seq_len, head_dim) tensor")
    return tuple(q.shape)


def _window(causal: bool, window) -> tuple[int, fa_window_t]:
    left, right = (-1, -1) if window is None else window
    return int(bool(causal)), fa_window_t(int(left), int(right))


def default_scale(d: int) -> float:
    """softmax_scale=None means 1/sqrt(head_dim)."""
    return 1.0 / math.sqrt(d)


# ------------------------------------------------------------------ raw entry points
def fa_fwd(q, k, v, o, lse, scale=None, causal=False, window=(-1, -1), stream=None) -> None:
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, s, c, w,
                         _stream(stream)), "fa_fwd")


def fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, scale=None, causal=False,
               window=(-1, -1), stream=None) -> None:
    """The forward on e4m3 tensors (torch.float8_e4m3fn or uint8 bytes) with per-tensor
    descales; o is bf16."""
    B, H, N, d = _shape(q8)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), float(q_scale), float(k_scale),
                             float(v_scale), _ptr(o), _ptr(lse), B, H, N, d, s, c, w,
                             _stream(stream)), "fa_fwd_fp8")


def attention_forward_fp8(q8, k8, v8, q_scale=1.0, k_scale=1.0, v_scale=1.0, scale=None,
                          causal=False, window=(-1, -1), stream=None):
    """Returns (O, LSE) of the attention of q8*q_scale, k8*k_scale, v8*v_scale for e4m3 CUDA
    tensors of shape (B, H, N, 128); O is bf16."""
    for t in (q8, k8, v8):
        if not t.is_cuda or t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError("q8, k8, v8 must be float8_e4m3fn (or uint8) CUDA tensors")
        if not t.is_contiguous() or t.shape != q8.shape:
            raise ValueError("q8, k8, v8 must be contiguous and share one shape")
    other = _other_stream(stream, q8.device)
    if other is not None:
        return _on_stream(other, attention_forward_fp8, q8, k8, v8, q_scale, k_scale, v_scale,
                          scale, causal, window)
    B, H, N, d = _shape(q8)
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, scale, causal, window, stream)
    return o, lse


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(_lib().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd_workspace_bytes_ex(B: int, H: int, N: int, d: int, opt=None) -> int:
    return int(_lib().fa_bwd_workspace_bytes_ex(B, H, N, d, _opt_ref(opt)))


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale=None, causal=False,
           window=(-1, -1), stream=None) -> None:
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                         _ptr(dk), _ptr(dv), B, H, N, d, s, c, w, _ptr(workspace), nbytes,
                         _stream(stream)), "fa_bwd")


def fa_fwd_alibi(q, k, v, o, lse, alibi_slopes, scale=None, causal=False, window=(-1, -1),
                 stream=None) -> None:
    """fa_fwd with the linear bias -alibi_slopes[h] * |i - j| (alibi_slopes: H fp32 values
    on the device)."""
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_fwd_alibi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, s, c,
                               w, _ptr(alibi_slopes), _stream(stream)), "fa_fwd_alibi")


def fa_bwd_alibi(q, k, v, o, do, lse, dq, dk, dv, workspace, alibi_slopes, scale=None,
                 causal=False, window=(-1, -1), stream=None) -> None:
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().fa_bwd_alibi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                               _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, s, c, w,
                               _ptr(alibi_slopes), _ptr(workspace), nbytes, _stream(stream)),
           "fa_bwd_alibi")


def _opt_ref(opt):
    return None if opt is None else ctypes.byref(opt)


def fa_fwd_ex(q, k, v, o, lse, opt=None, scale=None, causal=False, window=(-1, -1),
              stream=None, dims=None) -> None:
    """fa_fwd with an fa_options_t (see options()); `dims` = (B, H, N, d) for a packed batch."""
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, s, c, w,
                            _opt_ref(opt), _stream(stream)), "fa_fwd_ex")


def fa_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, workspace, opt=None, scale=None, causal=False,
              window=(-1, -1), stream=None, dims=None) -> None:
    """fa_bwd with an fa_options_t (see options()); `dims` = (B, H, N, d) for a packed batch."""
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().fa_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                            _ptr(dk), _ptr(dv), B, H, N, d, s, c, w, _opt_ref(opt),
                            _ptr(workspace), nbytes, _stream(stream)), "fa_bwd_ex")


def fa_fwd_score(q, k, v, o, lse, opt=None, score=None, scale=None, causal=False,
                 window=(-1, -1), stream=None, dims=None) -> None:
    """fa_fwd_ex with an fa_score_t (a cap of the scores, prefix lengths)."""
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_fwd_score(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, s, c, w,
                               _opt_ref(opt), _opt_ref(score), _stream(stream)), "fa_fwd_score")


def fa_bwd_score(q, k, v, o, do, lse, dq, dk, dv, workspace, opt=None, score=None, scale=None,
                 causal=False, window=(-1, -1), stream=None, dims=None) -> None:
    """fa_bwd_ex with the fa_score_t the forward had."""
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().fa_bwd_score(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), B, H, N, d, s, c, w, _opt_ref(opt),
                               _opt_ref(score), _ptr(workspace), nbytes, _stream(stream)),
           "fa_bwd_score")


def fa_bwd_preprocess(o, do, lse, workspace, opt=None, stream=None, dims=None) -> None:
    B, H, N, d = _shape(o, dims)
    _check(_lib().fa_bwd_preprocess(_ptr(o), _ptr(do), _ptr(lse), _ptr(workspace), B, H, N, d,
                                    _opt_ref(opt), _stream(stream)), "fa_bwd_preprocess")


def fa_bwd_dkdv(q, k, v, do, workspace, dk, dv, scale=None, causal=False, window=(-1, -1),
                stream=None, opt=None, dims=None) -> None:
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(workspace), _ptr(dk),
                              _ptr(dv), B, H, N, d, s, c, w, _opt_ref(opt), _stream(stream)),
           "fa_bwd_dkdv")


def fa_bwd_fused(q, k, v, do, workspace, dk, dv, scale=None, causal=False, window=(-1, -1),
                 stream=None, opt=None) -> None:
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_bwd_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(workspace), _ptr(dk),
                               _ptr(dv), B, H, N, d, s, c, w, _opt_ref(opt), _stream(stream)),
           "fa_bwd_fused")


def fa_bwd_dq_convert(workspace, dq, scale=None, stream=None) -> None:
    B, H, N, d = _shape(dq)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_bwd_dq_convert(_ptr(workspace), _ptr(dq), B, H, N, d, s, _stream(stream)),
           "fa_bwd_dq_convert")


def fa_bwd_dq(q, k, v, do, workspace, dq, scale=None, causal=False, window=(-1, -1),
              stream=None, opt=None, dims=None) -> None:
    B, H, N, d = _shape(q, dims)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(workspace), _ptr(dq),
                            B, H, N, d, s, c, w, _opt_ref(opt), _stream(stream)), "fa_bwd_dq")


def fa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, scale=None, causal=False, window=(-1, -1),
                   stream=None) -> None:
    """fa_bwd without a workspace argument: for callers that cannot allocate device
    memory; the library's own fixed device array holds the row statistics."""
    B, H, N, d = _shape(q)
    c, w = _window(causal, window)
    s = default_scale(d) if scale is None else float(scale)
    _check(_lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, s, c, w,
                                 _stream(stream)), "fa_bwd_noalloc")


def fa_qk_norm_rope_fwd(q, k, v, q_out, k_out, v_out, B, N, d, params, stream=None) -> None:
    """q .. v_out: fa_heads_t or None; params: fa_norm_rope_t."""
    _check(_lib().fa_qk_norm_rope_fwd(q, k, v, q_out, k_out, v_out, B, N, d, params,
                                      _stream(stream)), "fa_qk_norm_rope_fwd")


def fa_qk_norm_rope_workspace_bytes(d: int) -> int:
    return int(_lib().fa_qk_norm_rope_workspace_bytes(d))


def fa_qk_norm_rope_bwd(dq, dk, dv, q, k, gq, gk, gv, gq_weight, gk_weight, B, N, d, params,
                        workspace=None, stream=None) -> None:
    """dq .. gv: fa_heads_t or None; gq_weight, gk_weight: fp32 tensors or None."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().fa_qk_norm_rope_bwd(dq, dk, dv, q, k, gq, gk, gv, _ptr(gq_weight),
                                      _ptr(gk_weight), B, N, d, params, _ptr(workspace), nbytes,
                                      _stream(stream)), "fa_qk_norm_rope_bwd")


def fa_status_string(status: int) -> str:
    return _lib().fa_status_string(int(status)).decode()


def fa_debug_status(stream=None) -> int:
    return int(_lib().fa_debug_status(_stream(stream)))


def fa_debug_set_fault(fault: int) -> None:
    """Test hook: 1 makes later fa_fwd launches time out on purpose (see include/fa.h)."""
    _check(_lib().fa_debug_set_fault(int(fault)), "fa_debug_set_fault")


def fa_version() -> int:
    return int(_lib().fa_version())


# ------------------------------------------------------------------ allocating helpers
def _elsewhere(t):
    """Whether `t` lives on another CUDA device than the current one (the library launches on
    the current device)."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return t.get_device() != torch.cuda.current_device()


def _other_stream(stream, device):
    """`stream` where it is not the current stream of `device` (the current device), else None."""
    if stream is None or _stream(stream) == _stream(None):
        return None
    if not isinstance(stream, torch.cuda.Stream):
        return torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError("stream must be a stream of the tensors' device")
    return stream


def _on_stream(stream, call, *args):
    """`call(*args)` with `stream` as the current stream: what the call allocates is then memory of
    that stream, whose earlier users are ordered before the call's kernels (a block of the current
    stream may still be in use there). The arguments stay out of the allocator's hands until
    `stream`, the results until the caller's stream, has passed what is queued on it."""
    home = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        res = call(*args)
    for group, user in ((args, stream), (res, home)):
        for x in group:
            for t in x if isinstance(x, (list, tuple)) else (x,):
                if isinstance(t, torch.Tensor):
                    t.record_stream(user)
    return res


def _scratch(nbytes, device):
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


def _check_inputs(*ts):
    shape = ts[0].shape
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if t.dtype is not torch.bfloat16:
            raise ValueError("tensors must be bf16")
        if t.get_device() != ts[0].get_device():
            raise ValueError("tensors must be on one device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous (B, H, N, d)")
        if t.shape != shape:
            raise ValueError("q, k, v (and dO) must share one shape")


def _check_device(t, name, q):
    """The kernels read `t` by its address on the queries' device."""
    if t.get_device() != q.get_device():
        raise ValueError("%s must be on the queries' device" % name)


def _check_slopes(alibi_slopes, q):
    if not alibi_slopes.is_cuda or alibi_slopes.dtype != torch.float32:
        raise ValueError("alibi_slopes must be an fp32 CUDA tensor")
    _check_device(alibi_slopes, "alibi_slopes", q)
    if alibi_slopes.numel() != q.shape[1] or not alibi_slopes.is_contiguous():
        raise ValueError("alibi_slopes must hold one slope per head, contiguous")


def _check_padding(key_padding, q, B, N):
    if not key_padding.is_cuda or key_padding.dtype not in (torch.bool, torch.uint8):
        raise ValueError("key_padding must be a bool or uint8 CUDA tensor")
    _check_device(key_padding, "key_padding", q)
    if tuple(key_padding.shape) != (B, N) or not key_padding.is_contiguous():
        raise ValueError("key_padding must be a contiguous (batch, seq_len) tensor")


def _check_lengths(seq_lengths, q):
    if not seq_lengths.is_cuda or seq_lengths.dtype != torch.int32:
        raise ValueError("seq_lengths must be an int32 CUDA tensor")
    _check_device(seq_lengths, "seq_lengths", q)
    if seq_lengths.numel() != q.shape[0] or not seq_lengths.is_contiguous():
        raise ValueError("seq_lengths must hold one length per batch entry, contiguous")


def _packed_dims(q, cu_seqlens, max_seqlen, seq_lengths):
    """(B, H, N, d) of a packed batch: q is (total, H, d), cu_seqlens B + 1 int32 offsets."""
    if seq_lengths is not None:
        raise ValueError("seq_lengths and cu_seqlens exclude each other")
    if not cu_seqlens.is_cuda or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 CUDA tensor")
    _check_device(cu_seqlens, "cu_seqlens", q)
    if cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must hold B + 1 >= 2 offsets, contiguous")
    if q.dim() != 3:
        raise ValueError("a packed batch takes (total_tokens, heads, head_dim) tensors")
    if max_seqlen is None or int(max_seqlen) < 1:
        raise ValueError("a packed batch needs max_seqlen >= 1 (the longest sequence)")
    return cu_seqlens.numel() - 1, int(q.shape[1]), int(max_seqlen), int(q.shape[2])


def _score(softcap, prefix_lengths, q, B):
    """The fa_score_t of a cap and prefix lengths, or None without either."""
    if prefix_lengths is not None:
        if not prefix_lengths.is_cuda or prefix_lengths.dtype != torch.int32:
            raise ValueError("prefix_lengths must be an int32 CUDA tensor")
        if tuple(prefix_lengths.shape) != (B,) or not prefix_lengths.is_contiguous():
            raise ValueError("prefix_lengths must hold one length per sequence, contiguous")
        _check_device(prefix_lengths, "prefix_lengths", q)
    elif softcap is None or softcap == 0.0:
        return None
    return fa_score_t(_ptr(prefix_lengths), 0.0 if softcap is None else float(softcap))


def attention_forward(q, k, v, scale=None, causal=False, window=(-1, -1), stream=None,
                      alibi_slopes=None, key_padding=None, keep_residual=False, dropout=None,
                      seq_lengths=None, cu_seqlens=None, max_seqlen=None, softcap=0.0,
                      prefix_lengths=None):
    """Returns (O, LSE) for bf16 CUDA tensors q, k, v of shape (B, H, N, d), or
    (O, LSE, O_low) with keep_residual: O_low = O_fp32 - bf16(O) in bf16, which
    attention_backward uses to form rowsum(dO o O) from O to about 16 bits.
    alibi_slopes (H fp32 values): the scores carry the bias -alibi_slopes[h] * |i - j|.
    key_padding ((B, N) bool or uint8, True = padded key): padded keys are masked out
    for every head and query. dropout: (p, seed, offset) drops each attention weight with
    probability p (rounded to a multiple of 1/256) after the softmax and scales the kept
    ones by 1 / (1 - p); the backward needs the same triple. seq_lengths ((B,) int32):
    entry b holds seq_lengths[b] real tokens; rows past it are zero (LSE -inf) and tiles
    wholly past it are not computed. cu_seqlens ((B + 1,) int32) with max_seqlen: a packed
    batch, q, k, v of shape (total, H, d) holding sequence b at tokens cu_seqlens[b] ..
    cu_seqlens[b+1]-1; O is (total, H, d) and LSE (H, total), not written for tokens that no
    sequence covers (nor are their gradients by attention_backward). softcap (c > 0): the scaled scores
    s become c tanh(s / c). prefix_lengths ((B,) int32), for causal problems: query i of sequence b
    also sees every key j < prefix_lengths[b]."""
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return attention_forward(q, k, v, scale, causal, window, stream, alibi_slopes,
                                     key_padding, keep_residual, dropout, seq_lengths, cu_seqlens,
                                     max_seqlen, softcap, prefix_lengths)
    other = _other_stream(stream, q.device)
    if other is not None:
        return _on_stream(other, attention_forward, q, k, v, scale, causal, window, None,
                          alibi_slopes, key_padding, keep_residual, dropout, seq_lengths,
                          cu_seqlens, max_seqlen, softcap, prefix_lengths)
    _check_inputs(q, k, v)
    if cu_seqlens is not None:
        B, H, N, d = _packed_dims(q, cu_seqlens, max_seqlen, seq_lengths)
        lse = q.new_empty((H, q.shape[0]), dtype=torch.float32)
    else:
        B, H, N, d = _shape(q)
        lse = q.new_empty((B, H, N), dtype=torch.float32)
    o = torch.empty_like(q)
    o_low = torch.empty_like(q) if keep_residual else None
    if alibi_slopes is not None:
        _check_slopes(alibi_slopes, q)
    if key_padding is not None:
        _check_padding(key_padding, q, B, N)
    if seq_lengths is not None:
        _check_lengths(seq_lengths, q)
    score = _score(softcap, prefix_lengths, q, B)
    opt = None
    if (alibi_slopes is not None or key_padding is not None or o_low is not None
            or dropout is not None or seq_lengths is not None or cu_seqlens is not None):
        opt = options(alibi_slopes, key_padding, o_low, *(dropout or ()),
                      seq_lengths=seq_lengths, cu_seqlens=cu_seqlens,
                      total_tokens=q.shape[0] if cu_seqlens is not None else 0)
    if score is not None:
        fa_fwd_score(q, k, v, o, lse, opt, score, scale, causal, window, stream,
                     dims=(B, H, N, d))
    elif opt is not None:
        fa_fwd_ex(q, k, v, o, lse, opt, scale, causal, window, stream, dims=(B, H, N, d))
    else:
        fa_fwd(q, k, v, o, lse, scale, causal, window, stream)
    return (o, lse, o_low) if keep_residual else (o, lse)


def attention_backward(q, k, v, o, lse, do, scale=None, causal=False, window=(-1, -1),
                       stream=None, alibi_slopes=None, key_padding=None, o_low=None,
                       dropout=None, fused=False, seq_lengths=None, cu_seqlens=None,
                       max_seqlen=None, softcap=0.0, prefix_lengths=None):
    """Returns (dQ, dK, dV): the gradient of <O, dO>; lse (and o_low, if kept) come from
    attention_forward with the same alibi_slopes, key_padding, dropout, seq_lengths, softcap and
    prefix_lengths.
    fused: at head_dim 64, the backward in one pass over key tiles with dQ added up in fp32
    in no fixed order (see FA_BWD_FUSED); otherwise the deterministic dK/dV and dQ passes."""
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return attention_backward(q, k, v, o, lse, do, scale, causal, window, stream,
                                      alibi_slopes, key_padding, o_low, dropout, fused,
                                      seq_lengths, cu_seqlens, max_seqlen, softcap,
                                      prefix_lengths)
    other = _other_stream(stream, q.device)
    if other is not None:
        return _on_stream(other, attention_backward, q, k, v, o, lse, do, scale, causal, window,
                          None, alibi_slopes, key_padding, o_low, dropout, fused, seq_lengths,
                          cu_seqlens, max_seqlen, softcap, prefix_lengths)
    _check_inputs(q, k, v, o, do)
    if cu_seqlens is not None:
        B, H, N, d = _packed_dims(q, cu_seqlens, max_seqlen, seq_lengths)
    else:
        B, H, N, d = _shape(q)
    total = q.shape[0] if cu_seqlens is not None else 0
    dq = torch.empty_like(q)
    dk = torch.empty_like(q)
    dv = torch.empty_like(q)
    if alibi_slopes is not None:
        _check_slopes(alibi_slopes, q)
    if key_padding is not None:
        _check_padding(key_padding, q, B, N)
    if o_low is not None:
        _check_inputs(q, o_low)
    if seq_lengths is not None:
        _check_lengths(seq_lengths, q)
    score = _score(softcap, prefix_lengths, q, B)
    opt = None
    if (alibi_slopes is not None or key_padding is not None or o_low is not None
            or dropout is not None or fused or seq_lengths is not None
            or cu_seqlens is not None):
        opt = options(alibi_slopes, key_padding, o_low, *(dropout or ()),
                      fused=fused, seq_lengths=seq_lengths, cu_seqlens=cu_seqlens,
                      total_tokens=total)
    ws = _scratch(fa_bwd_workspace_bytes_ex(B, H, N, d, opt), q.device)
    if score is not None:
        fa_bwd_score(q, k, v, o, do, lse, dq, dk, dv, ws, opt, score, scale, causal, window,
                     stream, dims=(B, H, N, d))
    elif opt is not None:
        fa_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, ws, opt, scale, causal, window, stream,
                  dims=(B, H, N, d))
    else:
        fa_bwd(q, k, v, o, do, lse, dq, dk, dv, ws, scale, causal, window, stream)
    return dq, dk, dv


# ------------------------------------------------- per-head norm and rotary positions
_BF16 = torch.bfloat16


def _rows(t, name, tokens, d, device, heads_at):
    """The fa_heads_t of a bf16 tensor of any strides, token-major (B, N, heads, d), head-major
    (B, heads, N, d) (heads_at 2, 1) or packed (total, heads, d) (heads_at 1), checked to have
    the given tokens and head_dim, d consecutive, on CUDA device number `device`; None for None."""
    if t is None:
        return None
    if t.dtype is not _BF16 or t.get_device() != device:
        raise ValueError("%s must be a bf16 tensor on the queries' CUDA device" % name)
    shape, st = t.shape, t.stride()
    if len(shape) != len(tokens) + 2 or shape[0] != tokens[0] or (
            len(shape) == 4 and shape[3 - heads_at] != tokens[1]):
        raise ValueError("%s must have the queries' tokens" % name)
    if shape[-1] != d or st[-1] != 1:
        raise ValueError("%s must hold head_dim consecutive values per head" % name)
    if len(shape) == 4:
        return fa_heads_t(t.data_ptr(), shape[heads_at], st[0], st[3 - heads_at], st[heads_at])
    return fa_heads_t(t.data_ptr(), shape[1], 0, st[0], st[1])


def _aux(t, name, dtype, device, shape):
    """The address of a contiguous tensor of the given type and shape on CUDA device number
    `device`; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on the queries' device"
                         % (name, str(dtype).replace("torch.", "")))
    if t.shape != shape:
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return t.data_ptr()


def _norm_rope_params(device, tokens, d, q_weight, k_weight, eps, norm, inv_freq, positions,
                      pair_axis, interleaved, seq_lengths, cu_seqlens, max_seqlen):
    """(B, N, fa_norm_rope_t) of a call on rows of `tokens`."""
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("q_weight and k_weight are gains of the norm")
    rot, axes = 0, 1
    freq = pos = axis = lens = cu = None
    if inv_freq is not None:
        half = inv_freq.numel()
        rot = 2 * half
        freq = _aux(inv_freq, "inv_freq", torch.float32, device, (half,))
        if positions is not None:
            if positions.dim() == len(tokens) + 1:
                axes = positions.shape[0]
                pos = _aux(positions, "positions", torch.int32, device, (axes,) + tokens)
            else:
                pos = _aux(positions, "positions", torch.int32, device, tokens)
        axis = _aux(pair_axis, "pair_axis", torch.uint8, device, (half,))
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    total = 0
    if cu_seqlens is not None:
        if seq_lengths is not None:
            raise ValueError("seq_lengths and cu_seqlens exclude each other")
        if len(tokens) != 1:
            raise ValueError("a packed batch takes (total_tokens, heads, head_dim) tensors")
        B = cu_seqlens.numel() - 1
        cu = _aux(cu_seqlens, "cu_seqlens", torch.int32, device, (B + 1,))
        if B < 1:
            raise ValueError("cu_seqlens must hold B + 1 >= 2 offsets")
        if max_seqlen is None or int(max_seqlen) < 1:
            raise ValueError("a packed batch needs max_seqlen >= 1 (the longest sequence)")
        N, total = int(max_seqlen), tokens[0]
    else:
        if len(tokens) != 2:
            raise ValueError("(total_tokens, heads, head_dim) tensors need cu_seqlens")
        B, N = tokens
        lens = _aux(seq_lengths, "seq_lengths", torch.int32, device, (B,))
    return B, N, fa_norm_rope_t(_aux(q_weight, "q_weight", torch.float32, device, (d,)),
                                _aux(k_weight, "k_weight", torch.float32, device, (d,)),
                                freq, axis, pos, lens, cu, eps, 1 if norm else 0, rot, axes,
                                1 if interleaved else 0, total)


def qk_norm_rope_forward(q, k, v=None, q_weight=None, k_weight=None, eps=1e-6, norm=True,
                         inv_freq=None, positions=None, pair_axis=None, interleaved=False,
                         seq_lengths=None, cu_seqlens=None, max_seqlen=None, stream=None):
    """Queries and keys normalised per head and rotated by their positions, with the values, in
    the layout attention_forward takes. q, k, v: bf16 CUDA tensors (B, N, heads, d) of any token
    and head strides (views of a fused projection), d 64 or 128; returns contiguous
    (B, heads, N, d) tensors (Q, K), or (Q, K, V) with v; k may be None (then K is). A packed batch (cu_seqlens with
    max_seqlen, as in attention_forward) takes and returns (total, heads, d).
    norm: each row divided by sqrt(mean of squares + eps), times the gain q_weight / k_weight
    (d fp32 values; None = ones). inv_freq (rotary_dim / 2 fp32): rotation p turns values
    (p, p + rotary_dim / 2), or (2p, 2p + 1) when interleaved, by position * inv_freq[p]; None =
    no rotation. positions ((B, N) or (total,) int32; None = the place in the sequence): with
    several axes (axes, B, N) or (axes, total), and pair_axis (rotary_dim / 2 uint8) names each
    rotation's axis. seq_lengths ((B,) int32): rows past a length are zero, as are tokens of a
    packed batch that no sequence covers (before the first, behind the last, past max_seqlen)."""
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return qk_norm_rope_forward(q, k, v, q_weight, k_weight, eps, norm, inv_freq,
                                        positions, pair_axis, interleaved, seq_lengths,
                                        cu_seqlens, max_seqlen, stream)
    other = _other_stream(stream, q.device)
    if other is not None:
        return _on_stream(other, qk_norm_rope_forward, q, k, v, q_weight, k_weight, eps, norm,
                          inv_freq, positions, pair_axis, interleaved, seq_lengths, cu_seqlens,
                          max_seqlen)
    if q.dim() not in (3, 4):
        raise ValueError("q must be (B, N, heads, d) or packed (total, heads, d)")
    tokens, d, device = tuple(q.shape[:-2]), q.shape[-1], q.get_device()
    at = len(tokens)
    ins = (_rows(q, "q", tokens, d, device, at), _rows(k, "k", tokens, d, device, at),
           _rows(v, "v", tokens, d, device, at))
    B, N, params = _norm_rope_params(device, tokens, d, q_weight, k_weight, eps, norm, inv_freq,
                                     positions, pair_axis, interleaved, seq_lengths, cu_seqlens,
                                     max_seqlen)
    res, outs = [], []
    for r in ins:
        h = 0 if r is None else r.heads
        if r is None:
            t = out = None
        elif at == 2:
            t = q.new_empty((B, h, N, d))
            out = fa_heads_t(t.data_ptr(), h, h * N * d, d, N * d)
        else:
            t = q.new_empty((tokens[0], h, d))
            out = fa_heads_t(t.data_ptr(), h, 0, h * d, d)
        res.append(t)
        outs.append(out)
    params.fill_uncovered = 1  # (of memory that nothing has written yet)
    fa_qk_norm_rope_fwd(*ins, *outs, B, N, d, params, stream)
    return tuple(res) if v is not None else tuple(res[:2])


def qk_norm_rope_backward(dq, dk, dv=None, q=None, k=None, q_weight=None, k_weight=None, eps=1e-6,
                          norm=True, inv_freq=None, positions=None, pair_axis=None,
                          interleaved=False, seq_lengths=None, cu_seqlens=None, max_seqlen=None,
                          stream=None, out=None):
    """The gradient of qk_norm_rope_forward from those of its outputs, (B, heads, N, d) or packed
    (total, heads, d) (as attention_backward returns them): (gq, gk, gv, gq_weight, gk_weight),
    gk and gv None without dk and dv, the gains' None for a gain that is None. q, k: the forward's
    inputs (needed with norm). out: three tensors (None without dk, dv) of the forward's input
    shapes, of any strides that do not overlap, to write gq, gk, gv to (tokens of a packed batch
    that no sequence covers are left as they are there); by default they are views of one new
    (B, N, heads of all, d) or (total, heads of all, d) tensor, zero for such tokens."""
    if _elsewhere(dq):
        with torch.cuda.device(dq.device):
            return qk_norm_rope_backward(dq, dk, dv, q, k, q_weight, k_weight, eps, norm,
                                         inv_freq, positions, pair_axis, interleaved, seq_lengths,
                                         cu_seqlens, max_seqlen, stream, out)
    other = _other_stream(stream, dq.device)
    if other is not None:
        return _on_stream(other, qk_norm_rope_backward, dq, dk, dv, q, k, q_weight, k_weight, eps,
                          norm, inv_freq, positions, pair_axis, interleaved, seq_lengths,
                          cu_seqlens, max_seqlen, None, out)
    if dq.dim() == 4:
        tokens = (dq.shape[0], dq.shape[2])
    elif dq.dim() == 3:
        tokens = (dq.shape[0],)
    else:
        raise ValueError("dq must be (B, heads, N, d) or packed (total, heads, d)")
    d, device, at = dq.shape[-1], dq.get_device(), len(tokens)
    grads = [_rows(t, n, tokens, d, device, 1) for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"))]
    if norm and (q is None or (k is None and dk is not None)):
        raise ValueError("the norm's gradient needs q and k")
    xq = _rows(q, "q", tokens, d, device, at) if norm else None
    xk = _rows(k, "k", tokens, d, device, at) if norm else None
    B, N, params = _norm_rope_params(device, tokens, d, q_weight, k_weight, eps, norm, inv_freq,
                                     positions, pair_axis, interleaved, seq_lengths, cu_seqlens,
                                     max_seqlen)
    heads = [0 if r is None else r.heads for r in grads]
    if norm and [0 if r is None else r.heads for r in (xq, xk)] != heads[:2]:
        raise ValueError("q and k must have their gradients' heads")
    if out is None:
        out = list(dq.new_empty(tokens + (sum(heads), d)).split(heads, -2))
        out = [None if r is None else t for t, r in zip(out, grads)]
        params.fill_uncovered = 1
    else:
        out = list(out) + [None] * (3 - len(out))
        out = [None if r is None else t for t, r in zip(out, grads)]
    outs = [_rows(t, "out", tokens, d, device, at) for t in out]
    if [0 if r is None else r.heads for r in outs] != heads:
        raise ValueError("out must hold tensors of the forward's input shapes")
    gqw = torch.empty_like(q_weight) if q_weight is not None else None
    gkw = torch.empty_like(k_weight) if k_weight is not None else None
    ws = None
    if gqw is not None or gkw is not None:
        ws = _scratch(fa_qk_norm_rope_workspace_bytes(d), dq.device)
    fa_qk_norm_rope_bwd(*grads, xq, xk, *outs, gqw, gkw, B, N, d, params, ws, stream)
    return out[0], out[1], out[2], gqw, gkw
