"""Thin ctypes binding of libcollider (``include/collider.h``).

Argument marshalling only: every step of the filtered backward runs in the
library's CUDA kernels.  Each function takes the same arguments as the C entry
point of the same name; buffers may be torch tensors (their ``data_ptr()`` is
passed), plain integers (device addresses) or None (NULL).  ``stream``
defaults to torch's current CUDA stream.  A non-OK status raises
:class:`ColliderError` carrying the library's message.  There is no fallback:
if ``libcollider.so`` is missing, importing the binding's entry points fails.
"""
from __future__ import annotations

import ctypes as C
import os

__all__ = [
    "ColliderError", "lib", "LIB_PATH", "ROWS_FULL", "ROWS_COMPACT", "F32", "BF16",
    "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_CUDA", "ERR_TIMEOUT",
    "ARCH_LLAMA", "ARCH_PHI", "NORM_RMS", "NORM_LAYER", "ACT_SWIGLU", "ACT_GELU_TANH",
    "CKPT_E4M3", "CKPT_INT8", "Ckpt", "ckpt", "ResidualNormDesc", "ResidualNormParams", "ResidualNormOut", "ResidualNormSaved",
    "ResidualNormGrads", "residual_norm_params", "residual_norm_out", "residual_norm_saved", "residual_norm_grads",
    "collider_ckpt_pack", "collider_ckpt_unpack", "collider_linear_ckpt_workspace_size", "collider_linear_bwd_ckpt",
    "LayerSavedCkpt", "layer_saved_ckpt", "collider_layer_ckpt_workspace_size", "collider_layer_bwd_ckpt",
    "collider_residual_norm_fwd", "collider_residual_norm_bwd_workspace_size", "collider_residual_norm_bwd",
    "LayerDesc", "LayerWeights", "LayerSaved", "LayerGrads", "LayerParams", "LayerActs", "EXPORTED",
    "collider_last_error", "collider_check", "collider_selftest_wait_timeout", "collider_launch_count",
    "collider_profile_enable", "collider_profile_count", "collider_profile_get", "collider_profile_get_span",
    "collider_select_keep", "collider_compact_workspace_size", "collider_compact", "collider_compact_noalloc",
    "collider_gather_rows",
    "collider_scatter_rows", "collider_linear_workspace_size", "collider_linear_bwd",
    "collider_attn_workspace_size", "collider_attn_bwd", "collider_layer_workspace_size",
    "collider_layer_bwd", "collider_layer_fwd_workspace_size", "collider_layer_fwd",
    "collider_stack_workspace_size", "collider_stack_bwd",
    "GLU_SILU", "GLU_GELU_TANH", "GRAD_NORM_L2", "GRAD_NORM_MAX", "FfnDesc", "Grad", "grad_list",
    "collider_ffn_fwd_workspace_size", "collider_ffn_fwd", "collider_ffn_bwd_workspace_size", "collider_ffn_bwd",
    "collider_grad_norm_workspace_size", "collider_grad_norm", "collider_grad_clip",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcollider.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = range(5)
_STATUS = {1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}
F32, BF16 = 0, 1
ROWS_FULL, ROWS_COMPACT = 0, 1
ARCH_LLAMA, ARCH_PHI = 0, 1
NORM_RMS, NORM_LAYER = 0, 1
ACT_SWIGLU, ACT_GELU_TANH = 0, 1
CKPT_E4M3, CKPT_INT8 = 0, 1
GLU_SILU, GLU_GELU_TANH = 0, 1
GRAD_NORM_L2, GRAD_NORM_MAX = 0, 1


class ColliderError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"COLLIDER_ERR_{_STATUS.get(status, status)}: {msg}")
        self.status = status


class LayerDesc(C.Structure):
    _fields_ = [("arch", C.c_int), ("B", C.c_int), ("T", C.c_int), ("D", C.c_int), ("H", C.c_int),
                ("Hkv", C.c_int), ("dh", C.c_int), ("F", C.c_int), ("rotary_dim", C.c_int),
                ("rope_base", C.c_float), ("norm", C.c_int), ("eps", C.c_float), ("act", C.c_int),
                ("qkv_bias", C.c_int), ("out_bias", C.c_int), ("mlp_bias", C.c_int)]


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("norm1_w", "w_qkv", "w_o", "norm2_w", "w_up", "w_down")]


class LayerSaved(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "a", "mean1", "rstd1", "qkv", "o", "lse", "h", "b",
                                          "rstd2", "up", "s")]


class LayerGrads(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dx", "dnorm1_w", "dnorm1_b", "dw_qkv", "db_qkv", "dw_o",
                                          "db_o", "dnorm2_w", "dw_up", "db_up", "dw_down", "db_down")]


class LayerParams(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("norm1_w", "norm1_b", "w_qkv", "b_qkv", "w_o", "b_o", "norm2_w",
                                          "w_up", "b_up", "w_down", "b_down")]


class LayerActs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("a", "mean1", "rstd1", "qkv", "o", "lse", "h", "b", "rstd2", "up",
                                          "s")]


class Ckpt(C.Structure):
    """An 8-bit checkpoint (``collider_ckpt``); see :func:`ckpt`."""
    _fields_ = [("format", C.c_int), ("code", C.c_void_p), ("exps", C.c_void_p), ("code_ld", C.c_size_t),
                ("exp_ld", C.c_size_t)]


class LayerSavedCkpt(C.Structure):
    _fields_ = ([("rows", C.c_int)] + [(n, Ckpt) for n in ("x", "a", "qkv", "o", "h", "up")] +
                [(n, C.c_void_p) for n in ("mean1", "rstd1", "lse", "rstd2")])


class ResidualNormDesc(C.Structure):
    _fields_ = [("dtype", C.c_int), ("B", C.c_int), ("T", C.c_int), ("D", C.c_int), ("norm", C.c_int),
                ("post", C.c_int), ("pre", C.c_int), ("eps", C.c_float), ("res_scale", C.c_float),
                ("gate_rows", C.c_int), ("x_ld", C.c_int), ("y_ld", C.c_int), ("h_ld", C.c_int), ("a_ld", C.c_int)]


class ResidualNormParams(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("post_w", "post_b", "gate", "res_w", "pre_w", "pre_b")]


class ResidualNormOut(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("h", "a", "mean_y", "rstd_y", "mean_h", "rstd_h")]


class ResidualNormSaved(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("h", C.c_void_p), ("y_ckpt", C.POINTER(Ckpt)),
                ("h_ckpt", C.POINTER(Ckpt)), ("mean_y", C.c_void_p), ("rstd_y", C.c_void_p), ("mean_h", C.c_void_p),
                ("rstd_h", C.c_void_p)]


class ResidualNormGrads(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dx", "dy", "dpost_w", "dpost_b", "dgate", "dres_w", "dpre_w", "dpre_b")]


class FfnDesc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("M", "D", "F", "act", "grad_dtype", "x_ld", "up_ld", "y_ld")]


class Grad(C.Structure):
    """One gradient of a list (``collider_grad``); see :func:`grad_list`."""
    _fields_ = [("data", C.c_void_p), ("n", C.c_longlong), ("dtype", C.c_int)]


P = C.c_void_p
I = C.c_int
SZ = C.c_size_t
# name -> (restype, argtypes)
_SIGS = {
    "collider_last_error": (C.c_char_p, []),
    "collider_check": (I, [P]),
    "collider_selftest_wait_timeout": (I, [P]),
    "collider_launch_count": (C.c_longlong, [I]),
    "collider_profile_enable": (I, [I]),
    "collider_profile_count": (I, []),
    "collider_profile_get": (I, [I, C.POINTER(C.c_char_p), C.POINTER(C.c_longlong), C.POINTER(C.c_float)]),
    "collider_profile_get_span": (I, [I, C.POINTER(C.c_float), C.POINTER(C.c_float), C.POINTER(C.c_int)]),
    "collider_select_keep": (I, [P, I, I, I, P, P]),
    "collider_compact_workspace_size": (SZ, [I, I]),
    "collider_compact": (I, [P, I, I, P, P, P, P, SZ, P]),
    "collider_compact_noalloc": (I, [P, I, I, P, P, P, P]),
    "collider_gather_rows": (I, [P, SZ, P, SZ, SZ, I, P, P, P]),
    "collider_scatter_rows": (I, [P, SZ, P, SZ, SZ, I, P, P, P]),
    "collider_linear_workspace_size": (SZ, [I, I, I, I]),
    "collider_linear_bwd": (I, [I, I, I, I, P, I, P, P, I, P, P, P, I, P, P, P, SZ, P]),
    "collider_ckpt_pack": (I, [I, P, SZ, I, I, P, P, C.POINTER(Ckpt), P]),
    "collider_ckpt_unpack": (I, [I, C.POINTER(Ckpt), I, I, I, P, P, P, SZ, I, P]),
    "collider_linear_ckpt_workspace_size": (SZ, [I, I, I]),
    "collider_linear_bwd_ckpt": (I, [I, I, I, C.POINTER(Ckpt), I, P, P, I, P, P, P, I, P, P, P, SZ, P]),
    "collider_layer_ckpt_workspace_size": (SZ, [C.POINTER(LayerDesc)]),
    "collider_layer_bwd_ckpt": (I, [C.POINTER(LayerDesc), C.POINTER(LayerWeights), C.POINTER(LayerSavedCkpt), P, I,
                                    P, P, P, C.POINTER(LayerGrads), I, P, SZ, P]),
    "collider_residual_norm_fwd": (I, [C.POINTER(ResidualNormDesc), C.POINTER(ResidualNormParams), P, P,
                                       C.POINTER(ResidualNormOut), P]),
    "collider_residual_norm_bwd_workspace_size": (SZ, [C.POINTER(ResidualNormDesc)]),
    "collider_residual_norm_bwd": (I, [C.POINTER(ResidualNormDesc), C.POINTER(ResidualNormParams),
                                       C.POINTER(ResidualNormSaved), I, P, P, I, P, P, P,
                                       C.POINTER(ResidualNormGrads), I, P, SZ, P]),
    "collider_attn_workspace_size": (SZ, [I, I, I, I, I]),
    "collider_attn_bwd": (I, [I, I, I, I, I, I, C.c_float, I, C.c_float, P, P, P, P, P, I, I, I, I, P,
                              P, P, P, P, P, P, I, P, SZ, P]),
    "collider_layer_workspace_size": (SZ, [C.POINTER(LayerDesc)]),
    "collider_layer_bwd": (I, [C.POINTER(LayerDesc), C.POINTER(LayerWeights), C.POINTER(LayerSaved), P, I,
                               P, P, P, C.POINTER(LayerGrads), I, P, SZ, P]),
    "collider_layer_fwd_workspace_size": (SZ, [C.POINTER(LayerDesc)]),
    "collider_layer_fwd": (I, [C.POINTER(LayerDesc), C.POINTER(LayerParams), P, P, C.POINTER(LayerActs), P, SZ,
                               P]),
    "collider_stack_workspace_size": (SZ, [C.POINTER(LayerDesc), I, I]),
    "collider_stack_bwd": (I, [C.POINTER(LayerDesc), I, I, C.POINTER(LayerWeights), C.POINTER(LayerSaved),
                               P, P, P, P, P, P, P, P, P, P, P, C.POINTER(LayerGrads), P, P, P, P, SZ, P]),
    "collider_ffn_fwd_workspace_size": (SZ, [C.POINTER(FfnDesc)]),
    "collider_ffn_fwd": (I, [C.POINTER(FfnDesc), P, P, P, P, P, P, SZ, P]),
    "collider_ffn_bwd_workspace_size": (SZ, [C.POINTER(FfnDesc)]),
    "collider_ffn_bwd": (I, [C.POINTER(FfnDesc), P, P, P, P, I, P, I, P, P, P, I, P, P, P, SZ, P]),
    "collider_grad_norm_workspace_size": (SZ, [C.POINTER(Grad), I]),
    "collider_grad_norm": (I, [C.POINTER(Grad), I, I, C.c_float, P, P, P, SZ, P]),
    "collider_grad_clip": (I, [C.POINTER(Grad), I, I, C.c_float, C.c_float, P, P, P, P, SZ, P]),
}
EXPORTED = tuple(_SIGS)

_lib = None


def lib() -> C.CDLL:
    """Load libcollider.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_backward_gemm_gb300.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(s):
    if s is None:
        import torch
        # (0.3 us a call against 2.9 with a Stream object; the function is not public, so it may be missing)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int):
    if status != OK:
        raise ColliderError(status, lib().collider_last_error().decode())


def _nbytes(ws):
    if ws is None:
        return 0
    if hasattr(ws, "numel"):
        return ws.numel() * ws.element_size()
    raise TypeError("pass the workspace as a tensor (its size is taken from it)")


# --------------------------------------------------------------------------
def collider_last_error() -> str:
    return lib().collider_last_error().decode()


def collider_check(stream=None) -> None:
    _check(lib().collider_check(_stream(stream)))


def collider_selftest_wait_timeout(stream=None) -> None:
    _check(lib().collider_selftest_wait_timeout(_stream(stream)))


def collider_launch_count(reset: int = 0) -> int:
    return lib().collider_launch_count(reset)


def collider_profile_enable(on: int) -> None:
    lib().collider_profile_enable(int(on))


def collider_profile_count() -> int:
    return lib().collider_profile_count()


def collider_profile_get_span(i: int):
    """Returns (start_ms, end_ms, stream_index) of profile record i on the timeline of record 0."""
    a, b, k = C.c_float(), C.c_float(), C.c_int()
    if lib().collider_profile_get_span(i, C.byref(a), C.byref(b), C.byref(k)) != 0:
        raise IndexError(i)
    return a.value, b.value, k.value


def collider_profile_get(i: int):
    """Returns (name, (M, N, K, dyn), ms) of profile record i."""
    name = C.c_char_p()
    mnk = (C.c_longlong * 4)()
    ms = C.c_float()
    if lib().collider_profile_get(i, C.byref(name), mnk, C.byref(ms)) != 0:
        raise IndexError(i)
    return name.value.decode(), tuple(mnk), ms.value


def collider_select_keep(scores, B, T, n_filter, mask, stream=None) -> None:
    _check(lib().collider_select_keep(_ptr(scores), B, T, n_filter, _ptr(mask), _stream(stream)))


def collider_compact_workspace_size(B: int, T: int) -> int:
    return lib().collider_compact_workspace_size(B, T)


def collider_compact(mask, B, T, idx, cu_kept, n_kept, ws=None, stream=None) -> None:
    _check(lib().collider_compact(_ptr(mask), B, T, _ptr(idx), _ptr(cu_kept), _ptr(n_kept), _ptr(ws),
                                  _nbytes(ws), _stream(stream)))


def collider_compact_noalloc(mask, B, T, idx, cu_kept, n_kept, stream=None) -> None:
    """collider_compact without a workspace and without any allocation (scratch
    is a fixed array inside the library; B*T <= 2^30)."""
    _check(lib().collider_compact_noalloc(_ptr(mask), B, T, _ptr(idx), _ptr(cu_kept), _ptr(n_kept),
                                          _stream(stream)))


def collider_gather_rows(src, src_ld_bytes, dst, dst_ld_bytes, row_bytes, M, idx, n_kept, stream=None) -> None:
    _check(lib().collider_gather_rows(_ptr(src), src_ld_bytes, _ptr(dst), dst_ld_bytes, row_bytes, M, _ptr(idx),
                                      _ptr(n_kept), _stream(stream)))


def collider_scatter_rows(compact, compact_ld_bytes, full, full_ld_bytes, row_bytes, M, idx, n_kept,
                          stream=None) -> None:
    _check(lib().collider_scatter_rows(_ptr(compact), compact_ld_bytes, _ptr(full), full_ld_bytes, row_bytes, M,
                                       _ptr(idx), _ptr(n_kept), _stream(stream)))


def collider_linear_workspace_size(dtype, M, K, N) -> int:
    return lib().collider_linear_workspace_size(dtype, M, K, N)


def collider_linear_bwd(dtype, M, K, N, X, x_rows, W, dY, dy_rows, idx, n_kept, dX, dx_rows, dW, db, ws,
                        stream=None) -> None:
    _check(lib().collider_linear_bwd(dtype, M, K, N, _ptr(X), x_rows, _ptr(W), _ptr(dY), dy_rows, _ptr(idx),
                                     _ptr(n_kept), _ptr(dX), dx_rows, _ptr(dW), _ptr(db), _ptr(ws), _nbytes(ws),
                                     _stream(stream)))


def _filled(struct, tensors):
    """The struct with these buffers' addresses; it keeps the buffers alive."""
    unknown = set(tensors) - {f[0] for f in struct._fields_}
    if unknown:
        raise TypeError(f"{struct.__name__} has no field {sorted(unknown)[0]}")
    s = struct()
    s.buffers = tensors
    for k, v in tensors.items():
        if isinstance(v, Ckpt):
            setattr(s, k, C.pointer(v))
        elif v is not None:
            setattr(s, k, _ptr(v))
    return s


def ckpt(format, code, exps) -> Ckpt:
    """The 8-bit checkpoint whose codes and exponent bytes are the rows of two uint8 tensors ``[rows, N]`` and
    ``[rows, N // 32]`` (a row's bytes adjacent)."""
    for t in (code, exps):
        if t.dim() != 2 or t.element_size() != 1 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise TypeError("codes and exponents are 2-D tensors of bytes, a row's bytes adjacent")
    q = Ckpt(format=format, code=code.data_ptr(), exps=exps.data_ptr(), code_ld=code.stride(0), exp_ld=exps.stride(0))
    q.buffers = (code, exps)
    return q


def layer_saved_ckpt(rows, **fields) -> LayerSavedCkpt:
    """LayerSavedCkpt from :func:`ckpt` checkpoints (x, qkv, o, up, h or a) and f32 tensors (rstd1, lse, ...)."""
    s = LayerSavedCkpt(rows=rows)
    s.buffers = fields
    for k, v in fields.items():
        if k not in {f[0] for f in LayerSavedCkpt._fields_}:
            raise TypeError(f"LayerSavedCkpt has no field {k}")
        if v is not None:
            setattr(s, k, v if isinstance(v, Ckpt) else _ptr(v))
    return s


def residual_norm_params(**tensors) -> ResidualNormParams:
    """ResidualNormParams from tensors by field name (None or absent: NULL)."""
    return _filled(ResidualNormParams, tensors)


def residual_norm_out(**tensors) -> ResidualNormOut:
    return _filled(ResidualNormOut, tensors)


def residual_norm_saved(**tensors) -> ResidualNormSaved:
    """ResidualNormSaved from tensors and :func:`ckpt` checkpoints (y_ckpt, h_ckpt) by field name."""
    return _filled(ResidualNormSaved, tensors)


def residual_norm_grads(**tensors) -> ResidualNormGrads:
    return _filled(ResidualNormGrads, tensors)


def collider_ckpt_pack(dtype, src, src_ld, M, N, idx, n_kept, out, stream=None) -> None:
    _check(lib().collider_ckpt_pack(dtype, _ptr(src), src_ld, M, N, _ptr(idx), _ptr(n_kept), C.byref(out),
                                  _stream(stream)))


def collider_ckpt_unpack(dtype, src, src_rows, M, N, idx, n_kept, dst, dst_ld, dst_rows, stream=None) -> None:
    _check(lib().collider_ckpt_unpack(dtype, C.byref(src), src_rows, M, N, _ptr(idx), _ptr(n_kept), _ptr(dst), dst_ld,
                                    dst_rows, _stream(stream)))


def collider_linear_ckpt_workspace_size(M, K, N) -> int:
    return lib().collider_linear_ckpt_workspace_size(M, K, N)


def collider_linear_bwd_ckpt(M, K, N, X, x_rows, W, dY, dy_rows, idx, n_kept, dX, dx_rows, dW, db, ws,
                           stream=None) -> None:
    _check(lib().collider_linear_bwd_ckpt(M, K, N, None if X is None else C.byref(X), x_rows, _ptr(W), _ptr(dY), dy_rows,
                                        _ptr(idx), _ptr(n_kept), _ptr(dX), dx_rows, _ptr(dW), _ptr(db), _ptr(ws),
                                        _nbytes(ws), _stream(stream)))


def collider_residual_norm_fwd(desc, params, x, y, out, stream=None) -> None:
    _check(lib().collider_residual_norm_fwd(C.byref(desc), C.byref(params), _ptr(x), _ptr(y), C.byref(out),
                                            _stream(stream)))


def collider_residual_norm_bwd_workspace_size(desc) -> int:
    return lib().collider_residual_norm_bwd_workspace_size(C.byref(desc))


def collider_residual_norm_bwd(desc, params, saved, saved_rows, da, dh, in_rows, idx, cu_kept, n_kept, grads, out_rows,
                               ws, stream=None) -> None:
    _check(lib().collider_residual_norm_bwd(C.byref(desc), C.byref(params), C.byref(saved), saved_rows, _ptr(da),
                                            _ptr(dh), in_rows, _ptr(idx), _ptr(cu_kept), _ptr(n_kept), C.byref(grads),
                                            out_rows, _ptr(ws), _nbytes(ws), _stream(stream)))


def collider_attn_workspace_size(B, T, H, Hkv, dh) -> int:
    return lib().collider_attn_workspace_size(B, T, H, Hkv, dh)


def collider_attn_bwd(B, T, H, Hkv, dh, causal, scale, rotary_dim, rope_base, Q, K, V, O, dO, q_ld, kv_ld, do_ld,
                      in_rows, lse, idx, cu_kept, n_kept, dQ, dK, dV, out_rows, ws, stream=None) -> None:
    _check(lib().collider_attn_bwd(B, T, H, Hkv, dh, causal, scale, rotary_dim, rope_base, _ptr(Q), _ptr(K),
                                   _ptr(V), _ptr(O), _ptr(dO), q_ld, kv_ld, do_ld, in_rows, _ptr(lse), _ptr(idx),
                                   _ptr(cu_kept), _ptr(n_kept), _ptr(dQ), _ptr(dK), _ptr(dV), out_rows, _ptr(ws),
                                   _nbytes(ws), _stream(stream)))


def collider_layer_workspace_size(desc: LayerDesc) -> int:
    return lib().collider_layer_workspace_size(C.byref(desc))


def collider_layer_bwd(desc, weights, saved, dOut, dout_rows, idx, cu_kept, n_kept, grads, dx_rows, ws,
                       stream=None) -> None:
    _check(lib().collider_layer_bwd(C.byref(desc), C.byref(weights), C.byref(saved), _ptr(dOut), dout_rows,
                                    _ptr(idx), _ptr(cu_kept), _ptr(n_kept), C.byref(grads), dx_rows, _ptr(ws),
                                    _nbytes(ws), _stream(stream)))


def collider_layer_ckpt_workspace_size(desc: LayerDesc) -> int:
    return lib().collider_layer_ckpt_workspace_size(C.byref(desc))


def collider_layer_bwd_ckpt(desc, weights, saved, dOut, dout_rows, idx, cu_kept, n_kept, grads, dx_rows, ws,
                            stream=None) -> None:
    _check(lib().collider_layer_bwd_ckpt(C.byref(desc), C.byref(weights), C.byref(saved), _ptr(dOut), dout_rows,
                                         _ptr(idx), _ptr(cu_kept), _ptr(n_kept), C.byref(grads), dx_rows, _ptr(ws),
                                         _nbytes(ws), _stream(stream)))


def collider_layer_fwd_workspace_size(desc: LayerDesc) -> int:
    return lib().collider_layer_fwd_workspace_size(C.byref(desc))


def collider_layer_fwd(desc, params, x, y, acts, ws, stream=None) -> None:
    _check(lib().collider_layer_fwd(C.byref(desc), C.byref(params), _ptr(x), _ptr(y), C.byref(acts), _ptr(ws),
                                    _nbytes(ws), _stream(stream)))


def collider_stack_workspace_size(desc: LayerDesc, L: int, V: int) -> int:
    return lib().collider_stack_workspace_size(C.byref(desc), L, V)


def collider_stack_bwd(desc, L, V, weights, saved, logits, targets, ids, y, xL, rstdf, normf_w, w_lm, idx,
                       cu_kept, n_kept, grads, dnormf_w, dw_lm, dE, ws, stream=None) -> None:
    """weights / saved / grads: ctypes arrays of LayerWeights / LayerSaved / LayerGrads (length L)."""
    _check(lib().collider_stack_bwd(C.byref(desc), L, V, weights, saved, _ptr(logits), _ptr(targets), _ptr(ids),
                                    _ptr(y), _ptr(xL), _ptr(rstdf), _ptr(normf_w), _ptr(w_lm), _ptr(idx),
                                    _ptr(cu_kept), _ptr(n_kept), grads, _ptr(dnormf_w), _ptr(dw_lm), _ptr(dE),
                                    _ptr(ws), _nbytes(ws), _stream(stream)))


def collider_ffn_fwd_workspace_size(desc: FfnDesc) -> int:
    return lib().collider_ffn_fwd_workspace_size(C.byref(desc))


def collider_ffn_fwd(desc, x, w_up, w_down, up, y, ws, stream=None) -> None:
    _check(lib().collider_ffn_fwd(C.byref(desc), _ptr(x), _ptr(w_up), _ptr(w_down), _ptr(up), _ptr(y), _ptr(ws),
                                  _nbytes(ws), _stream(stream)))


def collider_ffn_bwd_workspace_size(desc: FfnDesc) -> int:
    return lib().collider_ffn_bwd_workspace_size(C.byref(desc))


def collider_ffn_bwd(desc, w_up, w_down, x, up, saved_rows, dy, dy_rows, idx, n_kept, dx, dx_rows, dw_up, dw_down, ws,
                     stream=None) -> None:
    _check(lib().collider_ffn_bwd(C.byref(desc), _ptr(w_up), _ptr(w_down), _ptr(x), _ptr(up), saved_rows, _ptr(dy),
                                  dy_rows, _ptr(idx), _ptr(n_kept), _ptr(dx), dx_rows, _ptr(dw_up), _ptr(dw_down),
                                  _ptr(ws), _nbytes(ws), _stream(stream)))


def grad_list(tensors):
    """The array of :class:`Grad` of these contiguous f32 or bf16 tensors; it keeps them alive."""
    import torch
    dtypes = {torch.float32: F32, torch.bfloat16: BF16}
    for t in tensors:
        if t.dtype not in dtypes or not t.is_contiguous():
            raise TypeError("gradients are contiguous f32 or bf16 tensors")
    a = (Grad * len(tensors))(*[Grad(t.data_ptr(), t.numel(), dtypes[t.dtype]) for t in tensors])
    a.buffers = tuple(tensors)
    return a


def collider_grad_norm_workspace_size(grads, count) -> int:
    return lib().collider_grad_norm_workspace_size(grads, count)


def _listed(grads, count):
    if isinstance(grads, C.Array) and count > len(grads):
        raise ColliderError(ERR_INVALID_ARG, f"a count of {count} gradients beyond a list of {len(grads)}")


def collider_grad_norm(grads, count, kind, scale, norm, norms, ws, stream=None) -> None:
    _listed(grads, count)
    _check(lib().collider_grad_norm(grads, count, kind, scale, _ptr(norm), _ptr(norms), _ptr(ws), _nbytes(ws),
                                    _stream(stream)))


def collider_grad_clip(grads, count, kind, scale, max_norm, norm, norms, coef, ws, stream=None) -> None:
    _listed(grads, count)
    _check(lib().collider_grad_clip(grads, count, kind, scale, max_norm, _ptr(norm), _ptr(norms), _ptr(coef), _ptr(ws),
                                    _nbytes(ws), _stream(stream)))
