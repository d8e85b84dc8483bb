"""Thin ctypes binding over librmsnorm.so (C ABI in include/rmsnorm.h).

Same entry-point names as the C ABI. Argument marshalling only: tensors are
checked (CUDA, contiguous or row-strided, dtype, shape), outputs that the
caller did not pass are allocated with torch, and raw device pointers, row
strides and the current torch CUDA stream are handed to the library. Every arithmetic step runs in the
CUDA kernels. If the library has not been built this module raises at load
time; there is no fallback. The 8-bit calls and those on attention heads are
marshalled in C++ (csrc/fp8/fp8_torch.cpp, csrc/heads/heads_torch.cpp) for
their time on the host.
"""
import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "librmsnorm.so")

RMSNORM_F32, RMSNORM_BF16, RMSNORM_F16 = 0, 1, 2
DTYPES = {torch.float32: RMSNORM_F32, torch.bfloat16: RMSNORM_BF16,
          torch.float16: RMSNORM_F16}
MAX_H = 16384
PATH_AUTO, PATH_ROWS, PATH_SPLIT, PATH_SCALAR, PATH_STREAM = 0, 1, 2, 3, 4
PATH_GEMV = 5            # reported by last_path() after rmsnorm_gemv_fwd: the
PATH_GEMV_TMA = 6        # weight in registers (5), fed by bulk copies (6), or
PATH_GEMV_UMMA = 7       # the product on tcgen05 (7); 6 and 7 also force it
PATH_GEMV_TC = 8         # persistent tcgen05 kernel, y held per CTA (8; forces it)
PATH_FP8_ROWS, PATH_FP8_BLOCKS = 9, 10            # reported only
PATH_FP8_GEMM, PATH_FP8_PAIR = 11, 12             # the 8-bit product's kernels
PATH_ROPE, PATH_ROPE_APPEND, PATH_KV4_READ = 13, 14, 15                  # reported only
PATH_KV4_ATTENTION, PATH_KV4_PROMPT = 16, 17

# Entry points of include/rmsnorm.h with their ctypes signatures.
_i64, _vp, _sz, _int, _f = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                            ctypes.c_int, ctypes.c_float)
SIGNATURES = {
    "rmsnorm_fwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i64, _i64,
                           _f, _int, _vp]),
    "rmsnorm_residual_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                    _f, _int, _vp]),
    "rmsnorm_residual_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _sz, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_bwd_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "rmsnorm_status_string": (ctypes.c_char_p, [_int]),
    "rmsnorm_last_cuda_error": (_int, []),
    "rmsnorm_set_path_override": (None, [_int]),
    "rmsnorm_last_path": (_int, []),
    "rmsnorm_bwd_static_scratch": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                          _i64, _f, _int, _vp]),
    "rmsnorm_set_static_scratch_test_limit": (None, [_sz]),
    "rmsnorm_wait_timeouts": (_int, [ctypes.POINTER(ctypes.c_uint), _int]),
    "rmsnorm_set_stream_test_fault": (None, [ctypes.c_uint, ctypes.c_uint]),
    "rmsnorm_set_gemv_cluster_test": (None, [_int]),
    "rmsnorm_bwd_ex": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i64,
                              _i64, _f, _int, _int, _vp]),
    "rmsnorm_fwd_strided": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp,
                                   _i64, _vp, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_bwd_strided": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp,
                                   _vp, _i64, _vp, _vp, _sz, _i64, _i64, _f,
                                   _int, _int, _vp]),
    "rmsnorm_bwd_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _sz, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_gemv_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                _i64, _i64, _f, _int, _int, _vp]),
    "rmsnorm_fwd_fp8": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp,
                               _i64, _vp, _i64, _i64, _f, _int, _int, _vp]),
    "rmsnorm_quant_fp8": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _int,
                                 _int, _int, _vp]),
    "rmsnorm_set_gemm_fp8_test": (None, [_int]),
    "rmsnorm_gemm_fp8": (_int, [_vp, _i64, _vp, _int, _vp, _i64, _vp, _int, _vp,
                                _i64, _i64, _i64, _i64, _int, _int, _vp]),
}

SIGNATURES.update({
    "rmsnorm_rope_fwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_rope_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _sz, _i64, _i64, _f, _int, _vp]),
    "rmsnorm_rope_bwd_workspace_bytes": (_sz, [_i64]),
    "rmsnorm_rope_append": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _i64, _i64,
                                   _i64, _f, _int, _vp]),
    "rmsnorm_rope_append_kv4": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _vp, _vp,
                                       _i64, _i64, _f, _int, _vp]),
    "rmsnorm_kv4_attention": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64,
                                     _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64,
                                     _f, _vp, _sz, _int, _vp]),
    "rmsnorm_kv4_attention_workspace_bytes": (_sz, [_i64]),
    "rmsnorm_set_kv4_test": (None, [_int]),
    "rmsnorm_kv4_read": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _int, _i64, _vp, _vp, _vp, _vp,
                                _vp]),
})

BWD_ACCUMULATE_DW = 1


class RmsNormError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().rmsnorm_status_string(status).decode()
        if status == -8:
            msg += f" (cudaError {lib().rmsnorm_last_cuda_error()})"
        super().__init__(f"{where}: status {status}: {msg}")


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "(there is no CPU fallback)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(status, where):
    if status != 0:
        raise RmsNormError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _rows(name, t, H, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[-1] != H:
        raise ValueError(f"{name} last dim must be {H}")
    return t.numel() // H if H else 0


def _strided(name, t, H, dtype=None):
    """(M, ld) of a 2-D [M, H] CUDA tensor with unit column stride; ld is its
    row stride in elements (H for one row)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or t.shape[1] != H:
        raise ValueError(f"{name} must be 2-D [M, {H}]")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    M = t.shape[0]
    if H > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = t.stride(0) if M > 1 else H
    return M, ld


def as_rows(t, H):
    """t viewed as [M, H] rows without a copy when its strides allow it
    (any row stride, unit column stride), else a contiguous copy."""
    if t.shape[-1] == H and (H == 1 or t.stride(-1) == 1):
        try:
            return t.view(-1, H)
        except RuntimeError:
            pass
    return t.contiguous().view(-1, H)


def _dtype_code(t):
    if t.dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return DTYPES[t.dtype]


def set_path_override(path: int):
    lib().rmsnorm_set_path_override(int(path))


def last_path() -> int:
    return lib().rmsnorm_last_path()


def wait_timeouts(reset: bool = False) -> int:
    """Streamed-kernel waits that ran out on the current device (0 when all
    is well); synchronous diagnostic."""
    c = ctypes.c_uint(0)
    _check(lib().rmsnorm_wait_timeouts(ctypes.byref(c), int(reset)),
           "rmsnorm_wait_timeouts")
    return int(c.value)


def set_stream_test_fault(extra_tx_bytes: int, wait_limit_us: int):
    """Test hook: make the streamed kernels' waits run out (see rmsnorm.h)."""
    lib().rmsnorm_set_stream_test_fault(int(extra_tx_bytes), int(wait_limit_us))


def set_gemv_cluster_test(cluster_size: int):
    """Test hook: force the persistent projection kernel's cluster size (0:
    the plan's choice; see rmsnorm.h)."""
    lib().rmsnorm_set_gemv_cluster_test(int(cluster_size))


def bwd_workspace_bytes(M: int, H: int, dtype: torch.dtype) -> int:
    return lib().rmsnorm_bwd_workspace_bytes(int(M), int(H), DTYPES[dtype])


def rmsnorm_fwd(x, w, y=None, rstd=None, eps=1e-6, want_rstd=True, stream=None):
    """y = RMSNorm(x) * w over the last dim; returns (y, rstd or None)."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("w", w.view(-1), H, x.dtype)
    if y is None:
        y = torch.empty_like(x)
    _rows("y", y, H, x.dtype)
    if rstd is None and want_rstd:
        rstd = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    if rstd is not None and rstd.dtype != torch.float32:
        raise ValueError("rstd must be float32")
    _check(lib().rmsnorm_fwd(_ptr(x), _ptr(w), _ptr(y), _ptr(rstd), M, H,
                             float(eps), _dtype_code(x), _stream(stream)),
           "rmsnorm_fwd")
    return y, rstd


def rmsnorm_bwd(dy, x, w, rstd=None, dx=None, dw=None, workspace=None,
                eps=1e-6, stream=None):
    """(dx, dw) of the RMSNorm; rstd=None recomputes it from x."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("dy", dy, H, x.dtype)
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        dw = torch.empty(H, device=x.device, dtype=torch.float32)
    need = bwd_workspace_bytes(M, H, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    _check(lib().rmsnorm_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dx),
                             _ptr(dw), _ptr(workspace), workspace.numel()
                             * workspace.element_size(), M, H, float(eps),
                             _dtype_code(x), _stream(stream)), "rmsnorm_bwd")
    return dx, dw


def rmsnorm_residual_fwd(x, r, w, h=None, y=None, rstd=None, eps=1e-6,
                         want_rstd=True, stream=None):
    """h = x + r (rounded to the dtype), y = RMSNorm(h) * w; returns
    (h, y, rstd or None)."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("r", r, H, x.dtype)
    if h is None:
        h = torch.empty_like(x)
    if y is None:
        y = torch.empty_like(x)
    if rstd is None and want_rstd:
        rstd = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    _check(lib().rmsnorm_residual_fwd(_ptr(x), _ptr(r), _ptr(w), _ptr(h),
                                      _ptr(y), _ptr(rstd), M, H, float(eps),
                                      _dtype_code(x), _stream(stream)),
           "rmsnorm_residual_fwd")
    return h, y, rstd


def rmsnorm_residual_bwd(dy, dh_out, h, w, rstd=None, dx=None, dw=None,
                         workspace=None, eps=1e-6, stream=None):
    """(dx, dw): dx is the gradient of both the input and the residual."""
    H = w.numel()
    M = _rows("h", h, H)
    _rows("dy", dy, H, h.dtype)
    if dh_out is not None:
        _rows("dh_out", dh_out, H, h.dtype)
    if dx is None:
        dx = torch.empty_like(h)
    if dw is None:
        dw = torch.empty(H, device=h.device, dtype=torch.float32)
    need = bwd_workspace_bytes(M, H, h.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=h.device, dtype=torch.uint8)
    _check(lib().rmsnorm_residual_bwd(
        _ptr(dy), _ptr(dh_out), _ptr(h), _ptr(w), _ptr(rstd), _ptr(dx),
        _ptr(dw), _ptr(workspace), workspace.numel() * workspace.element_size(),
        M, H, float(eps), _dtype_code(h), _stream(stream)),
        "rmsnorm_residual_bwd")
    return dx, dw


def rmsnorm_bwd_ex(dy, x, w, rstd=None, dh_out=None, dx=None, dw=None,
                   workspace=None, eps=1e-6, accumulate_dw=False, stream=None):
    """(dx, dw) of the plain (dh_out None) or residual backward; with
    accumulate_dw the call adds its dw into the given dw buffer."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("dy", dy, H, x.dtype)
    if dh_out is not None:
        _rows("dh_out", dh_out, H, x.dtype)
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        if accumulate_dw:
            raise ValueError("accumulate_dw needs the dw buffer to add into")
        dw = torch.empty(H, device=x.device, dtype=torch.float32)
    need = bwd_workspace_bytes(M, H, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    _check(lib().rmsnorm_bwd_ex(
        _ptr(dy), _ptr(dh_out), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dx), _ptr(dw),
        _ptr(workspace), workspace.numel() * workspace.element_size(), M, H,
        float(eps), _dtype_code(x), BWD_ACCUMULATE_DW if accumulate_dw else 0,
        _stream(stream)), "rmsnorm_bwd_ex")
    return dx, dw


def rmsnorm_fwd_strided(x, w, y=None, r=None, h=None, rstd=None, eps=1e-6,
                        want_rstd=True, stream=None):
    """Forward on row-strided 2-D tensors (each with its own row stride).
    Without r: returns (y, rstd); with r (residual variant): (h, y, rstd).
    Outputs the caller does not pass are allocated dense."""
    H = w.numel()
    M, ldx = _strided("x", x, H)
    _rows("w", w.view(-1), H, x.dtype)
    if y is None:
        y = torch.empty(M, H, device=x.device, dtype=x.dtype)
    _, ldy = _strided("y", y, H, x.dtype)
    ldr = ldh = H
    if r is not None:
        _, ldr = _strided("r", r, H, x.dtype)
        if h is None:
            h = torch.empty(M, H, device=x.device, dtype=x.dtype)
        _, ldh = _strided("h", h, H, x.dtype)
    elif h is not None:
        raise ValueError("h is the residual variant's output: pass r too")
    if rstd is None and want_rstd:
        rstd = torch.empty(M, device=x.device, dtype=torch.float32)
    _check(lib().rmsnorm_fwd_strided(
        _ptr(x), ldx, _ptr(r), ldr, _ptr(w), _ptr(y), ldy, _ptr(h), ldh,
        _ptr(rstd), M, H, float(eps), _dtype_code(x), _stream(stream)),
        "rmsnorm_fwd_strided")
    return (y, rstd) if r is None else (h, y, rstd)


def rmsnorm_bwd_strided(dy, x, w, rstd=None, dh_out=None, dx=None, dw=None,
                        workspace=None, eps=1e-6, accumulate_dw=False,
                        stream=None):
    """(dx, dw) of the plain (dh_out None) or residual backward on row-strided
    2-D tensors; dx is allocated dense unless given."""
    H = w.numel()
    M, ldx = _strided("x", x, H)
    _, lddy = _strided("dy", dy, H, x.dtype)
    lddh = H
    if dh_out is not None:
        _, lddh = _strided("dh_out", dh_out, H, x.dtype)
    if dx is None:
        dx = torch.empty(M, H, device=x.device, dtype=x.dtype)
    _, lddx = _strided("dx", dx, H, x.dtype)
    if dw is None:
        if accumulate_dw:
            raise ValueError("accumulate_dw needs the dw buffer to add into")
        dw = torch.empty(H, device=x.device, dtype=torch.float32)
    need = bwd_workspace_bytes(M, H, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    _check(lib().rmsnorm_bwd_strided(
        _ptr(dy), lddy, _ptr(dh_out), lddh, _ptr(x), ldx, _ptr(w), _ptr(rstd),
        _ptr(dx), lddx, _ptr(dw), _ptr(workspace),
        workspace.numel() * workspace.element_size(), M, H, float(eps),
        _dtype_code(x), BWD_ACCUMULATE_DW if accumulate_dw else 0,
        _stream(stream)), "rmsnorm_bwd_strided")
    return dx, dw


def rmsnorm_bwd_bwd(dy, x, w, rstd=None, gdx=None, gdw=None, ddy=None, dx2=None,
                    dw2=None, workspace=None, eps=1e-6, stream=None):
    """(ddy, dx2, dw2): gradients of sum(gdx * dx) + sum(gdw * dw) with
    respect to the backward's dy, x and w (see rmsnorm.h). gdx in x's dtype
    or None, gdw float32 or None; dw2 is float32."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("dy", dy, H, x.dtype)
    if gdx is not None:
        _rows("gdx", gdx, H, x.dtype)
    if gdw is not None and (gdw.dtype != torch.float32 or not gdw.is_contiguous()):
        raise ValueError("gdw must be a contiguous float32 tensor")
    if ddy is None:
        ddy = torch.empty_like(x)
    if dx2 is None:
        dx2 = torch.empty_like(x)
    if dw2 is None:
        dw2 = torch.empty(H, device=x.device, dtype=torch.float32)
    need = bwd_workspace_bytes(M, H, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    _check(lib().rmsnorm_bwd_bwd(
        _ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(gdx), _ptr(gdw), _ptr(ddy),
        _ptr(dx2), _ptr(dw2), _ptr(workspace),
        workspace.numel() * workspace.element_size(), M, H, float(eps),
        _dtype_code(x), _stream(stream)), "rmsnorm_bwd_bwd")
    return ddy, dx2, dw2


GEMV_STATIC_WEIGHTS = 1


def rmsnorm_gemv_fwd(x, w, A, r=None, out=None, h=None, want_h=True, y=None,
                     rstd=None, eps=1e-6, static_weights=False, stream=None):
    """out = round(RMSNorm(x [+ r]) * w) @ A^T for decode-sized x [M, H]
    (M <= 64) and a row-major weight A [N, H]. Returns (out, h or None,
    rstd or None); y (the norm's output) is written only into a given
    buffer. With r, h (the residual sum) is allocated unless want_h is
    False. static_weights: nothing in flight on the stream writes w or A
    (see RMSNORM_GEMV_STATIC_WEIGHTS)."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("w", w.view(-1), H, x.dtype)
    if A.dim() != 2:
        raise ValueError("A must be 2-D [N, H]")
    N = _rows("A", A, H, x.dtype)
    if r is not None:
        _rows("r", r, H, x.dtype)
        if h is None and want_h:
            h = torch.empty_like(x)
    elif h is not None:
        raise ValueError("h is the residual variant's output: pass r too")
    if out is None:
        out = torch.empty(x.shape[:-1] + (N,), device=x.device, dtype=x.dtype)
    _rows("out", out, N, x.dtype)
    if y is not None:
        _rows("y", y, H, x.dtype)
    _check(lib().rmsnorm_gemv_fwd(
        _ptr(x), _ptr(r), _ptr(w), _ptr(A), _ptr(out), _ptr(h), _ptr(y),
        _ptr(rstd), M, H, N, float(eps), _dtype_code(x),
        GEMV_STATIC_WEIGHTS if static_weights else 0, _stream(stream)),
        "rmsnorm_gemv_fwd")
    return out, h, rstd


FP8_GROUP = 128
FP8_TYPES = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}   # rmsnorm_fp8_type
FP8_MAX_K, FP8_MAX_ROWS = 1 << 24, 1 << 30
GEMM_FP8_STATIC_WEIGHTS = 1


# The 8-bit calls of a decode step, and those on its heads, run for 2 to 4 us
# on the GPU. Their checks, output allocation and marshalling are in small C++
# modules over the C ABI (csrc/fp8/fp8_torch.cpp, csrc/heads/heads_torch.cpp);
# in Python they took 13 to 18 us a call.
FP8_LIB_PATH = os.path.join(PKG, "_fp8_torch.so")
HEADS_LIB_PATH = os.path.join(PKG, "_heads_torch.so")
_fp8_mod = _heads_mod = None


def _binding(path, functions):
    """The loaded binding at `path`, handed the library's functions (raises if
    it was not built)."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(there is no CPU fallback)")
    name = os.path.basename(path)[:-3]
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
    loader.exec_module(mod)
    mod.init(*(ctypes.cast(getattr(lib(), f), _vp).value for f in functions), _check)
    return mod


def _fp8():
    global _fp8_mod
    if _fp8_mod is None:
        _fp8_mod = _binding(FP8_LIB_PATH, ("rmsnorm_fwd_fp8", "rmsnorm_quant_fp8", "rmsnorm_gemm_fp8"))
    return _fp8_mod


def _heads():
    global _heads_mod
    if _heads_mod is None:
        _heads_mod = _binding(HEADS_LIB_PATH, (
            "rmsnorm_rope_fwd", "rmsnorm_rope_bwd", "rmsnorm_rope_bwd_workspace_bytes",
            "rmsnorm_rope_append", "rmsnorm_rope_append_kv4", "rmsnorm_kv4_read",
            "rmsnorm_kv4_attention", "rmsnorm_kv4_attention_workspace_bytes"))
    return _heads_mod


def _on_stream(t, stream):
    """The context in which a call on tensor t runs on `stream`: what the
    binding allocates then belongs to that stream."""
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def rmsnorm_fwd_fp8(x, w, r=None, q=None, scale=None, h=None, rstd=None, eps=1e-6,
                    qdtype=torch.float8_e4m3fn, want_rstd=True, stream=None):
    """RMSNorm(x [+ r]) * w rounded to 8 bits, with one fp32 scale for each
    128 columns of a row (see rmsnorm.h). x [M, H] with any row stride.
    Returns (q, scale, rstd or None), with r (h, q, scale, rstd or None). q
    is [M, H] of qdtype (float8_e4m3fn or float8_e5m2), scale [M, ceil(H /
    128)]; q times its group's scale is the norm's output. The outputs that
    are not passed share one allocation where they take 256 KB or less
    together: keeping one keeps all of it, and torch.save, which refuses
    tensors of two types in one storage, wants clones of them."""
    if stream is not None:
        with _on_stream(x, stream):
            return _fp8().fwd_fp8(x, w, r, q, scale, h, rstd, eps, qdtype, want_rstd)
    return _fp8().fwd_fp8(x, w, r, q, scale, h, rstd, eps, qdtype, want_rstd)


def rmsnorm_quant_fp8(x, q=None, scale=None, block_rows=1, qdtype=torch.float8_e4m3fn,
                      stream=None):
    """x [M, H] (any row stride) rounded to 8 bits: (q, scale), with one fp32
    scale for each 128 columns of a row (block_rows=1, activations) or each
    block of 128 x 128 (block_rows=128, weights); see rmsnorm.h. An output
    that is not passed has an allocation of its own, of any size."""
    if stream is not None:
        with _on_stream(x, stream):
            return _fp8().quant_fp8(x, q, scale, block_rows, qdtype)
    return _fp8().quant_fp8(x, q, scale, block_rows, qdtype)


def set_gemm_fp8_test(path: int):
    """Test hook: run the 8-bit product's tile kernel (PATH_FP8_GEMM) or its
    paired one (PATH_FP8_PAIR) at any size (0: by size; see rmsnorm.h)."""
    lib().rmsnorm_set_gemm_fp8_test(int(path))


def rmsnorm_gemm_fp8(a, a_scale, b, b_scale, out=None, out_dtype=torch.bfloat16,
                     static_weights=False, stream=None):
    """out [M, N] = A B^T of 8-bit a [M, K] with a_scale [M, ceil(K / 128)]
    and b [N, K] with b_scale [ceil(N / 128), ceil(K / 128)], as
    rmsnorm_fwd_fp8 / rmsnorm_quant_fp8 return them (rows that start at
    multiples of 16 bytes). out: any row stride; out_dtype float32, bfloat16
    or float16 when it is not given. static_weights: nothing in flight on the
    stream writes b or b_scale (see RMSNORM_GEMM_FP8_STATIC_WEIGHTS)."""
    if stream is not None:
        with _on_stream(a, stream):
            return _fp8().gemm_fp8(a, a_scale, b, b_scale, out, out_dtype, static_weights)
    return _fp8().gemm_fp8(a, a_scale, b, b_scale, out, out_dtype, static_weights)


ROPE_MAX_D = 256
KV4_TILE = 16                       # tokens of a 4-bit cache stored together


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=None,
                     beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freq, amplitude) of a rotation of `rot` columns: freq is a float64
    tensor [rot / 2] of radians a position, base^(-2i / rot), for contexts
    longer than `original` positions scaled by `factor`:
    None       as they are;
    "linear"   positions compressed: every frequency / factor;
    "ntk"      another base, base * factor^(rot / (rot - 2)), which leaves the
               fastest pair alone and slows the slowest by `factor`;
    "yarn"     pairs that turn more than beta_fast times in `original`
               positions as they are, those that turn fewer than beta_slow
               times / factor, a ramp over the pairs between them; amplitude
               0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    n, amplitude = rot // 2, 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if original is None or original <= 0:
            raise ValueError("'yarn' needs original, the positions that the model was trained on")
        if not (base > 1 and beta_fast > 0 and beta_slow > 0):
            raise ValueError("'yarn' needs a base above 1, beta_fast and beta_slow above 0")

        def pair(turns):        # the pair (as a real number) that turns so often in `original`
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(n)]
        freq = [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)]
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return torch.tensor(freq, dtype=torch.float64, device=device), amplitude


def rmsnorm_rope_fwd(q, positions, freq, k=None, wq=None, wk=None, yq=None, yk=None, eps=1e-6,
                     interleaved=False, amplitude=1.0, want_rstd=True, stream=None):
    """Heads q [T, heads, D] (and k) after the heads' RMSNorm, where wq (wk)
    is given, turned by their positions (see rmsnorm.h). Any strides over
    tokens and heads. positions [T] int32 or int64; freq float64 [rot / 2]
    radians a position (rope_frequencies), which turns the first rot columns
    in pairs (i, i + rot / 2), or (2i, 2i + 1) when interleaved. positions and
    freq None: no rotation. Returns (yq, yk or None, rstd or None); rstd
    [T, q heads + k heads] is what the backward wants of a norm (rows of heads
    without one hold anything). Outputs that are not passed are dense; yq and
    yk share one allocation where they take 256 KB or less together."""
    if stream is not None:
        with _on_stream(q, stream):
            return _heads().rope_fwd(q, positions, freq, k, wq, wk, yq, yk, eps, interleaved, amplitude,
                                     want_rstd)
    return _heads().rope_fwd(q, positions, freq, k, wq, wk, yq, yk, eps, interleaved, amplitude, want_rstd)


def rmsnorm_rope_bwd(dyq, q, positions, freq, dyk=None, k=None, wq=None, wk=None, rstd=None, dq=None,
                     dk=None, eps=1e-6, interleaved=False, amplitude=1.0, stream=None):
    """(dq, dk or None, dwq or None, dwk or None) of rmsnorm_rope_fwd for the
    gradients dyq and dyk of its outputs; dw in float32. q (k) is read only
    where it has a norm, and may be None without one; rstd None: computed
    again."""
    if stream is not None:
        with _on_stream(dyq, stream):
            return _heads().rope_bwd(dyq, q, positions, freq, dyk, k, wq, wk, rstd, dq, dk, eps,
                                     interleaved, amplitude)
    return _heads().rope_bwd(dyq, q, positions, freq, dyk, k, wq, wk, rstd, dq, dk, eps, interleaved,
                             amplitude)


def rmsnorm_rope_append(k, v, positions, freq, slots, cache_k, cache_v, q=None, wq=None, wk=None, yq=None,
                        eps=1e-6, interleaved=False, amplitude=1.0, stream=None):
    """k and v [T, heads, D] into the slots of a paged cache, k (and q) on the
    way through rmsnorm_rope_fwd. cache_k, cache_v [pages, page_size, heads,
    D] of k's dtype, any strides but the last. slots [T] int32 or int64: page
    * page_size + place, distinct; tokens with a negative slot, or one past the
    cache, are not stored. Returns q's output (yq), or None without q."""
    if stream is not None:
        with _on_stream(k, stream):
            return _heads().append(k, v, positions, freq, slots, cache_k, cache_v, q, wq, wk, yq, eps,
                                   interleaved, amplitude, None, None, False)
    return _heads().append(k, v, positions, freq, slots, cache_k, cache_v, q, wq, wk, yq, eps, interleaved,
                           amplitude, None, None, False)


def kv4_cache(pages, heads, page_size, head_dim, device="cuda"):
    """A 4-bit cache of zeros for rmsnorm_rope_append_kv4: uint8 [pages,
    heads, page_size / 16, 18 head_dim] (the layout is in rmsnorm.h)."""
    if page_size < 1 or page_size % KV4_TILE:
        raise ValueError(f"page_size must be a multiple of {KV4_TILE}, got {page_size}")
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
    return torch.zeros(pages, heads, page_size // KV4_TILE, 18 * head_dim, dtype=torch.uint8, device=device)


def rmsnorm_rope_append_kv4(k, v, positions, freq, slots, cache, q=None, wq=None, wk=None, yq=None, eps=1e-6,
                            interleaved=False, amplitude=1.0, k_scale=None, v_scale=None, stream=None):
    """rmsnorm_rope_append into a 4-bit cache (kv4_cache): e2m1 codes with an
    e4m3 scale for each 16 features of a row, and an optional float32 scale
    for each head (k_scale, v_scale [heads]); see rmsnorm.h."""
    if stream is not None:
        with _on_stream(k, stream):
            return _heads().append(k, v, positions, freq, slots, cache, None, q, wq, wk, yq, eps,
                                   interleaved, amplitude, k_scale, v_scale, True)
    return _heads().append(k, v, positions, freq, slots, cache, None, q, wq, wk, yq, eps, interleaved,
                           amplitude, k_scale, v_scale, True)


def rmsnorm_kv4_read(cache, slots, stream=None):
    """Rows of a 4-bit cache as 8-bit rows: (k, k_scale, v, v_scale), all
    float8_e4m3fn and exact, k and v [n, heads, D], the scales [n, heads,
    D / 16]; zeros for slots outside the cache."""
    if stream is not None:
        with _on_stream(cache, stream):
            return _heads().kv4_read(cache, slots)
    return _heads().kv4_read(cache, slots)


def set_kv4_test(kernel: int):
    """Test hook: attention over a 4-bit cache by the kernel for few rows a
    sequence with its work list (1) or by clusters where the segments are few
    enough (3), or, with q_starts, by the one for pieces of prompts (2), at
    any size (0: by size)."""
    lib().rmsnorm_set_kv4_test(int(kernel))


def rmsnorm_kv4_attention(q, cache, block_table, seq_lens, q_starts=None, k_scale=None, v_scale=None,
                          scale=None, out=None, lse=None, want_lse=False, workspace=None, stream=None):
    """(out, lse or None): attention of q [T, heads, D] (bfloat16 or float16)
    over the 4-bit cache that rmsnorm_rope_append_kv4 writes; see rmsnorm.h.
    block_table [B, blocks] and seq_lens [B] int32; q_starts [B + 1] int32
    where sequences have other than one query token each, the last ones
    cached, each of which sees the tokens up to itself. scale: 1 / sqrt(D)
    where it is None. Rows of no sequence are not written (in an out that was
    not passed they hold anything). lse [T, heads] float32."""
    if stream is not None:
        with _on_stream(q, stream):
            return _heads().kv4_attention(q, cache, block_table, seq_lens, q_starts, k_scale, v_scale, scale,
                                          out, lse, want_lse, workspace)
    return _heads().kv4_attention(q, cache, block_table, seq_lens, q_starts, k_scale, v_scale, scale, out, lse,
                                  want_lse, workspace)


STATIC_SCRATCH_BYTES = 16 << 20     # RMSNORM_STATIC_SCRATCH_BYTES
ERR_SCRATCH_LIMIT = -10             # RMSNORM_ERR_SCRATCH_LIMIT


def rmsnorm_bwd_static_scratch(dy, x, w, rstd=None, dx=None, dw=None, eps=1e-6,
                               stream=None):
    """(dx, dw) like rmsnorm_bwd, but the library keeps the dw partial rows
    in its own fixed device array instead of a workspace, so the call itself
    allocates nothing (outputs the caller does not pass are still allocated
    here by torch). For callers that cannot allocate device memory; calls
    that overlap on the GPU share that array and race (see rmsnorm.h)."""
    H = w.numel()
    M = _rows("x", x, H)
    _rows("dy", dy, H, x.dtype)
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        dw = torch.empty(H, device=x.device, dtype=torch.float32)
    _check(lib().rmsnorm_bwd_static_scratch(
        _ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dx), _ptr(dw), M, H,
        float(eps), _dtype_code(x), _stream(stream)),
        "rmsnorm_bwd_static_scratch")
    return dx, dw


def set_static_scratch_test_limit(nbytes):
    """Test hook: rmsnorm_bwd_static_scratch treats its array as holding only
    nbytes (0: the full RMSNORM_STATIC_SCRATCH_BYTES)."""
    lib().rmsnorm_set_static_scratch_test_limit(int(nbytes))
