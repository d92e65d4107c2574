"""MI355X (gfx950) LLM.int8() mixed-precision linear layer.

Thin ctypes binding over libllmint8.so (include/llmint8.h). The Python
functions carry the C entry points' names and do argument marshalling only:
they check dtypes/devices, allocate outputs as torch tensors (PyTorch supplies
device memory and the current HIP stream) and call the library, which runs
every step of the layer in its own HIP kernels. There is no CPU fallback: if
the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes as C
import math
import os
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libllmint8.so")
_DEFAULT_LIB = LIB_PATH
# filled when the library is loaded: source digest, compiler and flags it was built with
build_record: dict = {}

LLMINT8_OK = 0
LLMINT8_ERR_INVALID_ARG = 1
LLMINT8_ERR_UNSUPPORTED = 2
LLMINT8_ERR_OVERFLOW = 3
LLMINT8_ERR_WORKSPACE = 4
LLMINT8_ERR_HIP = 5
LLMINT8_MAX_K = 133144
LLMINT8_NOALLOC_SCRATCH_BYTES = 32 << 20

LLMINT8_FP16 = 0
LLMINT8_BF16 = 1
LLMINT8_ACT_NONE = 0
LLMINT8_ACT_RELU = 1
LLMINT8_ACT_GELU = 2
LLMINT8_ACT_GELU_TANH = 3
LLMINT8_ACT_SILU = 4

_lib = None


LLMINT8_OUTLIER_W_FP16 = 0
LLMINT8_OUTLIER_W_INT8 = 1


class LinearOpts(C.Structure):
    """Mirror of llmint8_linear_opts."""
    _fields_ = [("struct_size", C.c_size_t), ("gemm_begin_event", C.c_void_p),
                ("gemm_end_event", C.c_void_p), ("outlier_weights", C.c_int),
                ("bias", C.c_void_p), ("y_col_absmax", C.c_void_p),
                ("x_col_absmax", C.c_void_p)]

    def __init__(self, **kw):
        super().__init__(struct_size=C.sizeof(LinearOpts), **kw)


class SavedMatrix(C.Structure):
    """Mirror of llmint8_saved."""
    _fields_ = [("data", C.c_void_p), ("ld", C.c_int64), ("scales", C.c_void_p),
                ("ld_scales", C.c_int64)]


class MatmulOpts(C.Structure):
    """Mirror of llmint8_matmul_opts."""
    _fields_ = [("struct_size", C.c_size_t), ("activation", C.c_int), ("bias", C.c_void_p),
                ("residual", C.c_void_p), ("ldr", C.c_int64), ("Z", C.c_void_p),
                ("ldz", C.c_int64)]


class Llmint8Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def lib() -> C.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build the HIP library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        if LIB_PATH == _DEFAULT_LIB:
            # the in-tree library must be the recorded build of the current sources
            from . import build as _build
            build_record.update(_build.check_record())
        L = C.CDLL(LIB_PATH)
        p, i64, f32, sz = C.c_void_p, C.c_int64, C.c_float, C.c_size_t
        L.llmint8_quantize_colwise.argtypes = [p, i64, i64, i64, p, p, p]
        L.llmint8_find_outliers_workspace_size.argtypes = [i64, i64]
        L.llmint8_find_outliers_workspace_size.restype = sz
        L.llmint8_find_outliers.argtypes = [p, i64, i64, i64, f32, p, p, p, sz, p]
        L.llmint8_quantize_rowwise.argtypes = [p, i64, i64, i64, p, p, p, p, p]
        L.llmint8_workspace_size.argtypes = [i64, i64, i64]
        L.llmint8_workspace_size.restype = sz
        L.llmint8_linear.argtypes = [p, i64, i64, i64, p, p, p, i64, i64, f32, p, i64, p, p, p,
                                     sz, p]
        L.llmint8_linear_ex.argtypes = L.llmint8_linear.argtypes + [p]
        L.llmint8_linear_noalloc.argtypes = [p, i64, i64, i64, p, p, p, i64, i64, f32, p, i64,
                                             p, p, p]
        L.llmint8_quantize_tensorwise_workspace_size.argtypes = [i64, i64]
        L.llmint8_quantize_tensorwise_workspace_size.restype = sz
        L.llmint8_quantize_tensorwise.argtypes = [p, i64, i64, i64, p, p, p, sz, p]
        L.llmint8_linear_tensorwise_workspace_size.argtypes = [i64, i64, i64]
        L.llmint8_linear_tensorwise_workspace_size.restype = sz
        L.llmint8_linear_tensorwise.argtypes = [p, i64, i64, i64, p, p, i64, p, p, i64, p, p, p,
                                                sz, p]
        L.llmint8_quantize_colwise_fp8.argtypes = [p, i64, i64, i64, p, p, p]
        L.llmint8_quantize_rowwise_fp8.argtypes = [p, i64, i64, i64, p, p, p, p, p]
        L.llmint8_linear_fp8_workspace_size.argtypes = [i64, i64, i64]
        L.llmint8_linear_fp8_workspace_size.restype = sz
        L.llmint8_linear_fp8.argtypes = L.llmint8_linear_ex.argtypes
        i = C.c_int
        L.llmint8_checkpoint_pack.argtypes = [p, i64, i64, i64, i, p, p]
        L.llmint8_checkpoint_unpack.argtypes = [p, i64, i64, i, p, i64, p]
        L.llmint8_matmul.argtypes = [p, i64, i64, i64, p, i64, i64, i, p, i64, p, p, sz, p]
        L.llmint8_matmul_backward.argtypes = [p, i64, i64, i64, p, i64, p, i64, p, i64, i, i, p,
                                              i64, p, i64, p, p, sz, p]
        L.llmint8_gated.argtypes = [p, i64, i64, i64, p, p, i64, i64, i, i, p, i64, p, p, p, sz, p]
        L.llmint8_gated_backward.argtypes = [p, i64, i64, i64, p, i64, p, p, i64, p, p, i, i, p,
                                             i64, p, p, i64, p, sz, p]
        for name in ("matmul", "matmul_backward", "gated", "gated_backward"):
            query = getattr(L, f"llmint8_{name}_workspace_size")
            query.argtypes, query.restype = [i64, i64, i64], sz
        L.llmint8_status_string.argtypes = [C.c_int]
        L.llmint8_status_string.restype = C.c_char_p
        for name in ("llmint8_quantize_colwise", "llmint8_find_outliers",
                     "llmint8_quantize_rowwise", "llmint8_linear", "llmint8_linear_ex",
                     "llmint8_linear_noalloc",
                     "llmint8_quantize_tensorwise", "llmint8_linear_tensorwise",
                     "llmint8_quantize_colwise_fp8", "llmint8_quantize_rowwise_fp8",
                     "llmint8_linear_fp8", "llmint8_checkpoint_pack",
                     "llmint8_checkpoint_unpack", "llmint8_matmul", "llmint8_matmul_backward",
                     "llmint8_gated", "llmint8_gated_backward"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def llmint8_status_string(status: int) -> str:
    return lib().llmint8_status_string(int(status)).decode()


def _check(status: int):
    if status != LLMINT8_OK:
        raise Llmint8Error(status, llmint8_status_string(status))


def _launch(call, t: torch.Tensor, *args, opts=()):
    """call(*args, stream, *opts) with torch's current stream of t's device, and that device
    the current one: a default stream's handle names no device, and the launches behind it
    go to the current one, where t's addresses mean nothing."""
    index = t.get_device()
    if index == torch._C._cuda_getDevice():
        status = call(*args, torch._C._cuda_getCurrentRawStream(index), *opts)
    else:
        with torch.cuda.device(index):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index), *opts)
    _check(status)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else C.c_void_p(None)


def _need(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if ndim == 2 and t.numel() == 0:
        # the C calls take M, K, N >= 1 (LLMINT8_ERR_INVALID_ARG otherwise)
        raise ValueError(f"{name} is empty ({tuple(t.shape)}); every dimension must be >= 1")


def _need_shape(t: torch.Tensor, name: str, shape: tuple, contiguous: bool = False):
    """Reject a buffer whose shape differs from the one the kernels write (or
    read) with the pitches the call passes: they would run past its end."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_vec(t: torch.Tensor, name: str, dtype, n: int, exact: bool = True):
    """A contiguous vector of n elements (at least n when exact is False)."""
    _need(t, name, dtype)
    if not t.is_contiguous() or (t.numel() != n if exact else t.numel() < n):
        raise ValueError(f"{name} must be a contiguous vector of {'' if exact else 'at least '}"
                         f"{n} elements, got {tuple(t.shape)}")


def _ws(workspace: torch.Tensor):
    """(pointer, size in bytes) of a caller-supplied device workspace."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise ValueError("workspace must be a GPU tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def _ld(t: torch.Tensor, name: str) -> int:
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    # a single row has no meaningful row stride (numpy and torch may report 0)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def llmint8_quantize_colwise(W: torch.Tensor):
    """fp16 W [K, N] -> (Wq int8 [N, K], col_absmax fp32 [N])."""
    _need(W, "W", torch.float16, 2)
    K, N = W.shape
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    s = torch.empty((N,), dtype=torch.float32, device=W.device)
    _launch(lib().llmint8_quantize_colwise, W, _ptr(W), K, N, _ld(W, "W"), _ptr(Wq), _ptr(s))
    return Wq, s


def llmint8_find_outliers_workspace_size(M: int, K: int) -> int:
    return int(lib().llmint8_find_outliers_workspace_size(M, K))


def llmint8_find_outliers(X: torch.Tensor, threshold: float = 6.0, workspace=None):
    """fp16 X [M, K] -> (idx int32 [K] ascending in idx[:count], count int32 [1]) on device."""
    _need(X, "X", torch.float16, 2)
    M, K = X.shape
    idx = torch.empty((K,), dtype=torch.int32, device=X.device)
    count = torch.empty((1,), dtype=torch.int32, device=X.device)
    need = llmint8_find_outliers_workspace_size(M, K)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=X.device)
    _launch(lib().llmint8_find_outliers, X, _ptr(X), M, K, _ld(X, "X"), float(threshold), _ptr(idx),
            _ptr(count), *_ws(workspace))
    return idx, count


def llmint8_quantize_rowwise(X: torch.Tensor, idx: torch.Tensor | None = None,
                             count: torch.Tensor | None = None):
    """fp16 X [M, K] (+ outlier idx/count on device) -> (Xq int8 [M, K], row_absmax fp32 [M])."""
    _need(X, "X", torch.float16, 2)
    if (idx is None) != (count is None):
        raise ValueError("idx and count go together")
    M, K = X.shape
    if idx is not None:
        _need_vec(idx, "idx", torch.int32, K, exact=False)
        _need_vec(count, "count", torch.int32, 1, exact=False)
    Xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    m = torch.empty((M,), dtype=torch.float32, device=X.device)
    _launch(lib().llmint8_quantize_rowwise, X, _ptr(X), M, K, _ld(X, "X"), _ptr(idx), _ptr(count),
            _ptr(Xq), _ptr(m))
    return Xq, m


def llmint8_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_workspace_size(M, K, N))


def llmint8_linear(X: torch.Tensor, Wq: torch.Tensor, col_absmax: torch.Tensor,
                   W: torch.Tensor | None, threshold: float = 6.0, *, Y=None, workspace=None,
                   outlier_count: torch.Tensor | None = None,
                   C_debug: torch.Tensor | None = None,
                   opts: LinearOpts | None = None, outlier_weights: str = "fp16",
                   bias: torch.Tensor | None = None,
                   y_col_absmax: torch.Tensor | None = None,
                   x_col_absmax: torch.Tensor | None = None) -> torch.Tensor:
    """The whole LLM.int8() layer: fp16 X [M, K] with Wq [N, K], col_absmax [N] and the
    fp16 weight W [K, N] (rows in the outlier set feed the 16-bit product) -> fp16 Y [M, N].

    outlier_weights "int8" takes the outlier rows from the codes Wq * col_absmax / 127
    instead (W may then be None); bias [N] fp16 is added to Y; y_col_absmax [N] fp32
    receives max_i |Y[i, n]|; x_col_absmax [K] fp32, if given, is taken as X's column
    absmax and decides the outlier columns without a scan of X."""
    _need(X, "X", torch.float16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or not Wq.is_contiguous():
        raise ValueError("Wq must be contiguous [N, K]")
    _need_vec(col_absmax, "col_absmax", torch.float32, N)
    if outlier_weights not in ("fp16", "int8"):
        raise ValueError("outlier_weights is 'fp16' or 'int8'")
    if W is not None:
        _need(W, "W", torch.float16, 2)
        if tuple(W.shape) != (K, N):
            raise ValueError("W must be [K, N]")
    elif outlier_weights == "fp16" and not (math.isinf(threshold) and threshold > 0):
        raise ValueError("W may be omitted only with threshold=+inf or int8 outlier weights")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(Y, "Y", torch.float16, 2)
    _need_shape(Y, "Y", (M, N))
    if outlier_count is not None:
        _need_vec(outlier_count, "outlier_count", torch.int32, 1, exact=False)
    if C_debug is not None:
        _need(C_debug, "C_debug", torch.int32)
        _need_shape(C_debug, "C_debug", (M, N), contiguous=True)
    for name, t, dt, n in (("bias", bias, torch.float16, N),
                           ("y_col_absmax", y_col_absmax, torch.float32, N),
                           ("x_col_absmax", x_col_absmax, torch.float32, K)):
        if t is not None:
            _need(t, name, dt, 1)
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous vector of {n}")
    if workspace is None:
        workspace = torch.empty((llmint8_workspace_size(M, K, N),), dtype=torch.uint8,
                                device=X.device)
    extra = (outlier_weights != "fp16" or bias is not None or y_col_absmax is not None
             or x_col_absmax is not None)
    if extra:
        o = LinearOpts(gemm_begin_event=opts.gemm_begin_event if opts else None,
                       gemm_end_event=opts.gemm_end_event if opts else None,
                       outlier_weights=(LLMINT8_OUTLIER_W_INT8 if outlier_weights == "int8"
                                        else LLMINT8_OUTLIER_W_FP16),
                       bias=bias.data_ptr() if bias is not None else None,
                       y_col_absmax=y_col_absmax.data_ptr() if y_col_absmax is not None else None,
                       x_col_absmax=x_col_absmax.data_ptr() if x_col_absmax is not None else None)
        opts = o
    args = (_ptr(X), M, K, _ld(X, "X"), _ptr(Wq), _ptr(col_absmax), _ptr(W),
            _ld(W, "W") if W is not None else N, N, float(threshold), _ptr(Y), _ld(Y, "Y"),
            _ptr(outlier_count), _ptr(C_debug), *_ws(workspace))
    if opts is None:
        _launch(lib().llmint8_linear, X, *args)
    else:
        _launch(lib().llmint8_linear_ex, X, *args, opts=(C.byref(opts),))
    return Y


def llmint8_linear_noalloc(X: torch.Tensor, Wq: torch.Tensor, col_absmax: torch.Tensor,
                           W: torch.Tensor | None, threshold: float = 6.0, *, Y=None,
                           outlier_count: torch.Tensor | None = None,
                           C_debug: torch.Tensor | None = None) -> torch.Tensor:
    """llmint8_linear without a workspace: the library's per-GPU scratch array
    (LLMINT8_NOALLOC_SCRATCH_BYTES) takes its place, so the C call allocates
    nothing (pass Y to allocate nothing here either). Shapes whose workspace
    would exceed the scratch raise Llmint8Error (LLMINT8_ERR_WORKSPACE); calls
    that may overlap on one GPU race on the shared scratch."""
    _need(X, "X", torch.float16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or not Wq.is_contiguous():
        raise ValueError("Wq must be contiguous [N, K]")
    _need_vec(col_absmax, "col_absmax", torch.float32, N)
    if W is not None:
        _need(W, "W", torch.float16, 2)
        if tuple(W.shape) != (K, N):
            raise ValueError("W must be [K, N]")
    elif not (math.isinf(threshold) and threshold > 0):
        raise ValueError("W may be omitted only with threshold=+inf")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(Y, "Y", torch.float16, 2)
    _need_shape(Y, "Y", (M, N))
    if outlier_count is not None:
        _need_vec(outlier_count, "outlier_count", torch.int32, 1, exact=False)
    if C_debug is not None:
        _need(C_debug, "C_debug", torch.int32)
        _need_shape(C_debug, "C_debug", (M, N), contiguous=True)
    _launch(lib().llmint8_linear_noalloc, X, _ptr(X), M, K, _ld(X, "X"), _ptr(Wq), _ptr(col_absmax),
            _ptr(W), _ld(W, "W") if W is not None else N, N, float(threshold), _ptr(Y), _ld(Y, "Y"),
            _ptr(outlier_count), _ptr(C_debug))
    return Y


def llmint8_quantize_tensorwise_workspace_size(K: int, N: int) -> int:
    return int(lib().llmint8_quantize_tensorwise_workspace_size(K, N))


def llmint8_quantize_tensorwise(W: torch.Tensor, workspace=None):
    """fp16 W [K, N] -> (Wq int8 [N, K], w_absmax fp32 [1]): one scale for all of W."""
    _need(W, "W", torch.float16, 2)
    K, N = W.shape
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sw = torch.empty((1,), dtype=torch.float32, device=W.device)
    if workspace is None:
        workspace = torch.empty((max(llmint8_quantize_tensorwise_workspace_size(K, N), 1),),
                                dtype=torch.uint8, device=W.device)
    _launch(lib().llmint8_quantize_tensorwise, W, _ptr(W), K, N, _ld(W, "W"), _ptr(Wq), _ptr(sw),
            *_ws(workspace))
    return Wq, sw


def llmint8_linear_tensorwise_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_linear_tensorwise_workspace_size(M, K, N))


def llmint8_linear_tensorwise(X: torch.Tensor, Wq: torch.Tensor, w_absmax: torch.Tensor, *,
                              bias: torch.Tensor | None = None, Y=None, workspace=None,
                              x_absmax: torch.Tensor | None = None,
                              C_debug: torch.Tensor | None = None) -> torch.Tensor:
    """The traditional per-tensor int8 layer: fp16 X [M, K], Wq [N, K] and w_absmax [1]
    from llmint8_quantize_tensorwise -> fp16 Y [M, N] (no outlier decomposition)."""
    _need(X, "X", torch.float16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    _need_vec(w_absmax, "w_absmax", torch.float32, 1, exact=False)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or not Wq.is_contiguous():
        raise ValueError("Wq must be contiguous [N, K]")
    if bias is not None:
        _need_vec(bias, "bias", torch.float16, N)
    if x_absmax is not None:
        _need_vec(x_absmax, "x_absmax", torch.float32, 1, exact=False)
    if C_debug is not None:
        _need(C_debug, "C_debug", torch.int32)
        _need_shape(C_debug, "C_debug", (M, N), contiguous=True)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(Y, "Y", torch.float16, 2)
    _need_shape(Y, "Y", (M, N))
    if workspace is None:
        workspace = torch.empty((llmint8_linear_tensorwise_workspace_size(M, K, N),),
                                dtype=torch.uint8, device=X.device)
    _launch(lib().llmint8_linear_tensorwise, X, _ptr(X), M, K, _ld(X, "X"), _ptr(Wq),
            _ptr(w_absmax), N, _ptr(bias), _ptr(Y), _ld(Y, "Y"), _ptr(x_absmax), _ptr(C_debug),
            *_ws(workspace))
    return Y


# ---- FP8 (E4M3) variant --------------------------------------------------------------

def llmint8_quantize_colwise_fp8(W: torch.Tensor):
    """fp16 W [K, N] -> (Wq8 uint8 E4M3 codes [N, K], col_absmax fp32 [N])."""
    _need(W, "W", torch.float16, 2)
    K, N = W.shape
    Wq = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    s = torch.empty((N,), dtype=torch.float32, device=W.device)
    _launch(lib().llmint8_quantize_colwise_fp8, W, _ptr(W), K, N, _ld(W, "W"), _ptr(Wq), _ptr(s))
    return Wq, s


def llmint8_quantize_rowwise_fp8(X: torch.Tensor, idx: torch.Tensor | None = None,
                                 count: torch.Tensor | None = None):
    """fp16 X [M, K] (+ outlier idx/count) -> (Xq8 uint8 E4M3 codes [M, K], row_absmax [M])."""
    _need(X, "X", torch.float16, 2)
    if (idx is None) != (count is None):
        raise ValueError("idx and count go together")
    M, K = X.shape
    if idx is not None:
        _need_vec(idx, "idx", torch.int32, K, exact=False)
        _need_vec(count, "count", torch.int32, 1, exact=False)
    Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    m = torch.empty((M,), dtype=torch.float32, device=X.device)
    _launch(lib().llmint8_quantize_rowwise_fp8, X, _ptr(X), M, K, _ld(X, "X"), _ptr(idx),
            _ptr(count), _ptr(Xq), _ptr(m))
    return Xq, m


def llmint8_linear_fp8_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_linear_fp8_workspace_size(M, K, N))


def llmint8_linear_fp8(X: torch.Tensor, Wq8: torch.Tensor, col_absmax: torch.Tensor,
                       W: torch.Tensor | None, threshold: float = 6.0, *, Y=None, workspace=None,
                       outlier_count: torch.Tensor | None = None,
                       C_debug: torch.Tensor | None = None, opts: LinearOpts | None = None,
                       bias: torch.Tensor | None = None,
                       y_col_absmax: torch.Tensor | None = None,
                       x_col_absmax: torch.Tensor | None = None) -> torch.Tensor:
    """The FP8 (E4M3) variant of the layer: fp16 X [M, K] with Wq8 [N, K] and col_absmax
    from llmint8_quantize_colwise_fp8 and the fp16 weight W [K, N] -> fp16 Y [M, N].
    C_debug, if given, is an fp32 [M, N] tensor receiving the 8-bit product."""
    _need(X, "X", torch.float16, 2)
    _need(Wq8, "Wq8", torch.uint8, 2)
    M, K = X.shape
    N = Wq8.shape[0]
    if Wq8.shape[1] != K or not Wq8.is_contiguous():
        raise ValueError("Wq8 must be contiguous [N, K]")
    _need_vec(col_absmax, "col_absmax", torch.float32, N)
    if W is not None:
        _need(W, "W", torch.float16, 2)
        if tuple(W.shape) != (K, N):
            raise ValueError("W must be [K, N]")
    elif not (math.isinf(threshold) and threshold > 0):
        raise ValueError("W may be omitted only with threshold=+inf")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(Y, "Y", torch.float16, 2)
    _need_shape(Y, "Y", (M, N))
    if outlier_count is not None:
        _need_vec(outlier_count, "outlier_count", torch.int32, 1, exact=False)
    if C_debug is not None:
        _need(C_debug, "C_debug", torch.float32)
        _need_shape(C_debug, "C_debug", (M, N), contiguous=True)
    for name, t, dt, n in (("bias", bias, torch.float16, N),
                           ("y_col_absmax", y_col_absmax, torch.float32, N),
                           ("x_col_absmax", x_col_absmax, torch.float32, K)):
        if t is not None:
            _need(t, name, dt, 1)
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous vector of {n}")
    if workspace is None:
        workspace = torch.empty((llmint8_linear_fp8_workspace_size(M, K, N),), dtype=torch.uint8,
                                device=X.device)
    o = LinearOpts(gemm_begin_event=opts.gemm_begin_event if opts else None,
                   gemm_end_event=opts.gemm_end_event if opts else None,
                   outlier_weights=LLMINT8_OUTLIER_W_FP16,
                   bias=bias.data_ptr() if bias is not None else None,
                   y_col_absmax=y_col_absmax.data_ptr() if y_col_absmax is not None else None,
                   x_col_absmax=x_col_absmax.data_ptr() if x_col_absmax is not None else None)
    _launch(lib().llmint8_linear_fp8, X, _ptr(X), M, K, _ld(X, "X"), _ptr(Wq8), _ptr(col_absmax),
            _ptr(W), _ld(W, "W") if W is not None else N, N, float(threshold), _ptr(Y), _ld(Y, "Y"),
            _ptr(outlier_count), _ptr(C_debug), *_ws(workspace), opts=(C.byref(o),))
    return Y


# ---- 16-bit feed-forward operators ---------------------------------------------------
# As the calls above, these record nothing for autograd: a result has no grad_fn, also where
# an input requires grad. The backward functions are called explicitly.

_DTYPES = {torch.float16: LLMINT8_FP16, torch.bfloat16: LLMINT8_BF16}
_ACTIVATIONS = {"none": LLMINT8_ACT_NONE, "relu": LLMINT8_ACT_RELU, "gelu": LLMINT8_ACT_GELU,
                "gelu_tanh": LLMINT8_ACT_GELU_TANH, "silu": LLMINT8_ACT_SILU}
CHECKPOINT_BLOCK = 32


class Checkpoint(NamedTuple):
    """An 8-bit activation checkpoint: int8 codes [M, K] (row pitch a multiple of 16) and
    the scale bytes [M, ceil(K / 32)]; an entry stands for code * 2^(byte - 127)."""
    codes: torch.Tensor
    scales: torch.Tensor


def _dtype_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    return _DTYPES[t.dtype]


def _activation(name: str) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation is one of {sorted(_ACTIVATIONS)}, got {name!r}")
    return _ACTIVATIONS[name]


def _matrix(t, name: str, like: torch.Tensor, shape=None) -> int:
    """The leading dimension of a matrix of like's dtype and device."""
    # what a valid matrix passes, by the cheapest queries (a call is a few microseconds);
    # the named errors below
    if isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.dim() == 2:
        device, got = t.get_device(), t.shape
        if device >= 0 and device == like.get_device() and (shape is None or got == shape):
            M, N = got
            if M and N:
                if t.is_contiguous():
                    return N
                s0, s1 = t.stride()
                if s1 == 1:
                    return s0 if M > 1 else N
    _need(t, name, like.dtype, 2)
    if shape is not None:
        _need_shape(t, name, shape)
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    return _ld(t, name)


def _vector(t, name: str, dtype, n: int, like: torch.Tensor) -> int:
    """The address of a contiguous vector of n elements on like's device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n
            and t.is_contiguous() and t.get_device() == like.get_device()):
        _need_vec(t, name, dtype, n)
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    return t.data_ptr()


def _out(t, name: str, like: torch.Tensor, shape):
    """(tensor, leading dimension) of an output, allocated here if not given."""
    if t is None:
        return like.new_empty(shape), shape[1]
    return t, _matrix(t, name, like, shape)


def _address(t):
    return None if t is None else t.data_ptr()


def _new_checkpoint(M: int, K: int, device) -> Checkpoint:
    codes = torch.empty((M, (K + 15) // 16 * 16), dtype=torch.int8, device=device)
    if K % 16:
        codes = codes[:, :K]
    return Checkpoint(codes, torch.empty((M, -(-K // CHECKPOINT_BLOCK)), dtype=torch.uint8,
                                         device=device))


def _c_checkpoint(c: Checkpoint) -> SavedMatrix:
    """The C view of a checkpoint from _new_checkpoint."""
    nb = c.scales.shape[1]
    return SavedMatrix(c.codes.data_ptr(), (c.codes.shape[1] + 15) // 16 * 16,
                       c.scales.data_ptr(), nb)


def _checkpoint(c, name: str, device, shape=None) -> SavedMatrix:
    """The C view of a checkpoint, after checking it."""
    codes, scales = c
    # as in _matrix, what a valid one passes first
    if (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor)
            and codes.dtype is torch.int8 and scales.dtype is torch.uint8 and codes.dim() == 2):
        index, got = codes.get_device(), codes.shape
        if (index >= 0 and index == device.index and scales.get_device() == index
                and (shape is None or got == shape)):
            M, K = got
            (s0, s1), blocks = codes.stride(), -(-K // CHECKPOINT_BLOCK)
            if (M > 1 and K and s1 == 1 and s0 >= (K + 15) // 16 * 16
                    and scales.shape == (M, blocks) and scales.is_contiguous()):
                return SavedMatrix(codes.data_ptr(), s0, scales.data_ptr(), blocks)
    _need(codes, f"{name}.codes", torch.int8, 2)
    if shape is not None:
        _need_shape(codes, f"{name}.codes", shape)
    M, K = codes.shape
    _need(scales, f"{name}.scales", torch.uint8, 2)
    _need_shape(scales, f"{name}.scales", (M, -(-K // CHECKPOINT_BLOCK)))
    if codes.device != device or scales.device != device:
        raise ValueError(f"{name} must be on {device}")
    s0, s1 = codes.stride()
    pad = (K + 15) // 16 * 16
    ld = s0 if M > 1 else pad
    if (K > 1 and s1 != 1) or ld < pad:
        raise ValueError(f"{name}.codes must have unit stride and rows padded to 16 entries")
    return SavedMatrix(codes.data_ptr(), ld, scales.data_ptr(), _ld(scales, f"{name}.scales"))


def _saved(t, name: str, like: torch.Tensor, shape) -> SavedMatrix:
    """The C view of a matrix held in 16 bits or as a checkpoint."""
    if isinstance(t, tuple):
        return _checkpoint(t, name, like.device, shape)
    return SavedMatrix(t.data_ptr() if isinstance(t, torch.Tensor) else None,
                       _matrix(t, name, like, shape), None, 0)


def _workspace(workspace, need: int, like: torch.Tensor):
    """(pointer, size, tensor) of the caller's workspace, or of one allocated here."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty((need,), dtype=torch.uint8, device=like.device)
        return workspace.data_ptr(), need, workspace
    ws = *_ws(workspace), workspace
    if workspace.get_device() != like.get_device():
        raise ValueError(f"workspace must be on {like.device}, got {workspace.device}")
    return ws


def llmint8_checkpoint_pack(X: torch.Tensor) -> Checkpoint:
    """fp16 or bf16 X [M, K] -> its 8-bit checkpoint."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    c = _new_checkpoint(M, K, X.device)
    _launch(lib().llmint8_checkpoint_pack, X, X.data_ptr(), M, K, ldx, dt,
            C.byref(_c_checkpoint(c)))
    return c


def llmint8_checkpoint_unpack(checkpoint: Checkpoint, dtype=torch.float16, *,
                              X=None) -> torch.Tensor:
    """What a checkpoint stands for, as a 16-bit matrix [M, K] of `dtype`. Exact in bf16, and
    in fp16 if it was packed from fp16; rounded (to infinity from 65520 on) otherwise."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
    codes = checkpoint[0]
    _need(codes, "checkpoint.codes", torch.int8, 2)
    saved = _checkpoint(checkpoint, "checkpoint", codes.device)
    M, K = codes.shape
    if X is None:
        X, ldx = torch.empty((M, K), dtype=dtype, device=codes.device), K
    else:
        ldx = _matrix(X, "X", torch.empty((0,), dtype=dtype, device=codes.device), (M, K))
    _launch(lib().llmint8_checkpoint_unpack, X, C.byref(saved), M, K, _DTYPES[dtype], X.data_ptr(),
            ldx)
    return X


_MATMUL_OPTS_SIZE = C.sizeof(MatmulOpts)


def llmint8_matmul_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_matmul_workspace_size(M, K, N))


def llmint8_matmul(X: torch.Tensor, W: torch.Tensor, *, bias: torch.Tensor | None = None,
                   activation: str = "none", residual: torch.Tensor | None = None,
                   Y=None, Z=None, workspace=None) -> torch.Tensor:
    """Y = act(X W + bias) + residual in one product: fp16 or bf16 X [M, K], W [K, N],
    bias [N] and residual [M, N] of the same dtype -> Y [M, N].

    activation is "none", "relu", "gelu", "gelu_tanh" or "silu". Z, if given, receives the
    pre-activations X W + bias [M, N] that llmint8_matmul_backward takes. Autograd does not
    see the call: gradients come from llmint8_matmul_backward."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    ldw = _matrix(W, "W", X)
    kw, N = W.shape
    if kw != K:
        raise ValueError(f"W must be [{K}, N], got {tuple(W.shape)}")
    act = _activation(activation)
    Y, ldy = _out(Y, "Y", X, (M, N))
    opts = None
    if act or bias is not None or residual is not None or Z is not None:
        b = r = z = None
        ldr = ldz = 0
        if bias is not None:
            b = _vector(bias, "bias", X.dtype, N, X)
        if residual is not None:
            ldr, r = _matrix(residual, "residual", X, (M, N)), residual.data_ptr()
        if Z is not None:
            ldz, z = _matrix(Z, "Z", X, (M, N)), Z.data_ptr()
        opts = C.byref(MatmulOpts(_MATMUL_OPTS_SIZE, act, b, r, ldr, z, ldz))
    L = lib()
    ws, nb, keep = _workspace(workspace, L.llmint8_matmul_workspace_size(M, K, N), X)
    _launch(L.llmint8_matmul, X, X.data_ptr(), M, K, ldx, W.data_ptr(), ldw, N, dt, Y.data_ptr(),
            ldy, opts, ws, nb)
    return Y


def llmint8_matmul_backward_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_matmul_backward_workspace_size(M, K, N))


def llmint8_matmul_backward(dY: torch.Tensor, X, W: torch.Tensor | None, *,
                            Z: torch.Tensor | None = None, activation: str = "none",
                            need_dX: bool = True, need_dW: bool = True, need_dbias: bool = False,
                            dX=None, dW=None, dbias=None, workspace=None):
    """Gradients of llmint8_matmul from dY [M, N]: (dX [M, K], dW [K, N], dbias fp32 [N]),
    None where not needed (the residual's gradient is dY).

    X [M, K] is the 16-bit input or its Checkpoint, read for dW; W [K, N] is read for dX;
    either may be None where it is not read, but one of them gives K. Z [M, N] holds the
    pre-activations and is needed unless activation is "none"."""
    dt = _dtype_of(dY, "dY")
    lddy = _matrix(dY, "dY", dY)
    M, N = dY.shape
    act = _activation(activation)
    if W is not None:
        ldw = _matrix(W, "W", dY)
        K = W.shape[0]
        if W.shape[1] != N:
            raise ValueError(f"W must be [K, {N}], got {tuple(W.shape)}")
    elif need_dX:
        raise ValueError("dX needs W")
    elif X is None:
        raise ValueError("one of X and W is needed")
    else:
        K, ldw = (X[0] if isinstance(X, tuple) else X).shape[1], N
    if need_dW and X is None:
        raise ValueError("dW needs X")
    if not (need_dX or need_dW or need_dbias):
        raise ValueError("no gradient is asked for")
    x = C.byref(_saved(X, "X", dY, (M, K))) if need_dW else None
    z, ldz = None, 0
    if act != LLMINT8_ACT_NONE:
        if Z is None:
            raise ValueError("Z is needed with an activation")
        ldz, z = _matrix(Z, "Z", dY, (M, N)), Z.data_ptr()
    dX, lddx = _out(dX, "dX", dY, (M, K)) if need_dX else (None, 0)
    dW, lddw = _out(dW, "dW", dY, (K, N)) if need_dW else (None, 0)
    if not need_dbias:
        dbias = None
    elif dbias is None:
        dbias = torch.empty((N,), dtype=torch.float32, device=dY.device)
    else:
        _vector(dbias, "dbias", torch.float32, N, dY)
    L = lib()
    ws, nb, keep = _workspace(workspace, L.llmint8_matmul_backward_workspace_size(M, K, N), dY)
    _launch(L.llmint8_matmul_backward, dY, dY.data_ptr(), M, N, lddy, x, K, _address(W), ldw, z,
            ldz, act, dt, _address(dX), lddx, _address(dW), lddw, _address(dbias), ws, nb)
    return dX, dW, dbias


def llmint8_gated_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_gated_workspace_size(M, K, N))


def _gate_weights(Wg, Wu, like: torch.Tensor):
    ldw = _matrix(Wg, "Wg", like)
    if _matrix(Wu, "Wu", like, tuple(Wg.shape)) != ldw:
        raise ValueError("Wg and Wu must have the same row stride")
    return ldw


def llmint8_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, *,
                  activation: str = "silu", save: str = "none", H=None, workspace=None):
    """The gated feed-forward block H = act(X Wg) * (X Wu) in one kernel: fp16 or bf16
    X [M, K], Wg and Wu [K, N] -> H [M, N].

    save "none" returns H; "full" returns (H, G, U) with the pre-activations G = X Wg and
    U = X Wu in 16 bits, "8bit" returns them as Checkpoints. Autograd does not see the call:
    gradients come from llmint8_gated_backward."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    ldw = _gate_weights(Wg, Wu, X)
    kw, N = Wg.shape
    if kw != K:
        raise ValueError(f"Wg and Wu must be [{K}, N], got {tuple(Wg.shape)}")
    act = _activation(activation)
    if save not in ("none", "full", "8bit"):
        raise ValueError(f"save is 'none', 'full' or '8bit', got {save!r}")
    H, ldh = _out(H, "H", X, (M, N))
    G = U = g = u = None
    if save == "full":
        G, U = X.new_empty((M, N)), X.new_empty((M, N))
        g, u = (C.byref(SavedMatrix(t.data_ptr(), N, None, 0)) for t in (G, U))
    elif save == "8bit":
        G, U = _new_checkpoint(M, N, X.device), _new_checkpoint(M, N, X.device)
        g, u = C.byref(_c_checkpoint(G)), C.byref(_c_checkpoint(U))
    L = lib()
    ws, nb, keep = _workspace(workspace, L.llmint8_gated_workspace_size(M, K, N), X)
    _launch(L.llmint8_gated, X, X.data_ptr(), M, K, ldx, Wg.data_ptr(), Wu.data_ptr(), ldw, N, act,
            dt, H.data_ptr(), ldh, g, u, ws, nb)
    return H if save == "none" else (H, G, U)


def llmint8_gated_backward_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_gated_backward_workspace_size(M, K, N))


def llmint8_gated_backward(dH: torch.Tensor, X, Wg: torch.Tensor, Wu: torch.Tensor, G, U, *,
                           activation: str = "silu", need_dX: bool = True, need_dW: bool = True,
                           dX=None, dWg=None, dWu=None, workspace=None):
    """Gradients of llmint8_gated from dH [M, N]: (dX [M, K], dWg [K, N], dWu [K, N]), None
    where not needed. X, G and U are 16-bit matrices or Checkpoints (G and U alike); X may be
    None without need_dW."""
    dt = _dtype_of(dH, "dH")
    lddh = _matrix(dH, "dH", dH)
    M, N = dH.shape
    ldw = _gate_weights(Wg, Wu, dH)
    K = Wg.shape[0]
    if Wg.shape[1] != N:
        raise ValueError(f"Wg and Wu must be [K, {N}], got {tuple(Wg.shape)}")
    act = _activation(activation)
    if need_dW and X is None:
        raise ValueError("dWg and dWu need X")
    if not (need_dX or need_dW):
        raise ValueError("no gradient is asked for")
    if isinstance(G, tuple) != isinstance(U, tuple):
        raise ValueError("G and U are both 16-bit matrices or both Checkpoints")
    x = C.byref(_saved(X, "X", dH, (M, K))) if need_dW else None
    g, u = _saved(G, "G", dH, (M, N)), _saved(U, "U", dH, (M, N))
    dX, lddx = _out(dX, "dX", dH, (M, K)) if need_dX else (None, 0)
    lddw = 0
    if need_dW:
        dWg, lddw = _out(dWg, "dWg", dH, (K, N))
        dWu, ldu = _out(dWu, "dWu", dH, (K, N))
        if ldu != lddw:
            raise ValueError("dWg and dWu must have the same row stride")
    else:
        dWg = dWu = None
    L = lib()
    ws, nb, keep = _workspace(workspace, L.llmint8_gated_backward_workspace_size(M, K, N), dH)
    _launch(L.llmint8_gated_backward, dH, dH.data_ptr(), M, N, lddh, x, K, Wg.data_ptr(),
            Wu.data_ptr(), ldw, C.byref(g), C.byref(u), act, dt, _address(dX), lddx, _address(dWg),
            _address(dWu), lddw, ws, nb)
    return dX, dWg, dWu
