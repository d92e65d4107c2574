"""MI355X (gfx950) LLM.int8() mixed-precision linear layer, the 16-bit feed-forward layers
beside it (dense and routed to experts, forward and backward) and their FP8 forms.

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
LLMINT8_FP32 = 2
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


class RouteOpts(C.Structure):
    """Mirror of llmint8_route_opts."""
    _fields_ = [("struct_size", C.c_size_t), ("scores", C.c_int), ("renormalize", C.c_int),
                ("scale", C.c_float), ("groups", C.c_int), ("top_groups", C.c_int),
                ("group_best", C.c_int), ("bias", C.c_void_p)]


class ExpertRows(C.Structure):
    """Mirror of llmint8_expert_rows."""
    _fields_ = [("offsets", C.c_void_p), ("order", C.c_void_p), ("places", C.c_void_p),
                ("E", C.c_int64), ("k", C.c_int64)]


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
        L.llmint8_route.argtypes = [p, i64, i64, i64, i, i64, p, p, p, p]
        L.llmint8_route_backward.argtypes = [p, p, i64, i64, i64, i, i64, p, p, p, i64, p]
        L.llmint8_expert_plan.argtypes = [p, i64, i64, i64, p, p, p, p, sz, p]
        L.llmint8_expert_plan_workspace_size.argtypes = [i64, i64, i64]
        L.llmint8_expert_plan_workspace_size.restype = sz
        L.llmint8_experts_gated.argtypes = [p, i64, i64, i64, p, p, i64, i64, i64, p, p, i, i, p,
                                            i64, p, p, i64, p, sz, p]
        L.llmint8_experts_gated_backward.argtypes = [p, i64, i64, i64, p, i64, i64, p, p, i64, i64,
                                                     p, p, i64, p, p, i, i, p, i64, p, p, i64,
                                                     i64, p, p, sz, p]
        L.llmint8_experts_matmul.argtypes = [p, i64, i64, i64, p, i64, i64, i64, p, p, i64, i, p,
                                             i64, p, sz, p]
        L.llmint8_experts_matmul_backward.argtypes = [p, i64, i64, i64, p, i64, i64, p, i64, i64,
                                                      p, i, p, i64, p, i64, i64, p, sz, p]
        L.llmint8_quantize_blockwise_fp8.argtypes = [p, i64, i64, i64, i, p, p, p]
        L.llmint8_quantize_rowblock_fp8.argtypes = [p, i64, i64, i64, i, p, p, i64, p]
        L.llmint8_linear_blockwise_fp8.argtypes = [p, i64, i64, i64, p, p, i64, i64, i, p, p, i64,
                                                   p, sz, p]
        L.llmint8_linear_blockwise_fp8_workspace_size.argtypes = [i64, i64, i64]
        L.llmint8_linear_blockwise_fp8_workspace_size.restype = sz
        for name in ("gated", "gated_backward", "matmul", "matmul_backward"):
            query = getattr(L, f"llmint8_experts_{name}_workspace_size")
            query.argtypes, query.restype = [i64] * 5, sz
        L.llmint8_status_string.argtypes = [C.c_int]
        L.llmint8_status_string.restype = C.c_char_p
        for name in ("llmint8_quantize_colwise", "llmint8_find_outliers",
                     "llmint8_quantize_rowwise", "llmint8_linear", "llmint8_linear_ex",
                     "llmint8_linear_noalloc",
                     "llmint8_quantize_tensorwise", "llmint8_linear_tensorwise",
                     "llmint8_quantize_colwise_fp8", "llmint8_quantize_rowwise_fp8",
                     "llmint8_linear_fp8", "llmint8_checkpoint_pack",
                     "llmint8_checkpoint_unpack", "llmint8_matmul", "llmint8_matmul_backward",
                     "llmint8_gated", "llmint8_gated_backward", "llmint8_route",
                     "llmint8_route_backward", "llmint8_expert_plan", "llmint8_experts_gated",
                     "llmint8_experts_gated_backward", "llmint8_experts_matmul",
                     "llmint8_experts_matmul_backward", "llmint8_quantize_blockwise_fp8",
                     "llmint8_quantize_rowblock_fp8", "llmint8_linear_blockwise_fp8"):
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


# ---- routed feed-forward layers ------------------------------------------------------
# A router sends each token to k of E experts. As above, autograd does not see the calls.

_SCORES = {"softmax": 0, "sigmoid": 1}
_LOGIT_TYPES = {**_DTYPES, torch.float32: LLMINT8_FP32}


class ExpertPlan(NamedTuple):
    """The (token, expert) pairs in the experts' order, int32: expert e has the rows
    offsets[e] .. offsets[e + 1] - 1 (offsets [E + 1]); order [M k] is the pair i k + j of each
    row, -1 behind the last; places [M, k] the row of each pair, -1 where it has none."""
    offsets: torch.Tensor
    order: torch.Tensor
    places: torch.Tensor


def _logits(logits) -> int:
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in _LOGIT_TYPES:
        raise TypeError("logits must be torch.float16, torch.bfloat16 or torch.float32, got "
                        f"{logits.dtype}")
    return _matrix(logits, "logits", logits)


def _route_opts(logits, scores, bias, groups, top_groups, group_best, renormalize, scale):
    if scores not in _SCORES:
        raise ValueError(f"scores is 'softmax' or 'sigmoid', got {scores!r}")
    E = logits.shape[1]
    b = None if bias is None else _vector(bias, "bias", torch.float32, E, logits)
    return C.byref(RouteOpts(C.sizeof(RouteOpts), _SCORES[scores], bool(renormalize), scale, groups,
                             groups if top_groups is None else top_groups, group_best, b))


def _table(t, name: str, dtype, shape, like: torch.Tensor) -> int:
    """The address of a contiguous matrix of this type and shape on like's device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == like.get_device()):
        _need(t, name, dtype, len(shape))
        _need_shape(t, name, shape, contiguous=True)
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    return t.data_ptr()


def llmint8_route(logits: torch.Tensor, k: int, *, scores: str = "softmax",
                  bias: torch.Tensor | None = None, groups: int = 1,
                  top_groups: int | None = None, group_best: int = 1, renormalize: bool = False,
                  scale: float = 1.0):
    """The k experts of each token: fp16, bf16 or fp32 logits [M, E] -> (ids int32 [M, k],
    weights fp32 [M, k]).

    scores is "softmax" (over the row) or "sigmoid". The k largest of score + bias (fp32 [E])
    are chosen, ties to the lower index, in falling order; with groups > 1 out of the top_groups
    best of `groups` equal runs of experts, a run's value being the sum of its group_best (1 or 2)
    largest. weights are the scores of the chosen, divided by their sum with `renormalize`, times
    `scale`. An expert whose logit is -inf or NaN is out, and one whose bias is: where fewer than k
    are left, the id is -1 and the weight 0."""
    ld = _logits(logits)
    M, E = logits.shape
    if not 1 <= k <= min(E, 64):
        raise ValueError(f"k must be from 1 to {min(E, 64)}, got {k}")
    if groups < 1 or E % groups:
        raise ValueError(f"groups must divide the {E} experts, got {groups}")
    opts = _route_opts(logits, scores, bias, groups, top_groups, group_best, renormalize, scale)
    ids = logits.new_empty((M, k), dtype=torch.int32)
    weights = logits.new_empty((M, k), dtype=torch.float32)
    _launch(lib().llmint8_route, logits, logits.data_ptr(), M, E, ld, _LOGIT_TYPES[logits.dtype],
            k, opts, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def llmint8_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *,
                           scores: str = "softmax", renormalize: bool = False, scale: float = 1.0,
                           dlogits=None) -> torch.Tensor:
    """The logits' gradient [M, E] (of their type) from dweights fp32 [M, k] and the ids of
    llmint8_route; scores, renormalize and scale as there. The choice has no gradient."""
    ld = _logits(logits)
    M, E = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be [M, k]")
    k = ids.shape[1]
    i = _table(ids, "ids", torch.int32, (M, k), logits)
    d = _table(dweights, "dweights", torch.float32, (M, k), logits)
    opts = _route_opts(logits, scores, None, 1, None, 1, renormalize, scale)
    dlogits, ldd = _out(dlogits, "dlogits", logits, (M, E))
    _launch(lib().llmint8_route_backward, logits, d, logits.data_ptr(), M, E, ld,
            _LOGIT_TYPES[logits.dtype], k, i, opts, dlogits.data_ptr(), ldd)
    return dlogits


def llmint8_expert_plan(ids: torch.Tensor, experts: int) -> ExpertPlan:
    """The experts' order of the pairs that ids int32 [M, k] name (ids outside 0 .. experts - 1:
    none, as on a rank that holds some of the experts). `experts` is at least k: a rank with fewer
    passes k and repeats an expert's weights (W.expand) for those that no id names. The plan
    serves every call on these ids, the backward ones too."""
    _need(ids, "ids", torch.int32, 2)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    if not 1 <= experts <= 1024:
        raise ValueError(f"experts must be from 1 to 1024, got {experts}")
    M, k = ids.shape
    need = lib().llmint8_expert_plan_workspace_size(M, k, experts)
    # one allocation: the parts, the workspace first, begin at multiples of 16 bytes
    w, a, b = (need + 15) // 16 * 4, (experts + 4) // 4 * 4, (M * k + 3) // 4 * 4
    held = ids.new_empty((w + a + 2 * b,))
    plan = ExpertPlan(held.as_strided((experts + 1,), (1,), w),
                      held.as_strided((M * k,), (1,), w + a),
                      held.as_strided((M, k), (k, 1), w + a + b))
    at = held.data_ptr()
    _launch(lib().llmint8_expert_plan, ids, ids.data_ptr(), M, k, experts, at + 4 * w,
            at + 4 * (w + a), at + 4 * (w + a + b), at if need else None, need)
    return plan


def _rows(plan, like: torch.Tensor, M: int | None = None) -> tuple:
    """(the C view of a plan, its tokens, experts and choices of a token)"""
    if not (isinstance(plan, tuple) and len(plan) == 3
            and all(isinstance(t, torch.Tensor) for t in plan)):
        raise TypeError("plan must be an ExpertPlan")
    offsets, order, places = plan
    if places.dim() != 2:
        raise ValueError("plan.places must be [M, k]")
    tokens, k = places.shape
    if M is not None and tokens != M:
        raise ValueError(f"the plan is of {tokens} tokens, not {M}")
    E = offsets.numel() - 1
    return C.byref(ExpertRows(_vector(offsets, "plan.offsets", torch.int32, E + 1, like),
                              _vector(order, "plan.order", torch.int32, tokens * k, like),
                              _table(places, "plan.places", torch.int32, (tokens, k), like), E,
                              k)), tokens, E, k


def _expert_weights(W, name: str, like: torch.Tensor, shape) -> tuple:
    """(row stride, stride from expert to expert) of weights [E, rows, columns]."""
    if not isinstance(W, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (W.dtype is like.dtype and W.shape == shape and W.get_device() == like.get_device()
            and W.is_contiguous()):
        _need(W, name, like.dtype, 3)
        _need_shape(W, name, shape)
        if W.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, got {W.device}")
        if W.numel() == 0:
            raise ValueError(f"{name} is empty ({tuple(W.shape)}); every dimension must be >= 1")
    se, ld, s1 = W.stride()
    E, rows, cols = shape
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    ld = ld if rows > 1 else cols
    return ld, se if E > 1 else rows * ld


def _gate_experts(Wg, Wu, like: torch.Tensor, shape) -> tuple:
    strides = _expert_weights(Wg, "Wg", like, shape)
    if _expert_weights(Wu, "Wu", like, shape) != strides:
        raise ValueError("Wg and Wu must have the same strides")
    return strides


def _out_experts(t, name: str, like: torch.Tensor, shape) -> tuple:
    if t is None:
        return like.new_empty(shape), shape[2], shape[1] * shape[2]
    return t, *_expert_weights(t, name, like, shape)


def _last_dims(W, name: str) -> tuple:
    if not isinstance(W, torch.Tensor) or W.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions")
    return W.shape[1:]


def _experts_workspace(name: str, workspace, sizes, like: torch.Tensor):
    need = getattr(lib(), f"llmint8_experts_{name}_workspace_size")(*sizes)
    return _workspace(workspace, need, like)


def llmint8_experts_gated_workspace_size(M: int, K: int, N: int, E: int, k: int) -> int:
    return int(lib().llmint8_experts_gated_workspace_size(M, K, N, E, k))


def llmint8_experts_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, plan: ExpertPlan, *,
                          weights: torch.Tensor | None = None, activation: str = "silu",
                          save: str = "none", H=None, workspace=None):
    """The experts' gated blocks, H[r] = w act(x Wg_e) * (x Wu_e) for every row r of the plan:
    fp16 or bf16 X [M, K], Wg and Wu [E, K, N], weights fp32 [M, k] (none: 1) -> H [M k, N].

    Rows behind plan.offsets[E] are left as they were (uninitialized in an H made here). save
    "full" returns (H, G, U) with the pre-activations in 16 bits, for
    llmint8_experts_gated_backward."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    rows, _, E, k = _rows(plan, X, M)
    N = _last_dims(Wg, "Wg")[1]
    ldw, sw = _gate_experts(Wg, Wu, X, (E, K, N))
    act = _activation(activation)
    if save not in ("none", "full"):
        raise ValueError(f"save is 'none' or 'full', got {save!r}")
    w = None if weights is None else _table(weights, "weights", torch.float32, (M, k), X)
    H, ldh = _out(H, "H", X, (M * k, N))
    G = U = None
    if save == "full":
        G, U = X.new_empty((M * k, N)), X.new_empty((M * k, N))
    ws, nb, keep = _experts_workspace("gated", workspace, (M, K, N, E, k), X)
    _launch(lib().llmint8_experts_gated, X, X.data_ptr(), M, K, ldx, Wg.data_ptr(), Wu.data_ptr(),
            ldw, sw, N, rows, w, act, dt, H.data_ptr(), ldh, _address(G), _address(U), N, ws, nb)
    return H if save == "none" else (H, G, U)


def llmint8_experts_gated_backward_workspace_size(M: int, K: int, N: int, E: int, k: int) -> int:
    return int(lib().llmint8_experts_gated_backward_workspace_size(M, K, N, E, k))


def llmint8_experts_gated_backward(dH: torch.Tensor, X: torch.Tensor | None, Wg: torch.Tensor,
                                   Wu: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                                   plan: ExpertPlan, *, weights: torch.Tensor | None = None,
                                   activation: str = "silu", need_dX: bool = True,
                                   need_dW: bool = True, need_dweights: bool = True, dX=None,
                                   dWg=None, dWu=None, dweights=None, workspace=None):
    """Gradients of llmint8_experts_gated from dH [M k, N]: (dX [M, K], dWg [E, K, N],
    dWu [E, K, N], dweights fp32 [M, k]), None where not needed. X may be None without need_dW."""
    dt = _dtype_of(dH, "dH")
    lddh = _matrix(dH, "dH", dH)
    rows, M, E, k = _rows(plan, dH)
    K, N = _last_dims(Wg, "Wg")
    _need_shape(dH, "dH", (M * k, N))
    ldw, sw = _gate_experts(Wg, Wu, dH, (E, K, N))
    act = _activation(activation)
    ldx = K
    if need_dW:
        if X is None:
            raise ValueError("dWg and dWu need X")
        ldx = _matrix(X, "X", dH, (M, K))
    if not (need_dX or need_dW or need_dweights):
        raise ValueError("no gradient is asked for")
    ldz = _matrix(G, "G", dH, (M * k, N))
    if _matrix(U, "U", dH, (M * k, N)) != ldz:
        raise ValueError("G and U must have the same row stride")
    w = None if weights is None else _table(weights, "weights", torch.float32, (M, k), dH)
    dX, lddx = _out(dX, "dX", dH, (M, K)) if need_dX else (None, 0)
    lddw = sdw = 0
    if need_dW:
        dWg, lddw, sdw = _out_experts(dWg, "dWg", dH, (E, K, N))
        dWu, *other = _out_experts(dWu, "dWu", dH, (E, K, N))
        if other != [lddw, sdw]:
            raise ValueError("dWg and dWu must have the same strides")
    else:
        dWg = dWu = None
    if not need_dweights:
        dweights = None
    elif dweights is None:
        dweights = torch.empty((M, k), dtype=torch.float32, device=dH.device)
    else:
        _table(dweights, "dweights", torch.float32, (M, k), dH)
    ws, nb, keep = _experts_workspace("gated_backward", workspace, (M, K, N, E, k), dH)
    _launch(lib().llmint8_experts_gated_backward, dH, dH.data_ptr(), M, N, lddh,
            X.data_ptr() if need_dW else None, K, ldx, Wg.data_ptr(), Wu.data_ptr(), ldw, sw,
            G.data_ptr(), U.data_ptr(), ldz, rows, w, act, dt, _address(dX), lddx, _address(dWg),
            _address(dWu), lddw, sdw, _address(dweights), ws, nb)
    return dX, dWg, dWu, dweights


def llmint8_experts_matmul_workspace_size(M: int, K: int, N: int, E: int, k: int) -> int:
    return int(lib().llmint8_experts_matmul_workspace_size(M, K, N, E, k))


def llmint8_experts_matmul(H: torch.Tensor, Wd: torch.Tensor, plan: ExpertPlan, *,
                           residual: torch.Tensor | None = None, Y=None,
                           workspace=None) -> torch.Tensor:
    """The experts' second product, summed over each token's experts: fp16 or bf16
    H [M k, N] in the plan's order, Wd [E, N, K] -> Y [M, K] = residual + sum of H[r] Wd_e."""
    dt = _dtype_of(H, "H")
    ldh = _matrix(H, "H", H)
    rows, M, E, k = _rows(plan, H)
    N, K = _last_dims(Wd, "Wd")
    _need_shape(H, "H", (M * k, N))
    ldw, sw = _expert_weights(Wd, "Wd", H, (E, N, K))
    r, ldr = None, 0
    if residual is not None:
        ldr, r = _matrix(residual, "residual", H, (M, K)), residual.data_ptr()
    Y, ldy = _out(Y, "Y", H, (M, K))
    ws, nb, keep = _experts_workspace("matmul", workspace, (M, K, N, E, k), H)
    _launch(lib().llmint8_experts_matmul, H, H.data_ptr(), M, N, ldh, Wd.data_ptr(), ldw, sw, K,
            rows, r, ldr, dt, Y.data_ptr(), ldy, ws, nb)
    return Y


def llmint8_experts_matmul_backward_workspace_size(M: int, K: int, N: int, E: int, k: int) -> int:
    return int(lib().llmint8_experts_matmul_backward_workspace_size(M, K, N, E, k))


def llmint8_experts_matmul_backward(dY: torch.Tensor, H: torch.Tensor | None, Wd: torch.Tensor,
                                    plan: ExpertPlan, *, need_dH: bool = True,
                                    need_dW: bool = True, dH=None, dWd=None, workspace=None):
    """Gradients of llmint8_experts_matmul from dY [M, K]: (dH [M k, N], dWd [E, N, K]), None
    where not needed (the residual's gradient is dY). H may be None without need_dW. Rows of dH
    behind the plan's last are left as they were."""
    dt = _dtype_of(dY, "dY")
    lddy = _matrix(dY, "dY", dY)
    M, K = dY.shape
    rows, _, E, k = _rows(plan, dY, M)
    N = _last_dims(Wd, "Wd")[0]
    ldw, sw = _expert_weights(Wd, "Wd", dY, (E, N, K))
    if not (need_dH or need_dW):
        raise ValueError("no gradient is asked for")
    ldh = N
    if need_dW:
        if H is None:
            raise ValueError("dWd needs H")
        ldh = _matrix(H, "H", dY, (M * k, N))
    dH, lddh = _out(dH, "dH", dY, (M * k, N)) if need_dH else (None, 0)
    dWd, lddw, sdw = _out_experts(dWd, "dWd", dY, (E, N, K)) if need_dW else (None, 0, 0)
    ws, nb, keep = _experts_workspace("matmul_backward", workspace, (M, K, N, E, k), dY)
    _launch(lib().llmint8_experts_matmul_backward, dY, dY.data_ptr(), M, K, lddy,
            H.data_ptr() if need_dW else None, N, ldh, Wd.data_ptr(), ldw, sw, rows, dt,
            _address(dH), lddh, _address(dWd), lddw, sdw, ws, nb)
    return dH, dWd


# ---- block-scaled FP8 ----------------------------------------------------------------
# E4M3 codes in blocks of 128 along the reduction that share a power-of-two scale 2^(byte - 127).

FP8_BLOCK = 128


def llmint8_quantize_blockwise_fp8(W: torch.Tensor):
    """fp16 or bf16 W [K, N] -> (Wq8 uint8 E4M3 codes [N, K], scale bytes uint8
    [ceil(N / 128), ceil(K / 128)]): 128 x 128 entries share a scale."""
    dt = _dtype_of(W, "W")
    ldw = _matrix(W, "W", W)
    K, N = W.shape
    Wq = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    sw = torch.empty((-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)), dtype=torch.uint8, device=W.device)
    _launch(lib().llmint8_quantize_blockwise_fp8, W, W.data_ptr(), K, N, ldw, dt, Wq.data_ptr(),
            sw.data_ptr())
    return Wq, sw


def llmint8_quantize_rowblock_fp8(X: torch.Tensor):
    """fp16 or bf16 X [M, K] -> (Xq8 uint8 E4M3 codes [M, K], scale bytes uint8
    [M, ceil(K / 128)]): 128 entries of a row share a scale. This is how
    llmint8_linear_blockwise_fp8 codes its X."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    pitch = -(-K // (4 * FP8_BLOCK)) * 4
    sx = torch.empty((M, pitch), dtype=torch.uint8, device=X.device)
    _launch(lib().llmint8_quantize_rowblock_fp8, X, X.data_ptr(), M, K, ldx, dt, Xq.data_ptr(),
            sx.data_ptr(), pitch)
    return Xq, sx[:, :-(-K // FP8_BLOCK)]


def llmint8_linear_blockwise_fp8_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().llmint8_linear_blockwise_fp8_workspace_size(M, K, N))


def llmint8_linear_blockwise_fp8(X: torch.Tensor, Wq8: torch.Tensor, scales: torch.Tensor, *,
                                 bias: torch.Tensor | None = None, Y=None,
                                 workspace=None) -> torch.Tensor:
    """Y = X W + bias in block-scaled FP8: fp16 or bf16 X [M, K], which the call codes by rows,
    Wq8 [N, K] and scales from llmint8_quantize_blockwise_fp8 -> Y [M, N] of X's type."""
    dt = _dtype_of(X, "X")
    ldx = _matrix(X, "X", X)
    M, K = X.shape
    if not isinstance(Wq8, torch.Tensor) or Wq8.dim() != 2:
        raise ValueError("Wq8 must be contiguous [N, K]")
    N = Wq8.shape[0]
    w = _table(Wq8, "Wq8", torch.uint8, (N, K), X)
    blocks = (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK))
    if not (isinstance(scales, torch.Tensor) and scales.dtype is torch.uint8
            and scales.shape == blocks and scales.get_device() == X.get_device()):
        _need(scales, "scales", torch.uint8, 2)
        _need_shape(scales, "scales", blocks)
        raise ValueError(f"scales must be on {X.device}, got {scales.device}")
    lds = _ld(scales, "scales")
    b = None if bias is None else _vector(bias, "bias", X.dtype, N, X)
    Y, ldy = _out(Y, "Y", X, (M, N))
    L = lib()
    ws, nb, keep = _workspace(workspace,
                              L.llmint8_linear_blockwise_fp8_workspace_size(M, K, N), X)
    _launch(L.llmint8_linear_blockwise_fp8, X, X.data_ptr(), M, K, ldx, w, scales.data_ptr(), lds,
            N, dt, b, Y.data_ptr(), ldy, ws, nb)
    return Y
