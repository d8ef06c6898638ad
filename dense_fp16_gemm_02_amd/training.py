"""The operators of a training step around the projections (include/tg_grouped.h,
include/tg_embed.h, include/tg_adamw.h).

    tg_grouped_f16 / _bf16(...), tg_grouped_dx_*(...), tg_grouped_dw_*(...)  -> status
    tg_grouped_workspace_bytes(...), tg_grouped_plan(...)
    tg_embedding_f32 / _f16 / _bf16(...), tg_embedding_bwd_*(...)            -> status
    tg_embedding_bwd_workspace_bytes(...)
    tg_adamw(tensors, config, stream)                                       -> status
    grouped_linear(X, W, ends)               torch, differentiable
    embedding(tokens, W, ...)                torch, differentiable
    adamw(params, grads, ...), adamw_8bit(params, grads, ...), adamw_8bit_state(p)   torch

Argument marshalling, checks and autograd glue only, as in the package.
"""
from __future__ import annotations

import array
import ctypes
import functools
import math

from .projection import _lib, _p, _pkg, _refuse_modes, _row_stride, _rows, _s

TG_GROUPED_Y = 0  # include/tg_grouped.h
TG_GROUPED_DX = 1
TG_GROUPED_DW = 2
TG_ADAMW_BLOCK = 256  # include/tg_adamw.h
TG_ADAMW_F32 = 0
TG_ADAMW_F16 = 1
TG_ADAMW_BF16 = 2


class tg_adamw_tensor(ctypes.Structure):
    """One tensor of tg_adamw: addresses and the number of elements."""

    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64)]


class tg_adamw_config(ctypes.Structure):
    """What all tensors of a tg_adamw call share."""

    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("lr_at", ctypes.c_void_p), ("step_at", ctypes.c_void_p), ("g_scale", ctypes.c_void_p),
                ("p_type", ctypes.c_int), ("g_type", ctypes.c_int), ("copy_type", ctypes.c_int),
                ("bits", ctypes.c_int)]


def declare(lib) -> None:
    """Argument types of the entry points (called once by the package's load())."""
    i64, vp, ci, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.tg_grouped_workspace_bytes.restype = i64
    lib.tg_grouped_workspace_bytes.argtypes = [ci, vp, vp] + [i64] * 7
    lib.tg_grouped_plan.restype = ci
    lib.tg_grouped_plan.argtypes = [ci, vp, vp] + [i64] * 7 + [ctypes.c_char_p, i64]
    for what in ("", "dx_", "dw_"):
        for dtype in ("f16", "bf16"):
            fn = getattr(lib, f"tg_grouped_{what}{dtype}")
            fn.restype, fn.argtypes = ci, [vp] * 4 + [i64] * 8 + [vp, i64, vp]
    for dtype in ("f32", "f16", "bf16"):
        fn = getattr(lib, f"tg_embedding_{dtype}")
        fn.restype, fn.argtypes = ci, [vp] * 3 + [i64] * 5 + [cf, vp]
        fn = getattr(lib, f"tg_embedding_bwd_{dtype}")
        fn.restype, fn.argtypes = ci, [vp] * 3 + [i64] * 5 + [cf, i64, vp, i64, vp]
    lib.tg_embedding_bwd_workspace_bytes.restype = i64
    lib.tg_embedding_bwd_workspace_bytes.argtypes = [i64] * 3
    lib.tg_adamw.restype = ci
    lib.tg_adamw.argtypes = [vp, i64, ctypes.POINTER(tg_adamw_config), vp]


# ------------------------------------------------------------------ grouped
def tg_grouped_workspace_bytes(product: int, A, B, M: int, E: int, N: int, K: int, lda: int, ldb: int,
                               w_stride: int) -> int:
    """Workspace bytes of a grouped product (TG_GROUPED_*) for these arguments (-1: refused)."""
    return _lib().tg_grouped_workspace_bytes(product, _p(A), _p(B), M, E, N, K, lda, ldb, w_stride)


def tg_grouped_plan(product: int, A, B, M: int, E: int, N: int, K: int, lda: int, ldb: int, w_stride: int):
    """Host-only: (status, kernel names)."""
    buf = ctypes.create_string_buffer(128)
    st = _lib().tg_grouped_plan(product, _p(A), _p(B), M, E, N, K, lda, ldb, w_stride, buf, 128)
    return st, buf.value.decode()


def _grouped(name, A, B, ends, D, M, E, N, K, lda, ldb, stride, ldd, workspace, workspace_bytes, stream):
    return getattr(_lib(), name)(_p(A), _p(B), _p(ends), _p(D), M, E, N, K, lda, ldb, stride, ldd, _p(workspace),
                                 workspace_bytes, _s(stream))


def tg_grouped_f16(X, W, ends, Y, M: int, E: int, N: int, K: int, ldx: int, ldw: int, w_stride: int, ldy: int,
                   workspace, workspace_bytes: int, stream=None) -> int:
    """Enqueue Y[i] = X[i]·W[e]ᵀ (binary16); returns the C status code."""
    return _grouped("tg_grouped_f16", X, W, ends, Y, M, E, N, K, ldx, ldw, w_stride, ldy, workspace, workspace_bytes,
                    stream)


def tg_grouped_bf16(X, W, ends, Y, M: int, E: int, N: int, K: int, ldx: int, ldw: int, w_stride: int, ldy: int,
                    workspace, workspace_bytes: int, stream=None) -> int:
    """tg_grouped_f16 for bfloat16 operands."""
    return _grouped("tg_grouped_bf16", X, W, ends, Y, M, E, N, K, ldx, ldw, w_stride, ldy, workspace,
                    workspace_bytes, stream)


def tg_grouped_dx_f16(dY, W, ends, dX, M: int, E: int, N: int, K: int, lddy: int, ldw: int, w_stride: int, lddx: int,
                      workspace, workspace_bytes: int, stream=None) -> int:
    """Enqueue dX[i] = dY[i]·W[e] (binary16); returns the C status code."""
    return _grouped("tg_grouped_dx_f16", dY, W, ends, dX, M, E, N, K, lddy, ldw, w_stride, lddx, workspace,
                    workspace_bytes, stream)


def tg_grouped_dx_bf16(dY, W, ends, dX, M: int, E: int, N: int, K: int, lddy: int, ldw: int, w_stride: int,
                       lddx: int, workspace, workspace_bytes: int, stream=None) -> int:
    """tg_grouped_dx_f16 for bfloat16 operands."""
    return _grouped("tg_grouped_dx_bf16", dY, W, ends, dX, M, E, N, K, lddy, ldw, w_stride, lddx, workspace,
                    workspace_bytes, stream)


def _grouped_dw(name, dY, X, ends, dW, M, E, N, K, lddy, ldx, lddw, dw_stride, workspace, workspace_bytes, stream):
    return getattr(_lib(), name)(_p(dY), _p(X), _p(ends), _p(dW), M, E, N, K, lddy, ldx, lddw, dw_stride,
                                 _p(workspace), workspace_bytes, _s(stream))


def tg_grouped_dw_f16(dY, X, ends, dW, M: int, E: int, N: int, K: int, lddy: int, ldx: int, lddw: int,
                      dw_stride: int, workspace, workspace_bytes: int, stream=None) -> int:
    """Enqueue dW[e] = Σ dY[i]ᵀ·X[i] (binary16); returns the C status code."""
    return _grouped_dw("tg_grouped_dw_f16", dY, X, ends, dW, M, E, N, K, lddy, ldx, lddw, dw_stride, workspace,
                       workspace_bytes, stream)


def tg_grouped_dw_bf16(dY, X, ends, dW, M: int, E: int, N: int, K: int, lddy: int, ldx: int, lddw: int,
                       dw_stride: int, workspace, workspace_bytes: int, stream=None) -> int:
    """tg_grouped_dw_f16 for bfloat16 operands."""
    return _grouped_dw("tg_grouped_dw_bf16", dY, X, ends, dW, M, E, N, K, lddy, ldx, lddw, dw_stride, workspace,
                       workspace_bytes, stream)


# ---------------------------------------------------------------- embedding
def _embedding(name, tokens, W, Y, M, V, K, ldw, ldy, scale, stream):
    return getattr(_lib(), name)(_p(tokens), _p(W), _p(Y), M, V, K, ldw, ldy, scale, _s(stream))


def tg_embedding_f32(tokens, W, Y, M: int, V: int, K: int, ldw: int, ldy: int, scale: float, stream=None) -> int:
    """Enqueue Y[i] = scale·W[tokens[i]] (fp32); returns the C status code."""
    return _embedding("tg_embedding_f32", tokens, W, Y, M, V, K, ldw, ldy, scale, stream)


def tg_embedding_f16(tokens, W, Y, M: int, V: int, K: int, ldw: int, ldy: int, scale: float, stream=None) -> int:
    """tg_embedding_f32 for binary16 rows."""
    return _embedding("tg_embedding_f16", tokens, W, Y, M, V, K, ldw, ldy, scale, stream)


def tg_embedding_bf16(tokens, W, Y, M: int, V: int, K: int, ldw: int, ldy: int, scale: float, stream=None) -> int:
    """tg_embedding_f32 for bfloat16 rows."""
    return _embedding("tg_embedding_bf16", tokens, W, Y, M, V, K, ldw, ldy, scale, stream)


def tg_embedding_bwd_workspace_bytes(M: int, V: int, K: int) -> int:
    """Workspace bytes of tg_embedding_bwd_* for these sizes (-1: refused)."""
    return _lib().tg_embedding_bwd_workspace_bytes(M, V, K)


def _embedding_bwd(name, tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace, workspace_bytes, stream):
    return getattr(_lib(), name)(_p(tokens), _p(dY), _p(dW), M, V, K, lddy, lddw, scale, padding, _p(workspace),
                                 workspace_bytes, _s(stream))


def tg_embedding_bwd_f32(tokens, dY, dW, M: int, V: int, K: int, lddy: int, lddw: int, scale: float, padding: int,
                         workspace, workspace_bytes: int, stream=None) -> int:
    """Enqueue dW[v] = scale·Σ dY[i] over the rows of token v (fp32); returns the C status code."""
    return _embedding_bwd("tg_embedding_bwd_f32", tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace,
                          workspace_bytes, stream)


def tg_embedding_bwd_f16(tokens, dY, dW, M: int, V: int, K: int, lddy: int, lddw: int, scale: float, padding: int,
                         workspace, workspace_bytes: int, stream=None) -> int:
    """tg_embedding_bwd_f32 for binary16 rows."""
    return _embedding_bwd("tg_embedding_bwd_f16", tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace,
                          workspace_bytes, stream)


def tg_embedding_bwd_bf16(tokens, dY, dW, M: int, V: int, K: int, lddy: int, lddw: int, scale: float, padding: int,
                          workspace, workspace_bytes: int, stream=None) -> int:
    """tg_embedding_bwd_f32 for bfloat16 rows."""
    return _embedding_bwd("tg_embedding_bwd_bf16", tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace,
                          workspace_bytes, stream)


# ------------------------------------------------------------------- adamw
def tg_adamw(tensors, config: tg_adamw_config, stream=None) -> int:
    """Enqueue one step over a sequence (or ctypes array) of tg_adamw_tensor; returns the C status code."""
    if not isinstance(tensors, ctypes.Array):
        tensors = (tg_adamw_tensor * len(tensors))(*tensors)
    return _lib().tg_adamw(ctypes.addressof(tensors) if len(tensors) else None, len(tensors), ctypes.byref(config),
                           _s(stream))


# ------------------------------------------------------------------ torch
@functools.lru_cache(maxsize=None)
def _cuda():
    """torch's current stream (as an address) and current device by index: what
    torch.cuda.current_stream and current_device look up, without the objects around
    it (2 of some 10 us of a small call)."""
    import torch

    return torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


@functools.lru_cache(maxsize=None)
def _queries():
    """torch.jit.is_tracing, whether any dispatch mode is on, and forward mode's levels."""
    import torch
    from torch.autograd import forward_ad
    from torch.utils._python_dispatch import is_in_torch_dispatch_mode

    return torch.jit.is_tracing, is_in_torch_dispatch_mode, forward_ad


def _refuse(what, *tensors):
    """_refuse_modes where there is any mode to refuse: a trace, or a level of dual tensors."""
    is_tracing, in_any_mode, forward_ad = _queries()
    if is_tracing() or in_any_mode() or forward_ad._current_level >= 0:
        _refuse_modes(what, *tensors)


def _call(index, fn, args, what):
    """fn(*args, stream) on torch's current stream of device ``index``, as the current device."""
    stream, device = _cuda()
    if device() == index:
        st = fn(*args, stream(index))
    else:
        import torch

        with torch.cuda.device(index):
            st = fn(*args, stream(index))
    if st:
        raise _pkg().TgError(st, what)


@functools.lru_cache(maxsize=1024)
def _grouped_plan(product, dtype, a_aligned, b_aligned, M, E, N, K, lda, ldb, w_stride):
    """Entry point and workspace bytes; of the pointers only their alignment counts."""
    import torch

    name = ("tg_grouped_", "tg_grouped_dx_", "tg_grouped_dw_")[product] + ("f16" if dtype == torch.float16 else "bf16")
    size = _lib().tg_grouped_workspace_bytes(product, 4096 if a_aligned else 4098, 4096 if b_aligned else 4098, M, E,
                                             N, K, lda, ldb, w_stride)
    return getattr(_lib(), name), max(0, size)


def _grouped_call(product, A, B, lda, ldb, w_stride, ends, D, N, K, ldd, d_stride=0):
    """Workspace, stream and device around one product of the library."""
    a, b = A.data_ptr(), B.data_ptr()
    M, E = A.shape[0], ends.shape[0]
    fn, size = _grouped_plan(product, A.dtype, a % 16 == 0, b % 16 == 0, M, E, N, K, lda, ldb, w_stride)
    ws = _bytes(A, size) if size else None
    last = (ldd, d_stride) if product == TG_GROUPED_DW else (w_stride, ldd)
    _call(A.get_device(), fn, (a, b, ends.data_ptr(), D.data_ptr(), M, E, N, K, lda, ldb, *last, _p(ws), size),
          "grouped_linear (backward)" if product else "grouped_linear")


@functools.lru_cache(maxsize=None)
def _uint8():
    import torch

    return torch.uint8


def _bytes(like, size):
    """A workspace on the device of ``like``."""
    return like.new_empty((size,), dtype=_uint8())


def _grouped_strides(X, W, ends, dev):
    """Row strides of X and W and the expert stride of W, of operands that are checked: all on
    the GPU ``dev`` (None: X is on none)."""
    import torch

    if X.dtype != W.dtype or X.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("X and W must both be float16 or both bfloat16")
    if ends.dtype != torch.int64:
        raise TypeError("ends must be int64")
    if not X.device == W.device == ends.device == dev:
        raise ValueError("X, W and ends must be GPU tensors on the same device")
    if X.dim() != 2 or W.dim() != 3 or ends.dim() != 1:
        raise ValueError("X must be 2-D, W 3-D and ends 1-D")
    if X.shape[1] != W.shape[2]:
        raise ValueError(f"K mismatch: X is {tuple(X.shape)}, W is {tuple(W.shape)}")
    if ends.shape[0] != W.shape[0]:
        raise ValueError(f"{ends.shape[0]} ends for {W.shape[0]} experts")
    return (_row_stride(X, "X", X.shape[1]), *_weight_strides(W))


def _weight_strides(W):
    """Row and expert strides of the weights; experts may share memory, rows may not."""
    E, N, K = W.shape
    stride = W.stride()
    if K > 1 and stride[2] != 1:
        raise ValueError("W must have a contiguous last dimension")
    ldw = stride[1] if N > 1 else max(K, 1)
    if ldw < K:
        raise ValueError(f"W has row stride {ldw} < row length {K}; pass a tensor with non-overlapping rows")
    return ldw, stride[0] if E > 1 else N * ldw


def _grouped_forward(X, W, ends, strides):
    N, K = W.shape[1:]
    Y = X.new_empty((X.shape[0], N))
    _grouped_call(TG_GROUPED_Y, X, W, *strides, ends, Y, N, K, max(N, 1))
    return Y


def _grouped_backward(X, W, ends, dY, strides, need_x, need_w):
    N, K = W.shape[1:]
    ldx, ldw, w_stride = strides
    ldy, ldk = N or 1, K or 1
    if not dY.is_contiguous():
        dY = _rows(dY)
        ldy = _row_stride(dY, "dY", N)
    dX = dW = None
    if need_x:
        dX = X.new_empty(X.shape)
        _grouped_call(TG_GROUPED_DX, dY, W, ldy, ldw, w_stride, ends, dX, N, K, ldk)
    if need_w:
        dW = W.new_empty(W.shape)
        _grouped_call(TG_GROUPED_DW, dY, X, ldy, ldx, 0, ends, dW, N, K, ldk, N * ldk)
    return dX, dW


def _grouped_layout(X, W, ends):
    """What a call of the library takes from its operands besides their addresses."""
    return (X.stride(), W.stride(), ends.stride(), X.shape, W.shape, ends.shape, X.dtype, W.dtype, ends.dtype,
            X.get_device(), W.get_device(), ends.get_device())


def _grouped_saved(X, W, ends, dY):
    """What the forward pass saved, and its strides, where hooks on saved tensors (offloading)
    brought it back in other memory than it was in."""
    if X.dim() == 2:
        X = _rows(X)
    if W.dim() == 3 and ((W.shape[2] > 1 and W.stride(2) != 1) or (W.shape[1] > 1 and W.stride(1) < W.shape[2])):
        W = W.contiguous()
    ends = ends.contiguous()
    strides = _grouped_strides(X, W, ends, dY.device)
    if dY.dtype != X.dtype or dY.shape != (X.shape[0], W.shape[1]):
        raise ValueError("X or W comes back from its hook as another tensor than was saved")
    return X, W, ends, strides


@functools.lru_cache(maxsize=None)
def _grouped_function():
    import torch

    class Gradients(torch.autograd.Function):
        """dX and dW as values with a graph, for create_graph: what depends on them
        would need second derivatives, which there are none of, and raises."""

        @staticmethod
        def forward(ctx, X, W, ends, dY, *how):
            return _grouped_backward(X, W, ends, dY, *how)

        @staticmethod
        def backward(ctx, *_):
            raise RuntimeError("grouped_linear can be differentiated once")

    class GroupedLinear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, ends, strides):
            ctx.save_for_backward(X, W, ends)
            ctx.layout, ctx.strides = _grouped_layout(X, W, ends), strides
            return _grouped_forward(X, W, ends, strides)

        @staticmethod
        def backward(ctx, dY):
            X, W, ends = ctx.saved_tensors
            strides = ctx.strides
            # (one comparison: every question here costs twice, on autograd's own thread)
            if _grouped_layout(X, W, ends) != ctx.layout:
                X, W, ends, strides = _grouped_saved(X, W, ends, dY)
            _refuse("grouped_linear (backward)", dY)
            gradients = Gradients.apply if torch.is_grad_enabled() else _grouped_backward
            need = ctx.needs_input_grad
            return (*gradients(X, W, ends, dY, strides, need[0], need[1]), None, None)

    return GroupedLinear


def grouped_linear(X, W, ends):
    """Rows grouped by expert times their expert's weight: Y[i] = X[i]·W[e]ᵀ for
    ends[e-1] <= i < ends[e] (ends[-1] taken as 0); rows from the last end on are 0.

    X (M×K, rows sorted by expert) and W (E×N×K, one weight as ``gemm`` takes its B
    for each expert) are fp16 or bf16 GPU tensors of one dtype on one device, with a
    contiguous last dimension and non-overlapping rows; ``ends`` holds E int64
    values on that device, e.g. ``torch.bincount(expert, minlength=E).cumsum(0)``. It
    is read there and nowhere checked: a value counts as at least the one before it
    and as 0 to M.  Returns Y (M×N) of that dtype, fp32 sums rounded once; it can be
    differentiated with respect to X and W, once (under create_graph, what depends on
    the gradients raises RuntimeError).  An expert without rows has a gradient of 0,
    rows behind the last end have one of 0 and reach no gradient.

    Runs on torch's current stream, never waits for the device, and takes its
    workspace (for operands without 16-byte aligned rows, and for sums cut into parts)
    from torch's allocator; it may be captured into a graph, whose replays read ``ends``
    anew, its backward pass with torch.autograd.grad, or with .backward() where no
    eager graph of the same leaves is alive (autograd would accumulate on that graph's
    stream, which ends the capture).  Under torch.compile it runs between the
    compiled parts.  Raises TypeError / ValueError on tensors it cannot take,
    NotImplementedError on dual tensors (there is no forward-mode derivative) and
    while torch.jit.trace or make_fx records (they would not see the call), and
    TgError on a non-zero status.
    """
    import torch

    if torch.compiler.is_dynamo_compiling():  # the call stays between the compiled parts
        return torch.compiler.disable(grouped_linear)(X, W, ends)
    strides = _grouped_strides(X, W, ends, X.device if X.is_cuda else None)
    _refuse("grouped_linear", X, W)
    ends = ends.contiguous()
    if torch.is_grad_enabled() and (X.requires_grad or W.requires_grad):
        return _grouped_function().apply(X, W, ends, strides)
    return _grouped_forward(X, W, ends, strides)


@functools.lru_cache(maxsize=None)
def _embedding_names():
    import torch

    return {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


@functools.lru_cache(maxsize=8)
def _embedding_entry(dtype, backward):
    return getattr(_lib(), ("tg_embedding_bwd_" if backward else "tg_embedding_") + _embedding_names()[dtype])


def _embedding_forward(tokens, W, ldw, scale):
    V, K = W.shape
    Y = W.new_empty((*tokens.shape, K))
    _call(W.get_device(), _embedding_entry(W.dtype, False),
          (tokens.data_ptr(), W.data_ptr(), Y.data_ptr(), tokens.numel(), V, K, ldw, max(K, 1), scale), "embedding")
    return Y


@functools.lru_cache(maxsize=1024)
def _embedding_size(M, V, K):
    return max(0, _lib().tg_embedding_bwd_workspace_bytes(M, V, K))


def _embedding_backward(tokens, dY, V, scale, padding):
    M, K = tokens.numel(), dY.shape[-1]
    lddy = K
    if not dY.is_contiguous():
        dY = _rows(dY.reshape(M, K))
        lddy = _row_stride(dY, "dY", K)
    dW = dY.new_empty((V, K))
    size = _embedding_size(M, V, K)
    ws = _bytes(dY, size)
    _call(dY.get_device(), _embedding_entry(dY.dtype, True),
          (tokens.data_ptr(), dY.data_ptr(), dW.data_ptr(), M, V, K, lddy, K, scale, padding, ws.data_ptr(), size),
          "embedding (backward)")
    return dW


@functools.lru_cache(maxsize=None)
def _embedding_function():
    import torch

    class Gradient(torch.autograd.Function):
        """dW as a value with a graph, for create_graph: what depends on it would
        need a second derivative, which there is none of, and raises."""

        @staticmethod
        def forward(ctx, *how):
            return _embedding_backward(*how)

        @staticmethod
        def backward(ctx, *_):
            raise RuntimeError("embedding can be differentiated once")

    class Embedding(torch.autograd.Function):
        @staticmethod
        def forward(ctx, tokens, W, ldw, scale, padding):
            ctx.save_for_backward(tokens)
            ctx.how = W.shape[0], scale, padding
            return _embedding_forward(tokens, W, ldw, scale)

        @staticmethod
        def backward(ctx, dY):
            tokens = ctx.saved_tensors[0].contiguous()  # a hook may have brought them back in other memory
            if tokens.dtype != torch.int64 or tokens.shape != dY.shape[:-1] or \
                    tokens.get_device() != dY.get_device():
                raise ValueError("tokens come back from their hook as another tensor than was saved")
            _refuse("embedding (backward)", dY)
            gradient = Gradient.apply if torch.is_grad_enabled() else _embedding_backward
            return None, gradient(tokens, dY, *ctx.how), None, None, None

    return Embedding


def embedding(tokens, W, scale: float = 1.0, padding_idx: int | None = None):
    """Embedding lookup: Y[...] = scale·W[tokens[...]].

    ``tokens`` holds int64 indices in any shape, W (V×K) is a fp32, fp16 or bf16 GPU
    tensor on the same device with a contiguous last dimension and non-overlapping
    rows; the result has the shape of tokens and K behind it, and W's dtype.  It can be
    differentiated with respect to W, once (under create_graph, what depends on the
    gradient raises RuntimeError): dW[v] = scale·Σ dY over the tokens v, summed in
    fp32 in the order of the tokens and rounded once, so that it is the same at every
    call.  Row ``padding_idx``, from 0 to V - 1, gets no gradient (its row of Y is read as
    any other).
    A token outside [0, V) makes its row NaN and adds to no gradient.

    It gathers any rows: the tokens' hidden states in the order that ``grouped_linear``
    takes them, with a gradient that adds up what a token's experts send back.

    Runs on torch's current stream, never waits for the device, and takes its
    workspace from torch's allocator; capture into graphs, torch.compile and the
    exceptions are as for ``grouped_linear``.
    """
    import torch

    if torch.compiler.is_dynamo_compiling():  # the call stays between the compiled parts
        return torch.compiler.disable(embedding)(tokens, W, scale, padding_idx)
    if W.dtype not in _embedding_names():
        raise TypeError("W must be float32, float16 or bfloat16")
    if tokens.dtype != torch.int64:
        raise TypeError("tokens must be int64")
    if not W.is_cuda or tokens.device != W.device:
        raise ValueError("tokens and W must be GPU tensors on the same device")
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    V, K = W.shape
    if not math.isfinite(scale) or abs(scale) > 3.4028234663852886e38:
        raise ValueError("scale must be a finite fp32 number")
    if padding_idx is not None and not 0 <= padding_idx < V:
        raise ValueError(f"padding_idx must be in [0, {V})")
    ldw = _row_stride(W, "W", K)
    _refuse("embedding", W)
    tokens = tokens.contiguous()
    if torch.is_grad_enabled() and W.requires_grad:
        return _embedding_function().apply(tokens, W, ldw, float(scale), -1 if padding_idx is None else padding_idx)
    return _embedding_forward(tokens, W, ldw, float(scale))


@functools.lru_cache(maxsize=None)
def _adamw_types():
    import torch

    return {torch.float32: TG_ADAMW_F32, torch.float16: TG_ADAMW_F16, torch.bfloat16: TG_ADAMW_BF16}


def _same_dtype(ts, name, allowed):
    """The dtype that all of ts have, one of ``allowed``."""
    dtypes = {t.dtype for t in ts}
    dtype = dtypes.pop()
    if dtypes or dtype not in allowed:
        raise TypeError(f"{name} must all be of one dtype among "
                        f"{', '.join(sorted(str(d).replace('torch.', '') for d in allowed))}")
    return dtype


def _scalar(x, name, dtype, dev):
    """The address of a one-element GPU tensor, or None for a number."""
    import torch

    if not isinstance(x, torch.Tensor):
        return None
    if x.dtype != dtype or x.numel() != 1 or x.device != dev:
        raise ValueError(f"{name} must be a number or a one-element {str(dtype).replace('torch.', '')} tensor on the "
                         "device of the parameters")
    return x.data_ptr()


def _adamw(what, params, grads, moments, scales, step, lr, betas, eps, weight_decay, g_scale, copies):
    import torch

    if torch.compiler.is_dynamo_compiling():  # the call stays between the compiled parts
        return torch.compiler.disable(_adamw)(what, params, grads, moments, scales, step, lr, betas, eps,
                                              weight_decay, g_scale, copies)
    bits = 8 if scales else 32
    lists = [list(params), list(grads)] + [list(x) for x in moments + scales] + ([list(copies)] if copies is not None else [])
    params, grads = lists[:2]
    count = len(params)
    if any([len(x) != count for x in lists]):
        raise ValueError("there must be as many gradients, moments and copies as parameters")
    if count == 0:
        return
    dev = params[0].device
    if not params[0].is_cuda:
        raise ValueError("params must be GPU tensors")
    try:
        dense = not any([t.is_sparse for t in grads])
    except AttributeError:  # None, where a parameter has no gradient
        dense = False
    if not dense:
        raise TypeError("grads must be dense tensors")
    f32, half = torch.float32, (torch.float16, torch.bfloat16)
    p_type = _same_dtype(params, "params", (f32, *half))
    g_type = _same_dtype(grads, "grads", (f32, *half) if p_type is f32 else (p_type,))
    held = f32 if bits == 32 else torch.float8_e4m3fn
    _same_dtype(lists[2], "exp_avgs", (held,))
    _same_dtype(lists[3], "exp_avg_sqs" if bits == 32 else "roots", (held,))
    if scales:
        _same_dtype(lists[4] + lists[5], "exp_avg_scales and root_scales", (f32,))
    copy_type = None
    if copies is not None:
        if p_type is not f32:
            raise ValueError("copies are for float32 parameters")
        copy_type = _same_dtype(lists[-1], "copies", half)
    _refuse(what, *params, *grads)
    # every list's tensors in a row, so that each question is asked in one pass
    index, sizes = dev.index, [p.numel() for p in params]
    every, want = [t for x in lists for t in x], sizes * len(lists)
    if scales:
        want[4 * count:6 * count] = [(n + TG_ADAMW_BLOCK - 1) // TG_ADAMW_BLOCK for n in sizes] * 2
    if [t.numel() for t in every] != want:
        raise ValueError("gradients, moments and copies must have as many elements as their parameter"
                         + (f", scales one for each {TG_ADAMW_BLOCK} of them" if scales else ""))
    if not all([t.is_contiguous() for t in every]):
        raise ValueError("parameters, gradients, moments and copies must be contiguous")
    if {t.get_device() for t in every} != {index}:
        raise ValueError("all tensors must be on one GPU")
    if [g.shape for g in grads] != [p.shape for p in params]:
        raise ValueError("a gradient has another shape than its parameter")
    written = params + every[2 * count:]
    if torch.is_grad_enabled() and not all([t.is_leaf for t in written if t.requires_grad]):
        raise ValueError("params, moments and copies that are results of autograd cannot be updated in place")
    types = _adamw_types()
    b1, b2 = betas
    lr_at, step_at = _scalar(lr, "lr", f32, dev), _scalar(step, "step", torch.int64, dev)
    config = tg_adamw_config(0.0 if lr_at else lr, b1, b2, eps, weight_decay, 1 if step_at else step, lr_at, step_at,
                             _scalar(g_scale, "grad_scale", f32, dev), types[p_type], types[g_type],
                             types[copy_type] if copy_type else 0, bits)
    if g_scale is not None and not isinstance(g_scale, torch.Tensor):
        raise TypeError("grad_scale must be a tensor")
    # tg_adamw_tensor structures: eight words each, a word of all of them at a time
    table, at = array.array("q", bytes(64 * count)), array.array("q", [t.data_ptr() for t in every])
    for k, word in enumerate((0, 1, 2, 3, 4, 5, 6) if scales else (0, 1, 2, 3, 6)):
        if k < len(lists):
            table[word::8] = at[k * count:(k + 1) * count]
    table[7::8] = array.array("q", sizes)
    _call(index, _lib().tg_adamw, (table.buffer_info()[0], count, ctypes.byref(config)), what)
    torch.autograd.graph.increment_version(written)


def adamw(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
          weight_decay: float = 1e-2, grad_scale=None, copies=None) -> None:
    """One AdamW step over lists of tensors, in place:

        m ← β1·m + (1 − β1)·g,   v ← β2·v + (1 − β2)·g²
        p ← (1 − lr·wd)·p − lr/(1 − β1^step)·m / (√v/√(1 − β2^step) + eps)

    ``params`` are contiguous fp32, fp16 or bf16 GPU tensors of one dtype on one
    device, ``grads`` tensors of their shapes and dtype (or any one of the three where
    the parameters are fp32), ``exp_avgs`` and ``exp_avg_sqs`` the moments m and v,
    fp32 and zeros before the first step.  ``step`` counts from 1.  ``copies``, where
    given, are fp16 or bf16 tensors of fp32 parameters' sizes that receive them rounded.
    ``grad_scale``, a one-element fp32 tensor on the device, multiplies the gradients
    (the factor that clips their norm, or a loss scale's inverse).  An ``eps`` below 2^-126
    counts as 0, with which an element whose moments are 0 becomes NaN.

    ``lr`` and ``step`` may be one-element tensors on the device (fp32 and int64): a
    call captured into a graph reads them anew at each replay.  Nothing is advanced
    here.  All tensors are taken in few launches; the arithmetic is fp32 throughout
    (include/tg_adamw.h).  Parameters may require grad; what is written counts as
    modified in place.

    Runs on torch's current stream without a workspace.  Under torch.compile it runs
    between the compiled parts.  Raises TypeError / ValueError on tensors it cannot
    take, NotImplementedError on dual tensors and while torch.jit.trace or make_fx
    records, and TgError on a non-zero status, among them tensors that share memory.
    """
    _adamw("adamw", params, grads, [exp_avgs, exp_avg_sqs], [], step, lr, betas, eps, weight_decay, grad_scale, copies)


def adamw_8bit_state(p):
    """The moments of one parameter before the first ``adamw_8bit`` step: (exp_avg,
    exp_avg_scale, root, root_scale), zeros.  A moment's values are those of the E4M3
    tensor times their block's scale: ``exp_avg.float().flatten() *
    exp_avg_scale.repeat_interleave(256)[:p.numel()]``, and the second moment is the square of the root's."""
    import torch

    blocks = (p.numel() + TG_ADAMW_BLOCK - 1) // TG_ADAMW_BLOCK

    def codes():
        return torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn)

    def scales():
        return torch.zeros(blocks, dtype=torch.float32, device=p.device)

    return codes(), scales(), codes(), scales()


def adamw_8bit(params, grads, exp_avgs, exp_avg_scales, roots, root_scales, step, lr=1e-3, betas=(0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 1e-2, grad_scale=None, copies=None) -> None:
    """``adamw`` with moments held in 8 bits: E4M3 tensors of the parameters' sizes
    with one fp32 scale for each 256 elements, of m and of √v (``adamw_8bit_state``
    makes them).  The step itself uses the moments before they are rounded; a rounding
    is at most 2^-4 of the value.  Large updates take a fifth longer with ``lr`` or ``step`` on
    the device.  include/tg_adamw.h says what is held of small,
    infinite and NaN values.  Everything else is as for ``adamw``."""
    _adamw("adamw_8bit", params, grads, [exp_avgs, roots], [exp_avg_scales, root_scales], step, lr, betas, eps,
           weight_decay, grad_scale, copies)
