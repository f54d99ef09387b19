"""Bindings of ``libmi355fused.so`` (``include/mi355fused.h``): the products of
a language model with the work around them folded in.

    gemm_gated(X, Wg, Wu, H, act="silu", G=None, U=None)
                                  # H = act(X@Wg.T) * (X@Wu.T)
    gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX=None, dWg=None, dWu=None, act="silu")
                                  # its gradients
    gemm_w4(X, Wq, scales, C, group=128, zeros=None, ...)
                                  # C = act(X@W.T + bias) + residual, W in 4 bits
    gemm_xent(X, W, targets, loss, lse)      # cross entropy of X@W.T, no logits kept
    gemm_xent_bwd(X, W, targets, lse, dloss, dX=None, dW=None)
                                  # its gradients

As for the calls of the package itself: the outputs are the caller's tensors,
work is enqueued on ``stream`` (default: torch's current stream) and nothing is
synchronised.  All tensors of a call live on one GPU, which need not be the
current one; ``stream``, if given, belongs to that GPU.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import (ACTS, HERE, INT_MAX, _check, _current_stream_handle, _epilogue_args, _matrix,
               _torch_module, _workspace)

LIB_PATH = os.path.join(HERE, "libmi355fused.so")
_lock = threading.Lock()
_lib = None


def load_library() -> ctypes.CDLL:
    """Load ``libmi355fused.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError("%s is missing: build it with `python -m dense_gemm_sgemm_amd.build` "
                              "(or __graft_entry__.build())" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        i, p, u64, i64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_ulonglong, ctypes.c_longlong
        mat = [p, i]

        def declare(name, args, restype=i):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, restype

        declare("gemm_gated", [i] * 5 + mat * 6 + [p, u64, p])
        declare("gemm_gated_workspace", [i] * 4 + mat * 3, u64)
        declare("gemm_gated_bwd", [i] * 5 + mat * 9 + [p, u64, p])
        declare("gemm_gated_bwd_workspace", [i] * 4 + mat * 3 + [i, i], u64)
        declare("gemm_w4", [i] * 5 + mat * 4 + [p, i] + mat * 2 + [p])
        declare("gemm_xent", [i] * 4 + mat * 2 + [p, i64, p, p, p, u64, p])
        declare("gemm_xent_workspace", [i] * 4 + mat * 2, u64)
        declare("gemm_xent_bwd", [i] * 4 + mat * 2 + [p, i64, p, p] + mat * 2 + [p, u64, p])
        declare("gemm_xent_bwd_workspace", [i] * 4 + mat * 2 + [i, i], u64)
        _lib = lib
        return lib


_Tensor = None   # torch.Tensor, once a call has needed it


def _first(t):
    """(dtype, GEMM_TYPE_*, GPU index, rows, columns, pointer, leading dimension)
    of the call's X; the other operands are held to its type and GPU."""
    global _Tensor
    torch = _torch_module()
    _Tensor = torch.Tensor
    dtype = t.dtype if isinstance(t, _Tensor) else None
    if dtype is torch.bfloat16:
        typ = 1
    elif dtype is torch.float16:
        typ = 0
    else:
        raise TypeError("X must be a float16 or bfloat16 tensor")
    rows, cols, ld, ptr = _matrix(t, "X", dtype)
    return dtype, typ, t.get_device(), rows, cols, ptr, ld


def _rows(t, name) -> int:
    if not isinstance(t, _Tensor) or t.dim() != 2:
        raise TypeError("%s must be a 2-D torch tensor" % name)
    rows = t.shape[0]
    if rows > INT_MAX:
        raise ValueError("%s: sizes must be below 2^31" % name)
    return rows


def _shaped(t, name, dtype, index, rows, cols):
    """(device pointer or None, leading dimension) of a rows x cols matrix on GPU
    ``index``.  Runs for every operand of every call: the usual case is told by
    the cheapest queries, and anything else by _matrix, which says what is wrong."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == (rows, cols) and \
            t.get_device() == index and rows > 1 and cols > 1:
        s0, s1 = t.stride()
        if s1 == 1 and s0 <= INT_MAX:
            return t.data_ptr(), s0
    r, c, ld, ptr = _matrix(t, name, dtype)
    if r != rows or c != cols:
        raise ValueError("%s must be %d x %d, got %s" % (name, rows, cols, tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("all tensors of a call must live on one GPU")
    return ptr, ld


def _optional(t, name, dtype, index, rows, cols):
    return (None, 0) if t is None else _shaped(t, name, dtype, index, rows, cols)


def _vector(t, name, dtype, index, n):
    torch = _torch_module()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or t.dim() != 1 or \
            t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s GPU vector of length %d" % (name, dtype, n))
    if t.get_device() != index:
        raise ValueError("all tensors of a call must live on one GPU")
    return t.data_ptr() if n else None


def _current_gpu() -> int:
    torch = _torch_module()
    get = getattr(torch._C, "_cuda_getDevice", None)   # as torch.cuda.current_device, less set-up
    return get() if get is not None else torch.cuda.current_device()


def _run(index, stream, fn, args, need=None, workspace=None):
    """``fn(*args[, workspace, bytes], stream)`` with GPU ``index`` current;
    ``need()`` gives the size of the workspace the call takes."""
    torch = _torch_module()
    if stream is not None and stream.device.index != index:
        raise ValueError("stream belongs to another GPU than the tensors")
    if index != _current_gpu():
        with torch.cuda.device(index):
            return _run(index, stream, fn, args, need, workspace)
    handle = stream.cuda_stream if stream is not None else _current_stream_handle()
    if need is None:
        status = fn(*args, handle)
    else:
        if workspace is not None and workspace.get_device() != index:
            raise ValueError("workspace must live on the GPU of the tensors")
        bytes_ = need() if workspace is None else 0
        if workspace is None and bytes_ == 0:
            status = fn(*args, None, 0, handle)
        else:
            pw, nw, _ws = _workspace(workspace, bytes_, "cuda:%d" % index, stream)
            status = fn(*args, pw, nw, handle)
    if status:
        _check(status)


def _act(act):
    if act not in ACTS:
        raise ValueError("act must be one of %s" % sorted(ACTS))
    return ACTS[act]


def gemm_gated(X, Wg, Wu, H, act: str = "silu", G=None, U=None, workspace=None, stream=None):
    """``H = act(X @ Wg.T) * (X @ Wu.T)`` for float16 or bfloat16 X[M,K], Wg[N,K],
    Wu[N,K] and H[M,N]; ``act`` "none", "relu" or "silu".  ``G`` and ``U``
    ([M,N], or None) receive the two products, which ``gemm_gated_bwd`` takes.
    ``workspace``: a contiguous GPU tensor of ``gated_workspace_bytes`` bytes, or
    None (taken from torch's allocator if the call needs one).  Returns H."""
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(Wg, "Wg")
    pg, ldg = _shaped(Wg, "Wg", dtype, at, N, K)
    pu, ldu = _shaped(Wu, "Wu", dtype, at, N, K)
    ph, ldh = _shaped(H, "H", dtype, at, M, N)
    pG, ldG = _optional(G, "G", dtype, at, M, N)
    pU, ldU = _optional(U, "U", dtype, at, M, N)
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_gated,
         (typ, _act(act), M, N, K, px, ldx, pg, ldg, pu, ldu, ph, ldh, pG, ldG, pU, ldU),
         lambda: lib.gemm_gated_workspace(typ, M, N, K, px, ldx, pg, ldg, pu, ldu), workspace)
    return H


def gated_workspace_bytes(X, Wg, Wu) -> int:
    """Workspace bytes ``gemm_gated`` needs for these tensors (0 when none)."""
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(Wg, "Wg")
    return load_library().gemm_gated_workspace(typ, M, N, K, px, ldx,
                                               *_shaped(Wg, "Wg", dtype, at, N, K),
                                               *_shaped(Wu, "Wu", dtype, at, N, K))


def gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX=None, dWg=None, dWu=None, act: str = "silu",
                   workspace=None, stream=None):
    """The gradients of ``gemm_gated`` for the gradient dH[M,N] of its result and
    the products G, U it stored: ``dX`` [M,K], ``dWg`` and ``dWu`` [N,K], each
    computed if given.  ``workspace``: ``gated_bwd_workspace_bytes`` bytes, or
    None.  Returns (dX, dWg, dWu)."""
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(Wg, "Wg")
    sizes = (M, N, K, px, ldx, *_shaped(Wg, "Wg", dtype, at, N, K),
             *_shaped(Wu, "Wu", dtype, at, N, K))
    ins = (*_shaped(G, "G", dtype, at, M, N), *_shaped(U, "U", dtype, at, M, N),
           *_shaped(dH, "dH", dtype, at, M, N))
    outs = (*_optional(dX, "dX", dtype, at, M, K), *_optional(dWg, "dWg", dtype, at, N, K),
            *_optional(dWu, "dWu", dtype, at, N, K))
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_gated_bwd, (typ, _act(act)) + sizes + ins + outs,
         lambda: lib.gemm_gated_bwd_workspace(typ, *sizes, dX is not None,
                                              dWg is not None or dWu is not None), workspace)
    return dX, dWg, dWu


def gated_bwd_workspace_bytes(X, Wg, Wu, want_dx: bool = True, want_dw: bool = True) -> int:
    """Workspace bytes ``gemm_gated_bwd`` needs for these tensors and gradients."""
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(Wg, "Wg")
    return load_library().gemm_gated_bwd_workspace(
        typ, M, N, K, px, ldx, *_shaped(Wg, "Wg", dtype, at, N, K),
        *_shaped(Wu, "Wu", dtype, at, N, K), bool(want_dx), bool(want_dw))


def gemm_w4(X, Wq, scales, C, group: int = 128, zeros=None, bias=None, act: str = "none",
            residual=None, stream=None):
    """``C = act(X @ W.T + bias) + residual`` with 4-bit weights,
    ``W[n,k] = (q[n,k] - zero[n,k//group]) * scale[n,k//group]``, for float16 or
    bfloat16 X[M,K] and C[M,N].  ``Wq``: uint8 [N, ceil(K/2)], q of even k in the
    low half of byte k // 2; ``group``: a multiple of 32; ``scales``: X's dtype,
    [N, ceil(K/group)]; ``zeros``: uint8 of the same shape with values 0 to 15,
    or None for 8.  Meant for the few rows of decode steps (the weights are
    streamed once for every 64 rows).  Returns C."""
    torch = _torch_module()
    dtype, typ, at, M, K, px, ldx = _first(X)
    if group <= 0 or group > INT_MAX:
        raise ValueError("group must be a positive multiple of 32 below 2^31")
    N = _rows(Wq, "Wq")
    groups = -(-K // group)
    pq, ldq = _shaped(Wq, "Wq", torch.uint8, at, N, (K + 1) // 2)
    ps, lds = _shaped(scales, "scales", dtype, at, N, groups)
    pz, ldz = _optional(zeros, "zeros", torch.uint8, at, N, groups)
    pc, ldc = _shaped(C, "C", dtype, at, M, N)
    if bias is None and residual is None:
        pbias, code, pres, ldr = None, _act(act), None, 0
    else:
        for t in (bias, residual):
            if t is not None and t.get_device() != at:
                raise ValueError("all tensors of a call must live on one GPU")
        pbias, code, pres, ldr = _epilogue_args(bias, act, residual, M, N, dtype)
    _run(at, stream, (_lib or load_library()).gemm_w4,
         (typ, M, N, K, group, px, ldx, pq, ldq, ps, lds, pz, ldz, pbias, code, pres, ldr, pc, ldc))
    return C


def _xent_args(X, W):
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(W, "W")
    return dtype, at, (typ, M, N, K, px, ldx, *_shaped(W, "W", dtype, at, N, K))


def gemm_xent(X, W, targets, loss, lse, ignore_index: int = -100, workspace=None, stream=None):
    """Softmax cross entropy of each row of ``X @ W.T`` (X[M,K], W[N,K], float16 or
    bfloat16) against the column ``targets[m]`` (int64 [M]), without storing the
    products: float32 [M] ``loss`` and ``lse`` (log of the sum of exponentials,
    which ``gemm_xent_bwd`` takes).  Rows with target ``ignore_index`` have loss
    0; a target outside [0, N) otherwise gives NaN.  ``workspace``:
    ``xent_workspace_bytes`` bytes, or None.  Returns loss."""
    torch = _torch_module()
    _, at, sizes = _xent_args(X, W)
    M = sizes[1]
    pt = _vector(targets, "targets", torch.int64, at, M)
    pl = _vector(loss, "loss", torch.float32, at, M)
    pe = _vector(lse, "lse", torch.float32, at, M)
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_xent, sizes + (pt, int(ignore_index), pl, pe),
         lambda: lib.gemm_xent_workspace(*sizes), workspace)
    return loss


def xent_workspace_bytes(X, W) -> int:
    """Workspace bytes ``gemm_xent`` needs for these tensors."""
    return load_library().gemm_xent_workspace(*_xent_args(X, W)[2])


def gemm_xent_bwd(X, W, targets, lse, dloss, dX=None, dW=None, ignore_index: int = -100,
                  workspace=None, stream=None):
    """The gradients of ``gemm_xent`` for the gradient ``dloss`` (float32 [M]) of
    each row's loss and the ``lse`` it stored: ``dX`` [M,K] and ``dW`` [N,K], each
    computed if given.  ``workspace``: ``xent_bwd_workspace_bytes`` bytes, or None.
    Returns (dX, dW)."""
    torch = _torch_module()
    dtype, at, sizes = _xent_args(X, W)
    M, N, K = sizes[1:4]
    pt = _vector(targets, "targets", torch.int64, at, M)
    pe = _vector(lse, "lse", torch.float32, at, M)
    pd = _vector(dloss, "dloss", torch.float32, at, M)
    outs = (*_optional(dX, "dX", dtype, at, M, K), *_optional(dW, "dW", dtype, at, N, K))
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_xent_bwd, sizes + (pt, int(ignore_index), pe, pd) + outs,
         lambda: lib.gemm_xent_bwd_workspace(*sizes, dX is not None, dW is not None), workspace)
    return dX, dW


def xent_bwd_workspace_bytes(X, W, want_dx: bool = True, want_dw: bool = True) -> int:
    """Workspace bytes ``gemm_xent_bwd`` needs for these tensors and gradients."""
    return load_library().gemm_xent_bwd_workspace(*_xent_args(X, W)[2], bool(want_dx),
                                                  bool(want_dw))
