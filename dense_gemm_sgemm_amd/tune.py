"""Bindings of ``libmi355tune.so`` (``include/mi355tune.h``): what fine tuning
needs next to a model's products.

    gemm_lora(X, W, A, B, ids, C, scales=None, T=None, ...)
                                  # C[m] = act(X[m]@W.T + scales[a] X[m]@A[a].T@B[a].T + bias)
                                  #        + residual[m], a = ids[m]
    gemm_lora_bwd(X, W, A, B, ids, T, dC, dX=None, dA=None, dB=None, scales=None)
                                  # its gradients, W frozen
    gemm_ortho(G, O, steps=5, coeffs=(a, b, c), eps=1e-7)
                                  # O = G orthogonalised by Newton-Schulz products

As for the other calls: the outputs are the caller's tensors, work is enqueued
on ``stream`` (default: torch's current stream) and nothing is synchronised.
All tensors of a call live on one GPU, which need not be the current one;
``stream``, if given, belongs to that GPU.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import HERE, INT_MAX, _epilogue_args, _torch_module
from .fused import _act, _first, _optional, _rows, _run, _shaped, _vector

LIB_PATH = os.path.join(HERE, "libmi355tune.so")
_lock = threading.Lock()
_lib = None


def load_library() -> ctypes.CDLL:
    """Load ``libmi355tune.so``; raises if it has not been built."""
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
        f = ctypes.c_float

        def declare(name, args, restype=i):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, restype

        mat, stack = [p, i], [p, i, i64]
        declare("gemm_lora", [i] * 6 + mat * 2 + stack * 2 + [p, p, p, i] + mat * 3 + [p, u64, p])
        declare("gemm_lora_workspace", [i] * 6 + mat * 2 + [i], u64)
        declare("gemm_lora_bwd",
                [i] * 6 + mat * 2 + stack * 2 + [p, p] + mat * 3 + stack * 2 + [p, u64, p])
        declare("gemm_lora_bwd_workspace", [i] * 6 + mat * 2 + [i] * 3, u64)
        declare("gemm_ortho", [i] * 5 + [p, i, i64, i, ctypes.POINTER(f), f, p, i, i64, p, u64, p])
        declare("gemm_ortho_workspace", [i] * 6, u64)
        _lib = lib
        return lib


_types = None


def _type_code(t, name):
    """GEMM_TYPE_* of a float tensor."""
    global _types
    torch = _torch_module()
    if _types is None:
        _types = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
    code = _types.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError("%s must be a float32, float16 or bfloat16 tensor" % name)
    return code


def _stack(t, name):
    """(matrices, rows, columns, leading dimension, distance between matrices,
    device pointer or None) of a row-major GPU matrix or a stack of them."""
    if t.dim() not in (2, 3):
        raise TypeError("%s must be a 2-D tensor or a 3-D stack of matrices" % name)
    if not t.is_cuda:
        raise TypeError("%s must live on the GPU" % name)
    shape, stride = tuple(t.shape), tuple(t.stride())
    if len(shape) == 2:
        shape, stride = (1,) + shape, (0,) + stride
    L, rows, cols = shape
    if cols > 1 and rows and L and stride[2] != 1:
        raise ValueError("%s must have unit stride along its rows (row-major)" % name)
    ld = stride[1] if rows > 1 and cols > 0 else max(1, cols)
    if max(L, rows, cols, ld) > INT_MAX:
        raise ValueError("%s: sizes and the distance between rows must be below 2^31" % name)
    return L, rows, cols, ld, (stride[0] if L > 1 else 0), (t.data_ptr() if t.numel() else None)


def _adapters(t, name, dtype, index, rows, cols, count=None):
    """(adapters, ranks or rows, pointer, leading dimension, distance between
    adapters) of a stack [S, rows, cols]; None of rows, cols or count is free.
    Runs for every stack of every call: the usual case is told by the cheapest
    queries."""
    torch = _torch_module()
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 3 and \
            t.get_device() == index:
        S, r, c = t.shape
        if r > 1 and c > 1 and S > 1 and (rows is None or r == rows) and \
                (cols is None or c == cols) and (count is None or S == count):
            s0, s1, s2 = t.stride()
            if s2 == 1 and c <= s1 <= INT_MAX:
                return S, r, t.data_ptr(), s1, s0
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise TypeError("%s must be a 3-D tensor, one matrix an adapter" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    S, r, c, ld, stride, ptr = _stack(t, name)
    for have, want in ((S, count), (r, rows), (c, cols)):
        if want is not None and have != want:
            raise ValueError("%s must be %s, got %s" % (name, [
                "adapters" if count is None else count, "ranks" if rows is None else rows,
                "ranks" if cols is None else cols], tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("all tensors of a call must live on one GPU")
    if ld < c and ptr is not None:
        raise ValueError("%s: the rows of an adapter must not overlap" % name)
    return S, r, ptr, max(ld, c), stride   # (no element: any distance)


def _scales(scales, index, S):
    return None if scales is None else _vector(scales, "scales", _torch_module().float32, index, S)


def gemm_lora(X, W, A, B, ids, C, scales=None, bias=None, act: str = "none", residual=None, T=None,
              workspace=None, stream=None):
    """``C[m] = act(X[m] @ W.T + scales[a] * X[m] @ A[a].T @ B[a].T + bias) + residual[m]``
    with ``a = ids[m]``: a projection shared by all rows beside the low-rank
    adapter that each row names.  float16 or bfloat16 X[M,K], W[N,K], A[S,R,K],
    B[S,N,R], C[M,N]; ``ids``: int64 [M], below 0 for rows without an adapter
    (S and more give NaN); ``scales``: float32 [S] or None for 1.  ``T``: float32
    [M,R] or None, receives ``X[m] @ A[a].T`` for ``gemm_lora_bwd``.  ``bias``,
    ``act`` and ``residual`` (which may be C) as for ``gemm_ex``.  ``workspace``:
    ``lora_workspace_bytes`` bytes, or None.  Returns C."""
    torch = _torch_module()
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(W, "W")
    pw, ldw = _shaped(W, "W", dtype, at, N, K)
    S, R, pa, lda, sa = _adapters(A, "A", dtype, at, None, K)
    _, _, pb, ldb, sb = _adapters(B, "B", dtype, at, N, R, S)
    pi = _vector(ids, "ids", torch.int64, at, M)
    ps = _scales(scales, at, S)
    pc, ldc = _shaped(C, "C", dtype, at, M, N)
    pt, ldt = _optional(T, "T", torch.float32, at, M, R)
    if bias is None and residual is None:
        pbias, code, pres, ldr = None, _act(act), None, 0
    else:
        for t in (bias, residual):
            if t is not None and t.get_device() != at:
                raise ValueError("all tensors of a call must live on one GPU")
        pbias, code, pres, ldr = _epilogue_args(bias, act, residual, M, N, dtype)
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_lora,
         (typ, M, N, K, R, S, px, ldx, pw, ldw, pa, lda, sa, pb, ldb, sb, pi, ps, pbias, code, pres,
          ldr, pc, ldc, pt, ldt),
         lambda: lib.gemm_lora_workspace(typ, M, N, K, R, S, px, ldx, pw, ldw, ldb), workspace)
    return C


def lora_workspace_bytes(X, W, A, B) -> int:
    """Workspace bytes ``gemm_lora`` needs for these tensors."""
    dtype, typ, at, M, K, px, ldx = _first(X)
    N = _rows(W, "W")
    S, R = _adapters(A, "A", dtype, at, None, K)[:2]
    ldb = _adapters(B, "B", dtype, at, N, R, S)[3]
    return load_library().gemm_lora_workspace(typ, M, N, K, R, S, px, ldx,
                                              *_shaped(W, "W", dtype, at, N, K), ldb)


def _none_or(t, name, *needed):
    """Whether ``t`` is missing; raises if one of ``needed`` (name, wanted) reads it."""
    if t is not None:
        return False
    for what, wanted in needed:
        if wanted is not None:
            raise ValueError("%s is needed for %s" % (name, what))
    return True


def _last(*tensors):
    """The length of the rows of the first tensor that there is."""
    torch = _torch_module()
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.dim():
            return t.shape[-1]
    raise ValueError("one of X, W and A must be given")


def gemm_lora_bwd(X, W, A, B, ids, T, dC, dX=None, dA=None, dB=None, scales=None, workspace=None,
                  stream=None):
    """The gradients of ``gemm_lora`` (act "none", W frozen) for the gradient dC
    [M,N] of its result and the T it stored: ``dX`` [M,K], ``dA`` [S,R,K] and
    ``dB`` [S,N,R], each computed if given; adapters that no row names get zeros.
    What the gradients asked for do not read may be None: X is read for dA, T for
    dB, W and A for dX, B for dX and dA (one of X, W and A is needed for its
    sizes).  ``workspace``: ``lora_bwd_workspace_bytes`` bytes, or None.  Returns
    (dX, dA, dB)."""
    torch = _torch_module()
    if _none_or(X, "X", ("dA", dA)):
        dtype, typ, at, M, N, pc, ldc = _first(dC, "dC")
        K, px, ldx = _last(W, A, dX), None, 0
    else:
        dtype, typ, at, M, K, px, ldx = _first(X)
        N = _rows(W, "W") if W is not None else _last(dC)
        pc, ldc = _shaped(dC, "dC", dtype, at, M, N)
    pw, ldw = (None, 0) if _none_or(W, "W", ("dX", dX)) else _shaped(W, "W", dtype, at, N, K)
    pa, lda, sa = pb, ldb, sb = pda, ldda, sda = pdb, lddb, sdb = None, 0, 0
    S = R = None
    if not _none_or(A, "A", ("dX", dX)):
        S, R, pa, lda, sa = _adapters(A, "A", dtype, at, R, K, S)
    if dA is not None:
        S, R, pda, ldda, sda = _adapters(dA, "dA", dtype, at, R, K, S)
    if dB is not None:
        R = _last(dB) if R is None else R
        S, _, pdb, lddb, sdb = _adapters(dB, "dB", dtype, at, N, R, S)
    if S is None:
        return dX, dA, dB
    if not _none_or(B, "B", ("dX", dX), ("dA", dA)):
        pb, ldb, sb = _adapters(B, "B", dtype, at, N, R, S)[2:]
    pi = _vector(ids, "ids", torch.int64, at, M)
    ps = _scales(scales, at, S)
    pt, ldt = (None, 0) if _none_or(T, "T", ("dB", dB)) else \
        _shaped(T, "T", torch.float32, at, M, R)
    pdx, lddx = _optional(dX, "dX", dtype, at, M, K)
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_lora_bwd,
         (typ, M, N, K, R, S, px, ldx, pw, ldw, pa, lda, sa, pb, ldb, sb, pi, ps, pt, ldt, pc, ldc,
          pdx, lddx, pda, ldda, sda, pdb, lddb, sdb),
         lambda: lib.gemm_lora_bwd_workspace(typ, M, N, K, R, S, pc, ldc, pw, ldw, pdx is not None,
                                             pda is not None, pdb is not None), workspace)
    return dX, dA, dB


def lora_bwd_workspace_bytes(X, W, A, dC, want_dx: bool = True, want_da: bool = True,
                             want_db: bool = True) -> int:
    """Workspace bytes ``gemm_lora_bwd`` needs for these tensors and gradients (X may
    be None, and W where dX is not wanted)."""
    dtype, typ, at, M, N, pc, ldc = _first(dC, "dC")
    S, R = _adapters(A, "A", dtype, at, None, None)[:2]
    K = _last(A)
    if X is not None:
        _shaped(X, "X", dtype, at, M, K)
    pw, ldw = (None, 0) if _none_or(W, "W", ("dX", want_dx or None)) else \
        _shaped(W, "W", dtype, at, N, K)
    return load_library().gemm_lora_bwd_workspace(typ, M, N, K, R, S, pc, ldc, pw, ldw,
                                                  bool(want_dx), bool(want_da), bool(want_db))


MUON = (3.4445, -4.7750, 2.0315)
_coeff_cache: dict = {}


def _numbers(v):
    """A number as a float, a sequence of them as a tuple of floats."""
    if isinstance(v, (tuple, list)) or getattr(v, "ndim", 0) == 1:
        return tuple(float(x) for x in v)
    if getattr(v, "ndim", 0) > 1:
        raise ValueError("coeffs must be three numbers, or three for each of the steps")
    return float(v)


def _coeffs(coeffs, steps):
    """The C array of ``coeffs``: one triple for all steps, or one for each.  Arrays
    are kept by the values alone: what holds them may change from call to call."""
    if coeffs is not MUON:
        coeffs = tuple(_numbers(v) for v in coeffs)
    key = (coeffs, steps)
    array = _coeff_cache.get(key)
    if array is None:
        flat = key[0]
        if len(flat) == 3 and not any(isinstance(v, tuple) for v in flat):
            flat = (flat,) * steps
        if len(flat) != steps or any(not isinstance(v, tuple) or len(v) != 3 for v in flat):
            raise ValueError("coeffs must be three numbers, or three for each of the steps")
        array = (ctypes.c_float * (3 * steps))(*[v for t in flat for v in t])
        if len(_coeff_cache) > 64:
            _coeff_cache.clear()
        _coeff_cache[key] = array
    return array


def _steps(steps):
    if not isinstance(steps, int) or not 1 <= steps <= 64:
        raise ValueError("steps must be 1 to 64")
    return steps


def gemm_ortho(G, O, steps: int = 5, coeffs=MUON, eps: float = 1e-7, workspace=None, stream=None):
    """``O = G`` orthogonalised by Newton-Schulz products: ``X = G / (|G| + eps)``,
    then ``steps`` times ``X = a X + b (X X^T) X + c (X X^T)^2 X``.  G and O: one
    matrix [m,n] or a stack [L,m,n] of them, float32, float16 or bfloat16 each
    (bfloat16 results of large matrices take a third of the products, float32 ones
    are the nearest to the formula).  ``coeffs``: (a, b, c), or one such triple a
    step; the singular values of every X must stay below 7, as they do for
    coefficients that converge from [0, 1]: iterates are held in 16-bit values, and
    larger ones become infinities.  ``workspace``: ``ortho_workspace_bytes`` bytes, or
    None.  Returns O."""
    tg, to = _type_code(G, "G"), _type_code(O, "O")
    L, m, n, ldg, stride_g, pg = _stack(G, "G")
    if O.shape != G.shape:
        raise ValueError("O must be %s like G, got %s" % (tuple(G.shape), tuple(O.shape)))
    _, _, _, ldo, stride_o, po = _stack(O, "O")
    at = G.get_device()
    if O.get_device() != at:
        raise ValueError("all tensors of a call must live on one GPU")
    steps = _steps(steps)
    lib = _lib or load_library()
    _run(at, stream, lib.gemm_ortho,
         (tg, to, L, m, n, pg, ldg, stride_g, steps, _coeffs(coeffs, steps), float(eps), po, ldo,
          stride_o),
         lambda: lib.gemm_ortho_workspace(tg, to, L, m, n, steps), workspace)
    return O


def ortho_workspace_bytes(G, O, steps: int = 5) -> int:
    """Workspace bytes ``gemm_ortho`` needs for these tensors."""
    L, m, n = _stack(G, "G")[:3]
    return load_library().gemm_ortho_workspace(_type_code(G, "G"), _type_code(O, "O"), L, m, n,
                                               _steps(steps))
