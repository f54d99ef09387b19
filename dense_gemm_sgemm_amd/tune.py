"""Bindings of ``libmi355tune.so`` (``include/mi355tune.h``): what fine tuning
needs next to a model's products.

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

from . import HERE, INT_MAX, _torch_module
from .fused import _run

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


MUON = (3.4445, -4.7750, 2.0315)
_coeff_cache: dict = {}


def _coeffs(coeffs, steps):
    """The C array of ``coeffs``: one triple for all steps, or one for each."""
    key = (coeffs if isinstance(coeffs, tuple) else tuple(map(tuple, coeffs)), steps)
    array = _coeff_cache.get(key)
    if array is None:
        flat = key[0]
        if len(flat) == 3 and not any(isinstance(v, (tuple, list)) for v in flat):
            flat = (flat,) * steps
        if len(flat) != steps or any(len(v) != 3 for v in flat):
            raise ValueError("coeffs must be three numbers, or three for each of the steps")
        array = (ctypes.c_float * (3 * steps))(*[float(v) for t in flat for v in t])
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
    (bfloat16 results take a third of the products).  ``coeffs``: (a, b, c), or
    one such triple a step.  ``workspace``: ``ortho_workspace_bytes`` bytes, or
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
