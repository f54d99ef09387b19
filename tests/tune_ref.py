"""Definitions of the operators of fine tuning in 64 bits, and the tolerances
their tests hold them to (fused_ref has the sums' and the roundings').

Adapters.  t (and dt, T) is used in two 16-bit values times a power of two that
brings the largest of its block to 2^13 .. 2^14.  hi is cut off: what is left is
less than 2^-7 of the value in bf16 (8 bits) and 2^-10 in fp16 (11 bits); lo is
it rounded, by half a step of those bits, which is 2^-16 or 2^-21 of the value;
where lo would be zero it is 2^-14, at most 2^-27 of the largest; below binary16's
normal range it is off by 2^-25, at most 2^-38 of the largest.  Together under
SPLIT of the block's largest.

Updates.  A step multiplies values that were rounded when they were stored, so
the distance from the formula is not the arithmetic's last bits: `rounded`
computes in 64 bits with exactly the documented roundings in the documented
places, `in_32_bits` in fp32.  Their distances from the definition are two
samples of the errors that the kernel may make; it may make twice both (another
order of sums, other ties), and round its output.
"""
from __future__ import annotations

import torch

from fused_ref import act, half_step, sum_error

SPLIT = {torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -20}
MUON = (3.4445, -4.7750, 2.0315)


def lora_ref(X, W, A, B, ids, scales=None):
    """(products, t, sums of sizes of x w, error of t's sums and values beside
    another, by row and column of the result) in 64 bits.  Rows with an unknown
    adapter are NaN."""
    dt = X.dtype
    x, w = X.double(), W.double()
    M, K = x.shape
    S, R = A.shape[:2]
    y, size = x @ w.T, x.abs() @ w.abs().T
    t = torch.zeros((M, R), dtype=torch.float64, device=X.device)
    dt_sum = torch.zeros_like(t)
    off = sum_error(K, size)
    for s in range(S):
        at = (ids == s).nonzero()[:, 0]
        if not len(at):
            continue
        a, b = A[s].double(), B[s].double()
        f = 1.0 if scales is None else float(scales[s])
        t[at] = x[at] @ a.T
        dt_sum[at] = sum_error(K, x[at].abs() @ a.abs().T)
        y[at] += f * t[at] @ b.T
        each = dt_sum[at] + SPLIT[dt] * t[at].abs().amax(1, keepdim=True)
        off[at] += abs(f) * (each @ b.abs().T + sum_error(2 * R, t[at].abs() @ b.abs().T))
    bad = ids >= S
    y[bad], t[bad] = float("nan"), float("nan")
    return y, t, off, dt_sum


def lora_result(y, off, dt, bias=None, name="none", residual=None):
    """The written-back result and its tolerance."""
    z = y if bias is None else y + bias.double()
    d = off + 2.0 ** -23 * (y.abs() + z.abs())
    h = act(z, name)
    d = 1.1 * d + 2.0 ** -20 * h.abs()
    if residual is not None:
        d = d + 2.0 ** -23 * (h.abs() + residual.double().abs())
        h = h + residual.double()
    return h, d + half_step(dt, h.abs() + d)


def lora_bwd_ref(X, W, A, B, ids, T, dC, scales=None):
    """((dX, tolerance), (dA, ...), (dB, ...)) in 64 bits."""
    dt = X.dtype
    x, w, d, T = X.double(), W.double(), dC.double(), T.double()
    M, K = x.shape
    N = w.shape[0]
    S, R = A.shape[:2]
    dx, off = d @ w, sum_error(N, d.abs() @ w.abs())
    out = []
    dA, dB = torch.zeros(A.shape, dtype=torch.float64, device=X.device), \
        torch.zeros(B.shape, dtype=torch.float64, device=X.device)
    offA, offB = torch.zeros_like(dA), torch.zeros_like(dB)
    for s in range(S):
        at = (ids == s).nonzero()[:, 0]
        if not len(at):
            continue
        a, b, n = A[s].double(), B[s].double(), len(at)
        f = 1.0 if scales is None else float(scales[s])
        g = f * d[at] @ b
        eg = abs(f) * sum_error(N, d[at].abs() @ b.abs()) + 2.0 ** -23 * g.abs()
        dx[at] += g @ a
        each = eg + SPLIT[dt] * g.abs().amax(1, keepdim=True)
        off[at] += each @ a.abs() + sum_error(2 * R, g.abs() @ a.abs())
        # (sums over rows: a step of 32, its two halves and its factor, each added in fp32)
        xa = x[at].abs()
        dA[s] = g.T @ x[at]
        offA[s] = (eg + SPLIT[dt] * g.abs().max()).T @ xa + sum_error(3 * n, g.abs().T @ xa)
        t, da = T[at] * f, d[at].abs()
        dB[s] = d[at].T @ t
        offB[s] = da.T @ (SPLIT[dt] * t.abs().max() + 2.0 ** -23 * t.abs()) + \
            sum_error(3 * n, da.T @ t.abs())
    dx[ids >= S] = float("nan")
    for v, o in ((dx, off), (dA, offA), (dB, offB)):
        out.append((v, o + half_step(dt, v.abs() + o)))
    return out


def _triples(coeffs, steps):
    return [coeffs] * steps if not isinstance(coeffs[0], (tuple, list)) else list(coeffs)


def ortho_ref(G, steps=5, coeffs=MUON, eps=1e-7, dtype=torch.float64):
    """The definition, in 64 bits (or as it is written in another type)."""
    X = G.to(dtype)
    X = X / (X.double().square().sum((-2, -1), keepdim=True).sqrt() + eps).to(dtype)
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT.contiguous() if tall else X
    for a, b, c in _triples(coeffs, steps):
        A = X @ X.mT.contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT.contiguous() if tall else X


def in_32_bits(G, steps=5, coeffs=MUON, eps=1e-7):
    return ortho_ref(G, steps, coeffs, eps, torch.float32)


def _one(v, scale):
    return (v * scale).half().double() / scale


def _two(v, scale):
    hi = _one(v, scale)
    return hi + _one(v - hi, scale)


def rounded(G, fine, steps=5, coeffs=MUON, eps=1e-7):
    """In 64 bits, with X, A and C rounded as they are stored: X times 2^12, A and
    C times 2^10, in two binary16 values (`fine`) or one, X's first three in two."""
    X = G.double()
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT.contiguous() if tall else X
    one = torch.eye(X.shape[-2], dtype=torch.float64, device=G.device)
    exact = G.dtype != torch.float32       # the first one is the input itself
    q = _two if fine else _one
    for k, (a, b, c) in enumerate(_triples(coeffs, steps)):
        if not (exact and k == 0):
            X = (_two if fine or (k < 3 and k + 1 < steps) else _one)(X, 4096.0)
        H = X if fine or (exact and k == 0) else _one(X, 4096.0)
        A = q(H @ H.mT, 1024.0)
        X = q(a * one + b * A + c * (A @ A), 1024.0) @ X
    return X.mT.contiguous() if tall else X


def ortho_check(got, G, what, steps=5, coeffs=MUON, eps=1e-7):
    """Matrix by matrix, in the 2-norm."""
    fine = got.dtype != torch.bfloat16
    # two values throughout for the smaller ones, whatever the output's type
    low = min(G.shape[-2:])
    small = low <= 64 or (low <= 1024 and G.numel() * (1.5 if low > 512 else 1) <= 2.5 * 2 ** 20)
    ref = ortho_ref(G, steps, coeffs, eps)
    off = (rounded(G, fine or small, steps, coeffs, eps) - ref).flatten(1).norm(dim=1) + \
        (in_32_bits(G, steps, coeffs, eps).double() - ref).flatten(1).norm(dim=1)
    size = ref.flatten(1).norm(dim=1)
    # (a matrix of few values samples its errors badly: 16 more steps of 2^-22)
    tol = 2 * off + (torch.finfo(got.dtype).eps / 2 + 2.0 ** -18) * size + \
        (2.0 ** -25 * ref[0].numel() ** 0.5 if got.dtype == torch.float16 else 1e-30)
    err = (got.double() - ref).flatten(1).norm(dim=1)
    worst = int((err - tol).argmax())
    assert bool((err <= tol).all()), "%s: matrix %d is off by %.3e, allowed %.3e of %.3e" % (
        what, worst, float(err[worst]), float(tol[worst]), float(size[worst]))
