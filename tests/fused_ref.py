"""Definitions of the fused operators in 64 bits, inputs for their tests, and
the tolerances the tests hold them to.

Tolerances.  An output is rounded once, by at most half a step: eps / 2
relative (eps = torch.finfo(type).eps; fp16 also half of its smallest step,
2^-25).  A sum of K products on the matrix cores goes 32 products at a time
into an fp32 accumulator: at most K / 32 additions of partial sums and a few
inside a step, each off by 2^-24 of a partial sum that is at most S = sum of
the products' sizes, so the sum is off by at most (K / 32 + 8) 2^-24 S.
Elementwise fp32 work (exponentials, reciprocals) is a few steps of 2^-24,
taken as 2^-20.  Gradients sum values that were rounded to 16 bits first: each
is off by eps / 2 of its size, so the sum is off by eps / 2 of the sum of the
sizes besides; over the whole output, in the 2-norm, such errors are
independent, which leaves eps / 2 of the norm beside the outputs' own eps / 2.
"""
from __future__ import annotations

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype, v):
    return torch.finfo(dtype).eps / 2 * v.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def sum_error(K, S):
    """The fp32 accumulation of K products whose sizes add up to S."""
    return (K / 32 + 8) * 2.0 ** -24 * S


def act(g, name):
    if name == "silu":
        return g * torch.sigmoid(g)
    return g.clamp(min=0) if name == "relu" else g


def act_slope(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    return (g > 0).double() if name == "relu" else torch.ones_like(g)


def close(got, ref, tol, what):
    """Elementwise: |got - ref| <= tol, and NaN and infinities where ref has them."""
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what + ": NaN elsewhere"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), what
    over = ((got - ref).abs() - tol)[fine]
    if over.numel():
        at = int(over.argmax())
        assert float(over.max()) <= 0, "%s: off by %.3e where %.3e is allowed (%d of %d over)" % (
            what, float((got - ref).abs()[fine][at]), float((tol + 0 * ref)[fine][at]),
            int((over > 0).sum()), over.numel())


def norm_close(got, ref, rel, what):
    """In the 2-norm.  A value below binary16's normal range is off by up to
    2^-25 whatever its size (half of the smallest step 2^-24), and n such
    values by up to 2^-25 sqrt(n) in the norm."""
    n = float(ref.norm())
    off = float((got.double() - ref).norm())
    least = 2.0 ** -25 * ref.numel() ** 0.5 if got.dtype == torch.float16 else 1e-30
    assert off <= rel * n + least, "%s: relative norm of the error %.3e > %.3e" % (
        what, off / max(n, 1e-300), rel)


def randn(shape, sd, dtype, gen):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * sd).to(dtype)


def place(t, pad=0, shift=0, device="cuda"):
    """A device copy of the matrix t whose rows lie ``pad`` elements further
    apart than needed and which starts ``shift`` elements into its storage;
    what lies between the rows is NaN (255 for bytes)."""
    r, c = t.shape
    fill = 255 if t.dtype == torch.uint8 else float("nan")
    buf = torch.full((shift + r * (c + pad) + pad + 8,), fill, dtype=t.dtype, device=device)
    v = buf[shift:shift + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


class Out:
    """An output matrix inside a sentinel-filled buffer."""

    def __init__(self, r, c, dtype, pad=0, shift=0, device="cuda"):
        self.buf = torch.full((shift + (r + 1) * (c + pad) + 8,), 777.0, dtype=dtype, device=device)
        self.t = self.buf[shift:shift + r * (c + pad)].view(r, c + pad)[:, :c]

    def check_frame(self, what):
        rest = self.buf.clone()
        o = rest[self.t.storage_offset():]
        torch.as_strided(rest, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(777.0)
        assert bool((rest == 777.0).all()), what + ": wrote outside its matrix"
        del o


def gated_ref(X, Wg, Wu, name):
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    g, u = x @ wg.T, x @ wu.T
    sg, su = x.abs() @ wg.abs().T, x.abs() @ wu.abs().T
    return g, u, act(g, name) * u, sg, su


def gated_tols(g, u, h, sg, su, name, K, dtype):
    """Elementwise tolerances of (G, U, H)."""
    dg, du = sum_error(K, sg), sum_error(K, su)
    th = 1.1 * dg * (u.abs() + du) + act(g, name).abs() * du + 2.0 ** -20 * h.abs()
    return dg + half_step(dtype, g), du + half_step(dtype, u), th + half_step(dtype, h.abs() + th)


def w4_weights(Wq, scales, zeros, group, K):
    """(q - z) and s, each [N][K] in 64 bits."""
    q = torch.stack((Wq & 15, Wq >> 4), -1).reshape(Wq.shape[0], -1)[:, :K].double()
    at = torch.arange(K, device=Wq.device) // group
    z = 8.0 if zeros is None else zeros.double()[:, at]
    return q - z, scales.double()[:, at]


def w4_norm_close(got, x, q, s, what):
    """X W^T in the 2-norm, W = q s (w4_weights), for x of random signs: an
    output's rounding, at most eps / 2 of each value, and the fp32 sums, whose
    additions are off by 2^-24 of partial sums of random signs: those stay within
    a few times the root of the sum of the squared products (4 of it are
    allowed), and their errors are independent, so that K / 32 + 8 additions are
    off by the root of that many.  The bf16 form has products of up to 143 |s x|
    in each of two sums, fp16's up to 15."""
    K, dt = x.shape[1], got.dtype
    x = x.double()
    ref = x @ (q * s).T
    root = ((x * x) @ (s * s).T).sum() ** 0.5 * (286.0 if dt == torch.bfloat16 else 15.0)
    off = 4 * (K / 32 + 8) ** 0.5 * 2.0 ** -24 * float(root)
    norm_close(got, ref, torch.finfo(dt).eps / 2 + off / float(ref.norm()), what)


def xent_ref(X, W, targets, ignore):
    """(z, lse, loss) in 64 bits; NaN loss for a target out of range."""
    z = X.double() @ W.double().T
    lse = torch.logsumexp(z, 1)
    N = W.shape[0]
    ok = (targets >= 0) & (targets < N)
    at = torch.where(ok, targets, 0)
    loss = lse - z.gather(1, at[:, None])[:, 0]
    loss = torch.where(ok, loss, torch.full_like(loss, float("nan")))
    return z, lse, torch.where(targets == ignore, torch.zeros_like(loss), loss)


def xent_tol(X, W, z, lse):
    """Tolerance of lse by row: the logits' sums, and fp32 exponentials of
    arguments down to the row's range and sums of them (a lane's 32 in turn,
    then pairwise and chunk by chunk: under 64 roundings)."""
    K = X.shape[1]
    dz = sum_error(K, (X.double().abs() @ W.double().abs().T).amax(1))
    spread = (z.amax(1) - z.amin(1)).clamp(max=100)
    return dz + (64 + 4 * spread) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
