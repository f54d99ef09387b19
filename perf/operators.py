"""The products with a model's work folded in, as they are measured.

Three families, each a product of activations with stored weights (row-major,
weights [out][in], as the library's A * B^T):

  gated   H = act(X Wg^T) * (X Wu^T), the first half of a gated feed-forward
          block, and its gradients dX, dWg, dWu from the saved products
          G = X Wg^T and U = X Wu^T
  w4      C = X W^T with W in 4 bits, a scale (and a zero point) for each
          group of K values of a row
  xent    the softmax cross entropy of X W^T against target columns, for each
          row, without keeping the logits; xent_step adds dX and dW

With ``own`` false, ``run`` computes them in elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100


def listed():
    return [
        # decoding: one token's hidden state through both projections of a block
        dict(name="gated one token", op="gated", type="bf16", act="silu", M=1, N=16384, K=4096,
             save=False),
        # decoding: a batch of two dozen sequences
        dict(name="gated small batch", op="gated", type="f16", act="silu", M=24, N=8192, K=2048,
             save=False),
        # a training step's forward pass, with the products kept for the backward pass
        dict(name="gated forward", op="gated", type="bf16", act="silu", M=4096, N=16384, K=4096,
             save=True),
        # nothing divides anything, and rows start at 2-byte addresses
        dict(name="gated forward ragged", op="gated", type="f16", act="relu", M=5000, N=3001,
             K=1537, save=False),
        # the same training step's backward pass
        dict(name="gated backward", op="gated_bwd", type="bf16", act="silu", M=4096, N=16384,
             K=4096),
        # packed sequences of a small model: ragged rows, an odd inner width
        dict(name="gated backward ragged", op="gated_bwd", type="f16", act="silu", M=1000, N=3001,
             K=768),
        # decoding one token with 4-bit weights
        dict(name="w4 one token", op="w4", type="f16", M=1, N=16384, K=4096, group=128,
             zeros=False),
        # a batch of sixteen on the way down, with zero points
        dict(name="w4 small batch", op="w4", type="bf16", M=16, N=4096, K=16384, group=64,
             zeros=True),
        # a small model's projection with an odd number of rows, short groups
        dict(name="w4 small odd", op="w4", type="f16", M=5, N=2305, K=768, group=32, zeros=True),
        # scoring 8192 tokens against a large vocabulary
        dict(name="xent forward", op="xent", type="bf16", M=8192, N=131072, K=4096),
        # a training step's head: the loss and both gradients
        dict(name="xent step", op="xent_step", type="bf16", M=4096, N=131072, K=2048),
        # a small model's head: few tokens, an odd vocabulary, scaled fp16 gradients
        dict(name="xent step small", op="xent_step", type="f16", M=333, N=50001, K=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "w4", "w4", "xent", "xent_step"])
    typ = rng.choice(["f16", "bf16"])
    if op in ("gated", "gated_bwd"):
        case = dict(op=op, type=typ, act=rng.choice(["silu", "silu", "relu"]),
                    M=_log(rng, 1, 4096), N=_log(rng, 200, 16384), K=_log(rng, 100, 4096))
        if op == "gated":
            case["save"] = rng.random() < 0.5
    elif op == "w4":
        group = rng.choice([32, 64, 128])
        case = dict(op=op, type=typ, M=_log(rng, 1, 64), N=_log(rng, 200, 16384),
                    K=group * max(1, _log(rng, 256, 16384) // group), group=group,
                    zeros=rng.random() < 0.5)
    else:
        case = dict(op=op, type=typ, M=_log(rng, 8, 8192), N=_log(rng, 1000, 131072),
                    K=_log(rng, 100, 4096))
        most = 1 << (42 if op == "xent" else 40)
        while case["M"] * case["N"] * case["K"] > most:
            case["M"] = max(8, case["M"] // 2 + rng.randrange(2))
    if rng.random() < 0.5:
        # half of the inner widths are whole 16-byte rows, as models choose them
        case["K"] = case["K"] if op == "w4" else max(8, case["K"] // 8 * 8)
    return case


def _normal(gen, shape, sd, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, sd, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dt = case["op"], DTYPES[case["type"]]
    M, N, K = case["M"], case["N"], case["K"]
    s = dict(case)
    s["X"] = _normal(gen, (M, K), 1.0, dt)
    if op in ("gated", "gated_bwd"):
        s["Wg"] = _normal(gen, (N, K), K ** -0.5, dt)
        s["Wu"] = _normal(gen, (N, K), K ** -0.5, dt)
        if op == "gated":
            s["H"] = torch.empty((M, N), device="cuda", dtype=dt)
            if case["save"]:
                s["G"], s["U"] = torch.empty_like(s["H"]), torch.empty_like(s["H"])
        else:
            # the products that the forward pass kept, and the gradient that comes back
            s["G"] = _normal(gen, (M, N), 1.0, dt)
            s["U"] = _normal(gen, (M, N), 1.0, dt)
            s["dH"] = _normal(gen, (M, N), 0.1, dt)
            s["dX"] = torch.empty_like(s["X"])
            s["dWg"], s["dWu"] = torch.empty_like(s["Wg"]), torch.empty_like(s["Wu"])
    elif op == "w4":
        groups = K // case["group"]
        s["Wq"] = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8,
                                generator=gen)
        scale = torch.rand((N, groups), device="cuda", generator=gen) + 0.5
        s["scales"] = (scale * (K ** -0.5 / 4.6)).to(dt)
        s["zero"] = torch.randint(5, 12, (N, groups), device="cuda", dtype=torch.uint8,
                                  generator=gen) if case["zeros"] else None
        s["C"] = torch.empty((M, N), device="cuda", dtype=dt)
    else:
        s["W"] = _normal(gen, (N, K), 2.0 * K ** -0.5, dt)
        t = torch.randint(0, N, (M,), device="cuda", generator=gen)
        # padding and prompt tokens have no target
        t[torch.rand((M,), device="cuda", generator=gen) < 0.05] = IGNORE
        s["targets"] = t
        s["loss"] = torch.empty((M,), device="cuda", dtype=torch.float32)
        s["lse"] = torch.empty_like(s["loss"])
        if op == "xent_step":
            # the mean over the rows that have a target, times fp16's loss scale
            count = (t != IGNORE).sum().clamp(min=1).float()
            s["dloss"] = ((1024.0 if case["type"] == "f16" else 1.0) / count).expand(M).contiguous()
            s["dX"], s["dW"] = torch.empty_like(s["X"]), torch.empty_like(s["W"])
    return s


# ---- the plain forms, in 32 bits, rounded once at the end

def _act(g, name):
    return g / (1.0 + torch.exp(-g)) if name == "silu" else torch.where(g > 0, g, torch.zeros_like(g))


def _act_slope(g, name):
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return sg * (1.0 + g * (1.0 - sg))
    return (g > 0).to(g.dtype)


def _gated(s):
    x, dt = s["X"].float(), s["X"].dtype
    g, u = x @ s["Wg"].float().T, x @ s["Wu"].float().T
    h = (_act(g, s["act"]) * u).to(dt)
    return (h, g.to(dt), u.to(dt)) if s["save"] else (h,)


def _gated_bwd(s):
    x, g, u, dh, dt = s["X"].float(), s["G"].float(), s["U"].float(), s["dH"].float(), s["X"].dtype
    dg = dh * u * _act_slope(g, s["act"])
    du = dh * _act(g, s["act"])
    dx = dg @ s["Wg"].float() + du @ s["Wu"].float()
    return dx.to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt)


def _w4(s):
    q = torch.stack((s["Wq"] & 15, s["Wq"] >> 4), -1).reshape(s["N"], -1, s["group"]).float()
    z = 8.0 if s["zero"] is None else s["zero"].float()[:, :, None]
    w = ((q - z) * s["scales"].float()[:, :, None]).reshape(s["N"], s["K"])
    return ((s["X"].float() @ w.T).to(s["X"].dtype),)


def _xent(s):
    x, w, t = s["X"].float(), s["W"].float(), s["targets"]
    z = x @ w.T
    top = z.max(1, keepdim=True).values
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    at = t.clamp(min=0)[:, None]
    live = t != IGNORE
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    if s["op"] == "xent":
        return loss, lse
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at, -torch.ones_like(at, dtype=d.dtype))
    d *= torch.where(live, s["dloss"], torch.zeros_like(lse))[:, None]
    return loss, lse, (d @ w).to(s["X"].dtype), (d.T @ x).to(s["X"].dtype)


def _library(s):
    import dense_gemm_sgemm_amd as dg

    op = s["op"]
    if op == "gated":
        if s["save"]:
            dg.gemm_gated(s["X"], s["Wg"], s["Wu"], s["H"], act=s["act"], G=s["G"], U=s["U"])
            return s["H"], s["G"], s["U"]
        return (dg.gemm_gated(s["X"], s["Wg"], s["Wu"], s["H"], act=s["act"]),)
    if op == "gated_bwd":
        dg.gemm_gated_bwd(s["X"], s["Wg"], s["Wu"], s["G"], s["U"], s["dH"], dX=s["dX"],
                          dWg=s["dWg"], dWu=s["dWu"], act=s["act"])
        return s["dX"], s["dWg"], s["dWu"]
    if op == "w4":
        return (dg.gemm_w4(s["X"], s["Wq"], s["scales"], s["C"], group=s["group"],
                           zeros=s["zero"]),)
    dg.gemm_xent(s["X"], s["W"], s["targets"], s["loss"], s["lse"], ignore_index=IGNORE)
    if op == "xent":
        return s["loss"], s["lse"]
    dg.gemm_xent_bwd(s["X"], s["W"], s["targets"], s["lse"], s["dloss"], dX=s["dX"], dW=s["dW"],
                     ignore_index=IGNORE)
    return s["loss"], s["lse"], s["dX"], s["dW"]


def run(state):
    if own:
        return _library(state)
    op = state["op"]
    if op == "gated":
        return _gated(state)
    if op == "gated_bwd":
        return _gated_bwd(state)
    if op == "w4":
        return _w4(state)
    return _xent(state)


def work(case):
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op == "gated":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N * (3 if case["save"] else 1)),
                "flops": 4 * M * N * K}
    if op == "gated_bwd":
        # X, both weights, G, U, dH in; dX and both weight gradients out
        return {"bytes": 2 * (2 * M * K + 4 * N * K + 3 * M * N), "flops": 8 * M * N * K}
    if op == "w4":
        groups = K // case["group"]
        return {"bytes": 2 * M * K + N * K // 2 + N * groups * (3 if case["zeros"] else 2)
                + 2 * M * N, "flops": 2 * M * N * K}
    if op == "xent":
        return {"bytes": 2 * (M * K + N * K) + 16 * M, "flops": 2 * M * N * K}
    # without the logits kept, the backward pass computes them again
    return {"bytes": 2 * (2 * M * K + 2 * N * K) + 20 * M, "flops": 8 * M * N * K}


# ---- the same from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, N, K = case["op"], case["N"], case["K"]
    x = s["X"].double()
    if op in ("gated", "gated_bwd"):
        wg, wu = s["Wg"].double(), s["Wu"].double()

        def gate(v):
            return v * torch.sigmoid(v) if case["act"] == "silu" else v.clamp(min=0.0)

        if op == "gated":
            g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            return (gate(g) * u, g, u) if case["save"] else (gate(g) * u,)
        g, u, dh = s["G"].double(), s["U"].double(), s["dH"].double()
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            slope = sig + g * sig * (1 - sig)
        else:
            slope = torch.heaviside(g, torch.zeros_like(g))
        dg, du = slope * u * dh, gate(g) * dh
        return (torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.t(), x), torch.mm(du.t(), x))
    if op == "w4":
        w = torch.empty((N, K), device="cuda", dtype=torch.float64)
        w[:, 0::2] = (s["Wq"] % 16).double()
        w[:, 1::2] = torch.div(s["Wq"], 16, rounding_mode="floor").double()
        zero = torch.full_like(s["scales"], 8).double() if s["zero"] is None else s["zero"].double()
        w -= zero.repeat_interleave(case["group"], 1)
        w *= s["scales"].double().repeat_interleave(case["group"], 1)
        return (torch.mm(x, w.t()),)
    w, t = s["W"].double(), s["targets"]
    loss, lse = [], []
    dx, dw = [], torch.zeros_like(w) if op == "xent_step" else None
    for i in range(0, case["M"], 1024):
        z = torch.mm(x[i:i + 1024], w.t())
        r = torch.arange(z.shape[0], device="cuda")
        ti = t[i:i + 1024]
        skip = ti == IGNORE
        safe = torch.where(skip, 0, ti)
        li = torch.logsumexp(z, 1)
        lse.append(li)
        loss.append((li - z[r, safe]).masked_fill(skip, 0.0))
        if dw is not None:
            z -= li[:, None]
            p = z.exp_()
            p[r, safe] -= 1.0
            p *= s["dloss"][i:i + 1024].double().masked_fill(skip, 0.0)[:, None]
            dx.append(torch.mm(p, w))
            dw += torch.mm(p.t(), x[i:i + 1024])
    if dw is None:
        return torch.cat(loss), torch.cat(lse)
    return torch.cat(loss), torch.cat(lse), torch.cat(dx), dw
