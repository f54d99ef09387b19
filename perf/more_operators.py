"""What fine tuning and serving many tuned models need next to the products, as
it is measured.

Two families:

  lora    Y = X W^T + scale_a (X A_a^T) B_a^T, a frozen projection shared by all
          rows of X beside the low-rank adapter a that each row names (or none);
          lora_bwd: the gradients of X and of every adapter's A and B
  ortho   an update orthogonalised by Newton-Schulz products, for L matrices of
          one size: X = G / (|G| + eps), then `steps` times
          X = a X + b (X X^T) X + c (X X^T)^2 X

With ``own`` false, ``run`` computes them in elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STEPS, COEFFS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


def listed():
    return [
        # decoding one token of one tuned model
        dict(name="lora one token", op="lora", type="bf16", M=1, N=4096, K=4096, R=16, S=8,
             rows="tokens"),
        # decoding: 48 sequences, almost every one with an adapter of its own
        dict(name="lora decode batch", op="lora", type="f16", M=48, N=4096, K=4096, R=16, S=64,
             rows="tokens"),
        # prompts of several requests behind each other, wider adapters
        dict(name="lora prompts", op="lora", type="bf16", M=4096, N=4096, K=4096, R=32, S=8,
             rows="requests"),
        # nothing divides anything, and rows start at 2-byte addresses
        dict(name="lora ragged", op="lora", type="f16", M=333, N=2305, K=769, R=12, S=3,
             rows="requests"),
        # a training step of one adapter: the gradients of a large projection
        dict(name="lora backward", op="lora_bwd", type="bf16", M=4096, N=4096, K=4096, R=16, S=1,
             rows="requests"),
        # several adapters trained side by side on a small model, odd width, packed rows
        dict(name="lora backward ragged", op="lora_bwd", type="f16", M=1000, N=3001, K=768, R=64,
             S=5, rows="requests"),
        # the update of one square projection, its momentum in 32 bits
        dict(name="ortho square", op="ortho", source="f32", type="bf16", L=1, m=4096, n=4096),
        # the up projections of four layers, momentum in 16 bits
        dict(name="ortho four layers", op="ortho", source="bf16", type="bf16", L=4, m=2048, n=8192),
        # a tall matrix of a small model, nothing a multiple of a tile
        dict(name="ortho tall odd", op="ortho", source="f32", type="f16", L=2, m=2305, n=769),
        # the factors of sixteen adapters
        dict(name="ortho adapters", op="ortho", source="f32", type="bf16", L=16, m=16, n=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora", "lora_bwd", "lora_bwd", "ortho", "ortho", "ortho"])
    typ = rng.choice(["f16", "bf16"])
    if op == "ortho":
        case = dict(op=op, source=rng.choice(["f32", typ]), type=typ, L=_log(rng, 1, 16),
                    m=_log(rng, 8, 4096), n=_log(rng, 64, 8192))
        if rng.random() < 0.5:
            case["m"], case["n"] = case["n"], case["m"]
        while case["L"] > 1 and _ortho_flops(case) > _ortho_flops(listed()[7]):
            case["L"] -= 1
        while _ortho_flops(case) > _ortho_flops(listed()[7]):
            case["m"], case["n"] = case["m"] * 3 // 4, case["n"] * 3 // 4
        return case
    case = dict(op=op, type=typ, M=_log(rng, 1 if op == "lora" else 16, 4096),
                N=_log(rng, 200, 8192), K=_log(rng, 200, 8192),
                R=rng.choice([4, 8, 8, 12, 16, 16, 32, 64, 128]), S=_log(rng, 1, 64),
                rows=rng.choice(["requests", "requests", "tokens"]))
    if rng.random() < 0.5:
        # half of the widths are whole 16-byte rows, as models choose them
        case["N"], case["K"] = case["N"] // 8 * 8, case["K"] // 8 * 8
    while case["M"] * case["N"] * case["K"] > 1 << 36:
        case["M"] = case["M"] // 2 + rng.randrange(2)
    while case["S"] * case["R"] > 1024:
        case["S"] //= 2
    return case


def _normal(gen, shape, sd, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, sd, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    dt = DTYPES[case["type"]]
    if case["op"] == "ortho":
        L, m, n = case["L"], case["m"], case["n"]
        # momentum: a few strong directions over noise
        g = torch.randn((L, m, n), device="cuda", generator=gen)
        k = min(8, m, n)
        strong = torch.randn((L, m, k), device="cuda", generator=gen)
        strong *= 3.0 * 0.75 ** torch.arange(k, device="cuda")
        g += torch.bmm(strong, torch.randn((L, k, n), device="cuda", generator=gen))
        s["G"] = (1e-3 * g).to(DTYPES[case["source"]])
        s["O"] = torch.empty((L, m, n), device="cuda", dtype=dt)
        return s
    M, N, K, R, S = (case[k] for k in "MNKRS")
    s["X"] = _normal(gen, (M, K), 1.0, dt)
    s["W"] = _normal(gen, (N, K), K ** -0.5, dt)
    s["A"] = _normal(gen, (S, R, K), K ** -0.5, dt)
    s["B"] = _normal(gen, (S, N, R), 0.3 * R ** -0.5, dt)
    s["scales"] = 0.5 + 1.5 * torch.rand((S,), device="cuda", generator=gen)
    # -1: a request of the model as it is, without an adapter
    ids = torch.randint(0, S, (M,), device="cuda", generator=gen)
    ids[torch.rand((M,), device="cuda", generator=gen) < 0.1] = -1
    if case["rows"] == "requests":
        # each request's tokens stand behind each other
        start = torch.rand((M,), device="cuda", generator=gen) < 8.0 / M
        ids = ids[torch.cumsum(start, 0).clamp(max=M - 1)].contiguous()
    s["ids"] = ids
    if case["op"] == "lora":
        s["C"] = torch.empty((M, N), device="cuda", dtype=dt)
    else:
        # what the forward pass kept, and the gradient that comes back
        s["T"] = _pick(s["X"].float(), s["A"].float(), ids)
        s["dC"] = _normal(gen, (M, N), 0.1, dt)
        s["dX"], s["dA"], s["dB"] = (torch.empty_like(s[k]) for k in "XAB")
    return s


# ---- the plain forms, in 32 bits, rounded once at the end

def _chosen(ids, S):
    """[M][S]: whether row m is adapter s's."""
    return ids[:, None] == torch.arange(S, device=ids.device)


def _pick(x, a, ids):
    """x[m] . a[ids[m]][r] for x [M][K] and a [S][R][K]; 0 for rows without."""
    S, R, K = a.shape
    t = (x @ a.reshape(S * R, K).T).reshape(-1, S, R)
    return torch.where(_chosen(ids, S)[:, :, None], t, torch.zeros_like(t)).sum(1)


def _spread(t, ids, S):
    """[M][S R]: row m's t in the place of its adapter, zeros in the others'."""
    t = t[:, None, :] * _chosen(ids, S)[:, :, None].to(t.dtype)
    return t.reshape(t.shape[0], -1)


def _by_row(s):
    """Each row's scale."""
    return torch.where(s["ids"] >= 0, s["scales"][s["ids"].clamp(min=0)], torch.zeros(()).cuda())


def _lora(s):
    x, b, S, R = s["X"].float(), s["B"].float(), s["S"], s["R"]
    t = _pick(x, s["A"].float(), s["ids"]) * _by_row(s)[:, None]
    y = x @ s["W"].float().T
    y += _spread(t, s["ids"], S) @ b.transpose(1, 2).reshape(S * R, -1)
    return (y.to(s["X"].dtype),)


def _lora_bwd(s):
    x, dc, a, S, R = s["X"].float(), s["dC"].float(), s["A"].float(), s["S"], s["R"]
    dt, scale = s["X"].dtype, _by_row(s)[:, None]
    dtt = _spread(_pick(dc, s["B"].float().transpose(1, 2), s["ids"]) * scale, s["ids"], S)
    dx = dc @ s["W"].float() + dtt @ a.reshape(S * R, -1)
    da = (dtt.T @ x).reshape(a.shape)
    db = (_spread(s["T"] * scale, s["ids"], S).T @ dc).reshape(S, R, -1).transpose(1, 2)
    return dx.to(dt), da.to(dt), db.to(dt).contiguous()


def _ortho(s):
    x = s["G"].float()
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
    tall = s["m"] > s["n"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFFS
    for _ in range(STEPS):
        g = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    if tall:
        x = x.transpose(1, 2)
    return (x.to(s["O"].dtype).contiguous(),)


def _library(s):
    import dense_gemm_sgemm_amd as dg

    if s["op"] == "ortho":
        return (dg.gemm_ortho(s["G"], s["O"], steps=STEPS, coeffs=COEFFS, eps=EPS),)
    if s["op"] == "lora":
        return (dg.gemm_lora(s["X"], s["W"], s["A"], s["B"], s["ids"], s["C"],
                             scales=s["scales"]),)
    dg.gemm_lora_bwd(s["X"], s["W"], s["A"], s["B"], s["ids"], s["T"], s["dC"], dX=s["dX"],
                     dA=s["dA"], dB=s["dB"], scales=s["scales"])
    return s["dX"], s["dA"], s["dB"]


def run(state):
    if own:
        return _library(state)
    op = state["op"]
    if op == "lora":
        return _lora(state)
    return _lora_bwd(state) if op == "lora_bwd" else _ortho(state)


def _ortho_flops(case):
    # X X^T and its square are symmetric: half of their products
    lo, hi = sorted((case["m"], case["n"]))
    return STEPS * case["L"] * (lo * lo * hi + lo * lo * lo + 2 * lo * lo * hi)


def work(case):
    if case["op"] == "ortho":
        size = 4 if case["source"] == "f32" else 2
        return {"bytes": case["L"] * case["m"] * case["n"] * (size + 2),
                "flops": _ortho_flops(case)}
    M, N, K, R, S = (case[k] for k in "MNKRS")
    used = min(S, M)   # adapters that a row can name
    if case["op"] == "lora":
        return {"bytes": 2 * (M * K + N * K + M * N + used * R * (N + K)) + 8 * M + 4 * S,
                "flops": 2 * M * (N * K + R * (N + K))}
    # X, W, dC, T and the adapters in; dX and the adapters' gradients out
    return {"bytes": 2 * (2 * M * K + N * K + M * N + 2 * used * R * (N + K)) + 4 * M * R + 8 * M
            + 4 * S, "flops": 2 * M * (N * K + 2 * R * (N + K))}


# ---- the same from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        out = []
        for g in s["G"].double():
            y = g / (g.norm() + EPS)
            y = y.t().contiguous() if case["m"] > case["n"] else y
            one = torch.eye(y.shape[0], device="cuda", dtype=torch.float64)
            for _ in range(STEPS):
                p = torch.mm(y, y.t())
                y = torch.mm(torch.addmm(COEFFS[0] * one + COEFFS[1] * p, p, p, alpha=COEFFS[2]), y)
            out.append(y.t() if case["m"] > case["n"] else y)
        return (torch.stack(out),)
    x, w, ids = s["X"].double(), s["W"].double(), s["ids"]
    if case["op"] == "lora":
        y = torch.mm(x, w.t())
        for a in range(case["S"]):
            at = (ids == a).nonzero()[:, 0]
            t = torch.mm(x[at], s["A"][a].double().t()) * s["scales"][a].double()
            y[at] += torch.mm(t, s["B"][a].double().t())
        return (y,)
    d = s["dC"].double()
    dx = torch.mm(d, w)
    da, db = s["A"].double().zero_(), s["B"].double().zero_()
    for a in range(case["S"]):
        at = (ids == a).nonzero()[:, 0]
        f = s["scales"][a].double()
        dt = torch.mm(d[at], s["B"][a].double()) * f
        dx[at] += torch.mm(dt, s["A"][a].double())
        da[a] = torch.mm(dt.t(), x[at])
        db[a] = torch.mm(d[at].t(), s["T"][at].double()) * f
    return dx, da, db
