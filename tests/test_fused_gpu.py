"""The fused operators (gated products, 4-bit weights, cross entropy) against
their definitions in 64 bits on the GPU's host."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_sgemm_amd as dg  # noqa: E402
from fused_ref import (DT, Out, act, act_slope, close, gated_ref, gated_tols, half_step,  # noqa: E402
                       norm_close, place, randn, sum_error, w4_norm_close, w4_weights, xent_ref,
                       xent_tol)

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def show(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------- gated

def gated_inputs(M, N, K, dt, seed=0, pad=0, shift=0):
    r = gen(seed)
    mats = (randn((M, K), 1.0, dt, r), randn((N, K), K ** -0.5, dt, r),
            randn((N, K), K ** -0.5, dt, r))
    return [place(t, pad, shift) for t in mats]


# one row to several tiles; N and K off every multiple; K below, at and past a slab
GATED = [(1, 16, 32), (1, 1, 1), (1, 200, 100), (3, 1000, 8), (16, 130, 65), (17, 96, 128),
         (33, 64, 264), (64, 513, 72), (65, 129, 127), (100, 64, 130), (128, 64, 128),
         (129, 257, 320), (300, 500, 264), (257, 1000, 72), (513, 640, 192), (700, 333, 1537),
         (370, 11009, 200), (570, 5001, 4090),
         (65, 5200, 127), (100, 6001, 130), (129, 5001, 320), (300, 2500, 264), (257, 3001, 72),
         (513, 1700, 192), (700, 1333, 1537), (2000, 400, 136), (5000, 100, 70)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", GATED)
def test_gated(M, N, K, typ):
    dt = DT[typ]
    name = ("silu", "relu", "none")[(M + N) % 3]
    X, Wg, Wu = gated_inputs(M, N, K, dt, M + N + K)
    H, G, U = (Out(M, N, dt) for _ in range(3))
    show("gated", M, N, K, typ, name)
    assert dg.gemm_gated(X, Wg, Wu, H.t, act=name, G=G.t, U=U.t) is H.t
    only = Out(M, N, dt)
    dg.gemm_gated(X, Wg, Wu, only.t, act=name)
    g, u, h, sg, su = gated_ref(X, Wg, Wu, name)
    tg, tu, th = gated_tols(g, u, h, sg, su, name, K, dt)
    close(G.t, g, tg, "G")
    close(U.t, u, tu, "U")
    close(H.t, h, th, "H")
    assert torch.equal(only.t, H.t)
    for o in (H, G, U, only):
        o.check_frame("gated")


@pytest.mark.parametrize("M,N,K,pad,shift", [(5, 70, 96, 3, 1), (150, 200, 160, 8, 8),
                                             (150, 200, 160, 5, 0), (200, 150, 136, 0, 1),
                                             (40, 300, 256, 16, 8)])
def test_gated_strides(M, N, K, pad, shift):
    """Rows further apart than their length, and at 2-byte addresses; what lies
    between the rows (NaN) is never read into a result, nor written."""
    dt = torch.bfloat16
    X, Wg, Wu = gated_inputs(M, N, K, dt, 3, pad, shift)
    H, G, U = Out(M, N, dt, pad, shift), Out(M, N, dt, 1, 1), Out(M, N, dt, 0, 3)
    show("gated strides", M, N, K, pad, shift)
    dg.gemm_gated(X, Wg, Wu, H.t, G=G.t, U=U.t)
    g, u, h, sg, su = gated_ref(X, Wg, Wu, "silu")
    tg, tu, th = gated_tols(g, u, h, sg, su, "silu", K, dt)
    close(H.t, h, th, "H")
    close(G.t, g, tg, "G")
    close(U.t, u, tu, "U")
    for o in (H, G, U):
        o.check_frame("gated strides")


def test_gated_halves_of_one_matrix():
    """Wg and Wu as the two halves of one weight, H, G and U beside each other."""
    M, N, K = 140, 192, 128
    r = gen(5)
    W = randn((2 * N, K), K ** -0.5, torch.float16, r).to(DEV)
    X = randn((M, K), 1.0, torch.float16, r).to(DEV)
    out = torch.empty((M, 3 * N), dtype=torch.float16, device=DEV)
    H, G, U = out[:, :N], out[:, N:2 * N], out[:, 2 * N:]
    dg.gemm_gated(X, W[:N], W[N:], H, G=G, U=U)
    g, u, h, sg, su = gated_ref(X, W[:N], W[N:], "silu")
    for got, ref, tol in zip((G, U, H), (g, u, h), gated_tols(g, u, h, sg, su, "silu", K,
                                                             torch.float16)):
        close(got, ref, tol, "half")


@pytest.mark.parametrize("M", [1, 20, 200])
def test_gated_empty_k_and_rows(M):
    H = torch.full((M, 70), 5.0, dtype=torch.float16, device=DEV)
    X, W = (torch.empty((n, 0), dtype=torch.float16, device=DEV) for n in (M, 70))
    dg.gemm_gated(X, W, W, H)
    assert bool((H == 0).all())
    none = torch.empty((0, 70), dtype=torch.float16, device=DEV)
    dg.gemm_gated(torch.empty((0, 64), dtype=torch.float16, device=DEV),
                  torch.ones((70, 64), dtype=torch.float16, device=DEV),
                  torch.ones((70, 64), dtype=torch.float16, device=DEV), none)


def gated_bwd_ref(X, Wg, Wu, G, U, dH, name, dt):
    """Gradients, their elementwise tolerances, and dG, dU."""
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    g, u, dh = G.double(), U.double(), dH.double()
    a, sl = act(g, name), act_slope(g, name)
    d_g, d_u = dh * u * sl, dh * a
    # rounding of dG, dU to the type; fp32 slope: 1 + g (1 - s) cancels to a few
    # 2^-24 of 1 + |g|
    half = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    e_g = half * d_g.abs() + 2.0 ** -20 * (dh * u).abs() * (1 + g.abs()) + tiny
    e_u = half * d_u.abs() + 2.0 ** -20 * d_u.abs() + tiny
    M, N = G.shape
    out = []
    dx = d_g @ wg + d_u @ wu
    sx = d_g.abs() @ wg.abs() + d_u.abs() @ wu.abs()
    out.append((dx, e_g @ wg.abs() + e_u @ wu.abs() + sum_error(2 * N, sx) + half_step(dt, dx)))
    for d, e in ((d_g, e_g), (d_u, e_u)):
        dw = d.T @ x
        out.append((dw, e.T @ x.abs() + sum_error(M, d.abs().T @ x.abs()) + half_step(dt, dw)))
    return out


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", GATED)
def test_gated_bwd(M, N, K, typ):
    dt = DT[typ]
    name = ("silu", "relu", "none")[(M + N) % 3]
    X, Wg, Wu = gated_inputs(M, N, K, dt, M + N + K)
    r = gen(9)
    G, U, dH = (randn((M, N), s, dt, r).to(DEV) for s in (1.5, 1.0, 0.5))
    G[0, 0] = 0.0   # ReLU's corner
    dX, dWg, dWu = Out(M, K, dt), Out(N, K, dt), Out(N, K, dt)
    show("gated_bwd", M, N, K, typ, name)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX=dX.t, dWg=dWg.t, dWu=dWu.t, act=name)
    refs = gated_bwd_ref(X, Wg, Wu, G, U, dH, name, dt)
    for o, (ref, tol), what in zip((dX, dWg, dWu), refs, ("dX", "dWg", "dWu")):
        close(o.t, ref, tol, what)
        if ref.numel() > 1000:
            norm_close(o.t, ref, torch.finfo(dt).eps, what)
        o.check_frame(what)
    # each gradient by itself is the same
    for k, o in (("dX", dX), ("dWg", dWg), ("dWu", dWu)):
        one = torch.empty_like(o.t).contiguous()
        dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, act=name, **{k: one})
        assert torch.equal(one, o.t), k


@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 0), (0, 1)])
def test_gated_bwd_strides(pad, shift):
    M, N, K, dt = 150, 201, 136, torch.float16
    X, Wg, Wu = gated_inputs(M, N, K, dt, 4, pad, shift)
    Wu = place(Wu.cpu(), pad + 8, 0)   # the two weights' rows differ
    r = gen(11)
    G, U, dH = (place(randn((M, N), 1.0, dt, r), pad, shift) for _ in range(3))
    outs = [Out(M, K, dt, pad, shift), Out(N, K, dt, pad + 1, 0), Out(N, K, dt, 0, 1)]
    show("gated_bwd strides", pad, shift)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *[o.t for o in outs])
    for o, (ref, tol) in zip(outs, gated_bwd_ref(X, Wg, Wu, G, U, dH, "silu", dt)):
        close(o.t, ref, tol, "strided gradient")
        o.check_frame("gated_bwd")


def test_gated_bwd_empty_sums():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    full = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    # no rows: the weights' gradients are zero
    dWg, dWu = full(70, 64), full(70, 64)
    dg.gemm_gated_bwd(e(0, 64), e(70, 64), e(70, 64), e(0, 70), e(0, 70), e(0, 70), dWg=dWg,
                      dWu=dWu)
    assert bool((dWg == 0).all()) and bool((dWu == 0).all())
    # no columns: dX is zero
    dX = full(5, 64)
    dg.gemm_gated_bwd(e(5, 64), e(0, 64), e(0, 64), e(5, 0), e(5, 0), e(5, 0), dX=dX)
    assert bool((dX == 0).all())


def test_gated_extreme_gates():
    """Large gates of either sign saturate SiLU and its slope without NaN."""
    M, N, K, dt = 130, 64, 128, torch.bfloat16
    X = torch.zeros((M, K), dtype=dt, device=DEV)
    X[:, 0] = torch.linspace(-300, 300, M)
    Wg = torch.zeros((N, K), dtype=dt, device=DEV)
    Wu = torch.zeros((N, K), dtype=dt, device=DEV)
    Wg[:, 0], Wu[:, 0] = 1.0, 0.5
    H, G, U = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(3))
    dg.gemm_gated(X, Wg, Wu, H, G=G, U=U)
    g, u, h, sg, su = gated_ref(X, Wg, Wu, "silu")
    close(H, h, gated_tols(g, u, h, sg, su, "silu", K, dt)[2] + 1e-30, "H")
    dX = torch.empty_like(X)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, torch.ones_like(H), dX=dX)
    ref, tol = gated_bwd_ref(X, Wg, Wu, G, U, torch.ones_like(H), "silu", dt)[0]
    close(dX, ref, tol + 1e-30, "dX")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("name", ["silu", "relu", "none"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 72), (5, 70, 130), (40, 33, 65), (200, 2700, 136),
                                   (129, 5001, 70)])
def test_gated_not_a_number(M, N, K, name, typ):
    """NaN gates give NaN (ReLU's too), an infinite x what the definition gives;
    outputs they do not enter keep their bits.  Few rows, tiles, padded copies."""
    dt = DT[typ]
    X, Wg, Wu = gated_inputs(M, N, K, dt, 23)
    base = [torch.empty((M, N), dtype=dt, device=DEV) for _ in range(3)]
    show("gated NaN", M, N, K, name, typ)
    dg.gemm_gated(X, Wg, Wu, base[0], act=name, G=base[1], U=base[2])
    nan_w = Wg.clone()
    nan_w[N // 2, K // 2] = float("nan")
    H, G, U = (Out(M, N, dt) for _ in range(3))
    dg.gemm_gated(X, nan_w, Wu, H.t, act=name, G=G.t, U=U.t)
    column = torch.arange(N, device=DEV) == N // 2
    assert bool(torch.isnan(H.t[:, column]).all()) and bool(torch.isnan(G.t[:, column]).all())
    for o, b in zip((H, G, U), base):
        assert torch.equal(o.t[:, ~column], b[:, ~column])
    assert torch.equal(U.t, base[2])
    inf_x = X.clone()
    inf_x[M // 2, K - 1] = float("inf")
    dg.gemm_gated(inf_x, Wg, Wu, H.t, act=name, G=G.t, U=U.t)
    g, u, h, sg, su = gated_ref(inf_x, Wg, Wu, name)
    tols = gated_tols(g, u, h, sg, su, name, K, dt)
    for o, ref, tol in zip((G, U, H), (g, u, h), tols):
        close(o.t, ref, tol, "beside an infinite row")
        o.check_frame("gated")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("name", ["silu", "relu", "none"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 72), (70, 130, 65), (200, 700, 136)])
def test_gated_bwd_not_a_number(M, N, K, name, typ):
    """A NaN gate reaches its row of dX and its rows of dWg (through the slope)
    and dWu, and nothing else."""
    dt = DT[typ]
    X, Wg, Wu = gated_inputs(M, N, K, dt, 24)
    r = gen(25)
    G, U, dH = (randn((M, N), 1.0, dt, r).to(DEV) for _ in range(3))
    base = [torch.empty_like(q) for q in (X, Wg, Wu)]
    show("gated_bwd NaN", M, N, K, name, typ)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *base, act=name)
    m, n = M // 2, N // 3
    G[m, n] = float("nan")
    got = [torch.empty_like(q) for q in base]
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *got, act=name)
    for o, b, row in zip(got, base, (m, None if name == "none" else n, n)):
        hit = torch.zeros(len(o), dtype=torch.bool, device=DEV)
        if row is not None:
            hit[row] = True
        assert bool(torch.isnan(o[hit]).all()) and torch.equal(o[~hit], b[~hit])


@pytest.mark.parametrize("size", ["small", "large"])
@pytest.mark.parametrize("want", ["dX", "dWg", "dWu", "dWg dWu", "dX dWg dWu"])
@pytest.mark.parametrize("M,N,K", [(300, 200, 136), (256, 512, 128), (1000, 130, 300),
                                   (70, 1000, 2100)])
def test_gated_bwd_fp16_range(M, N, K, want, size):
    """dG and dU outside binary16's range beside gradients inside it.  Small:
    dG = dU of 2e-6, the same in all rows of a column, as a rounding in
    binary16's subnormal range (up to 2^-25) would be.  Large: dG and dU of
    4e5.  A rounding of the factored values is eps / 2 at most and the outputs'
    own as much: eps in the norm."""
    dt = torch.float16
    r = gen(M + N)
    names = want.split()
    if size == "small":
        X = 30 + randn((M, K), 1.0, torch.float32, r)
        G = (0.04 * (1 + 0.3 * torch.rand((N,), generator=r))).expand(M, N)
        U = 0.5 * G
        dH = torch.full((M, N), 1e-4)
        W = [1000 * (1 + torch.rand((N, K), generator=r)) for _ in range(2)]
    else:
        X = randn((M, K), 1e-3, torch.float32, r)
        G = 100 * (1 + 0.1 * torch.rand((M, N), generator=r))
        U = 100 + randn((M, N), 1.0, torch.float32, r)
        dH = randn((M, N), 4000.0, torch.float32, r)
        W = [randn((N, K), 1e-4, torch.float32, r) for _ in range(2)]
    X, Wg, Wu, G, U, dH = (q.to(dt).to(DEV).contiguous() for q in (X, *W, G, U, dH))
    outs = {"dX": torch.empty_like(X), "dWg": torch.empty_like(Wg), "dWu": torch.empty_like(Wu)}
    show("gated_bwd range", M, N, K, want, size)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, **{k: outs[k] for k in names})
    refs = dict(zip(outs, gated_bwd_ref(X, Wg, Wu, G, U, dH, "silu", dt)))
    for k in names:
        ref = refs[k][0]
        assert 2.0 ** -10 < float(ref.abs().max()) < 6e4   # representable
        assert bool(torch.isfinite(outs[k]).all()), k
        norm_close(outs[k], ref, torch.finfo(dt).eps, k)


def test_gated_bwd_fp16_infinite():
    """An infinite dH takes its row of dX and its rows of dWg and dWu with it and
    leaves the others their bits; all of dH zero gives zeros."""
    M, N, K, dt = 150, 200, 136, torch.float16
    X, Wg, Wu = gated_inputs(M, N, K, dt, 26)
    r = gen(27)
    G, U = (1 + randn((M, N), 0.1, dt, r).to(DEV).abs() for _ in range(2))
    dH = 1 + randn((M, N), 0.1, dt, r).to(DEV).abs()
    base = [torch.empty_like(q) for q in (X, Wg, Wu)]
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *base)
    dH[40, 60] = float("inf")
    got = [torch.empty_like(q) for q in base]
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *got)
    for o, b, row in zip(got, base, (40, 60, 60)):
        rest = torch.arange(len(o), device=DEV) != row
        assert not bool(torch.isfinite(o[row]).any()) and torch.equal(o[rest], b[rest])
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, torch.zeros_like(dH), *got)
    assert all(bool((o == 0).all()) for o in got)


# ---------------------------------------------------------------- 4-bit weights

def w4_inputs(M, N, K, group, dt, zeros, seed=0, pad=0, shift=0):
    r = gen(seed)
    groups = -(-K // group)
    X = place(randn((M, K), 1.0, dt, r), pad, shift)
    Wq = place(torch.randint(0, 256, (N, (K + 1) // 2), generator=r, dtype=torch.uint8), pad, shift)
    s = place((torch.rand((N, groups), generator=r) + 0.5).to(dt), pad, shift)
    z = None
    if zeros:
        z = place(torch.randint(0, 16, (N, groups), generator=r, dtype=torch.uint8), pad, shift)
    return X, Wq, s, z


def w4_check(C, X, Wq, s, z, group, bias=None, name="none", res=None):
    K, dt = X.shape[1], X.dtype
    q, sc = w4_weights(Wq, s, z, group, K)
    x = X.double()
    y = x @ (q * sc).T
    # bf16 sums x (128 + q) and (128 + z) x apart: products of up to 143 |s x|
    size = 143.0 * 2 if dt == torch.bfloat16 else 15.0
    S = x.abs() @ (sc.abs() * size).T
    tol = sum_error(K, S) + 2.0 ** -22 * y.abs()
    if bias is not None:
        y = y + bias.double()
    y2 = act(y, name)
    tol = 1.1 * tol + 2.0 ** -20 * y2.abs()
    if res is not None:
        y2 = y2 + res.double()
    close(C, y2, tol + half_step(dt, y2.abs() + tol), "C")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 16, 128, 128, False), (1, 1, 1, 32, True), (1, 100, 4096, 128, True),
    (2, 33, 512, 32, True), (5, 2305, 768, 32, True), (3, 48, 1000, 64, True),
    (16, 64, 640, 64, False), (17, 70, 2048, 128, True), (7, 31, 333, 96, True),
    (31, 40, 1536, 256, True), (33, 50, 257, 128, True), (64, 96, 1024, 64, True),
    (65, 40, 520, 32, True), (130, 17, 300, 160, False), (1, 300, 16384, 128, True),
    (4, 20, 31, 128, True), (9, 65, 130, 1024, True), (3, 40, 8192, 64, True),
    (1, 33, 28000, 128, True), (20, 129, 2048, 64, True), (32, 300, 4100, 128, False),
    (40, 128, 16384, 128, True), (48, 257, 9000, 32, True), (100, 250, 3333, 96, True),
    (17, 16, 100, 32, False)])
def test_w4(M, N, K, group, zeros, typ):
    dt = DT[typ]
    X, Wq, s, z = w4_inputs(M, N, K, group, dt, zeros, M + N + K)
    C = Out(M, N, dt)
    show("w4", M, N, K, group, zeros, typ)
    assert dg.gemm_w4(X, Wq, s, C.t, group=group, zeros=z) is C.t
    w4_check(C.t, X, Wq, s, z, group)
    C.check_frame("w4")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128, 256, 96])
@pytest.mark.parametrize("M,N,K", [(1, 40, 16384), (2, 30, 9000), (5, 40, 16384), (16, 33, 17000),
                                   (64, 20, 16500)])
def test_w4_long(M, N, K, group, typ):
    """Few weight rows and a long K: the most waves a workgroup has."""
    dt = DT[typ]
    X, Wq, s, z = w4_inputs(M, N, K, group, dt, True, M + group)
    C = Out(M, N, dt)
    show("w4 long", M, N, K, group, typ)
    dg.gemm_w4(X, Wq, s, C.t, group=group, zeros=z)
    w4_check(C.t, X, Wq, s, z, group)
    C.check_frame("w4")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 96])
@pytest.mark.parametrize("M,N,K", [(1, 100, 16384), (3, 100, 9001), (5, 64, 16384), (16, 65, 17000),
                                   (16, 200, 300), (24, 64, 9000), (40, 50, 16400), (64, 64, 4100),
                                   (70, 40, 2050)])
def test_w4_in_norm(M, N, K, group, zeros, typ):
    """A bound that one wrong K value in a thousand exceeds (see
    test_fused_checks.py), at a long K too, where the elementwise one of bf16's
    two large sums is wide."""
    dt = DT[typ]
    X, Wq, s, z = w4_inputs(M, N, K, group, dt, zeros, M + K + group)
    C = torch.empty((M, N), dtype=dt, device=DEV)
    show("w4 in norm", M, N, K, group, zeros, typ)
    dg.gemm_w4(X, Wq, s, C, group=group, zeros=z)
    w4_norm_close(C, X, *w4_weights(Wq, s, z, group, K), "C")


@pytest.mark.parametrize("pad,shift", [(1, 1), (3, 0), (16, 16)])
@pytest.mark.parametrize("group", [32, 64, 128, 96])
def test_w4_strides(group, pad, shift):
    M, N, K, dt = 6, 37, 700, torch.float16
    X, Wq, s, z = w4_inputs(M, N, K, group, dt, True, 2, pad, shift)
    C = Out(M, N, dt, pad, shift)
    show("w4 strides", group, pad, shift)
    dg.gemm_w4(X, Wq, s, C.t, group=group, zeros=z)
    w4_check(C.t, X, Wq, s, z, group)
    C.check_frame("w4")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu"])
@pytest.mark.parametrize("M,K", [(2, 384), (9, 384), (33, 4096)])
def test_w4_write_back(M, K, name, typ):
    N, dt = 50, DT[typ]
    X, Wq, s, z = w4_inputs(M, N, K, 128, dt, True, 6)
    r = gen(7)
    bias, res = randn((N,), 5.0, dt, r).to(DEV), randn((M, N), 5.0, dt, r).to(DEV)
    C = torch.empty((M, N), dtype=dt, device=DEV)
    dg.gemm_w4(X, Wq, s, C, zeros=z, bias=bias, act=name, residual=res)
    w4_check(C, X, Wq, s, z, 128, bias, name, res)
    inplace = res.clone()
    dg.gemm_w4(X, Wq, s, inplace, zeros=z, bias=bias, act=name, residual=inplace)
    assert torch.equal(inplace, C)


def test_w4_offset_sums_cancel():
    """x of one sign: the bf16 form's two large sums cancel; scales over a wide
    range; every nibble at every place."""
    M, N, K, dt = 4, 16, 512, torch.bfloat16
    X = torch.full((M, K), 3.0, dtype=dt, device=DEV)
    nib = (torch.arange(N)[:, None] + torch.arange(K)[None, :]) % 16
    Wq = (nib[:, 0::2] | (nib[:, 1::2] << 4)).to(torch.uint8).to(DEV)
    s = torch.logspace(-3, 3, N * 4).reshape(N, 4).to(dt).to(DEV)
    z = torch.arange(N * 4).reshape(N, 4).remainder(16).to(torch.uint8).to(DEV)
    C = torch.empty((M, N), dtype=dt, device=DEV)
    dg.gemm_w4(X, Wq, s, C, zeros=z)
    w4_check(C, X, Wq, s, z, 128)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("M,N,K", [(1, 33, 700), (2, 30, 9000), (6, 40, 300), (16, 33, 17000),
                                   (20, 49, 2100), (64, 20, 4500), (70, 17, 513)])
def test_w4_infinite_and_huge(M, N, K, group, typ):
    """An infinite or NaN x gives its row what the definition gives (NaN only
    where the weight is zero, or where infinities meet), and bf16 values whose
    128-fold no fp32 holds are multiplied as any others; the other rows keep
    their bits."""
    dt = DT[typ]
    X, Wq, s, z = w4_inputs(M, N, K, group, dt, True, M + group)
    base = torch.empty((M, N), dtype=dt, device=DEV)
    dg.gemm_w4(X, Wq, s, base, group=group, zeros=z)
    m, inf = M // 2, float("inf")
    kinds = [{0: inf}, {K - 1: -inf}, {K // 2: inf, K // 3: inf}, {5: inf, K - 2: -inf},
             {K // 2: float("nan")}]
    if typ == "bf16":   # 15 x 1.5 x 3 x 2^121 < 2^128
        kinds += [{K // 3: 2.0 ** 121}, {0: -2.0 ** 121, K // 2: 2.0 ** 121, K - 1: 2.0 ** 121}]
    for kind in kinds:
        X2 = X.clone()
        for k, v in kind.items():
            X2[m, k] = v
        C = Out(M, N, dt)
        show("w4 infinite", M, N, K, group, typ, kind)
        dg.gemm_w4(X2, Wq, s, C.t, group=group, zeros=z)
        w4_check(C.t, X2, Wq, s, z, group)
        others = torch.arange(M, device=DEV) != m
        assert torch.equal(C.t[others], base[others]), kind
        C.check_frame("w4")


def test_w4_empty_k():
    C = torch.full((3, 20), 5.0, dtype=torch.float16, device=DEV)
    e = lambda r, dt: torch.empty((r, 0), dtype=dt, device=DEV)  # noqa: E731
    bias = torch.arange(20, device=DEV).half() - 10
    dg.gemm_w4(e(3, torch.float16), e(20, torch.uint8), e(20, torch.float16), C, bias=bias,
               act="relu")
    assert torch.equal(C, bias.clamp(min=0).expand(3, 20))


# ---------------------------------------------------------------- cross entropy

IGN = -100


def xent_inputs(M, N, K, dt, seed=0, pad=0, shift=0, sd=3.0):
    r = gen(seed)
    X = place(randn((M, K), 1.0, dt, r), pad, shift)
    W = place(randn((N, K), sd * K ** -0.5, dt, r), pad, shift)
    t = torch.randint(0, N, (M,), generator=r)
    t[torch.rand((M,), generator=r) < 0.1] = IGN
    t[0] = N - 1
    return X, W, t.to(DEV)


XENT = [(1, 1, 1), (1, 2, 8), (2, 127, 64), (5, 128, 128), (129, 129, 130), (200, 1000, 136),
        (128, 191, 65), (64, 300, 72), (333, 5001, 96), (300, 256, 1537), (513, 2050, 264),
        (370, 22001, 136), (370, 22001, 1032)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", XENT)
def test_xent(M, N, K, typ):
    dt = DT[typ]
    X, W, t = xent_inputs(M, N, K, dt, M + N)
    loss, lse = torch.full((M,), 9.0, device=DEV), torch.full((M,), 9.0, device=DEV)
    show("xent", M, N, K, typ)
    assert dg.gemm_xent(X, W, t, loss, lse) is loss
    z, rl, ro = xent_ref(X, W, t, IGN)
    tol = xent_tol(X, W, z, rl)
    close(lse, rl, tol, "lse")
    close(loss, ro, 2 * tol, "loss")
    assert bool((loss[t == IGN] == 0).all())


def xent_bwd_check(X, W, t, lse, dloss, dX, dW, ignore=IGN):
    dt, K = X.dtype, X.shape[1]
    M, N = X.shape[0], W.shape[0]
    x, w = X.double(), W.double()
    z = x @ w.T
    live = t != ignore
    rows = torch.arange(M, device=DEV)[live]
    d = torch.exp(z - lse.double()[:, None])
    e = d * (xent_tol(X, W, z, lse.double())[:, None] + 2.0 ** -18)   # exp of an inexact z - lse
    d[rows, t[live]] -= 1
    scale = torch.where(live, dloss.double(), torch.zeros_like(dloss.double()))[:, None]
    d, e = d * scale, e * scale.abs()
    eps = torch.finfo(dt).eps
    e = e + eps / 2 * d.abs()
    if dt == torch.float16:   # half of binary16's smallest step below the common factor
        e = e + 2.0 ** -25 * 2.0 ** -13 * float(scale.abs().max()) * live[:, None]
    if dX is not None:
        ref = d @ w
        close(dX, ref, e @ w.abs() + sum_error(N, d.abs() @ w.abs()) + half_step(dt, ref), "dX")
        if ref.numel() > 1000:
            norm_close(dX, ref, eps, "dX")
    if dW is not None:
        ref = d.T @ x
        close(dW, ref, e.T @ x.abs() + sum_error(M, d.abs().T @ x.abs()) + half_step(dt, ref),
              "dW")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", XENT)
def test_xent_bwd(M, N, K, typ):
    dt = DT[typ]
    X, W, t = xent_inputs(M, N, K, dt, M + N)
    lse = torch.logsumexp(X.double() @ W.double().T, 1).float()
    dloss = (torch.rand((M,), generator=gen(3)) + 0.5).to(DEV)
    dX, dW = Out(M, K, dt), Out(N, K, dt)
    show("xent_bwd", M, N, K, typ)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX.t, dW=dW.t)
    xent_bwd_check(X, W, t, lse, dloss, dX.t, dW.t)
    dX.check_frame("dX")
    dW.check_frame("dW")
    a, b = torch.empty_like(dX.t).contiguous(), torch.empty_like(dW.t).contiguous()
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=a)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dW=b)
    assert torch.equal(a, dX.t) and torch.equal(b, dW.t)


@pytest.mark.parametrize("M,N,K", [(4096, 40009, 128), (65536, 16394, 128), (33000, 4100, 136)])
def test_xent_bwd_in_pieces(M, N, K):
    """More columns than one piece: two of them; eight and a last one of ten
    columns, which starts early; two and a ragged one."""
    dt = torch.bfloat16
    X, W, t = xent_inputs(M, N, K, dt, 21)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    show("xent pieces", M, N, K)
    dg.gemm_xent(X, W, t, loss, lse)
    dloss = torch.full((M,), 1.0 / M, device=DEV)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX, dW=dW)
    # in 64 bits, by rows
    dx, dw = torch.empty_like(X, dtype=torch.float64), torch.zeros_like(W, dtype=torch.float64)
    w = W.double()
    for i in range(0, M, 4096):
        x, ti = X[i:i + 4096].double(), t[i:i + 4096]
        d = x @ w.T
        l64 = torch.logsumexp(d, 1)
        assert float((lse[i:i + 4096] - l64).abs().max()) < 1e-4
        d = torch.exp(d - l64[:, None])
        live = ti != IGN
        d[torch.arange(len(ti), device=DEV)[live], ti[live]] -= 1
        d *= live[:, None] / M
        dx[i:i + 4096] = d @ w
        dw += d.T @ x
    norm_close(dX, dx, torch.finfo(dt).eps, "dX")
    norm_close(dW, dw, torch.finfo(dt).eps, "dW")
    # row by row of W as well: each piece's rows, the shared ones of the last two among them
    rel = (dW.double() - dw).norm(dim=1) / dw.norm(dim=1)
    assert float(rel.max()) <= 2 * torch.finfo(dt).eps, int(rel.argmax())


@pytest.mark.parametrize("M,N,K", [(16384, 262154, 128), (8192, 524400, 72)])
def test_xent_bwd_last_piece_in_ranges(M, N, K):
    """A last piece of ten and of 112 columns (two slabs of 64) where the others'
    128 and 256 slabs are cut into ranges: ranges of one slab."""
    test_xent_bwd_in_pieces(M, N, K)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("N", [321, 832, 833, 1088, 1345, 1600])
def test_gated_bwd_ranges(N, typ):
    """Few outputs of dX over 12 to 50 slabs: last ranges of every length."""
    M, K, dt = 128, 128, DT[typ]
    X, Wg, Wu = gated_inputs(M, N, K, dt, N)
    r = gen(N)
    G, U, dH = (randn((M, N), 1.0, dt, r).to(DEV) for _ in range(3))
    outs = [Out(r, K, dt) for r in (M, N, N)]
    show("gated_bwd ranges", N, typ)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, *[o.t for o in outs])
    for o, (ref, tol) in zip(outs, gated_bwd_ref(X, Wg, Wu, G, U, dH, "silu", dt)):
        close(o.t, ref, tol, "gradient")
        norm_close(o.t, ref, torch.finfo(dt).eps, "gradient")
        o.check_frame("gated_bwd")


@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 8), (0, 1)])
def test_xent_strides(pad, shift):
    M, N, K, dt = 140, 333, 152, torch.float16
    X, W, t = xent_inputs(M, N, K, dt, 8, pad, shift)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    show("xent strides", pad, shift)
    dg.gemm_xent(X, W, t, loss, lse)
    z, rl, ro = xent_ref(X, W, t, IGN)
    tol = xent_tol(X, W, z, rl)
    close(loss, ro, 2 * tol, "loss")
    dloss = torch.rand((M,), device=DEV)
    dX, dW = Out(M, K, dt, pad, shift), Out(N, K, dt, pad, shift)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX.t, dW=dW.t)
    xent_bwd_check(X, W, t, lse, dloss, dX.t, dW.t)
    dX.check_frame("dX")
    dW.check_frame("dW")


@pytest.mark.parametrize("typ", TYPES)
def test_xent_targets(typ):
    """All rows ignored; an ignored class inside the vocabulary; targets out of
    range; ignored rows whose lse and dloss are NaN."""
    M, N, K, dt = 150, 300, 128, DT[typ]
    X, W, t = xent_inputs(M, N, K, dt, 12)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dX, dW = torch.full_like(X, 3.0), torch.full_like(W, 3.0)
    every = torch.full_like(t, IGN)
    dg.gemm_xent(X, W, every, loss, lse)
    assert bool((loss == 0).all())
    bad = torch.full((M,), float("nan"), device=DEV)
    dg.gemm_xent_bwd(X, W, every, bad, bad, dX=dX, dW=dW)
    assert bool((dX == 0).all()) and bool((dW == 0).all())
    # class 7 is the padding class
    t = torch.where(t == IGN, torch.full_like(t, 7), t)
    dg.gemm_xent(X, W, t, loss, lse, ignore_index=7)
    assert bool((loss[t == 7] == 0).all()) and bool((loss[t != 7] > 0).all())
    dloss = torch.ones((M,), device=DEV)
    dloss[t == 7] = float("nan")
    Xn = X.clone()
    Xn[t == 7] = float("nan")
    dg.gemm_xent_bwd(Xn, W, t, lse, dloss, dX=dX, dW=dW, ignore_index=7)
    xent_bwd_check(X, W, t, lse, torch.ones((M,), device=DEV), dX, dW, ignore=7)
    # out of range: the row's loss and dX are NaN, and so is dW
    t[3], t[140] = N, -1
    dg.gemm_xent(X, W, t, loss, lse, ignore_index=7)
    assert torch.isnan(loss).nonzero().flatten().tolist() == [3, 140]
    dg.gemm_xent_bwd(X, W, t, lse, torch.ones((M,), device=DEV), dX=dX, dW=dW, ignore_index=7)
    assert torch.isnan(dX).any(1).nonzero().flatten().tolist() == [3, 140]
    assert bool(torch.isnan(dW).all())


def test_xent_no_rows():
    W = torch.ones((200, 128), dtype=torch.float16, device=DEV)
    dW = torch.full_like(W, 4.0)
    e = torch.empty((0,), device=DEV)
    none = torch.empty((0,), dtype=torch.int64, device=DEV)
    X = torch.empty((0, 128), dtype=torch.float16, device=DEV)
    dg.gemm_xent(X, W, none, e, e.clone())
    dg.gemm_xent_bwd(X, W, none, e, e, dW=dW)
    assert bool((dW == 0).all())


@pytest.mark.parametrize("N,K", [(200, 100), (1000, 4095), (70, 128)])
def test_xent_bwd_no_rows_null_operands(N, K):
    """No rows, through the C entry point: dW = 0 with null operands, at sizes
    that would have padded copies."""
    from dense_gemm_sgemm_amd import fused

    dW = Out(N, K, torch.bfloat16, 3, 1)
    lib = fused.load_library()
    need = lib.gemm_xent_bwd_workspace(1, 0, N, K, None, K, None, K, 0, 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    show("xent_bwd without rows", N, K)
    status = lib.gemm_xent_bwd(1, 0, N, K, None, K, None, K, None, IGN, None, None, None, 0,
                               dW.t.data_ptr(), dW.t.stride(0), ws.data_ptr(), need,
                               torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    assert bool((dW.t == 0).all())
    dW.check_frame("dW")


def test_xent_no_columns_of_x():
    """K == 0: all logits are 0."""
    X, W = (torch.empty((n, 0), dtype=torch.bfloat16, device=DEV) for n in (5, 300))
    t = torch.tensor([0, 299, IGN, 7, 300], device=DEV)
    loss, lse = torch.empty((5,), device=DEV), torch.empty((5,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    log300 = torch.full((5,), 300.0, dtype=torch.float64, device=DEV).log()
    close(lse, log300, 64 * 2.0 ** -24 + 2.0 ** -22 * log300, "lse")
    want = log300.clone()
    want[2], want[4] = 0.0, float("nan")
    close(loss, want, 64 * 2.0 ** -24 + 2.0 ** -22 * log300, "loss")


def test_xent_infinite_logits():
    """A logit of +inf gives lse = +inf, one of -inf counts for nothing, NaN
    stays NaN, each in its row only."""
    M, N, K, dt = 130, 400, 128, torch.bfloat16
    X, W, t = xent_inputs(M, N, K, dt, 14)
    W[:, 0], X[:, 0] = 0.0, 0.0
    W[5, 0], t[:] = 1.0, 9
    X[0, 0], X[1, 0], X[2, 0] = float("inf"), float("-inf"), float("nan")
    W[:5, 0], W[6:, 0] = 2.0 ** -60, 2.0 ** -60
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    assert float(lse[0]) == float("inf") and float(lse[1]) == float("-inf")
    assert bool(torch.isnan(lse[2])) and bool(torch.isfinite(lse[3:]).all())
    X[1, 0], W[7, 0] = float("-inf"), -1.0     # one column of +inf beside columns of -inf
    dg.gemm_xent(X, W, t, loss, lse)
    assert float(lse[1]) == float("inf")


def test_xent_extreme_logits():
    """A row whose largest logit leaves nothing beside it, one with equal
    logits, and tiny fp16 gradients of a large mean."""
    M, N, K, dt = 130, 300, 128, torch.float16
    X = torch.zeros((M, K), dtype=dt, device=DEV)
    X[0, 0], X[1, 0] = 200.0, -200.0
    W = torch.zeros((N, K), dtype=dt, device=DEV)
    W[17, 0] = 200.0
    t = torch.full((M,), 17, device=DEV)
    t[1] = 299
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    z, rl, ro = xent_ref(X, W, t, IGN)
    close(loss, ro, 2 * xent_tol(X, W, z, rl), "loss")
    X, W, t = xent_inputs(M, N, K, dt, 13)
    dg.gemm_xent(X, W, t, loss, lse)
    for size in (1e-7, 1e4):   # gradients that fp16 could not hold, or not without the factor
        dloss = torch.full((M,), size, device=DEV)
        dX = torch.empty_like(X)
        dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX)
        xent_bwd_check(X, W, t, lse, dloss, dX, None)


@pytest.mark.parametrize("typ", TYPES)
def test_xent_bwd_one_dloss_for_all(typ):
    """A mean's dloss, just below halfway between two 16-bit values: its own
    rounding (up to half a step, the same way in every row) must not reach the
    gradients.  Their outputs' rounding is at most half a step each, evenly
    spread: 1 / sqrt(3) of it in the norm; the rounding of d adds as much of the
    probabilities' share, here a tenth (300 rows, 1000 columns)."""
    M, N, K, dt = 300, 1000, 128, DT[typ]
    X, W, t = xent_inputs(M, N, K, dt, 17, sd=1.0)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    half = torch.finfo(dt).eps / 2
    dloss = torch.full((M,), 1.0 + 0.99 * half, device=DEV)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX, dW=dW)
    d = torch.softmax(X.double() @ W.double().T, 1)
    live = t != IGN
    d[torch.arange(M, device=DEV)[live], t[live]] -= 1
    d *= live[:, None] * dloss.double()[:, None]
    for got, ref in ((dX, d @ W.double()), (dW, d.T @ X.double())):
        norm_close(got, ref, 1.2 * half / 3 ** 0.5, "one dloss")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_xent_bwd_infinite_dloss(value, typ):
    """A dloss that is no number takes its row of dX (and dW) with it; the other
    rows of dX keep their bits, also where fp16 needs the common factor."""
    M, N, K, dt = 150, 2000, 136, DT[typ]
    X, W, t = xent_inputs(M, N, K, dt, 18, sd=1.0)
    t[40] = 7
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    dloss = torch.full((M,), 1e-3, device=DEV)
    base, dX = torch.empty_like(X), torch.empty_like(X)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=base)
    dloss[40] = value
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX)
    rest = torch.arange(M, device=DEV) != 40
    assert not bool(torch.isfinite(dX[40]).any()) and torch.equal(dX[rest], base[rest])


# ---------------------------------------------------------------- how they are called

def test_run_together():
    """A training step of a block and its head -- gated product, projection down
    with the residual, cross entropy, and back -- against the same in 64 bits."""
    M, H, F, V, dt = 200, 256, 520, 1000, torch.bfloat16
    r = gen(31)
    X = randn((M, H), 1.0, dt, r).to(DEV)
    Wg, Wu = (randn((F, H), H ** -0.5, dt, r).to(DEV) for _ in range(2))
    Wd = randn((H, F), F ** -0.5, dt, r).to(DEV)
    Wv = randn((V, H), H ** -0.5, dt, r).to(DEV)
    t = torch.randint(0, V, (M,), generator=r).to(DEV)
    t[::9] = IGN
    new = lambda *s, d=dt: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    A, G, U, Y = new(M, F), new(M, F), new(M, F), new(M, H)
    loss, lse = new(M, d=torch.float32), new(M, d=torch.float32)
    dg.gemm_gated(X, Wg, Wu, A, G=G, U=U)
    dg.gemm_ex(A, Wd, Y, residual=X)
    dg.gemm_xent(Y, Wv, t, loss, lse)
    count = int((t != IGN).sum())
    dloss = torch.full((M,), 1.0 / count, device=DEV)
    dY, dWv, dA, dWd = new(M, H), new(V, H), new(M, F), new(H, F)
    dX, dWg, dWu = new(M, H), new(F, H), new(F, H)
    dg.gemm_xent_bwd(Y, Wv, t, lse, dloss, dX=dY, dW=dWv)
    dg.gemm_ex(dY, Wd, dA, op_b="n")
    dg.gemm_ex(dY, A, dWd, op_a="t", op_b="n")
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dA, dX=dX, dWg=dWg, dWu=dWu)
    dX = dX.double() + dY.double()   # the residual's path

    p = [q.detach().double().requires_grad_() for q in (X, Wg, Wu, Wd, Wv)]
    x, wg, wu, wd, wv = p
    g = x @ wg.T
    y = (g * torch.sigmoid(g) * (x @ wu.T)) @ wd.T + x
    z = y @ wv.T
    ref = torch.nn.functional.cross_entropy(z, t, ignore_index=IGN, reduction="sum") / count
    grads = torch.autograd.grad(ref, p)
    ref = ref.detach()
    mean = float(loss.double().sum() / count)
    # activations and gradients pass through up to seven roundings to bf16 (A,
    # Y, d, dY, dA, dG or dU, and the result), independent of each other
    eps = torch.finfo(dt).eps
    assert abs(mean - float(ref)) <= 2 * eps * float(ref)
    for got, want, what in zip((dX, dWg, dWu, dWd, dWv), grads, "dX dWg dWu dWd dWv".split()):
        norm_close(got, want, 7 ** 0.5 * eps, what)


def test_gradients_against_differences():
    """The change of the summed loss along a direction, from central
    differences in 64 bits, is the gradients' product with it."""
    M, N, K, dt = 60, 200, 136, torch.float16
    X, W, t = xent_inputs(M, N, K, dt, 41)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dg.gemm_xent_bwd(X, W, t, lse, torch.ones((M,), device=DEV), dX=dX, dW=dW)
    vx, vw = dX.double(), dW.double()   # along the gradient: no cancellation

    def total(h):
        return float(xent_ref(X.double() + h * vx, W.double() + h * vw, t, IGN)[2].sum())

    h = 1e-5
    slope = (total(h) - total(-h)) / (2 * h)
    along = float((vx * vx).sum() + (vw * vw).sum())
    assert abs(slope - along) <= 2 * torch.finfo(dt).eps * along

    Wg, Wu = (randn((N, K), K ** -0.5, dt, gen(s)).to(DEV) for s in (1, 2))
    H, G, U = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(3))
    R = randn((M, N), 1.0, dt, gen(3)).to(DEV)
    dg.gemm_gated(X, Wg, Wu, H, G=G, U=U)
    gs = [torch.empty_like(q) for q in (X, Wg, Wu)]
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, R, *gs)
    v = [q.double() for q in gs]

    def total2(h):
        a, b, c = (q.double() + h * d for q, d in zip((X, Wg, Wu), v))
        return float((gated_ref(a, b, c, "silu")[2] * R.double()).sum())

    h = 1e-6
    slope = (total2(h) - total2(-h)) / (2 * h)
    along = sum(float((d * d).sum()) for d in v)
    assert abs(slope - along) <= 4 * torch.finfo(dt).eps * along


def everything(M=200, N=2777, K=136, dt=torch.bfloat16, seed=0):
    """One call of each operator; returns (function, outputs)."""
    X, Wg, Wu = gated_inputs(M, N, K, dt, seed)
    r = gen(seed + 1)
    H, G, U = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(3))
    dH = randn((M, N), 1.0, dt, r).to(DEV)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    X4, Wq, s, z = w4_inputs(5, N, K, 32, dt, True, seed)
    C = torch.empty((5, N), dtype=dt, device=DEV)
    C1 = torch.empty((3, N), dtype=dt, device=DEV)
    Xx, W, t = xent_inputs(M, N, K, dt, seed)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dloss = torch.rand((M,), generator=r).to(DEV)
    dXx, dW = torch.empty_like(Xx), torch.empty_like(W)
    size = max(dg.gated_workspace_bytes(X, Wg, Wu), dg.gated_bwd_workspace_bytes(X, Wg, Wu),
               dg.xent_workspace_bytes(Xx, W), dg.xent_bwd_workspace_bytes(Xx, W))
    ws = torch.empty((size,), dtype=torch.uint8, device=DEV)

    def call(stream=None, ws=ws):
        dg.gemm_gated(X, Wg, Wu, H, G=G, U=U, workspace=ws, stream=stream)
        dg.gemm_gated(X[:3], Wg, Wu, C1, workspace=ws, stream=stream)
        dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX, dWg, dWu, workspace=ws, stream=stream)
        dg.gemm_w4(X4, Wq, s, C, group=32, zeros=z, stream=stream)
        dg.gemm_xent(Xx, W, t, loss, lse, workspace=ws, stream=stream)
        dg.gemm_xent_bwd(Xx, W, t, lse, dloss, dXx, dW, workspace=ws, stream=stream)

    return call, [H, G, U, C1, dX, dWg, dWu, C, loss, lse, dXx, dW], (X, Wg, Wu, X4, Xx, W, dH)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_captured_and_replayed(dt):
    """Two graphs with workspaces of their own, replayed in turn on new inputs
    with eager calls between, give the eager results bit for bit."""
    sides = [everything(dt=dt, seed=50), everything(180, 129, 200, dt, 60)]
    graphs = []
    for call, _, _ in sides:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for turn in range(3):
        wants = []
        for call, outs, ins in sides:
            for q in ins:
                q.mul_(-1.0 if turn % 2 else 0.5)
            call()
            torch.cuda.synchronize()
            wants.append([o.clone() for o in outs])
            for o in outs:
                o.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for want, (_, outs, _) in zip(wants, sides):
            for a, b in zip(want, outs):
                assert torch.equal(a, b)


def test_streams_and_repeats():
    """On a side stream, given or current, and again: the same bits."""
    call, outs, _ = everything(seed=70)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ws=None)      # workspaces from the graph's own pool
    first = [o.clone() for o in outs]
    for _ in range(3):
        for o in outs:
            o.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    for how in range(3):
        for o in outs:
            o.fill_(3)
        s.wait_stream(torch.cuda.current_stream())
        if how == 0:
            call(stream=s, ws=None)
        else:
            with torch.cuda.stream(s):
                call(ws=None)
        s.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_two_threads_at_once():
    import threading

    sides = [everything(seed=80), everything(120, 257, 144, torch.float16, 90)]
    wants = []
    for call, outs, _ in sides:
        call()
        torch.cuda.synchronize()
        wants.append([o.clone() for o in outs])
    errors = []

    def work(call):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                call(stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in sides]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for want, (_, outs, _) in zip(wants, sides):
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(200, 333, 136), (430, 2751, 1024), (926, 2749, 128),
                                   (65, 4098, 200), (300, 5004, 72), (129, 255, 65),
                                   (40000, 3715, 128)])
def test_what_a_workspace_holds(M, N, K, typ):
    """Nothing of a workspace is read before it is written: NaN everywhere in
    it (all bits set, in 16 and in 32 bits) gives the bits that zeros give."""
    dt = DT[typ]
    X, Wg, Wu = gated_inputs(M, N, K, dt, M)
    H, G, U = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(3))
    dH = randn((M, N), 1.0, dt, gen(1)).to(DEV)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    t = torch.randint(0, N, (M,), generator=gen(2)).to(DEV)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dloss = torch.rand((M,), generator=gen(3)).to(DEV)
    ops = [
        (lambda ws: dg.gemm_gated(X, Wg, Wu, H, G=G, U=U, workspace=ws),
         dg.gated_workspace_bytes(X, Wg, Wu), (H, G, U)),
        (lambda ws: dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX, dWg, dWu, workspace=ws),
         dg.gated_bwd_workspace_bytes(X, Wg, Wu), (dX, dWg, dWu)),
        (lambda ws: dg.gemm_xent(X, Wg, t, loss, lse, workspace=ws),
         dg.xent_workspace_bytes(X, Wg), (loss, lse)),
        (lambda ws: dg.gemm_xent_bwd(X, Wg, t, lse, dloss, dX, dWg, workspace=ws),
         dg.xent_bwd_workspace_bytes(X, Wg), (dX, dWg)),
    ]
    for i, (op, size, outs) in enumerate(ops):
        results = []
        for fill in (0, 255):
            ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
            op(ws)
            results.append([o.clone() for o in outs])
        for a, b in zip(*results):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), (i, M, N, K)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(256, 512, 128), (200, 333, 136), (70, 1345, 200)])
def test_some_gradients_captured(M, N, K, typ):
    """Single gradients and pairs: nothing of a workspace full of NaN is read, and
    a graph replayed on new inputs, eager calls between, gives the eager bits."""
    dt = DT[typ]
    X, Wg, Wu = gated_inputs(M, N, K, dt, M)
    G, U, dH = (randn((M, N), 1.0, dt, gen(s)).to(DEV) for s in (1, 2, 3))
    t = torch.randint(0, N, (M,), generator=gen(4)).to(DEV)
    lse = torch.logsumexp(X.double() @ Wg.double().T, 1).float()
    dloss = torch.rand((M,), generator=gen(5)).to(DEV)
    dX, dWg, dWu, dX2, dW2 = (torch.empty_like(q) for q in (X, Wg, Wu, X, Wg))
    names = dict(dX=dX, dWg=dWg, dWu=dWu)
    calls = []
    for want in ("dX", "dWg", "dWu", "dWg dWu", "dX dWu"):
        kw = {k: names[k] for k in want.split()}
        size = dg.gated_bwd_workspace_bytes(X, Wg, Wu, "dX" in kw, "dWg" in kw or "dWu" in kw)
        calls.append((lambda ws, kw=kw: dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, workspace=ws, **kw),
                      size, list(kw.values())))
    for kw in (dict(dX=dX2), dict(dW=dW2)):
        size = dg.xent_bwd_workspace_bytes(X, Wg, "dX" in kw, "dW" in kw)
        calls.append((lambda ws, kw=kw: dg.gemm_xent_bwd(X, Wg, t, lse, dloss, workspace=ws, **kw),
                      size, list(kw.values())))
    for i, (call, size, outs) in enumerate(calls):
        show("some gradients", M, N, K, typ, i)
        results = []
        for fill in (0, 255):
            ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
            call(ws)
            results.append([o.clone() for o in outs])
        for a, b in zip(*results):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), i
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(ws)
        for turn in range(3):
            dH.mul_(-1.0 if turn % 2 else 0.5)
            dloss.mul_(0.5)
            call(torch.empty_like(ws))
            torch.cuda.synchronize()
            want = [o.clone() for o in outs]
            for o in outs:
                o.fill_(7)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, outs):
                assert torch.equal(a, b), (i, turn)
        dH.mul_(-4.0)
        dloss.mul_(8.0)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 8), (0, 1), (2, 2)])
@pytest.mark.parametrize("M,N,K", [(7, 61, 200), (150, 333, 152), (200, 2700, 139)])
def test_strides_of_both_types(M, N, K, pad, shift, typ):
    """Every operator with rows further apart than their length or at 2-byte
    addresses, NaN (255 in bytes) between them."""
    dt = DT[typ]
    show("strides", M, N, K, pad, shift, typ)
    X, Wg, Wu = gated_inputs(M, N, K, dt, 5, pad, shift)
    H, G, U = (Out(M, N, dt, pad, shift) for _ in range(3))
    dg.gemm_gated(X, Wg, Wu, H.t, G=G.t, U=U.t)
    g, u, h, sg, su = gated_ref(X, Wg, Wu, "silu")
    for o, ref, tol in zip((G, U, H), (g, u, h), gated_tols(g, u, h, sg, su, "silu", K, dt)):
        close(o.t, ref, tol, "gated")
        o.check_frame("gated")
    dH = place(randn((M, N), 1.0, dt, gen(6)), pad, shift)
    outs = [Out(r, K, dt, pad, shift) for r in (M, N, N)]
    dg.gemm_gated_bwd(X, Wg, Wu, G.t, U.t, dH, *[o.t for o in outs])
    for o, (ref, tol) in zip(outs, gated_bwd_ref(X, Wg, Wu, G.t, U.t, dH, "silu", dt)):
        close(o.t, ref, tol, "gated_bwd")
        o.check_frame("gated_bwd")
    for group in (32, 64, 128, 96):
        X4, Wq, s, z = w4_inputs(M, N, K, group, dt, True, 7, pad, shift)
        C = Out(M, N, dt, pad, shift)
        dg.gemm_w4(X4, Wq, s, C.t, group=group, zeros=z)
        w4_check(C.t, X4, Wq, s, z, group)
        C.check_frame("w4")
    X, W, t = xent_inputs(M, N, K, dt, 8, pad, shift)
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dg.gemm_xent(X, W, t, loss, lse)
    z, rl, ro = xent_ref(X, W, t, IGN)
    close(loss, ro, 2 * xent_tol(X, W, z, rl), "loss")
    dX, dW = Out(M, K, dt, pad, shift), Out(N, K, dt, pad, shift)
    dloss = torch.rand((M,), generator=gen(9)).to(DEV)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX=dX.t, dW=dW.t)
    xent_bwd_check(X, W, t, lse, dloss, dX.t, dW.t)
    dX.check_frame("dX")
    dW.check_frame("dW")


# ---------------------------------------------------------------- past 2^31 elements

def big(shape, sd, dt, seed):
    """Random values made on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dt, device=DEV).normal_(0.0, sd, generator=g)


def some(n, k=97):
    """Indices of n: the first, the last, those around element 2^31, and some between."""
    at = {0, 1, n - 2, n - 1, *range(0, n, max(1, n // k))}
    return torch.tensor(sorted(i for i in at if 0 <= i < n), device=DEV)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (3, 530000, 4100),        # few rows: weights
    (200, 530000, 4104),      # tiles, operands in place: weights
    (130, 1100000, 2001),     # tiles, padded copies of both weights
    (70000, 32000, 136),      # the outputs
    (2100000, 130, 1040)])    # X
def test_gated_past_two_gibi_elements(M, N, K, typ):
    dt = DT[typ]
    X, Wg, Wu = big((M, K), 1.0, dt, 1), big((N, K), K ** -0.5, dt, 2), big((N, K), K ** -0.5, dt, 3)
    H, G, U = (torch.full((M, N), 7.0, dtype=dt, device=DEV) for _ in range(3))
    show("gated large", M, N, K, typ)
    dg.gemm_gated(X, Wg, Wu, H, G=G, U=U)
    m, n = some(M), some(N)
    g, u, h, sg, su = gated_ref(X[m], Wg[n], Wu[n], "silu")
    tg, tu, th = gated_tols(g, u, h, sg, su, "silu", K, dt)
    at = (m[:, None], n[None, :])
    close(G[at], g, tg, "G")
    close(U[at], u, tu, "U")
    close(H[at], h, th, "H")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(70000, 32000, 136), (200, 530000, 4104)])
def test_gated_bwd_past_two_gibi_elements(M, N, K, typ):
    dt = DT[typ]
    X, Wg, Wu = big((M, K), 1.0, dt, 1), big((N, K), N ** -0.5, dt, 2), big((N, K), N ** -0.5, dt, 3)
    G, U, dH = big((M, N), 1.0, dt, 4), big((M, N), 1.0, dt, 5), big((M, N), M ** -0.5, dt, 6)
    dX, dWg, dWu = (torch.full_like(q, 7.0) for q in (X, Wg, Wu))
    show("gated_bwd large", M, N, K, typ)
    dg.gemm_gated_bwd(X, Wg, Wu, G, U, dH, dX, dWg, dWu)
    m, n, eps = some(M, 40), some(N, 40), torch.finfo(dt).eps
    at = gated_bwd_ref(X[m], Wg, Wu, G[m], U[m], dH[m], "silu", dt)[0]
    norm_close(dX[m], at[0], eps, "dX")
    refs = gated_bwd_ref(X, Wg[n], Wu[n], *(q[:, n] for q in (G, U, dH)), "silu", dt)
    for got, (ref, _), what in zip((dWg[n], dWu[n]), refs[1:], ("dWg", "dWu")):
        norm_close(got, ref, eps, what)
        rows = (got.double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(rows.max()) <= 2 * eps, (what, int(rows.argmax()))


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 300000, 16384), (20, 300000, 16400), (34000, 66000, 64)])
def test_w4_past_two_gibi_elements(M, N, K, typ):
    """The packed weights, and the output."""
    dt, group = DT[typ], 64
    g = torch.Generator(device=DEV).manual_seed(5)
    X = big((M, K), 1.0, dt, 1)
    Wq = torch.randint(0, 256, (N, K // 2), device=DEV, dtype=torch.uint8, generator=g)
    s = (torch.rand((N, -(-K // group)), device=DEV, generator=g) + 0.5).to(dt)
    z = torch.randint(0, 16, s.shape, device=DEV, dtype=torch.uint8, generator=g)
    C = torch.full((M, N), 7.0, dtype=dt, device=DEV)
    show("w4 large", M, N, K, typ)
    dg.gemm_w4(X, Wq, s, C, group=group, zeros=z)
    m, n = some(M), some(N)
    got = C[m[:, None], n[None, :]]
    w4_check(got, X[m], Wq[n], s[n], z[n], group)
    w4_norm_close(got, X[m], *w4_weights(Wq[n], s[n], z[n], group, K), "C")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(150, 530000, 4104), (2100000, 257, 1032)])
def test_xent_past_two_gibi_elements(M, N, K, typ):
    """The vocabulary matrix and its gradient; X and its gradient."""
    dt = DT[typ]
    X, W = big((M, K), 1.0, dt, 1), big((N, K), 2.0 * K ** -0.5, dt, 2)
    t = torch.randint(0, N, (M,), generator=gen(3)).to(DEV)
    t[::7], t[-1] = IGN, N - 1
    loss, lse = torch.empty((M,), device=DEV), torch.empty((M,), device=DEV)
    dX, dW = torch.full_like(X, 7.0), torch.full_like(W, 7.0)
    dloss = torch.rand((M,), generator=gen(4)).to(DEV) + 0.5
    show("xent large", M, N, K, typ)
    dg.gemm_xent(X, W, t, loss, lse)
    dg.gemm_xent_bwd(X, W, t, lse, dloss, dX, dW)
    m, eps = some(M, 40), torch.finfo(dt).eps
    for i in m.split(8):   # rows of logits in 64 bits
        z, a, b = xent_ref(X[i], W, t[i], IGN)
        tol = xent_tol(X[i], W, z, a)
        close(lse[i], a, tol, "lse")
        close(loss[i], b, 2 * tol, "loss")
        p = torch.exp(z - a[:, None])
        live = t[i] != IGN
        p[torch.arange(len(i), device=DEV)[live], t[i][live]] -= 1
        p *= (live * dloss[i].double())[:, None]
        norm_close(dX[i], p @ W.double(), eps, "dX")
        assert bool((dX[i][~live] == 0).all())
    # columns of the logits for the rows of dW
    n = some(N, 40)
    p = torch.exp(X.double() @ W[n].double().T - lse.double()[:, None])
    p -= (t[:, None] == n[None, :]).double()
    p *= ((t != IGN) * dloss.double())[:, None]
    norm_close(dW[n], p.T @ X.double(), eps, "dW")
