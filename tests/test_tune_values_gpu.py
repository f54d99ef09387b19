"""The operators of fine tuning on values at the ends of their types' ranges, held
to fixed bounds."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_sgemm_amd as dg  # noqa: E402
from fused_ref import DT, close, randn  # noqa: E402
from test_tune_gpu import ALL, DEV, TYPES, gen, lora_inputs, ortho_input, show  # noqa: E402
from tune_ref import MUON, lora_bwd_ref, lora_ref, lora_result, ortho_ref  # noqa: E402

pytestmark = pytest.mark.gpu


# N: whole slabs of 64, whole 16-byte rows, neither; few rows and tiles of every
# shape; an infinity in the last slab, in what its copies read twice, and before
@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(40, 328, 136), (1500, 328, 264), (1500, 320, 264),
                                   (1500, 333, 264), (2304, 264, 2304), (1300, 200, 200)])
def test_infinite_weights(M, N, K, typ):
    """An infinity in W is one in the columns of dX and of the result that it
    belongs to, with the sign of what it is multiplied with, and reaches no other."""
    dt, inf, R, S = DT[typ], float("inf"), 8, 2
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, M + N)
    dC = randn((M, N), 0.1, dt, gen(M)).to(DEV)
    T = lora_ref(X, W, A, B, ids)[1].float()
    dX, dA, dB = torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)
    (ref, tol), _, _ = lora_bwd_ref(X, W, A, B, ids, T, dC, scales)
    at = sorted({N - 1, N - 63, N - 64, N // 64 * 64 - 1, N // 64 * 64 - 5, 3})
    W1, want = W.clone(), ref.clone()
    for i, n in enumerate(at):
        sign = -1.0 if i % 2 else 1.0
        W1[n, 7 * i + 1] = sign * inf
        want[:, 7 * i + 1] = sign * torch.sign(dC[:, n].double()) * inf
    show("infinite weights", M, N, K, typ, at)
    assert bool((dC[:, at] != 0).all())
    dg.gemm_lora_bwd(X, W1, A, B, ids, T, dC, dX, dA, dB, scales=scales)
    close(dX, want, tol, "dX")
    y, _, off, _ = lora_ref(X, W, A, B, ids, scales)
    want, tol = lora_result(y, off, dt)
    W1, C = W.clone(), torch.empty_like(dC)
    for i, k in enumerate(sorted({K - 1, K - 8, K - 63, K - 64, K // 64 * 64 - 1, 3})):
        W1[7 * i + 1, k] = inf
        assert bool((X[:, k] != 0).all())
        want[:, 7 * i + 1] = torch.sign(X[:, k].double()) * inf
    dg.gemm_lora(X, W1, A, B, ids, C, scales=scales)
    close(C, want, tol, "C")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(1500, 328, 264), (1500, 333, 264)])
def test_infinite_gradients(M, N, K, typ):
    """One in dC is one throughout its row of dX and in no other row."""
    dt, inf, R, S = DT[typ], float("inf"), 8, 2
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, M + N + 1)
    W[W == 0] = 1.0
    dC = randn((M, N), 0.1, dt, gen(M)).to(DEV)
    ids[:] = -1
    T = torch.zeros((M, R), device=DEV)
    (want, tol), _, _ = lora_bwd_ref(X, W, A, B, ids, T, dC, scales)
    dX = torch.empty_like(X)
    for m, n in enumerate(sorted({N - 1, N - 63, N - 64, N // 64 * 64 - 1, 3})):
        dC[m, n] = inf
        want[m] = torch.sign(W[n].double()) * inf
    show("infinite gradients", M, N, K, typ)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX, scales=scales)
    close(dX, want, tol, "dX")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(24, 96, 64), (500, 5000, 128)])
def test_small_values_beside_large_ones(M, N, K, typ):
    """What a rank adds is its own, however small it is beside the other ranks of its
    block: an infinity that it meets is one, and without the large one it is there to
    the last bits (fp16 holds values down to 2^-37 of the largest, bf16 all of them)."""
    dt, inf, R, S = DT[typ], float("inf"), 4, 1
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 5, "one")
    ids[0] = -1
    W[:] = 0
    scales[:] = 1.0
    X[:, 0], X[:, 1] = 1.0, 2.0 ** -14
    A[:] = 0
    A[0, 0, 0] = 8192.0                                  # t: 2^13,
    A[0, 1, 0], A[0, 1, 1] = 2.0 ** -9, 2.0 ** -16       # 2^-9 + 2^-30,
    A[0, 2, 0] = -2.0 ** -24                             # -2^-24,
    A[0, 3, 1] = 2.0 ** -20                              # 2^-34
    B[:] = 0
    B[0, 5, 1], B[0, 6, 2], B[0, 7, 3] = inf, inf, -inf
    B[0, 8, 1], B[0, 9, 2] = 512.0, 4096.0
    C, T = torch.empty((M, N), dtype=dt, device=DEV), torch.empty((M, R), device=DEV)
    show("small beside large", M, N, K, typ)
    dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
    want = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    want[1:, 5], want[1:, 6], want[1:, 7] = inf, -inf, -inf
    want[1:, 8], want[1:, 9] = 1.0 + 2.0 ** -21, -2.0 ** -12
    # the second product's values: 2^-37 of the largest, 2^13, times B
    tol = torch.zeros_like(want)
    tol[:, 8], tol[:, 9] = 512.0 * 2.0 ** -24, 4096.0 * 2.0 ** -24
    close(C, want, tol + torch.finfo(dt).eps / 2 * want.abs().clamp(max=2.0), "C")
    # gradients: dt = dC B and T of all rows of an adapter are scaled together
    d = torch.zeros((M, N), dtype=dt, device=DEV)
    B[:] = 0
    B[0, 0, 0], B[0, 1, 1], B[0, 2, 2], B[0, 3, 3] = 8192.0, 2.0 ** -9, -2.0 ** -24, 2.0 ** -14
    B[0, 4, 1], B[0, 5, 3] = 2.0 ** -14, 2.0 ** -14
    d[:, :4] = 1.0
    d[:, 4], d[:, 3], d[:, 5] = 2.0 ** -16, 2.0 ** -14, 2.0 ** -14
    X[:, 2:] = 0
    X[1, 2], X[2, 3] = inf, 0.0
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, d, None, dA, dB, scales=scales)
    assert dA[0, :, 2].tolist() == [inf, inf, -inf, inf]
    assert bool((dA[0, :, 3:] == 0).all())
    d[1, 11], d[1, 12] = inf, -inf
    dg.gemm_lora_bwd(X, W, A, B, ids, T, d, None, None, dB, scales=scales)
    assert dB[0, 11].tolist() == [inf, inf, -inf, inf] and dB[0, 12].tolist() == [-inf, -inf, inf, -inf]
    # (sums of 2^13 over the rows are past binary16's largest value, and no other one is)
    rest = (d[1:, :11].double().T @ T[1:].double()).to(dt)
    assert torch.equal(torch.isinf(dB[0, :11]), torch.isinf(rest))
    assert not bool(torch.isnan(dB[0, :11]).any()) and bool((dB[0, 13:] == 0).all())


@pytest.mark.parametrize("M,S", [(300, 1 << 20), (5000, 40000), (3000, 2049), (2, 1 << 22)])
def test_a_million_adapters(M, S):
    """Gradients of as many adapters as fit take the time of writing them."""
    dt, N, K, R = torch.bfloat16, 8, 16, 1
    g = gen(S)
    X, dC = randn((M, K), 1.0, dt, g).to(DEV), randn((M, N), 1.0, dt, g).to(DEV)
    W = randn((N, K), 1.0, dt, g).to(DEV)
    B = torch.ones((S, N, R), dtype=dt, device=DEV)
    A = torch.ones((S, R, K), dtype=dt, device=DEV)
    ids = torch.randint(-1, S, (M,), generator=g)
    ids[M // 3:M // 2] = S - 1                 # more than one step of 32 rows
    ids[0] = 0
    ids = ids.to(DEV)
    T = torch.rand((M, R), generator=g).to(DEV)
    dA, dB = torch.full_like(A, 3.0), torch.full_like(B, 3.0)
    show("many adapters", M, S)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, None, dA, dB)
    at, have = ids.clamp(min=0), (ids >= 0).double()[:, None]
    x, d = X.double(), dC.double() * have
    dt64 = d.sum(1, keepdim=True)
    each = lambda v: torch.zeros((S, v.shape[1]), dtype=torch.float64, device=DEV).index_add_(0, at, v)
    # (one step of bf16 for the result, and t's two values of 2^-15 each)
    wantA, sizeA = each(dt64 * x), each(dt64.abs() * x.abs())
    wantB, sizeB = each(d * T.double()), each(d.abs() * T.double())
    most = float(d.abs().sum(1).max())
    close(dA[:, 0], wantA, 2.0 ** -8 * wantA.abs() + 2.0 ** -14 * (sizeA + most * each(x.abs() * have)),
          "dA")
    close(dB[:, :, 0], wantB, 2.0 ** -8 * wantB.abs() + 2.0 ** -14 * each(d.abs()), "dB")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(33, 100, 264, 12, 4), (900, 520, 200, 16, 3)])
def test_gradients_without_what_they_do_not_read(M, N, K, R, S, typ):
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 18)
    dC, T = randn((M, N), 0.1, dt, gen(19)).to(DEV), lora_ref(X, W, A, B, ids)[1].float()
    dX, dA, dB = (torch.empty_like(v) for v in (X, A, B))
    eX, eA, eB = (torch.full_like(v, 9.0) for v in (X, A, B))
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX, dA, dB, scales=scales)
    show("gradients alone", M, N, K, R, S, typ)
    dg.gemm_lora_bwd(None, W, A, B, ids, None, dC, dX=eX, scales=scales)
    dg.gemm_lora_bwd(X, None, None, B, ids, None, dC, dA=eA, scales=scales)
    dg.gemm_lora_bwd(None, None, A, None, ids, T, dC, dB=eB, scales=scales)
    assert torch.equal(dX, eX) and torch.equal(dA, eA) and torch.equal(dB, eB)


# ---------------------------------------------------------------- updates

# each form: one launch a step, short tiles, the tile kernel (its ranges of K, a tall one)
FORMS = [(2, 24, 500), (2, 500, 40), (3, 140, 200), (2, 500, 150), (1, 1100, 1160), (2, 1300, 1100),
         (1, 1030, 5000)]
# the documented distance from the formula in the 2-norm, with a factor of 2 for
# "about", and half a step of the output's type, root of its squares' sum: an error of
# rounding is anywhere within it, so over many values half a step / sqrt(3) and more
# only where they crowd at one end of a power of two
FINE, BF16 = 2.0 ** -18, 2 * 0.0012


def bound(dtype, L, m, n):
    low, size = min(m, n), L * m * n
    two = low <= 64 or (low <= 1024 and (1.5 if low > 512 else 1) * size <= 2.5 * 2 ** 20)
    return (FINE if two or dtype != torch.bfloat16 else BF16) + torch.finfo(dtype).eps / 2


def ortho_off(O, ref):
    """Matrix by matrix, what is under binary16's normal range aside."""
    least = 2.0 ** -25 * ref[0].numel() ** 0.5 if O.dtype == torch.float16 else 0.0
    return ((O.double() - ref).flatten(1).norm(dim=1) - least) / ref.flatten(1).norm(dim=1)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,m,n", FORMS)
def test_ortho_far_below_eps(L, m, n, out):
    """A norm far below eps: the update is in proportion to it, and as near to the
    formula as any other."""
    G = ortho_input(L, m, n, "f32", 90)
    O = torch.empty(G.shape, dtype=ALL[out], device=DEV)
    norm = float(G.double().flatten(1).norm(dim=1).max())
    for ratio in (0.7, 0.1, 1e-2, 1e-4, 1e-6, 1e-9, 1e-20, 1e-30):
        eps = 1e-7 if ratio > 1e-9 else 1e3
        H = G * (ratio * eps / norm)
        for steps, coeffs in ((5, MUON), (1, MUON), (9, (1.5, -0.5, 0.0)), (3, (0.75, 0.5, 0.25))):
            show("below eps", L, m, n, out, ratio, steps)
            dg.gemm_ortho(H, O, steps=steps, coeffs=coeffs, eps=eps)
            off = ortho_off(O, ortho_ref(H, steps, coeffs, eps))
            assert float(off.max()) <= bound(ALL[out], L, m, n), (ratio, steps, off.tolist())


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,m,n", FORMS + [(1, 2048, 2048)])
def test_ortho_as_documented(L, m, n, out):
    """The documented distances from the formula: for noise, and, less well, for singular
    values spread evenly over a factor of 300 and for a few directions a hundred times
    the rest in the Frobenius norm, whose singular values are a thousand times the
    rest's.  A value held in two is off by 2^-23 of its size, so an iterate of norm 1 by
    2^-23 in the norm; what the step then adds to that by rounding C (a = 3.4 on its
    diagonal, and a gain of 3.4 for what is small: as much again), A (b / a = 1.4) and
    A^2 (c A / a, 1.2 at most) makes 4.6 of it.  The rest, of norm 0.01, gains as much
    as that error, and 3.4 a step, so that the iterates' errors add up to 1.42 of the
    first one's: 100 * 4.6 * 1.42 * 2^-23 = 7.8e-5 of the result, under 100 * 2^-20.
    Singular values spread evenly: the error of the norm 2^-23 gains as the directions
    do, in the root of their gains' mean square, which over the result's norm is
    158 / 4.6 for 24 of them and 323 / 37 for 2048."""
    O = torch.empty((L, m, n), dtype=ALL[out], device=DEV)
    g = gen(91)
    k = min(m, n)
    q, r = (torch.linalg.qr(torch.randn((L, v, k), generator=g).double().to(DEV))[0] for v in (m, n))
    values = torch.logspace(0, -2.477, k, dtype=torch.float64)
    first = last = values / values.norm()
    for _ in range(5):
        last = MUON[0] * last + MUON[1] * last ** 3 + MUON[2] * last ** 5
    gain = float((last / first).square().mean().sqrt() / last.norm())
    more = {"noise": 0.0, "strong": 100 * 2.0 ** -20, "spread": 4.6 * 1.42 * 2.0 ** -23 * gain}
    spread = (q * torch.logspace(0, -2.477, k, dtype=torch.float64, device=DEV)) @ r.mT.contiguous()
    for source in ("f32", "bf16"):
        for name, G in (("noise", ortho_input(L, m, n, source, 92)),
                        ("strong", ortho_input(L, m, n, source, 93, 100.0 / min(4, k) ** 0.5)),
                        ("spread", spread.to(ALL[source]))):
            show("as documented", L, m, n, source, out, name)
            dg.gemm_ortho(G, O)
            off = ortho_off(O, ortho_ref(G))
            show("  off", [("%.2e" % v) for v in off.tolist()])
            most = bound(ALL[out], L, m, n) + more[name]
            assert float(off.max()) <= most, (name, source, off.tolist())


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("L,m,n", FORMS)
def test_ortho_below_eps_and_growing(L, m, n, out):
    """One direction, smaller than 1 by eps, and coefficients by which it grows faster
    than small values do, or keeps its size while they shrink: 1 + 3 x^2 takes 0.3 to
    4.3 in four steps, 1 + 30 x^2 takes 0.05 to 3.24 in ten, 0.75 + 0.5 x^2 + 0.25 x^4 is
    1 at 0.6436.  An error grows with it, by 14 and 47 (relative to it), and by 1.58 a
    step, 61 in nine."""
    g = gen(94)
    u, v = (torch.randn((L, s, 1), generator=g).double().to(DEV) for s in (m, n))
    G = ((u / u.norm(dim=1, keepdim=True)) @ (v / v.norm(dim=1, keepdim=True)).mT).float()
    G *= 0.99                                  # (so that it is stored as it is)
    O = torch.empty(G.shape, dtype=ALL[out], device=DEV)
    for size, steps, coeffs, more in ((0.3, 4, (1.0, 3.0, 0.0), 14), (0.1, 6, (1.0, 3.0, 0.0), 2),
                                      (0.6436, 9, (0.75, 0.5, 0.25), 61), (0.05, 30, (1.0, 0.9, 0.0), 2),
                                      (0.05, 11, ((1.0, 30.0, 0.0),) * 10 + ((0.5, 0.0, 0.0),), 47),
                                      (0.03, 3, (0.0, 4.0, 0.0), 0)):
        eps = 0.99 / size - 0.99
        show("growing", L, m, n, out, size, steps)
        dg.gemm_ortho(G, O, steps=steps, coeffs=coeffs, eps=eps)
        ref = ortho_ref(G, steps, coeffs, eps)
        off = ortho_off(O, ref)
        assert bool(torch.isfinite(O).all()) and float(ref.abs().max()) > 0
        if more:
            most = more * (bound(ALL[out], L, m, n) - torch.finfo(O.dtype).eps / 2)
            assert float(off.max()) <= most + torch.finfo(O.dtype).eps / 2, (size, off.tolist())
