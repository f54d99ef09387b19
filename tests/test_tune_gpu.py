"""The operators of fine tuning (adapters, their gradients, orthogonalised
updates) against their definitions in 64 bits on the GPU's host."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_sgemm_amd as dg  # noqa: E402
from fused_ref import DT, Out, close, place, randn, sum_error  # noqa: E402
from tune_ref import (MUON, lora_bwd_ref, lora_ref, lora_result, ortho_check, ortho_ref)  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]
ALL = {"f32": torch.float32, **DT}
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def show(*a):
    print(*a, flush=True)


def place3(t, pad=0, shift=0, gap=0):
    """A stack whose rows lie ``pad`` elements further apart than needed, whose
    matrices ``gap`` rows, ``shift`` into its storage, NaN between."""
    S, r, c = t.shape
    ld = c + pad
    buf = torch.full((shift + S * (r + gap) * ld + 8,), float("nan"), dtype=t.dtype, device=DEV)
    v = torch.as_strided(buf, (S, r, c), ((r + gap) * ld, ld, 1), shift)
    v.copy_(t)
    return v


class Out3:
    """An output stack inside a sentinel-filled buffer."""

    def __init__(self, S, r, c, dtype, pad=0, shift=0, gap=0):
        ld = c + pad
        self.buf = torch.full((shift + S * (r + gap) * ld + 8,), 777.0, dtype=dtype, device=DEV)
        self.t = torch.as_strided(self.buf, (S, r, c), ((r + gap) * ld, ld, 1), shift)

    def check_frame(self, what):
        rest = self.buf.clone()
        torch.as_strided(rest, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(777.0)
        assert bool((rest == 777.0).all()), what + ": wrote outside its matrices"


# ---------------------------------------------------------------- adapters

def lora_inputs(M, N, K, R, S, dt, seed=0, order="any", pad=0, shift=0, gap=0):
    g = gen(seed)
    X = place(randn((M, K), 1.0, dt, g), pad, shift)
    W = place(randn((N, K), K ** -0.5, dt, g), pad, shift)
    A = place3(randn((S, R, K), K ** -0.5, dt, g), pad, shift, gap)
    B = place3(randn((S, N, R), R ** -0.5, dt, g), pad, shift, gap)
    ids = torch.randint(-1, S, (M,), generator=g)
    if order == "sorted":
        ids = ids.sort().values
    elif order == "one":
        ids = torch.full((M,), S - 1)
    return X, W, A, B, ids.to(DEV), (torch.rand((S,), generator=g) + 0.5).to(DEV)


# one row to many tiles, ranks off every multiple, one adapter to one a row
LORA = [(1, 16, 32, 4, 1), (1, 1, 1, 1, 1), (1, 4096, 512, 16, 3), (3, 100, 8, 8, 70),
        (5, 70, 96, 12, 4), (16, 130, 65, 5, 16), (17, 130, 65, 17, 5), (33, 64, 264, 16, 9),
        (48, 513, 1030, 32, 64), (64, 513, 72, 33, 64), (65, 129, 127, 8, 3), (100, 64, 130, 64, 2),
        (129, 5001, 320, 7, 7), (300, 500, 264, 100, 4), (257, 4096, 72, 16, 1), (500, 2800, 200, 24, 9),
        (700, 4333, 1537, 16, 6), (2000, 400, 136, 8, 5), (1100, 3000, 328, 128, 3),
        (1500, 2304, 136, 48, 40), (2304, 2304, 192, 16, 2), (4100, 4104, 72, 20, 3),
        (20, 90, 64, 1024, 2), (600, 2600, 136, 200, 2)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", LORA)
def test_lora(M, N, K, R, S, typ):
    dt = DT[typ]
    order = ("any", "sorted", "one")[(M + R) % 3] if M < 1500 else "sorted"
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, M + N + K, order)
    C, T = Out(M, N, dt), Out(M, R, torch.float32)
    show("lora", M, N, K, R, S, typ, order)
    assert dg.gemm_lora(X, W, A, B, ids, C.t, scales=scales, T=T.t) is C.t
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    close(T.t, t, dt_sum, "T")
    close(C.t, *lora_result(y, off, dt), "C")
    C.check_frame("C")
    T.check_frame("T")
    only = Out(M, N, dt)
    dg.gemm_lora(X, W, A, B, ids, only.t)
    y, _, off, _ = lora_ref(X, W, A, B, ids)
    close(only.t, *lora_result(y, off, dt), "C without scales")


def grads_check(X, W, A, B, ids, T, dC, scales, dX=None, dA=None, dB=None):
    for got, (ref, tol), what in zip((dX, dA, dB), lora_bwd_ref(X, W, A, B, ids, T, dC, scales),
                                     ("dX", "dA", "dB")):
        if got is not None:
            close(got, ref, tol, what)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", LORA)
def test_lora_bwd(M, N, K, R, S, typ):
    dt = DT[typ]
    order = ("one", "any", "sorted")[(M + R) % 3] if M < 1500 else "sorted"
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, M + N + K, order)
    dC = randn((M, N), 0.1, dt, gen(M)).to(DEV)
    T = lora_ref(X, W, A, B, ids)[1].float()
    dX, dA, dB = Out(M, K, dt), Out3(S, R, K, dt), Out3(S, N, R, dt)
    show("lora_bwd", M, N, K, R, S, typ, order)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX.t, dA.t, dB.t, scales=scales)
    grads_check(X, W, A, B, ids, T, dC, scales, dX.t, dA.t, dB.t)
    for o in (dX, dA, dB):
        o.check_frame("lora_bwd")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(7, 61, 200, 6, 3), (150, 333, 152, 24, 4),
                                       (200, 4700, 139, 12, 2), (300, 5000, 200, 16, 3)])
@pytest.mark.parametrize("pad,shift,gap", [(3, 1, 2), (8, 8, 0), (0, 1, 1), (2, 2, 3)])
def test_lora_strides(M, N, K, R, S, pad, shift, gap, typ):
    """Rows further apart than their length, adapters further than their size and
    all at 2-byte addresses, NaN between them."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 3, "any", pad, shift, gap)
    C, T = Out(M, N, dt, pad, shift), Out(M, R, torch.float32, pad, shift)
    show("lora strides", M, N, K, R, S, pad, shift, gap, typ)
    dg.gemm_lora(X, W, A, B, ids, C.t, scales=scales, T=T.t)
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    close(C.t, *lora_result(y, off, dt), "C")
    close(T.t, t, dt_sum, "T")
    dC = place(randn((M, N), 0.1, dt, gen(9)), pad, shift)
    dX, dA, dB = Out(M, K, dt, pad, shift), Out3(S, R, K, dt, pad, shift, gap), \
        Out3(S, N, R, dt, pad, shift, gap)
    dg.gemm_lora_bwd(X, W, A, B, ids, T.t, dC, dX.t, dA.t, dB.t, scales=scales)
    grads_check(X, W, A, B, ids, T.t, dC, scales, dX.t, dA.t, dB.t)
    for o in (C, T, dX, dA, dB):
        o.check_frame("lora strides")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu"])
@pytest.mark.parametrize("M,N,K,R", [(3, 77, 130, 8), (50, 1000, 264, 16), (600, 2500, 136, 12)])
def test_lora_write_back(M, N, K, R, name, typ):
    """Bias, activation, and a residual that is the result itself."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, 3, dt, 4)
    bias = randn((N,), 1.0, dt, gen(5)).to(DEV)
    res = randn((M, N), 1.0, dt, gen(6)).to(DEV)
    C = Out(M, N, dt, 3, 1)
    C.t.copy_(res)
    show("lora write-back", M, N, K, R, name, typ)
    dg.gemm_lora(X, W, A, B, ids, C.t, scales=scales, bias=bias, act=name, residual=C.t)
    y, _, off, _ = lora_ref(X, W, A, B, ids, scales)
    close(C.t, *lora_result(y, off, dt, bias, name, res), "C")
    C.check_frame("C")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(40, 300, 200, 16, 5), (700, 4096, 136, 24, 5)])
def test_lora_order_of_rows(M, N, K, R, S, typ):
    """A row's result does not depend on the rows beside it: another order of
    the rows gives the same bits."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 7, "sorted")
    C, D = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(2))
    T, U = (torch.empty((M, R), device=DEV) for _ in range(2))
    dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
    p = torch.randperm(M, generator=gen(8)).to(DEV)
    dg.gemm_lora(X[p].contiguous(), W, A, B, ids[p].contiguous(), D, scales=scales, T=U)
    assert torch.equal(D, C[p]) and torch.equal(U, T[p])


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(20, 130, 100, 8, 4), (64, 300, 264, 24, 6),
                                       (400, 6000, 136, 16, 4)])
def test_lora_rows_without_and_unknown(M, N, K, R, S, typ):
    """Rows without an adapter are the projection alone, whatever they hold they
    reach no gradient; ids past the last adapter make NaN of their rows only."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 11)
    ids[:] = torch.where(ids == 1, 0, ids)      # adapter 1 has no rows
    ids[0], ids[3], ids[M // 2], ids[5] = -7, -2 ** 40, S, 2 ** 40
    C, T = torch.empty((M, N), dtype=dt, device=DEV), torch.empty((M, R), device=DEV)
    show("lora without", M, N, K, R, S, typ)
    dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    close(C, *lora_result(y, off, dt), "C")
    close(T, t, dt_sum, "T")
    assert torch.isnan(C).any(1).nonzero().flatten().tolist() == sorted({5, M // 2})
    dC = randn((M, N), 0.1, dt, gen(12)).to(DEV)
    dX, dA, dB = torch.empty_like(X), torch.full_like(A, 3.0), torch.full_like(B, 3.0)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX, dA, dB, scales=scales)
    grads_check(X, W, A, B, ids, T, dC, scales, dX, dA, dB)
    assert bool((dA[1] == 0).all()) and bool((dB[1] == 0).all())
    # NaN in rows without an adapter: dA and dB are the same bits
    out = (ids < 0) | (ids >= S)
    Xn, dCn, Tn = X.clone(), dC.clone(), T.clone()
    Xn[out], dCn[out], Tn[out] = float("nan"), float("nan"), float("nan")
    eA, eB = torch.empty_like(A), torch.empty_like(B)
    dg.gemm_lora_bwd(Xn, W, A, B, ids, Tn, dCn, None, eA, eB, scales=scales)
    assert torch.equal(dA, eA) and torch.equal(dB, eB)
    # no row has one
    none = torch.full_like(ids, -1)
    dg.gemm_lora(X, W, A, B, none, C, T=T)
    y, _, off, _ = lora_ref(X, W, A, B, none)
    close(C, *lora_result(y, off, dt), "C without adapters")
    assert bool((T == 0).all())
    dg.gemm_lora_bwd(Xn, W, A, B, none, Tn, dCn, None, dA, dB)
    assert bool((dA == 0).all()) and bool((dB == 0).all())


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("R", [8, 16, 40])
@pytest.mark.parametrize("M,N,K", [(24, 96, 64), (500, 5000, 128)])
def test_lora_not_a_number(M, N, K, R, typ):
    """What one adapter holds, infinities and NaN too, reaches its own rows and
    gradients only; an infinity in it is one there, not a NaN."""
    dt, S, inf = DT[typ], 3, float("inf")
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 13)
    ids[:8] = torch.tensor([0, 1, 2, 1, 0, 2, -1, 1])
    B1, A1 = B.clone(), A.clone()
    B1[1, 5, 3], B1[1, 7, 0], B1[1, N - 1, R - 1] = inf, float("nan"), -inf
    C, T = torch.empty((M, N), dtype=dt, device=DEV), torch.empty((M, R), device=DEV)
    show("lora not a number", M, N, K, R, typ)
    dg.gemm_lora(X, W, A, B1, ids, C, scales=scales, T=T)
    y, t, off, _ = lora_ref(X, W, A, B, ids, scales)
    want, tol = lora_result(y, off, dt)
    own = ids == 1
    want[own, 5] = torch.sign(t[own, 3]) * inf
    want[own, 7] = float("nan")
    want[own, N - 1] = -torch.sign(t[own, R - 1]) * inf
    close(C, want, tol, "C")
    # an infinity in its first factor: t of its rows, and what comes of it
    A1[1, 2, 4] = inf
    dg.gemm_lora(X, W, A1, B, ids, C, scales=scales, T=T)
    want, _ = lora_result(y, off, dt)
    want[own] = torch.sign(X[own, 4].double())[:, None] * torch.sign(B[1, :, 2].double()) * inf
    close(C, want, tol, "C of an infinite t")
    # gradients: an infinite dC and X in rows of adapter 1
    T.copy_(t)
    dC = randn((M, N), 0.1, dt, gen(14)).to(DEV)
    dC1, X1 = dC.clone(), X.clone()
    at = int(own.nonzero()[0, 0])
    X1[at, 6] = inf
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    dg.gemm_lora_bwd(X1, W, A, B, ids, T, dC, None, dA, dB, scales=scales)
    ref = lora_bwd_ref(X, W, A, B, ids, T, dC, scales)
    want = ref[1][0].clone()
    g = (dC[at].double() @ B[1].double())
    want[1, :, 6] = torch.sign(g) * inf
    close(dA, want, ref[1][1], "dA")
    close(dB, *ref[2], "dB")
    dC1[at, 9] = inf
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC1, None, None, dB, scales=scales)
    want = ref[2][0].clone()
    want[1, 9] = torch.sign(t[at]) * inf
    close(dB, want, ref[2][1], "dB of an infinite dC")


@pytest.mark.parametrize("M,N,K,R", [(30, 200, 128, 16), (600, 4096, 128, 20)])
@pytest.mark.parametrize("size", [1e-4, 60.0])
def test_lora_fp16_range(M, N, K, R, size):
    """t far below binary16's normal range and far above its largest value, with
    results inside it; gradients alike."""
    dt, S = torch.float16, 2
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 15)
    X *= size
    A *= 0.02 if size < 1 else 600.0
    B *= 1.0 if size < 1 else 1e-4
    C, T = torch.empty((M, N), dtype=dt, device=DEV), torch.empty((M, R), device=DEV)
    show("lora fp16 range", M, N, K, R, size)
    dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    assert (float(t.abs().max()) < 2.0 ** -14) == (size < 1) and \
        (float(t.abs().max()) > 65504) == (size > 1)
    close(T, t, dt_sum, "T")
    close(C, *lora_result(y, off, dt), "C")
    dC = (randn((M, N), 0.1, dt, gen(16)) * (1e-3 if size < 1 else 1.0)).to(DEV)
    T = t.float()
    dX, dA, dB = torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX, dA, dB, scales=scales)
    ref = lora_bwd_ref(X, W, A, B, ids, T, dC, scales)
    for got, (r, tol), what in zip((dX, dA, dB), ref, ("dX", "dA", "dB")):
        if float(r.abs().max()) < 65504:
            close(got, r, tol, what)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_lora_empty_sums(M):
    dt, N, R, S = torch.bfloat16, 3000, 8, 2
    A, B = torch.empty((S, R, 0), dtype=dt, device=DEV), torch.ones((S, N, R), dtype=dt, device=DEV)
    X, W = (torch.empty((n, 0), dtype=dt, device=DEV) for n in (M, N))
    ids = torch.zeros((M,), dtype=torch.int64, device=DEV)
    C = torch.full((M, N), 5.0, dtype=dt, device=DEV)
    bias = torch.arange(N, device=DEV).to(dt)
    T = torch.full((M, R), 5.0, device=DEV)
    dg.gemm_lora(X, W, A, B, ids, C, bias=bias, T=T)            # K == 0
    assert bool((C == bias).all()) and bool((T == 0).all())
    # no adapters: the projection; N == 0: T alone
    X, W, A, B, _, _ = lora_inputs(M, N, 64, R, S, dt, 17)
    none = torch.empty((0, R, 64), dtype=dt, device=DEV), torch.empty((0, N, R), dtype=dt, device=DEV)
    dg.gemm_lora(X, W, *none, ids - 1, C, T=T)
    want = torch.empty_like(C)
    dg.gemm_lora(X, W, A, B, ids - 1, want)
    assert torch.equal(C, want) and bool((T == 0).all())
    dg.gemm_lora(X, W, *none, ids, C)
    assert bool(torch.isnan(C).all())
    dg.gemm_lora(X, W[:0], A, B[:, :0], ids, C[:, :0], T=T)
    close(T, X.double() @ A[0].double().T, sum_error(64, X.double().abs() @ A[0].double().abs().T), "T")
    # no rows: gradients of zero
    dA, dB = torch.full_like(A, 3.0), torch.full_like(B, 3.0)
    dg.gemm_lora_bwd(X[:0], W, A, B, ids[:0], T[:0], C[:0], X[:0], dA, dB)
    assert bool((dA == 0).all()) and bool((dB == 0).all())
    dg.gemm_lora(X[:0], W, A, B, ids[:0], C[:0])
    # N == 0: dX and dA are empty sums
    dX, dA = torch.full_like(X, 3.0), torch.full_like(A, 3.0)
    dg.gemm_lora_bwd(X, W[:0], A, B[:, :0], ids, T, C[:, :0], dX, dA)
    assert bool((dX == 0).all()) and bool((dA == 0).all())
    # no adapters: dX alone
    dC = torch.ones((M, N), dtype=dt, device=DEV)
    dg.gemm_lora_bwd(X, W, *none, ids - 1, T, dC, dX)
    want = torch.empty_like(dX)
    dg.gemm_lora_bwd(X, W, A, B, ids - 1, T, dC, want)
    assert torch.equal(dX, want)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(33, 100, 264, 12, 4), (300, 520, 200, 16, 3)])
def test_lora_gradients_apart(M, N, K, R, S, typ):
    """Each gradient alone and in pairs gives the bits of all three."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 18)
    dC, T = randn((M, N), 0.1, dt, gen(19)).to(DEV), lora_ref(X, W, A, B, ids)[1].float()
    every = [torch.empty_like(v) for v in (X, A, B)]
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, *every, scales=scales)
    for mask in range(1, 7):
        some = [torch.full_like(v, 9.0) if mask >> i & 1 else None for i, v in enumerate(every)]
        dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, *some, scales=scales)
        for a, b in zip(some, every):
            assert a is None or torch.equal(a, b), mask


def test_lora_gradients_against_differences():
    """<dC, C(theta + h d) - C(theta - h d)> / 2 h of the definition in 64 bits,
    along random directions of X, A and B, against the gradients' products with them."""
    M, N, K, R, S, dt = 40, 60, 48, 8, 3, torch.float16
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 20)
    dC = randn((M, N), 0.1, dt, gen(21)).to(DEV)
    T = torch.empty((M, R), device=DEV)
    dg.gemm_lora(X, W, A, B, ids, torch.empty_like(dC), scales=scales, T=T)
    grads = [torch.empty_like(v) for v in (X, A, B)]
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, *grads, scales=scales)
    f = torch.where(ids >= 0, scales[ids.clamp(min=0)], 0.0).double()

    def value(x, a, b):
        at = ids.clamp(min=0)
        t = (x[:, None, :] * a[at]).sum(2) * f[:, None]
        return (dC.double() * (x @ W.double().T + (b[at] * t[:, None, :]).sum(2))).sum()

    base = [v.double() for v in (X, A, B)]
    for i, (v, g) in enumerate(zip(base, grads)):
        d = torch.randn(v.shape, generator=gen(22 + i), dtype=torch.float64).to(DEV)
        h = 1e-4
        up, down = ([q + s * h * d if j == i else q for j, q in enumerate(base)] for s in (1, -1))
        slope = float((value(*up) - value(*down)) / (2 * h))
        # a sum of products with rounded gradients: eps / 2 of each, at random signs
        tol = 8 * torch.finfo(dt).eps / 2 * float((g.double() * d).norm()) + 1e-6
        assert abs(float((g.double() * d).sum()) - slope) <= tol, i


# ---------------------------------------------------------------- updates

def ortho_input(L, m, n, typ, seed=0, strong=0.0, pad=0, shift=0, gap=0):
    g = gen(seed)
    G = torch.randn((L, m, n), generator=g)
    if strong:
        k = min(4, m, n)
        G += strong * torch.randn((L, m, k), generator=g) @ torch.randn((L, k, n), generator=g)
    return place3((1e-3 * G).to(ALL[typ]), pad, shift, gap)


# short sides below and at the borders of the one-launch form, of padding, of the
# tiles; tiles of every shape, whole rounds and ranges
ORTHO = [(1, 1, 1), (2, 1, 300), (3, 5, 3), (1, 32, 32), (2, 33, 129), (4, 64, 1000), (1, 1500, 64),
         (2, 65, 65), (2, 65, 1030), (1, 127, 400), (1, 400, 129), (1, 192, 192), (3, 200, 264),
         (2, 513, 300), (1, 777, 1500), (1, 2100, 640), (5, 384, 384), (1, 1025, 1025)]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("source", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,m,n", ORTHO)
def test_ortho(L, m, n, source, out):
    G, O = ortho_input(L, m, n, source, L + m + n), Out3(L, m, n, ALL[out])
    show("ortho", L, m, n, source, out)
    assert dg.gemm_ortho(G, O.t) is O.t
    ortho_check(O.t, G, "ortho")
    O.check_frame("ortho")


@pytest.mark.parametrize("L,m,n,source,out", [(1, 4096, 4096, "f32", "bf16"),
                                              (4, 2048, 4096, "bf16", "bf16"),
                                              (1, 3000, 1300, "f32", "f32"),
                                              (6, 1100, 600, "f16", "f16"),
                                              (1, 5000, 1025, "bf16", "bf16")])
def test_ortho_large(L, m, n, source, out):
    test_ortho(L, m, n, source, out)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("strong", [1.0, 30.0])
@pytest.mark.parametrize("L,m,n", [(2, 48, 700), (1, 300, 200), (1, 700, 1500)])
def test_ortho_strong_directions(L, m, n, strong, out):
    """A few directions hold nearly all of the norm."""
    for source in ("f32", "bf16"):
        G, O = ortho_input(L, m, n, source, 3, strong), Out3(L, m, n, ALL[out])
        show("ortho strong", L, m, n, source, out, strong)
        dg.gemm_ortho(G, O.t)
        ortho_check(O.t, G, "ortho")


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("L,m,n", [(2, 40, 90), (1, 150, 300), (2, 300, 150)])
def test_ortho_steps_and_coefficients(L, m, n, steps):
    """Other numbers of steps, one triple for each, and the coefficients that
    converge: the result's singular values go to 1."""
    for source, out in (("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")):
        G = ortho_input(L, m, n, source, 5)
        O = torch.empty(G.shape, dtype=ALL[out], device=DEV)
        show("ortho steps", L, m, n, steps, source, out)
        dg.gemm_ortho(G, O, steps=steps)
        ortho_check(O, G, "ortho", steps)
        each = tuple((2.0 + 0.25 * k, -1.5 - 0.25 * k, 0.5) for k in range(steps))
        dg.gemm_ortho(G, O, steps=steps, coeffs=each)
        ortho_check(O, G, "ortho, a triple a step", steps, each)
    O = torch.empty(G.shape, device=DEV)
    dg.gemm_ortho(G, O, steps=40, coeffs=(1.5, -0.5, 0.0))
    sv = torch.linalg.svdvals(O.double().cpu())
    assert float((sv - 1).abs().max()) < 2.0 ** -16


@pytest.mark.parametrize("L,m,n", [(3, 20, 70), (3, 130, 200), (2, 300, 140)])
@pytest.mark.parametrize("pad,shift,gap", [(3, 1, 2), (8, 8, 0), (0, 1, 1)])
def test_ortho_strides(L, m, n, pad, shift, gap):
    for source, out in (("f32", "f32"), ("f16", "f16"), ("f32", "bf16")):
        G = ortho_input(L, m, n, source, 6, 0.0, pad, shift, gap)
        O = Out3(L, m, n, ALL[out], pad, shift, gap)
        show("ortho strides", L, m, n, source, out, pad, shift, gap)
        dg.gemm_ortho(G, O.t)
        ortho_check(O.t, G, "ortho")
        O.check_frame("ortho")
    # one matrix, and the same one for all
    dg.gemm_ortho(G[0], O.t[0])
    want = O.t[0].clone()
    O = torch.empty((L, m, n), dtype=ALL["bf16"], device=DEV)
    dg.gemm_ortho(G[:1].expand(L, m, n), O)
    assert all(torch.equal(o, want) for o in O)


@pytest.mark.parametrize("m,n", [(24, 500), (140, 200), (500, 150)])
def test_ortho_edges(m, n):
    """Zeros, one matrix with an infinity or a NaN, sizes from 1e-38 to 1e38, and
    an eps that counts; the other matrices keep their bits."""
    G = ortho_input(6, m, n, "f32", 7)
    for out in ("f32", "bf16"):
        O = torch.empty(G.shape, dtype=ALL[out], device=DEV)
        dg.gemm_ortho(G, O)
        H = G.clone()
        H[1] = 0.0
        H[2, 3, 5], H[4, 1, 2] = float("inf"), float("nan")
        P = torch.empty_like(O)
        show("ortho edges", m, n, out)
        dg.gemm_ortho(H, P)
        assert bool((P[1] == 0).all()) and bool(torch.isnan(P[2]).all()) and \
            bool(torch.isnan(P[4]).all())
        for l in (0, 3, 5):
            assert torch.equal(P[l], O[l])
        for size in (1e-35, 1e-20, 1e20, 1e35):
            H = G[:2] * 1e3 * size
            dg.gemm_ortho(H, P[:2], eps=0.0)
            ortho_check(P[:2], H, "ortho of size %g" % size, eps=0.0)
        H = G[:2] * 1e-6
        dg.gemm_ortho(H, P[:2], eps=1e-6)
        ortho_check(P[:2], H, "ortho with an eps", eps=1e-6)


def test_ortho_empty():
    for shape in ((0, 5, 7), (3, 0, 7), (3, 5, 0)):
        t = torch.empty(shape, device=DEV)
        dg.gemm_ortho(t, torch.empty_like(t))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("typ", TYPES)
def test_run_together(typ):
    """Two steps of training three adapters beside a frozen projection: forward,
    gradients, the factors' updates orthogonalised and applied. Gradients
    against autograd in 64 bits."""
    M, N, K, R, S, dt = 300, 256, 192, 16, 3, DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 30, "sorted")
    goal = randn((M, N), 1.0, dt, gen(31)).to(DEV)
    C, T = torch.empty_like(goal), torch.empty((M, R), device=DEV)
    dX, dA, dB = torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)
    oA, oB = (torch.empty(v.shape, dtype=torch.bfloat16, device=DEV) for v in (A, B))
    for step in range(2):
        dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
        dC = ((C.float() - goal.float()) / M).to(dt)
        dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX, dA, dB, scales=scales)
        x, a, b = (v.double().requires_grad_() for v in (X, A, B))
        at = ids.clamp(min=0)
        f = torch.where(ids >= 0, scales[at], 0.0).double()
        t = (x[:, None, :] * a[at]).sum(2)
        y = x @ W.double().T + (b[at] * (t * f[:, None])[:, None, :]).sum(2)
        want = torch.autograd.grad(y, (x, a, b), dC.double())
        refs = lora_bwd_ref(X, W, A, B, ids, t.detach(), dC, scales)
        close(C, *lora_result(y.detach(), lora_ref(X, W, A, B, ids, scales)[2], dt), "C")
        # (T is the kernel's, off by its sums)
        most = (X.double().abs() @ A.double().abs().flatten(0, 1).T).max()
        slack = 1.5 * sum_error(K, most) * dC.double().abs().sum(0).max()
        for got, g, (ref, tol), what in zip((dX, dA, dB), want, refs, ("dX", "dA", "dB")):
            assert float((g - ref).abs().max()) <= 1e-9 * float(ref.abs().max())
            close(got, ref, tol + (slack if what == "dB" else 0.0), what)
        for grad, o, v in ((dA, oA, A), (dB, oB, B)):
            dg.gemm_ortho(grad, o)
            ortho_check(o, grad, "update")
            v -= 0.02 * o.to(dt)


def calls(typ, sizes):
    """(call on a workspace, its bytes, outputs, an input to change) of every operator."""
    M, N, K, R, S = sizes
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 40)
    C, T = torch.empty((M, N), dtype=dt, device=DEV), torch.zeros((M, R), device=DEV)
    T0 = lora_ref(X, W, A, B, ids)[1].float()
    dC = randn((M, N), 0.1, dt, gen(41)).to(DEV)
    dX, dA, dB = torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)
    G = ortho_input(2, N // 4, K, "f32", 42)
    H = ortho_input(3, R, K, "f32", 43)
    O, P, Q = (torch.empty(v.shape, dtype=d, device=DEV)
               for v, d in ((G, dt), (H, dt), (G.mT.contiguous(), torch.bfloat16)))
    Gt = G.mT.contiguous()
    return [
        (lambda ws: dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T, workspace=ws),
         dg.lora_workspace_bytes(X, W, A, B), [C, T], X),
        (lambda ws: dg.gemm_lora_bwd(X, W, A, B, ids, T0, dC, dX, dA, dB, scales=scales, workspace=ws),
         dg.lora_bwd_workspace_bytes(X, W, A, dC), [dX, dA, dB], dC),
        (lambda ws: dg.gemm_ortho(G, O, workspace=ws), dg.ortho_workspace_bytes(G, O), [O], G),
        (lambda ws: dg.gemm_ortho(H, P, workspace=ws), dg.ortho_workspace_bytes(H, P), [P], H),
        (lambda ws: dg.gemm_ortho(Gt, Q, workspace=ws), dg.ortho_workspace_bytes(Gt, Q), [Q], Gt),
    ]


SIZES = [(40, 300, 200, 12, 5), (400, 4100, 328, 16, 3), (330, 5001, 139, 24, 2)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("sizes", SIZES)
def test_what_a_workspace_holds(sizes, typ):
    """Zeros or NaN throughout: the same bits; and one byte less is refused."""
    for i, (call, size, outs, _) in enumerate(calls(typ, sizes)):
        show("workspace", sizes, typ, i, size)
        results = []
        for fill in (0, 255):
            call(torch.full((size,), fill, dtype=torch.uint8, device=DEV))
            results.append([o.clone() for o in outs])
        for a, b in zip(*results):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), i
        with pytest.raises(dg.GemmError):
            call(torch.empty((size - 1,), dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("sizes", SIZES)
def test_captured_and_replayed(sizes, typ):
    """Graphs of all operators replayed on changed inputs, in turn, with eager calls
    between: the eager bits each time."""
    graphs = []
    every = calls(typ, sizes)
    for call, size, outs, _ in every:
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        call(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(ws)
        graphs.append((g, ws))
    for turn in range(3):
        for i, ((call, size, outs, change), (g, ws)) in enumerate(zip(every, graphs)):
            show("captured", sizes, typ, turn, i)
            change.mul_(-0.5 if turn % 2 else 2.0)
            call(None)
            torch.cuda.synchronize()
            want = [o.clone() for o in outs]
            for o in outs:
                o.fill_(7)
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, outs):
                assert torch.equal(a, b), (turn, i)


def test_streams_and_threads():
    """A side stream given and current, and two threads with a stream each: the
    bits of one call after another."""
    import threading

    sides = []
    for typ in TYPES:
        every = calls(typ, SIZES[1])
        for call, _, _, _ in every:
            call(None)
        torch.cuda.synchronize()
        sides.append((every, [[o.clone() for o in outs] for _, _, outs, _ in every],
                      torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(every, stream):
        with torch.cuda.stream(stream):
            for _ in range(5):
                for call, _, outs, _ in every:
                    for o in outs:
                        o.fill_(3)
                    call(None)

    threads = [threading.Thread(target=work, args=(e, s)) for e, _, s in sides]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for every, want, _ in sides:
        for (_, _, outs, _), w in zip(every, want):
            for a, b in zip(outs, w):
                assert torch.equal(a, b)
    side = torch.cuda.Stream()
    X, W, A, B, ids, _ = lora_inputs(20, 90, 64, 8, 3, torch.float16, 50)
    C, D = (torch.empty((20, 90), dtype=torch.float16, device=DEV) for _ in range(2))
    dg.gemm_lora(X, W, A, B, ids, C)
    torch.cuda.synchronize()
    dg.gemm_lora(X, W, A, B, ids, D, stream=side)
    G, O, P = (torch.randn((70, 80), device=DEV) for _ in range(3))
    dg.gemm_ortho(G, O)
    torch.cuda.synchronize()
    dg.gemm_ortho(G, P, stream=side)
    side.synchronize()
    assert torch.equal(C, D) and torch.equal(O, P)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,ldx,ldc", [(40, 200, 72, 1 << 26, 1 << 26), (300, 2500, 136, 1 << 23, 1 << 23)])
def test_lora_past_two_gibi_elements(M, N, K, ldx, ldc, typ):
    """Rows of X, C, dC and dX beyond 2^31 elements."""
    dt, R, S = DT[typ], 8, 2
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, 60)
    show("lora far", M, N, K, typ)
    big = torch.empty((M * ldx,), dtype=dt, device=DEV)
    Xf = torch.as_strided(big, (M, K), (ldx, 1))
    Cf = torch.as_strided(big, (M, N), (ldc, 1), 4096)
    dXf = torch.as_strided(big, (M, K), (ldx, 1), 16384)
    Xf.copy_(X)
    C, dX, T = torch.empty((M, N), dtype=dt, device=DEV), torch.empty_like(X), \
        torch.empty((M, R), device=DEV)
    dg.gemm_lora(X, W, A, B, ids, C, scales=scales, T=T)
    dg.gemm_lora(Xf, W, A, B, ids, Cf, scales=scales)
    y, _, off, _ = lora_ref(X, W, A, B, ids, scales)
    close(Cf, *lora_result(y, off, dt), "C")
    assert torch.equal(C, Cf)
    dA, dB, eA, eB = (torch.empty_like(v) for v in (A, B, A, B))
    dg.gemm_lora_bwd(X, W, A, B, ids, T, C, dX, dA, dB, scales=scales)
    dg.gemm_lora_bwd(Xf, W, A, B, ids, T, Cf, dXf, eA, eB, scales=scales)
    assert torch.equal(dX, dXf) and torch.equal(dA, eA) and torch.equal(dB, eB)


def test_stacks_past_two_gibi_elements():
    """Adapters and matrices that start beyond 2^31 elements."""
    dt, M, N, K, R = torch.bfloat16, 40, 90, 64, 8
    far = (1 << 31) + 4096
    buf = torch.empty((far + (1 << 20),), dtype=dt, device=DEV)
    A = torch.as_strided(buf, (2, R, K), (far, K, 1), 0)
    B = torch.as_strided(buf, (2, N, R), (far, R, 1), R * K)
    X, W, A0, B0, ids, _ = lora_inputs(M, N, K, R, 2, dt, 61)
    A.copy_(A0)
    B.copy_(B0)
    C, D = (torch.empty((M, N), dtype=dt, device=DEV) for _ in range(2))
    show("stacks far")
    dg.gemm_lora(X, W, A0, B0, ids, C)
    dg.gemm_lora(X, W, A, B, ids, D)
    assert torch.equal(C, D)
    dA = torch.as_strided(buf, (2, R, K), (far, K, 1), 8192)
    dB = torch.as_strided(buf, (2, N, R), (far, R, 1), 16384)
    T, eA, eB = torch.randn((M, R), device=DEV), torch.empty_like(A0), torch.empty_like(B0)
    dg.gemm_lora_bwd(X, W, A0, B0, ids, T, C, None, eA, eB)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, C, None, dA, dB)
    assert torch.equal(dA, eA) and torch.equal(dB, eB)
    for m, n in ((20, 300), (130, 140), (300, 150)):
        G = ortho_input(2, m, n, "bf16", 62)
        far_g = torch.as_strided(buf, (2, m, n), (far, n, 1), 0)
        far_o = torch.as_strided(buf, (2, m, n), (far, n, 1), 1 << 17)
        far_g.copy_(G)
        O = torch.empty_like(G)
        dg.gemm_ortho(G.contiguous(), O)
        dg.gemm_ortho(far_g, far_o)
        assert torch.equal(O, far_o)
    del buf


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K,R,S", [(300, 64, 72, 4, 2500), (20, 136, 200, 16, 2049),
                                       (900, 2600, 64, 4, 2300)])
def test_lora_thousands_of_adapters(M, N, K, R, S, typ):
    """More adapters than one workgroup counts, and ids past 32 bits."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, R, S, dt, M + S)
    ids[0], ids[M // 2], ids[M - 1] = (1 << 32) + 1, -(1 << 40), S - 1
    C, T = Out(M, N, dt), Out(M, R, torch.float32)
    show("lora", M, N, K, R, S, typ)
    dg.gemm_lora(X, W, A, B, ids, C.t, scales=scales, T=T.t)
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    assert bool(C.t[0].isnan().all()) and bool(T.t[0].isnan().all())
    close(T.t[1:], t[1:], dt_sum[1:], "T")
    ref, tol = lora_result(y, off, dt)
    close(C.t[1:], ref[1:], tol[1:], "C")
    dC = randn((M, N), 0.1, dt, gen(M)).to(DEV)
    T = t.float()
    T[0] = 0
    dX, dA, dB = Out(M, K, dt), Out3(S, R, K, dt), Out3(S, N, R, dt)
    dg.gemm_lora_bwd(X, W, A, B, ids, T, dC, dX.t, dA.t, dB.t, scales=scales)
    (rx, tx), (ra, ta), (rb, tb) = lora_bwd_ref(X, W, A, B, ids, T, dC, scales)
    assert bool(dX.t[0].isnan().all())
    close(dX.t[1:], rx[1:], tx[1:], "dX")
    close(dA.t, ra, ta, "dA")
    close(dB.t, rb, tb, "dB")


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("M,N,K", [(192, 4096, 264), (193, 4096, 264), (640, 264, 1024),
                                   (200, 2000, 7000), (641, 1000, 200), (65, 600, 64)])
def test_lora_at_the_rules(M, N, K, typ):
    """Sizes on both sides of what chooses the kernels for few rows."""
    dt = DT[typ]
    X, W, A, B, ids, scales = lora_inputs(M, N, K, 16, 6, dt, M + K)
    C, T = Out(M, N, dt), Out(M, 16, torch.float32)
    show("lora", M, N, K, typ)
    dg.gemm_lora(X, W, A, B, ids, C.t, scales=scales, T=T.t)
    y, t, off, dt_sum = lora_ref(X, W, A, B, ids, scales)
    close(C.t, *lora_result(y, off, dt), "C")
    close(T.t, t, dt_sum, "T")
    dC = randn((M, N), 0.1, dt, gen(M)).to(DEV)
    dX = Out(M, K, dt)
    dg.gemm_lora_bwd(X, W, A, B, ids, T.t, dC, dX.t, scales=scales)
    grads_check(X, W, A, B, ids, T.t, dC, scales, dX.t)
    C.check_frame("C")
    dX.check_frame("dX")
