"""The operators of fine tuning on values at the ends of their types' ranges, held
to fixed bounds."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_sgemm_amd as dg  # noqa: E402
from fused_ref import DT, close, randn  # noqa: E402
from test_tune_gpu import DEV, TYPES, gen, lora_inputs, show  # noqa: E402
from tune_ref import lora_bwd_ref, lora_ref, lora_result  # noqa: E402

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
