"""Calls of the operators of fine tuning that the binding or the plans have to
answer rightly, without a GPU: none of them reaches a kernel."""
from __future__ import annotations

import os

import pytest

import dense_gemm_sgemm_amd as dg
from dense_gemm_sgemm_amd import tune
from test_fused_abi import fake_gpu


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tune.LIB_PATH):
        from dense_gemm_sgemm_amd import build
        build.build()
    return tune.load_library()


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("S", [1, 5])
def test_stacks_whose_rows_overlap(lib, S):
    """Rows closer than their length (one row expanded to all, a sliding window)
    are no matrix that the kernels can read, and none that they may write."""
    x, w, out = fake_gpu((2, 64), (64, 1)), fake_gpu((3, 64), (64, 1)), fake_gpu((2, 3), (3, 1))
    a, b = fake_gpu((S, 4, 64), (256, 64, 1)), fake_gpu((S, 3, 4), (12, 4, 1))
    ids = fake_gpu((2,), (1,), dtype="int64")
    t = fake_gpu((2, 4), (4, 1), dtype="float32")
    for row in (0, 1, 63):
        A, B = fake_gpu((S, 4, 64), (1 << 20, row, 1)), fake_gpu((S, 3, 4), (1 << 20, row % 4, 1))
        for call in (lambda: dg.gemm_lora(x, w, A, b, ids, out),
                     lambda: dg.gemm_lora(x, w, a, B, ids, out),
                     lambda: dg.lora_workspace_bytes(x, w, A, b),
                     lambda: dg.lora_workspace_bytes(x, w, a, B),
                     lambda: dg.lora_bwd_workspace_bytes(x, w, A, out),
                     lambda: dg.gemm_lora_bwd(x, w, A, b, ids, t, out, dX=x),
                     lambda: dg.gemm_lora_bwd(x, w, a, B, ids, t, out, dX=x),
                     lambda: dg.gemm_lora_bwd(x, w, a, b, ids, t, out, dA=A),
                     lambda: dg.gemm_lora_bwd(x, w, a, b, ids, t, out, dB=B)):
            with pytest.raises(ValueError, match="overlap"):
                call()
                pytest.fail("rows %d elements apart" % row)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_stacks_with_one_row_or_no_element():
    """Where no row has another behind it, the distance between rows says nothing."""
    half, at = fake_gpu((1, 1), (1, 1)).dtype, 0
    assert tune._adapters(fake_gpu((3, 1, 64), (64, 0, 1)), "A", half, at, 1, 64)[3] == 64
    assert tune._adapters(fake_gpu((3, 4, 1), (4, 1, 1)), "B", half, at, 4, 1)[3] == 1
    assert tune._adapters(fake_gpu((0, 4, 64), (0, 0, 1)), "A", half, at, 4, 64)[:2] == (0, 4)
    assert tune._adapters(fake_gpu((2, 4, 0), (0, 0, 1)), "A", half, at, 4, 0)[:2] == (2, 4)


def test_coefficients_by_their_values():
    """Numbers held in tensors count as they are at the call, not as they were at an
    earlier one; a whole matrix of them, and numpy's, are taken too."""
    torch = pytest.importorskip("torch")
    np = pytest.importorskip("numpy")
    own = [torch.tensor(v) for v in (3.0, -4.0, 2.0)]
    assert list(tune._coeffs(own, 2)) == [3.0, -4.0, 2.0] * 2
    own[0].fill_(9.0)
    assert list(tune._coeffs(own, 2)) == [9.0, -4.0, 2.0] * 2
    own[1] -= 1.0
    assert list(tune._coeffs([own, own], 2)) == [9.0, -5.0, 2.0] * 2
    own[2].fill_(0.5)
    assert list(tune._coeffs([tuple(own), own], 2)) == [9.0, -5.0, 0.5] * 2
    rows = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]])
    for held in (rows, rows.numpy(), list(rows), tuple(rows.numpy())):
        assert list(tune._coeffs(held, 2)) == [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]
    rows[1, 2] = 7.0
    assert list(tune._coeffs(rows, 2)) == [1.0, 2.0, 3.0, 4.0, 5.0, 7.0]
    assert list(tune._coeffs(np.array([1.0, 2.0, 3.0]), 2)) == [1.0, 2.0, 3.0] * 2
    assert list(tune._coeffs(tune.MUON, 1)) == list(tune._coeffs(tuple(tune.MUON), 1))
    for wrong in (rows.T, torch.ones(2, 3, 1), torch.ones(2), torch.ones(4, 3)):
        with pytest.raises((ValueError, TypeError)):
            tune._coeffs(wrong, 2)
            pytest.fail(str(wrong))


def test_coefficients_do_not_hold_the_callers_objects():
    torch = pytest.importorskip("torch")
    import gc
    import weakref
    t = torch.tensor(2.0)
    alive = weakref.ref(t)
    tune._coeffs((t, 0.5, 0.25), 3)
    del t
    gc.collect()
    assert alive() is None


A, F16, BF16 = 0x100000, 0, 1     # a fake device address


def bwd_bytes(lib, M, N, K, R, S, dx=0, da=0, db=0):
    return lib.gemm_lora_bwd_workspace(BF16, M, N, K, R, S, A, max(1, N), A, max(1, K), dx, da, db)


def test_partial_sums_by_the_chunks(lib):
    """Only an adapter that goes on from one workgroup's steps to the next one's
    leaves partial sums, two of them a workgroup at most: the workspace does not
    grow by gradients in fp32 with the adapters that no row names."""
    M, N, K, R = 300, 4096, 4096, 64
    few, many = (bwd_bytes(lib, M, N, K, R, S, db=1) for S in (M, 8 * M))
    assert 0 <= many - few <= 2 * 4 * (7 * M + 128)              # rows of each, first steps
    few, many = (bwd_bytes(lib, M, N, K, R, S, da=1) for S in (M, 8 * M))
    assert 0 <= many - few <= 2 * 4 * (7 * M + 128) + 7 * M * R * 4096 * 2   # and B turned
    # one adapter keeps what it had: a place a chunk and one
    assert bwd_bytes(lib, 4096, 4096, 4096, 16, 1, da=1, db=1) < 10 << 20


def test_rows_times_adapters(lib):
    """Rows are listed by adapter in time that goes as M * min(M, S): where that is no
    longer a moment's work the gradients of adapters are refused, dX is not."""
    from ctypes import c_void_p
    a = c_void_p(A)

    def call(M, S, dx, da, db, ws=None, bytes=0):
        return lib.gemm_lora_bwd(F16, M, 8, 8, 1, S, a, 8, a, 8, a, 8, 8, a, 1, 8, a, None, a, 1, a,
                                 8, a if dx else None, 8, a if da else None, 8, 8, a if db else None,
                                 1, 8, ws, bytes, None)

    big = 1 << 20
    for da, db in ((1, 0), (0, 1), (1, 1)):
        assert call(big, big, 1, da, db) == -7                   # a workspace is missing
        assert call(big + 1, big, 1, da, db) == -6
        assert call(1 << 27, 1 << 13, 0, da, db) == -7 and call(1 << 27, 8193, 0, da, db) == -6
        assert bwd_bytes(lib, big, 8, 8, 1, big, 0, da, db) > 0
        assert bwd_bytes(lib, big + 1, 8, 8, 1, big, 0, da, db) == 0
    assert call(1 << 22, 1 << 22, 1, 0, 0) == -7 and bwd_bytes(lib, 1 << 22, 8, 8, 1, 1 << 22, 1) > 0
    assert call(4, 1 << 27, 0, 1, 1) == -7                       # few rows, any adapters


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_gradients_without_what_they_do_not_read(lib, monkeypatch):
    """X is read for dA alone, T for dB, W and A for dX, B for dX and dA: None will do
    elsewhere, and nothing of it reaches the library."""
    x, w, dc = fake_gpu((2, 64), (64, 1)), fake_gpu((3, 64), (64, 1)), fake_gpu((2, 3), (3, 1))
    a, b = fake_gpu((5, 4, 64), (256, 64, 1)), fake_gpu((5, 3, 4), (12, 4, 1))
    ids, t = fake_gpu((2,), (1,), dtype="int64"), fake_gpu((2, 4), (4, 1), dtype="float32")
    seen = []
    monkeypatch.setattr(tune, "_run", lambda at, stream, fn, args, need=None, ws=None: seen.append(args))

    def call(X=x, W=w, A=a, B=b, T=t, **out):
        assert dg.gemm_lora_bwd(X, W, A, B, ids, T, dc, **out) == (
            out.get("dX"), out.get("dA"), out.get("dB"))
        return seen.pop()

    # (type and sizes; leading dimensions of X, W, A, B, T)
    sizes, lds = slice(0, 6), lambda s: [s[i] for i in (7, 9, 11, 14, 19)]
    every = call(dX=x, dA=a, dB=b)
    assert every[sizes] == (0, 2, 3, 64, 4, 5) and lds(every) == [64, 64, 64, 4, 4]
    got = call(X=None, T=None, dX=x)
    assert got[sizes] == every[sizes] and lds(got) == [0, 64, 64, 4, 0]
    got = call(W=None, A=None, T=None, dA=a)
    assert got[sizes] == every[sizes] and lds(got) == [64, 0, 0, 4, 0]
    for keep in (dict(X=x), dict(W=w), dict(A=a)):      # one of them says how long rows are
        got = call(**{**dict(X=None, W=None, A=None, B=None), **keep}, dB=b)
        assert got[sizes] == every[sizes], list(keep)
    got = call(T=None, W=None, dA=a)
    assert got[sizes] == every[sizes]
    for kw in (dict(W=None, dX=x), dict(A=None, dX=x), dict(B=None, dX=x), dict(X=None, dA=a),
               dict(B=None, dA=a), dict(T=None, dB=b), dict(X=None, W=None, A=None, B=None, dB=b),
               dict(X=None, dA=a, dX=x), dict(W=fake_gpu((3, 63), (63, 1)), X=None, dB=b),
               dict(X=None, W=None, A=fake_gpu((5, 3, 64), (192, 64, 1)), dB=b),
               dict(X=fake_gpu((3, 64), (64, 1)), dB=b), dict(X=None, W=w, A=None, dB=w)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
            pytest.fail(str(list(kw)))
    need = dg.lora_bwd_workspace_bytes(x, w, a, dc, False, True, True)
    assert need == dg.lora_bwd_workspace_bytes(None, None, a, dc, False, True, True) > 0
    assert dg.lora_bwd_workspace_bytes(None, w, a, dc) == dg.lora_bwd_workspace_bytes(x, w, a, dc)
    with pytest.raises(ValueError):
        dg.lora_bwd_workspace_bytes(None, None, a, dc)


def test_singular_values_are_in_the_documentation():
    """What gemm_ortho's matrices must keep to is where a caller from Python reads it."""
    text = " ".join(dg.gemm_ortho.__doc__.split())
    assert "singular values" in text and "below 7" in text
