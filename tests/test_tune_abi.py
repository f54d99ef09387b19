"""The C ABI and binding of the operators of fine tuning without a GPU: exported
symbols, argument validation, workspace sizes.  None of these calls reaches a
kernel (validation returns before the device check, and there the calls end)."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest

import dense_gemm_sgemm_amd as dg
from dense_gemm_sgemm_amd import tune
from test_fused_abi import fake_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mi355tune.h")
p = ctypes.c_void_p
A = p(0x100000)          # a fake device address: only its alignment is looked at
ODD = p(0x100002)
F16, BF16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tune.LIB_PATH):
        from dense_gemm_sgemm_amd import build
        build.build()
    return tune.load_library()


def test_exports_exactly_the_header(lib):
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"MI355TUNE_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)))
    out = subprocess.run(["nm", "-D", "--defined-only", tune.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T " in l) == declared
    assert len(declared) == 6


def lora(lib, type=F16, M=4, N=8, K=16, R=4, S=2, X=A, ldx=16, W=A, ldw=16, A_=A, lda=16, sa=64,
         B=A, ldb=4, sb=32, ids=A, scales=None, bias=None, act=0, res=None, ldr=0, C=A, ldc=8,
         T=None, ldt=0, ws=None, bytes=0):
    return lib.gemm_lora(type, M, N, K, R, S, X, ldx, W, ldw, A_, lda, sa, B, ldb, sb, ids, scales,
                         bias, act, res, ldr, C, ldc, T, ldt, ws, bytes, None)


def test_lora_refusals(lib):
    for k in ("M", "N", "K", "R", "S"):
        assert lora(lib, **{k: -1}) == -1, k
    big = (1 << 27) + 1
    assert lora(lib, M=big) == -6 and lora(lib, S=big) == -6
    assert lora(lib, type=2) == -6 and lora(lib, act=3) == -6
    assert lora(lib, R=0) == -6 and lora(lib, R=1025, ldb=1025) == -6
    for k, v in (("ldx", 15), ("ldw", 15), ("lda", 15), ("ldb", 3), ("ldc", 7), ("sa", -1),
                 ("sb", -1)):
        assert lora(lib, **{k: v}) == -2, k
    assert lora(lib, res=A, ldr=7) == -2 and lora(lib, T=A, ldt=3) == -2
    for k in ("X", "W", "A_", "B", "ids", "C"):
        assert lora(lib, **{k: None}) == -3, k
    assert lora(lib) == -7                                      # no workspace
    need = lib.gemm_lora_workspace(F16, 4, 8, 16, 4, 2, A, 16, A, 16, 4)
    assert need == 4 * 32 * 2 + 256
    assert lora(lib, ws=A, bytes=need - 1) == -7
    assert lora(lib, ws=p(0x100008), bytes=need) == -7
    assert lora(lib, ws=A, bytes=need) == -4                    # no device here
    # nothing to do; what is not read may be missing
    assert lora(lib, M=0, X=None, ids=None, C=None) == 0
    assert lora(lib, N=0, W=None, B=None, C=None) == 0
    assert lora(lib, N=0, W=None, B=None, C=None, T=A, ldt=4, ws=A, bytes=need) == -4
    assert lora(lib, S=0, A_=None, B=None, ws=A, bytes=need) == -4
    assert lora(lib, K=0, X=None, W=None, A_=None, ws=A, bytes=need) == -4
    # adapters may be the same one, or lie inside each other: they are only read
    assert lora(lib, sa=0, sb=0, ws=A, bytes=need) == -4


def test_lora_workspace(lib):
    ws = lib.gemm_lora_workspace
    t = 4096 * 32 * 2 + 4096 * 4
    assert ws(BF16, 4096, 4096, 4096, 16, 8, A, 4096, A, 4096, 16) == t
    assert ws(BF16, 4096, 4096, 4096, 16, 8, ODD, 4096, A, 4096, 16) == t + 4096 * 4096 * 2
    # ranks that are no multiple of eight: B widened
    assert ws(BF16, 4096, 4096, 4096, 12, 8, A, 4096, A, 4096, 12) == t + 8 * 4096 * 16 * 2
    assert ws(BF16, 4096, 4096, 4096, 8, 8, A, 4096, A, 4096, 1 << 22) == t + 8 * 4096 * 16 * 2
    assert ws(BF16, 4096, 4096, 4096, 33, 8, A, 4096, A, 4096, 33) == \
        4096 * 96 * 2 + 4096 * 12 + 8 * 4096 * 48 * 2
    # few rows: operands as they are
    assert ws(BF16, 64, 4096, 4095, 12, 8, ODD, 4095, ODD, 4095, 12) == 64 * 64 + 256
    assert ws(BF16, 0, 4096, 4096, 16, 8, A, 4096, A, 4096, 16) == 0
    assert ws(7, 64, 4096, 4096, 16, 8, A, 4096, A, 4096, 16) == 0
    assert ws(BF16, 64, 4096, 4096, 0, 8, A, 4096, A, 4096, 16) == 0
    # sizes past 32 bits
    assert ws(BF16, 1 << 22, 4096, 4096, 1024, 8, A, 4096, A, 4096, 1024) == (1 << 34) + (1 << 30)


def bwd(lib, type=F16, M=4, N=8, K=16, R=4, S=2, X=A, ldx=16, W=A, ldw=16, A_=A, lda=16, sa=64,
        B=A, ldb=4, sb=32, ids=A, scales=None, T=A, ldt=4, dC=A, lddc=8, dX=A, lddx=16, dA=A,
        ldda=16, sda=64, dB=A, lddb=4, sdb=32, ws=None, bytes=0):
    return lib.gemm_lora_bwd(type, M, N, K, R, S, X, ldx, W, ldw, A_, lda, sa, B, ldb, sb, ids,
                             scales, T, ldt, dC, lddc, dX, lddx, dA, ldda, sda, dB, lddb, sdb, ws,
                             bytes, None)


def test_lora_bwd_refusals(lib):
    assert bwd(lib, M=-1) == -1 and bwd(lib, type=2) == -6 and bwd(lib, R=0) == -6
    for k, v in (("ldx", 15), ("ldw", 15), ("lda", 15), ("ldb", 3), ("ldt", 3), ("lddc", 7),
                 ("lddx", 15), ("ldda", 15), ("lddb", 3), ("sa", -1), ("sb", -1)):
        assert bwd(lib, **{k: v}) == -2, k
    # gradients of two adapters that would overlap
    assert bwd(lib, sda=63) == -2 and bwd(lib, sdb=31) == -2
    assert bwd(lib, S=1, sda=0, sdb=0) == -7
    for k in ("X", "W", "A_", "B", "ids", "T", "dC"):
        assert bwd(lib, **{k: None}) == -3, k
    assert bwd(lib) == -7
    # operands that the gradients asked for do not read may be missing
    assert bwd(lib, dX=None, W=None, ldw=0, A_=None, lda=0) == -7
    assert bwd(lib, dA=None, X=None, ldx=0) == -7
    assert bwd(lib, dB=None, T=None, ldt=0) == -7
    assert bwd(lib, dX=None, dA=None, W=None, A_=None, B=None, X=None) == -7
    assert bwd(lib, dX=None, dA=None, dB=None) == 0
    # no rows: gradients of zero are still work
    none = dict(M=0, X=None, ids=None, T=None, dC=None, W=None, A_=None, B=None)
    assert bwd(lib, **none) == -7 and bwd(lib, **none, dA=None, dB=None) == 0
    need = lib.gemm_lora_bwd_workspace(F16, 4, 8, 16, 4, 2, A, 8, A, 16, 1, 1, 1)
    assert bwd(lib, ws=A, bytes=need - 1) == -7 and bwd(lib, ws=A, bytes=need) == -4


def test_lora_bwd_workspace(lib):
    ws = lib.gemm_lora_bwd_workspace
    size = (BF16, 4096, 4096, 4096, 16, 2)
    dx = ws(*size, A, 4096, A, 4096, 1, 0, 0)
    t = 4096 * 32 * 2 + 4096 * 4
    factors = 2 * 4096 * 16 * 2
    assert dx == t + 2 * factors                                # both factors turned
    assert ws(*size, A, 4096, ODD, 4096, 1, 0, 0) == dx + 4096 * 4096 * 2
    assert ws(*size, A, 4104, A, 4096, 1, 0, 0) == dx
    # columns of dC that are no whole slab of 64: its last ones again
    assert ws(BF16, 4096, 4104, 4096, 16, 2, A, 4104, A, 4096, 1, 0, 0) == \
        t + factors + 2 * 16 * 4160 * 2 + 4096 * 128
    da = ws(*size, A, 4096, A, 4096, 0, 1, 0)
    assert da > factors + 4096 * 16 * 4 and ws(*size, A, 4096, A, 4096, 0, 0, 0) == 0
    assert ws(*size, A, 4096, A, 4096, 1, 1, 1) > max(dx, da)
    assert ws(BF16, 4096, 4096, 4096, 16, 0, A, 4096, A, 4096, 0, 1, 1) == 0


def ortho(lib, tg=F32, to=BF16, L=2, m=8, n=4, G=A, ldg=4, sg=32, steps=5, coeffs=True, eps=1e-7,
          O=A, ldo=4, so=32, ws=None, bytes=0):
    c = (ctypes.c_float * 192)(*([1.5, -0.5, 0.0] * 64)) if coeffs else None
    return lib.gemm_ortho(tg, to, L, m, n, G, ldg, sg, steps, c, eps, O, ldo, so, ws, bytes, None)


def test_ortho_refusals(lib):
    for k in ("L", "m", "n"):
        assert ortho(lib, **{k: -1}) == -1, k
        assert ortho(lib, **{k: (1 << 16) + 1}) == -6, k
    assert ortho(lib, tg=3) == -6 and ortho(lib, to=-1) == -6
    assert ortho(lib, steps=0) == -6 and ortho(lib, steps=65) == -6
    assert ortho(lib, eps=-1.0) == -6 and ortho(lib, eps=float("nan")) == -6
    assert ortho(lib, ldg=3) == -2 and ortho(lib, ldo=3) == -2 and ortho(lib, sg=-1) == -2
    assert ortho(lib, so=31) == -2                              # results that would overlap
    assert ortho(lib, G=None) == -3 and ortho(lib, O=None) == -3 and ortho(lib, coeffs=False) == -3
    assert ortho(lib) == -7
    need = lib.gemm_ortho_workspace(F32, BF16, 2, 8, 4, 5)
    assert ortho(lib, ws=A, bytes=need - 1) == -7 and ortho(lib, ws=p(0x100008), bytes=need) == -7
    assert ortho(lib, ws=A, bytes=need) == -4 and ortho(lib, sg=0, ws=A, bytes=need) == -4
    assert ortho(lib, L=1, sg=0, so=0, ws=A, bytes=need) == -4
    for k in ("L", "m", "n"):
        assert ortho(lib, **{k: 0}, G=None, O=None) == 0, k


def test_ortho_workspace(lib):
    ws = lib.gemm_ortho_workspace
    side = 4096 * 4096
    # two iterates in two values each, A and C; 253 tiles of 192 x 192 leave no ranges
    assert ws(F32, BF16, 1, 4096, 4096, 5) == 12 * side + 256 * 8 + 256
    # two values for A and C as well
    assert ws(F32, F16, 1, 4096, 4096, 5) == 16 * side + 256 * 8 + 256
    assert ws(F32, F32, 1, 4096, 4096, 5) == ws(F32, F16, 1, 4096, 4096, 5)
    # either way round; a single step of 16-bit matrices has no second value
    assert ws(BF16, BF16, 3, 300, 5000, 5) == ws(BF16, BF16, 3, 5000, 300, 5)
    assert ws(BF16, BF16, 1, 4096, 4096, 1) == 8 * side + 256 * 8 + 256
    # a short side: iterates of 32 or 64 rows, and sixteen parts of A (a norm's parts
    # are 1024 pieces of eight values)
    assert ws(F32, BF16, 16, 16, 4096, 5) == \
        16 * 8 * 8 + 256 + 4 * 16 * 4096 * 32 * 2 + 2 * 16 * 16 * 32 * 32 * 4
    assert ws(F32, BF16, 0, 16, 4096, 5) == 0 and ws(F32, BF16, 1, 16, 4096, 0) == 0
    assert ws(F32, F32, 1, 1 << 16, 1 << 16, 5) > 8 * (1 << 33)


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    h, i, f = torch.zeros(4, 64).half(), torch.zeros(4).long(), torch.zeros(4, 2)
    a, b = torch.zeros(2, 2, 64).half(), torch.zeros(2, 4, 2).half()
    with pytest.raises(TypeError):
        dg.gemm_lora(h, h, a, b, i, torch.zeros(4, 4).half())              # CPU tensors
    with pytest.raises(TypeError):
        dg.gemm_lora_bwd(h, h, a, b, i, f, torch.zeros(4, 4).half())
    with pytest.raises(TypeError):
        dg.gemm_ortho(h, h)
    with pytest.raises(TypeError):
        dg.gemm_ortho(i, h)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_binding_checks(lib):
    x, w, out = fake_gpu((2, 64), (64, 1)), fake_gpu((3, 64), (64, 1)), fake_gpu((2, 3), (3, 1))
    a, b = fake_gpu((5, 4, 64), (256, 64, 1)), fake_gpu((5, 3, 4), (12, 4, 1))
    ids = fake_gpu((2,), (1,), dtype="int64")
    t = fake_gpu((2, 4), (4, 1), dtype="float32")
    far = 2 ** 32 + 64

    def lora(**kw):
        k = dict(X=x, W=w, A=a, B=b, ids=ids, C=out)
        k.update(kw)
        return dg.gemm_lora(**k)

    for kw in (dict(A=fake_gpu((5, 4, 63), (252, 63, 1))), dict(B=fake_gpu((4, 3, 4), (12, 4, 1))),
               dict(B=fake_gpu((5, 2, 4), (8, 4, 1))), dict(B=fake_gpu((5, 3, 5), (15, 5, 1))),
               dict(A=fake_gpu((5, 4, 64), (256, 1, 4))), dict(ids=fake_gpu((3,), (1,), dtype="int64")),
               dict(ids=fake_gpu((2,), (1,), dtype="int32")), dict(C=w),
               dict(scales=fake_gpu((4,), (1,), dtype="float32")),
               dict(scales=fake_gpu((5,), (2,), dtype="float32")),
               dict(T=fake_gpu((2, 3), (3, 1), dtype="float32")), dict(act="gelu"),
               dict(A=fake_gpu((5, 4, 64), (256, far, 1))), dict(W=fake_gpu((3, 64), (far, 1)))):
        with pytest.raises(ValueError):
            lora(**kw)
            pytest.fail(str(list(kw)))
    for kw in (dict(A=fake_gpu((4, 64), (64, 1))), dict(T=fake_gpu((2, 4), (4, 1))),
               dict(A=fake_gpu((5, 4, 64), (256, 64, 1), dtype="bfloat16"))):
        with pytest.raises(TypeError):
            lora(**kw)
            pytest.fail(str(list(kw)))
    with pytest.raises(ValueError):
        dg.gemm_lora_bwd(x, w, a, b, ids, t, out, dA=fake_gpu((5, 3, 64), (192, 64, 1)))
    with pytest.raises(ValueError):
        dg.gemm_lora_bwd(x, w, a, b, ids, t, out, dB=fake_gpu((4, 3, 4), (12, 4, 1)))
    g = fake_gpu((2, 8, 4), (32, 4, 1), dtype="float32")
    with pytest.raises(ValueError):
        dg.gemm_ortho(g, fake_gpu((2, 8, 5), (40, 5, 1)))
    with pytest.raises(ValueError):
        dg.gemm_ortho(g, fake_gpu((2, 8, 4), (32, 1, 8)))
    with pytest.raises(TypeError):
        dg.gemm_ortho(fake_gpu((2, 8, 4), (32, 4, 1), dtype="float64"), g)
    for kw in (dict(steps=0), dict(steps=65), dict(coeffs=(1.0, 2.0)), dict(steps=2.0),
               dict(coeffs=((1.5, -0.5, 0.0),) * 4), dict(coeffs=((1.5, -0.5),) * 5)):
        with pytest.raises(ValueError):
            dg.gemm_ortho(g, g.clone(), **kw)
            pytest.fail(str(kw))


def test_coefficients_in_any_sequence():
    from dense_gemm_sgemm_amd import tune
    one = [3.0, -4.0, 2.0]
    for coeffs in (tuple(one), one):
        assert list(tune._coeffs(coeffs, 2)) == one * 2
    for coeffs in ((one, one), [one, one], [tuple(one), one], (tuple(one), tuple(one))):
        assert list(tune._coeffs(coeffs, 2)) == one * 2
    for coeffs in ((one, 1.0), [one], (1.0, 2.0), [one, one, one]):
        with pytest.raises(ValueError):
            tune._coeffs(coeffs, 2)
