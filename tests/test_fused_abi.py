"""The fused operators' C ABI and binding without a GPU: exported symbols,
argument validation, workspace sizes.  None of these calls reaches a kernel
(validation returns before the device check, and there the calls end)."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest

import dense_gemm_sgemm_amd as dg
from dense_gemm_sgemm_amd import fused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mi355fused.h")
p = ctypes.c_void_p
A = p(0x100000)          # a fake device address: only its alignment is looked at
ODD = p(0x100002)
F16, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fused.LIB_PATH):
        from dense_gemm_sgemm_amd import build
        build.build()
    return fused.load_library()


def declared():
    text = open(HEADER).read()
    return sorted(set(re.findall(r"MI355FUSED_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)))


def test_exports_exactly_the_header(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", fused.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T " in l) == declared()
    assert len(declared()) == 9


def gated(lib, type=F16, act=2, M=4, N=8, K=16, X=A, ldx=16, Wg=A, ldg=16, Wu=A, ldu=16, H=A,
          ldh=8, G=None, ldG=0, U=None, ldU=0, ws=None, bytes=0):
    return lib.gemm_gated(type, act, M, N, K, X, ldx, Wg, ldg, Wu, ldu, H, ldh, G, ldG, U, ldU, ws,
                          bytes, None)


def test_gated_refusals(lib):
    assert gated(lib, M=-1) == -1 and gated(lib, N=-1) == -1 and gated(lib, K=-1) == -1
    big = (1 << 27) + 1
    assert gated(lib, K=big, ldx=big, ldg=big, ldu=big) == -6 and gated(lib, M=big) == -6
    assert gated(lib, type=2) == -6 and gated(lib, act=3) == -6 and gated(lib, act=-1) == -6
    assert gated(lib, ldx=15) == -2 and gated(lib, ldg=15) == -2 and gated(lib, ldu=15) == -2
    assert gated(lib, ldh=7) == -2 and gated(lib, G=A, ldG=7) == -2 and gated(lib, U=A) == -2
    assert gated(lib, X=None) == -3 and gated(lib, Wu=None) == -3 and gated(lib, H=None) == -3
    assert gated(lib, M=0, X=None, H=None) == 0 and gated(lib, N=0, Wg=None, ldh=1) == 0
    # a padded copy is needed: no workspace, one too small, one misaligned
    big = dict(M=200, N=2600, K=20, ldx=20, ldg=20, ldu=20, ldh=2600)
    need = lib.gemm_gated_workspace(F16, 200, 2600, 20, A, 20, A, 20, A, 20)
    assert need == (200 + 2600 + 2600) * 128 * 2
    assert gated(lib, **big) == -7 and gated(lib, **big, ws=A, bytes=need - 1) == -7
    assert gated(lib, **big, ws=p(0x100008), bytes=need) == -7
    assert gated(lib, **big, ws=A, bytes=need) == -4      # no device here


def test_workspace_sizes(lib):
    ws = lib.gemm_gated_workspace
    assert ws(F16, 256, 2560, 128, A, 128, A, 128, A, 128) == 0
    copy = 2560 * 128 * 2
    assert ws(F16, 256, 2560, 128, A, 128, ODD, 128, A, 128) == copy     # address
    assert ws(F16, 256, 2560, 128, A, 128, A, 132, A, 128) == copy       # rows apart
    assert ws(F16, 256, 2560, 127, A, 127, A, 127, A, 127) == 256 * 256 + 2 * copy
    assert ws(F16, 256, 2560, 130, A, 130, A, 130, A, 130) == (256 + 2 * 2560) * 192 * 2
    # few outputs: none, fewer with odd rows
    assert ws(F16, 256, 2500, 130, A, 130, A, 130, A, 130) == 0
    assert ws(F16, 256, 1000, 127, A, 127, A, 127, A, 127) == 0
    assert ws(F16, 256, 1001, 127, A, 127, A, 127, A, 127) == (256 + 2 * 1001) * 256
    assert ws(F16, 0, 512, 127, A, 127, A, 127, A, 127) == 0
    assert ws(7, 256, 2560, 127, A, 127, A, 127, A, 127) == 0
    bwd = lib.gemm_gated_bwd_workspace
    # dW: dG and dU, and X transposed
    assert bwd(F16, 256, 512, 128, A, 128, A, 128, A, 128, 0, 1) == 256 * 1024 * 2 + 128 * 256 * 2
    assert bwd(F16, 256, 520, 128, A, 128, A, 128, A, 128, 0, 1) == 256 * 1152 * 2 + 128 * 256 * 2
    # dX: the last 64 columns of dG and dU again where N is no multiple of 64,
    # copies of weights whose rows are not equally far apart, fp32 sums where K
    # (here N of both weights) is cut into ranges: one of 256 x 128 for each
    d, sums = 256 * 1152 * 2 + 256 * 256, 256 * 128 * 4
    dx = bwd(F16, 256, 520, 128, A, 128, A, 128, A, 128, 1, 0)
    assert dx > d and (dx - d) % sums == 0 and (dx - d) // sums <= 64
    apart = bwd(F16, 256, 520, 128, A, 128, A, 128, A, 136, 1, 0)
    assert apart == dx + 2 * (520 * 128 * 2)
    assert bwd(F16, 256, 512, 128, A, 128, A, 128, A, 136, 0, 1) == 256 * 1024 * 2 + 128 * 256 * 2
    assert bwd(F16, 256, 512, 128, A, 128, A, 128, A, 128, 0, 0) == 0
    # enough tiles: no ranges
    assert bwd(BF16, 4096, 16384, 4096, A, 4096, A, 4096, A, 4096, 1, 0) == 4096 * 32768 * 2
    x = lib.gemm_xent_workspace
    assert x(BF16, 0, 1000, 128, A, 128, A, 128) == 0
    assert x(BF16, 200, 0, 128, A, 128, A, 128) == 0
    assert x(BF16, 200, 1000, 128, A, 128, A, 128) == 200 * 16 * 8 + 1024
    assert x(BF16, 8192, 131072, 128, A, 128, A, 128) == 8192 * 1024 * 8 + 8192 * 4
    xb = lib.gemm_xent_bwd_workspace
    # dW alone: d and X transposed (and 256 bytes for the factor)
    assert xb(BF16, 4096, 1024, 128, A, 128, A, 128, 0, 1) == 4096 * (1024 + 128) * 2 + 256
    # pieces: far less than the logits' 2^30 bytes
    large = xb(BF16, 4096, 131072, 128, A, 128, A, 128, 1, 1)
    assert 256 << 20 < large < 512 << 20
    assert xb(BF16, 4096, 1024, 128, A, 128, A, 128, 0, 0) == 0
    # sizes past 32 bits
    assert bwd(BF16, 1 << 20, 1 << 14, 4096, A, 4096, A, 4096, A, 4096, 1, 1) == \
        (1 << 36) + (1 << 33)


def bwd(lib, type=F16, act=2, M=4, N=8, K=16, X=A, ldx=16, Wg=A, ldg=16, Wu=A, ldu=16, G=A, ldG=8,
        U=A, ldU=8, dH=A, lddh=8, dX=A, lddx=16, dWg=A, lddg=16, dWu=A, lddu=16, ws=None, bytes=0):
    return lib.gemm_gated_bwd(type, act, M, N, K, X, ldx, Wg, ldg, Wu, ldu, G, ldG, U, ldU, dH,
                              lddh, dX, lddx, dWg, lddg, dWu, lddu, ws, bytes, None)


def test_gated_bwd_refusals(lib):
    assert bwd(lib, M=-1) == -1 and bwd(lib, type=5) == -6 and bwd(lib, act=9) == -6
    for k in ("ldx", "ldg", "ldu", "lddx", "lddg", "lddu"):
        assert bwd(lib, **{k: 15}) == -2, k
    for k in ("ldG", "ldU", "lddh"):
        assert bwd(lib, **{k: 7}) == -2, k
    for k in ("X", "Wg", "Wu", "G", "U", "dH"):
        assert bwd(lib, **{k: None}) == -3, k
    assert bwd(lib) == -7
    # operands that the gradients asked for do not read may be missing
    assert bwd(lib, dX=None, Wg=None, Wu=None, ldg=0) == -7
    assert bwd(lib, dWg=None, dWu=None, X=None, ldx=0) == -7
    assert bwd(lib, dX=None, dWg=None, dWu=None) == 0
    assert bwd(lib, K=0, ldx=1, ldg=1, ldu=1, lddx=1, lddg=1, lddu=1) == 0


def w4(lib, type=F16, M=4, N=8, K=64, group=32, X=A, ldx=64, Wq=A, ldq=32, s=A, lds=2, z=A, ldz=2,
       bias=None, act=0, res=None, ldr=0, C=A, ldc=8):
    return lib.gemm_w4(type, M, N, K, group, X, ldx, Wq, ldq, s, lds, z, ldz, bias, act, res, ldr,
                       C, ldc, None)


def test_w4_refusals(lib):
    assert w4(lib) == -4     # valid: ends at the device check
    assert w4(lib, M=-1) == -1 and w4(lib, type=2) == -6 and w4(lib, act=3) == -6
    for g in (0, -32, 16, 48):
        assert w4(lib, group=g) == -6, g
    for k, v in (("ldx", 63), ("ldq", 31), ("lds", 1), ("ldz", 1), ("ldc", 7)):
        assert w4(lib, **{k: v}) == -2, k
    assert w4(lib, res=A, ldr=7) == -2
    assert w4(lib, K=65, ldx=65, ldq=32, lds=3, ldz=3) == -2     # 33 bytes a row
    for k in ("X", "Wq", "s", "C"):
        assert w4(lib, **{k: None}) == -3, k
    assert w4(lib, z=None, ldz=0) == -4
    assert w4(lib, K=0, X=None, Wq=None, s=None) == -4 and w4(lib, N=0, C=None, Wq=None) == 0


def test_xent_refusals(lib):
    def fwd(type=F16, M=4, N=8, K=16, X=A, ldx=16, W=A, ldw=16, t=A, loss=A, lse=A, ws=None, n=0):
        return lib.gemm_xent(type, M, N, K, X, ldx, W, ldw, t, -100, loss, lse, ws, n, None)

    assert fwd(M=-1) == -1 and fwd(type=2) == -6 and fwd(N=0) == -6
    assert fwd(ldx=15) == -2 and fwd(ldw=15) == -2
    for k in ("X", "W", "t", "loss", "lse"):
        assert fwd(**{k: None}) == -3, k
    assert fwd() == -7 and fwd(M=0, X=None, t=None) == 0

    def back(type=F16, M=4, N=8, K=16, X=A, ldx=16, W=A, ldw=16, t=A, lse=A, dl=A, dX=A, lddx=16,
             dW=A, lddw=16, ws=None, n=0):
        return lib.gemm_xent_bwd(type, M, N, K, X, ldx, W, ldw, t, -100, lse, dl, dX, lddx, dW,
                                 lddw, ws, n, None)

    assert back(K=-1) == -1 and back(type=2) == -6 and back(N=0) == -6
    for k in ("ldx", "ldw", "lddx", "lddw"):
        assert back(**{k: 15}) == -2, k
    for k in ("X", "W", "t", "lse", "dl"):
        assert back(**{k: None}) == -3, k
    assert back() == -7 and back(dX=None, dW=None) == 0
    assert back(M=0, X=None, W=None, t=None, lse=None, dl=None) == -7      # dW = 0 is still work
    need = lib.gemm_xent_bwd_workspace(F16, 4, 8, 16, A, 16, A, 16, 1, 1)
    assert back(ws=A, n=need - 1) == -7 and back(ws=A, n=need) == -4


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    h, b, i = torch.zeros(4, 64).half(), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4).long()
    f = torch.zeros(4)
    with pytest.raises(TypeError):
        dg.gemm_gated(h, h, h, h)                         # CPU tensors
    with pytest.raises(TypeError):
        dg.gemm_gated(h.float(), h, h, h)
    with pytest.raises(TypeError):
        dg.gemm_gated_bwd(h, h, h, h, h, h)
    with pytest.raises(TypeError):
        dg.gemm_w4(h, b, h, h)
    with pytest.raises((TypeError, ValueError)):
        dg.gemm_xent(h, h, i, f, f)
    with pytest.raises((TypeError, ValueError)):
        dg.gemm_xent_bwd(h, h, i, f, f)


def test_xent_bwd_without_rows_reads_no_operand(lib):
    """M == 0: dW = 0 takes neither X nor W (either may be null), so nothing is
    copied, whatever their alignment and sizes: the workspace is d, the factor
    and the transposed X (zeros), 128 rows of each."""
    ws = lib.gemm_xent_bwd_workspace
    assert ws(BF16, 0, 200, 100, None, 100, None, 100, 0, 1) == 128 * 256 * 2 + 256 + 128 * 128 * 2
    for N, K in ((1, 1), (100, 256), (200, 100), (131072, 4095), (1000, 4096)):
        size = ws(BF16, 0, N, K, A, K, A, K, 1, 1)
        assert size == ws(BF16, 0, N, K, ODD, K + 1, ODD, K + 3, 1, 1)
        Np, Kp = max(N, 128), max((K + 63) // 64 * 64, 128)
        assert size == 128 * ((Np + 63) // 64 * 64) * 2 + 256 + Kp * 128 * 2, (N, K)


def fake_gpu(*size_stride, dtype="float16"):
    """A GPU tensor without memory (none of these calls gets as far as its data)."""
    torch = pytest.importorskip("torch")
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    with fake.FakeTensorMode():
        return torch.empty_strided(*size_stride, device="cuda", dtype=getattr(torch, dtype))


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_binding_refuses_what_an_int_does_not_hold(lib):
    """Rows 2^32 + 64 elements apart or 2^32 + 2 of them would reach the C calls
    as 64 and 2."""
    far, small = fake_gpu((2, 64), (2 ** 32 + 64, 1)), fake_gpu((2, 64), (64, 1))
    many = fake_gpu((2 ** 32 + 2, 64), (64, 1))
    out = fake_gpu((2, 2), (2, 1))
    far_out = fake_gpu((2, 2), (2 ** 32 + 2, 1))
    t, f = fake_gpu((2,), (1,), dtype="int64"), fake_gpu((2,), (1,), dtype="float32")
    q = fake_gpu((2, 32), (2 ** 32 + 32, 1), dtype="uint8")
    s = fake_gpu((2, 2), (2, 1))
    calls = [
        lambda: dg.gemm_gated(far, small, small, out),
        lambda: dg.gemm_gated(small, small, far, out),
        lambda: dg.gemm_gated(small, small, small, far_out),
        lambda: dg.gemm_gated(small, many, many, fake_gpu((2, 2 ** 32 + 2), (2 ** 32 + 2, 1))),
        lambda: dg.gated_workspace_bytes(many, small, small),
        lambda: dg.gemm_gated_bwd(small, small, small, out, out, far_out),
        lambda: dg.gemm_w4(small, q, s, out, group=32),
        lambda: dg.gemm_w4(small, fake_gpu((2, 32), (32, 1), dtype="uint8"),
                           fake_gpu((2, 1), (1, 1)), out, group=2 ** 32 + 64),
        lambda: dg.gemm_xent(small, far, t, f, f),
        lambda: dg.gemm_xent(small, many, t, f, f),
        lambda: dg.gemm_xent_bwd(small, small, t, f, f, dX=far),
        lambda: dg.gemm_ex(far, small, out),
        lambda: dg.gemm_f16_nt(small, small, far_out),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()
            pytest.fail("call %d" % i)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_binding_refuses_a_strided_bias(lib):
    """A column of a matrix as the bias, [N, 1]: its values are not N in a row."""
    x, q, s = fake_gpu((2, 64), (64, 1)), fake_gpu((3, 32), (32, 1), dtype="uint8"), \
        fake_gpu((3, 2), (2, 1))
    out, w = fake_gpu((2, 3), (3, 1)), fake_gpu((3, 64), (64, 1))
    for size_stride in (((3, 1), (5, 1)), ((1, 3), (3, 2)), ((3,), (2,)), ((3,), (0,))):
        bias = fake_gpu(*size_stride)
        with pytest.raises(ValueError, match="contiguous"):
            dg.gemm_w4(x, q, s, out, group=32, bias=bias)
        with pytest.raises(ValueError, match="contiguous"):
            dg.gemm_ex(x, w, out, bias=bias)
