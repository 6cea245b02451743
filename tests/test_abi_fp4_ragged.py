"""Host-side checks of the 4-bit and ragged entry points: bad arguments give the documented codes before
anything is launched (no GPU needed)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from fp8_block_scaled_grouped_amd import moe355
    if not os.path.exists(moe355.LIB_PATH):
        pytest.skip("libmoe355.so not built")
    return moe355.lib()


def _p(v=16):
    return ctypes.c_void_p(v)


def test_fp4_quant_codes(L):
    def quant(w=_p(), fp16=0, ld=256, rows=4, K=256, group=64, q=_p(), s=_p(), e8m0=0):
        return L.fp4_quant_groups(w, fp16, ld, rows, K, group, q, s, e8m0, None)

    def dequant(w=_p(), fp16=0, ld=256, rows=4, K=256, group=64, q=_p(), s=_p(), e8m0=0):
        return L.fp4_dequant_groups(q, s, e8m0, rows, K, group, w, fp16, ld, None)

    for f in (quant, dequant):
        assert f(group=48) == -2 and f(K=240, ld=240) == -2
        assert f(fp16=2) == -1 and f(e8m0=2) == -1 and f(ld=248) == -1 and f(rows=-1) == -1
        assert f(w=None) == -1 and f(q=None) == -1 and f(s=None) == -1
        assert f(w=_p(8)) == -3 and f(q=_p(8)) == -3 and f(ld=260) == -3 and f(s=_p(2)) == -3
        assert f(rows=0, w=None, q=None, s=None) == 0 and f(K=0, ld=0) == 0


def test_gemm_fp4_codes(L):
    def gemm(x=_p(), fp16=0, ldx=256, q=_p(), s=_p(), e8m0=0, group=64, M=4, N=33, K=256, c=_p(), ldc=33, ws=None, wsn=0):
        return L.gemm_fp4_groupscale(x, fp16, ldx, q, s, e8m0, group, M, N, K, c, ldc, ws, wsn, None)

    def grouped(x=_p(), fp16=0, ldx=256, q=_p(), s=_p(), e8m0=0, group=64, M=4, N=33, K=256, c=_p(), ldc=33, off=_p(), E=3):
        return L.grouped_gemm_fp4(x, fp16, ldx, q, s, e8m0, group, off, M, E, N, K, c, ldc, None)

    for f in (gemm, grouped):
        assert f(group=16) == -2 and f(K=264, ldx=264) == -2
        assert f(fp16=-1) == -1 and f(e8m0=3) == -1 and f(ldx=248) == -1 and f(ldc=32) == -1 and f(M=-1) == -1
        assert f(x=None) == -1 and f(q=None) == -1 and f(s=None) == -1 and f(c=None) == -1
        assert f(x=_p(8)) == -3 and f(q=_p(8)) == -3 and f(ldx=260) == -3 and f(c=_p(1)) == -3
        assert f(M=0, x=None, c=None) == 0 and f(N=0) == 0
        assert f(ldx=(1 << 21) + 8) == -2
    # a workspace that is given has to be large enough and aligned
    assert gemm(M=64, K=8192, ldx=8192, ws=_p(), wsn=64) == -1 and gemm(ws=_p(8)) == -3
    assert grouped(off=None) == -1 and grouped(off=_p(2)) == -3
    assert grouped(E=65536) == -2 and grouped(E=-1) == -1 and grouped(E=0, off=None) == 0


def test_ragged_codes(L):
    def fwd(a=_p(), fp16=0, lda=64, b=_p(), off=_p(), R=4, E=3, N=32, K=64, c=_p(), ldc=32):
        return L.grouped_gemm(a, fp16, lda, b, off, R, E, N, K, c, ldc, None)

    def dgrad(a=_p(), fp16=0, lda=64, b=_p(), off=_p(), R=4, E=3, N=64, K=32, c=_p(), ldc=32):
        return L.grouped_gemm_dgrad(a, fp16, lda, b, off, R, E, N, K, c, ldc, None)

    def wgrad(a=_p(), fp16=0, lda=64, b=_p(), off=_p(), R=4, E=3, N=64, K=32, c=_p(), ldc=32, out=1):
        return L.grouped_gemm_wgrad(a, fp16, lda, b, ldc, off, R, E, N, K, c, out, None)

    for f in (fwd, dgrad, wgrad):
        assert f(N=36, lda=64, ldc=40) == -2 and f(K=28) == -2 and f(E=65536) == -2
        assert f(lda=(1 << 21) + 8) == -2 and f(ldc=(1 << 21) + 8) == -2
        assert f(fp16=2) == -1 and f(lda=56) == -1 and f(ldc=24) == -1 and f(R=-1) == -1 and f(E=-1) == -1
        assert f(a=None) == -1 and f(b=None) == -1 and f(c=None) == -1 and f(off=None) == -1
        assert f(a=_p(8)) == -3 and f(b=_p(8)) == -3 and f(c=_p(8)) == -3 and f(lda=68) == -3 and f(ldc=36) == -3
        assert f(off=_p(2)) == -3
        assert f(E=0, off=None) == 0
    assert fwd(R=0, off=None) == 0 and dgrad(R=0) == 0 and wgrad(N=0) == 0 and wgrad(out=2) == -1


def test_gemm_fp4_workspace_query(L):
    from fp8_block_scaled_grouped_amd import moe355
    for M in (0, 1, 16):
        assert moe355.gemm_fp4_groupscale_workspace(M, 2048, 7168) == 0
    n = moe355.gemm_fp4_groupscale_workspace(64, 2048, 7168)
    assert n > 0 and n % (64 * 2048 * 4) == 0 and n // (64 * 2048 * 4) <= 7
    assert moe355.gemm_fp4_groupscale_workspace(64, 2048, 1024) == 0      # one run: nothing to split
    assert moe355.gemm_fp4_groupscale_workspace(64, 1 << 17, 7168) == 0   # columns enough for every CU
    for M, N, K, code in ((64, 2048, 48, -2), (-1, 2048, 64, -1)):
        with pytest.raises(moe355.Moe355Error) as e:
            moe355.gemm_fp4_groupscale_workspace(M, N, K)
        assert e.value.code == code
