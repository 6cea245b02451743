"""Host-side checks of the dispatch and FP8 ragged entry points: bad arguments give the documented codes before
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


def test_group_codes(L):
    n = ctypes.c_size_t(99)

    def size(T=8, k=2, E=4):
        return L.moe_group_workspace(T, k, E, ctypes.byref(n))

    assert size() == 0 and n.value == 0 and size(T=512, k=8) == 0 and n.value == 0
    assert size(T=513, k=8, E=256) == 0 and n.value == 2 * 256 * 4
    assert size(T=1 << 20, k=8, E=1024) == 0 and n.value == 256 * 1024 * 4
    assert size(T=-1) == -1 and size(k=0) == -1 and size(E=0) == -1 and size(E=1025) == -2 and size(T=1 << 28, k=8) == -2
    assert L.moe_group_workspace(1, 1, 1, None) == -1

    def group(ids=_p(), ld=2, T=8, k=2, E=4, off=_p(), rop=_p(), por=_p(), ws=None, wsn=0):
        return L.moe_group(ids, ld, T, k, E, off, rop, por, ws, wsn, None)

    assert group(ids=None) == -1 and group(off=None) == -1 and group(rop=None) == -1 and group(ld=1) == -1
    assert group(E=1025) == -2 and group(T=-1) == -1
    assert group(T=5000) == -1 and group(T=5000, ws=_p(), wsn=32) == -1 and group(T=5000, ws=_p(2), wsn=1 << 20) == -3
    assert group(ids=_p(2)) == -3 and group(off=_p(2)) == -3 and group(rop=_p(1)) == -3 and group(por=_p(1)) == -3


def test_rows_codes(L):
    def disp(x=_p(), dt=0, ldx=8, T=4, H=8, k=2, rop=_p(), R=8, rows=_p(), ldr=8):
        return L.moe_dispatch(x, dt, ldx, T, H, k, rop, R, rows, ldr, None)

    def comb(x=_p(), dt=0, ldx=8, T=4, H=8, k=2, rop=_p(), R=8, rows=_p(), ldr=8, w=None, ldw=2):
        return L.moe_combine(rows, dt, ldr, T, H, k, rop, R, w, ldw, x, ldx, None)

    def grad(x=_p(), dt=0, ldx=8, T=4, H=8, k=2, rop=_p(), R=8, rows=_p(), ldr=8, w=_p(), ldw=2, d=_p(), ldd=8, dw=_p()):
        return L.moe_combine_grad(x, ldx, rows, ldr, dt, T, H, k, rop, R, w, ldw, d, ldd, dw, None)

    for f in (disp, comb, grad):
        assert f(dt=4) == -1 and f(dt=-1) == -1 and f(T=-1) == -1 and f(H=-1) == -1 and f(k=0) == -1 and f(R=-1) == -1
        assert f(ldx=7) == -1 and f(ldr=7) == -1 and f(x=None) == -1 and f(rop=None) == -1 and f(rows=None) == -1
        assert f(x=_p(1)) == -3 and f(rows=_p(1)) == -3 and f(rop=_p(2)) == -3
        assert f(T=0, x=None, rop=None, rows=None) == 0
    assert comb(dt=3) == -1 and grad(dt=3) == -1 and comb(dt=2, x=_p(2)) == -3
    assert comb(w=_p(), ldw=1) == -1 and grad(ldw=1) == -1 and grad(w=None) == -1 and grad(ldd=7) == -1
    assert comb(w=_p(2)) == -3 and grad(w=_p(2)) == -3 and grad(d=_p(1)) == -3 and grad(dw=_p(2)) == -3
    assert grad(d=None, dw=None) == 0 and disp(R=0, rows=None) == 0 and disp(H=0, x=None) == 0
    assert disp(T=2 ** 31 - 1, H=65536, ldx=65536, ldr=65536) == -2 and grad(T=1 << 25) == -2


def test_quant_codes(L):
    def quant(x=_p(), f16=0, ldx=64, off=_p(), R=8, E=2, K=64, q=_p(), ldq=64, s=_p(), sm=1, sk=8, qt=_p(), ts=_p()):
        return L.fp8_quant_ragged(x, f16, ldx, off, R, E, K, q, ldq, s, sm, sk, qt, ts, None)

    assert quant(f16=2) == -1 and quant(R=-1) == -1 and quant(E=-1) == -1 and quant(K=-8) == -1 and quant(ldx=56) == -1 and quant(ldq=56) == -1
    assert quant(K=60) == -2 and quant(E=65536) == -2 and quant(K=1 << 30, ldx=1 << 30, ldq=1 << 30, R=1 << 20) == -2
    assert quant(x=None) == -1 and quant(q=None, qt=None) == -1 and quant(s=None) == -1 and quant(ts=None) == -1 and quant(off=None) == -1
    assert quant(sm=-1) == -1 and quant(sk=-1) == -1
    for bad in ({"x": _p(8)}, {"q": _p(8)}, {"qt": _p(8)}, {"ldx": 68}, {"ldq": 68}, {"ts": _p(1)}, {"off": _p(2)}):
        assert quant(**bad) == -3, bad
    assert quant(R=0, x=None) == 0 and quant(K=0, ldx=0) == 0 and quant(E=0) == 0

    def weights(w=_p(), f16=0, E=2, N=32, K=64, q=_p(), s=_p(), qt=_p(), ts=_p(), e8=1):
        return L.fp8_quant_128x128(w, f16, E, N, K, q, s, qt, ts, e8, None)

    assert weights(f16=-1) == -1 and weights(e8=2) == -1 and weights(E=-1) == -1 and weights(N=-1) == -1
    assert weights(K=60) == -2 and weights(N=24) == -2 and weights(E=4096, N=1 << 16, K=1 << 16) == -2
    assert weights(w=None) == -1 and weights(q=None) == -1 and weights(s=None) == -1 and weights(ts=None) == -1
    assert weights(w=_p(8)) == -3 and weights(q=_p(8)) == -3 and weights(qt=_p(8)) == -3 and weights(s=_p(2), e8=0) == -3
    assert weights(E=0, w=None) == 0 and weights(N=0) == 0
    n = ctypes.c_int64()
    assert L.fp8_ragged_blocks(1000, 5, ctypes.byref(n)) == 0 and n.value == 12
    assert L.fp8_ragged_blocks(-1, 5, ctypes.byref(n)) == -1 and L.fp8_ragged_blocks(1, 1, None) == -1


def test_product_codes(L):
    def gemm(x=_p(), xs=_p(), ldx=64, sm=1, sk=1, w=_p(), ws=_p(), e8=1, off=_p(), R=4, E=2, N=32, K=64, y=_p(), ldy=32, f16=0):
        return L.grouped_gemm_fp8(x, xs, ldx, sm, sk, w, ws, e8, off, R, E, N, K, y, ldy, f16, None)

    assert gemm(f16=2) == -1 and gemm(e8=2) == -1 and gemm(R=-1) == -1 and gemm(ldx=48) == -1 and gemm(ldy=24) == -1 and gemm(sm=-1) == -1
    assert gemm(K=56) == -2 and gemm(N=28) == -2 and gemm(E=65536) == -2 and gemm(ldx=(1 << 22) + 16) == -2
    for name in ("x", "xs", "w", "ws", "off", "y"):
        assert gemm(**{name: None}) == -1, name
    for bad in ({"x": _p(8)}, {"w": _p(8)}, {"y": _p(8)}, {"ldx": 72}, {"ldy": 36}, {"off": _p(2)}, {"xs": _p(2), "e8": 0}, {"ws": _p(2), "e8": 0}):
        assert gemm(**bad) == -3, bad
    assert gemm(R=0, x=None, y=None) == 0 and gemm(E=0) == 0 and gemm(N=0) == 0

    def wgrad(d=_p(), ds=_p(), x=_p(), xs=_p(), off=_p(), R=4, E=2, N=32, K=64, dw=_p(), out=2):
        return L.grouped_gemm_fp8_wgrad(d, ds, x, xs, off, R, E, N, K, dw, out, None)

    assert wgrad(out=3) == -1 and wgrad(R=-1) == -1 and wgrad(N=28) == -2 and wgrad(K=60) == -2 and wgrad(E=65536) == -2
    for name in ("d", "ds", "x", "xs", "off", "dw"):
        assert wgrad(**{name: None}) == -1, name
    for bad in ({"d": _p(8)}, {"x": _p(8)}, {"dw": _p(8)}, {"off": _p(2)}):
        assert wgrad(**bad) == -3, bad
    assert wgrad(E=0, dw=None) == 0 and wgrad(N=0) == 0 and wgrad(K=0) == 0


def test_tensors_off_the_gpu_are_refused(L):
    """Before anything is launched, also where there is no GPU."""
    import torch

    import fp8_block_scaled_grouped_amd as m
    ids, x, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 32), dtype=torch.bfloat16), torch.zeros((2, 16, 32), dtype=torch.bfloat16)
    off, q = torch.tensor([0, 2, 4], dtype=torch.int32), torch.zeros((4, 32), dtype=torch.uint8)
    for call in (lambda: m.moe_group(ids, 4), lambda: m.moe_dispatch(x, ids), lambda: m.moe_dispatch(x.float().requires_grad_(), ids),
                 lambda: m.moe_combine(x, ids), lambda: m.moe_combine_grad(x, x, ids, torch.ones(4, 2)), lambda: m.fp8_quant_ragged(x, off),
                 lambda: m.fp8_quant_128x128(w), lambda: m.grouped_linear_fp8(x, w, off),
                 lambda: m.grouped_gemm_fp8(q, torch.ones(4, 1), torch.zeros((2, 16, 32), dtype=torch.uint8), torch.ones(2, 1, 1), off),
                 lambda: m.grouped_gemm_fp8_wgrad(torch.zeros((2, 16, 128), dtype=torch.uint8), q, torch.zeros((2, 16, 128), dtype=torch.uint8), q, off, 4)):
        with pytest.raises(ValueError):
            call()
