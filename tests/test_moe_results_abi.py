"""Refusals of the row calls that also zero the rows that no slot names: every
call below fails its checks on the host, or is an empty call, before anything is
launched, so no GPU is needed and the addresses are never used."""
import ctypes
import os

import pytest

from bit_gemm_quantize_b200 import _native

OK, INVALID, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
A, U = 0x10000, 0x10001
BIG = (1 << 31) - 1


def P(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from bit_gemm_quantize_b200 import build

        build.build()
    return _native.load()


def test_zeroed_row_call_refusals(lib):
    def di(x=A, dt=_native.BF16, T=4, H=64, ldx=64, sr=A, k=2, R=8, out=A):
        return lib.moe_dispatch_zeroed(P(x), dt, T, H, ldx, P(sr), k, R, P(out), None)

    def ba(x=A, ddt=_native.BF16, ldx=64, y=A, dt=_native.F16, R=8, H=64, ldy=64, sr=A, w=A, T=4, k=2, out=A, dw=A):
        return lib.moe_combine_backward_zeroed(P(x), ddt, ldx, P(y), dt, R, H, ldy, P(sr), P(w), T, k, P(out), P(dw),
                                               None)

    for f in (di, ba):
        for kw in (dict(T=-1), dict(k=0), dict(k=33), dict(H=0), dict(R=-1), dict(R=BIG + 1), dict(T=BIG), dict(ldx=63),
                   dict(R=9), dict(T=0)):  # more rows than slots are not cleared
            assert f(**kw) == SHAPE, (f, kw)
        assert f(T=0, R=0) == OK
        assert f(dt=_native.I32) == DTYPE
        for n in ("x", "out"):
            assert f(**{n: 0}) == INVALID and f(**{n: U}) == ALIGN, n
        assert f(sr=U) == ALIGN
    assert di(sr=0) == INVALID
    assert ba(sr=0, R=7) == SHAPE  # slot order needs every slot's row
    for n in ("y", "w", "dw"):
        assert ba(**{n: 0}) == INVALID and ba(**{n: U}) == ALIGN, n
