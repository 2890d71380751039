"""bitlinear_linear_plan on the host: its refusals, and the calls that go to the
CUDA cores, which need no device."""
import ctypes

import pytest

from test_between_cpu import FAKE, linear
from ternary_weight_bit_bitlinear_b200 import _lib, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_refusals(L):
    t, p = ctypes.c_int(-1), ctypes.c_int(-1)

    def call(N=4, count=1, tokens=t, pairs=p, **kw):
        return L.bitlinear_linear_plan((_lib.LinearProblem * 1)(linear(**kw)), count, N, tokens,
                                       pairs)
    assert L.bitlinear_linear_plan(None, 1, 4, t, p) == _lib.ERR_INVALID_ARG
    assert call(count=0) == _lib.ERR_INVALID_ARG and call(N=0) == _lib.ERR_INVALID_ARG
    assert call(tokens=None) == _lib.ERR_INVALID_ARG and call(pairs=None) == _lib.ERR_INVALID_ARG
    assert call(K=200) == _lib.ERR_UNSUPPORTED_SHAPE
    assert call(N=1 << 31) == _lib.ERR_UNSUPPORTED_SHAPE
    assert call(ldy=127) == _lib.ERR_INVALID_ARG
    assert call(xq=FAKE + 4) == _lib.ERR_MISALIGNED
    assert (t.value, p.value) == (-1, -1)


def test_cuda_cores(L):
    arr = (_lib.LinearProblem * 2)(linear(), linear())
    for N in (1, 2, 8):
        assert _lib.bitlinear_linear_plan(arr, 2, N) == (0, 0)
    big = (_lib.LinearProblem * 1)(linear(M=8192, K=28672, ldy=8192, ldr=8192))
    assert _lib.bitlinear_linear_plan(big, 1, 2) == (0, 0)
