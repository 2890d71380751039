"""Refusals of the operators between two products, and the arithmetic of their
test reference, on the CPU: every call below fails validation before the
library touches CUDA.
"""
import ctypes

import numpy as np
import pytest
import torch

import between64 as ref
from ternary_weight_bit_bitlinear_b200 import _lib, api, build

FAKE = 0x10000          # 16-byte aligned, never dereferenced
MISALIGNED = 0x10004
ODD = 0x10001


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def norm(**kw):
    a = dict(x=FAKE, residual=0, h=0, weight=FAKE, xq=FAKE, amax=FAKE, xsum=FAKE, N=4, K=256,
             ldx=256, ldr=256, ldh=256, eps=1e-5, dtype=_lib.BF16, normalize=1)
    a.update(kw)
    return _lib.Norm(*[a[n] for n, _ in _lib.Norm._fields_])


def gated(**kw):
    a = dict(gate=FAKE, up=FAKE, weight=FAKE, xq=FAKE, amax=FAKE, xsum=FAKE, N=4, K=256, ldg=256,
             ldu=256, eps=1e-5, dtype=_lib.BF16, activation=_lib.ACT_SILU, normalize=1)
    a.update(kw)
    return _lib.GatedNorm(*[a[n] for n, _ in _lib.GatedNorm._fields_])


def linear(**kw):
    a = dict(packed=FAKE, alpha=FAKE, M=128, K=256, xq=FAKE, amax=FAKE, xsum=FAKE, bias=FAKE,
             residual=FAKE, y=FAKE + 4096, ldr=128, ldy=128, dtype=_lib.F32,
             activation=_lib.ACT_NONE)
    a.update(kw)
    return _lib.LinearProblem(*[a[n] for n, _ in _lib.LinearProblem._fields_])


def test_norm_quant_argument_errors(L):
    f = L.bitlinear_norm_quant

    def call(**kw):
        return f(norm(**kw), None)

    assert f(None, None) == _lib.ERR_INVALID_ARG
    assert call(N=0) == _lib.OK
    assert call(N=-1) == _lib.ERR_INVALID_ARG
    for K in (0, 8, 250, 131072 + 16):
        assert call(K=K, ldx=K) == _lib.ERR_UNSUPPORTED_SHAPE
    assert call(N=1 << 31) == _lib.ERR_UNSUPPORTED_SHAPE
    for k in ("x", "xq", "amax"):
        assert call(**{k: 0}) == _lib.ERR_INVALID_ARG
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert call(eps=eps) == _lib.ERR_INVALID_ARG
        assert call(eps=eps, N=0) == _lib.ERR_INVALID_ARG
    assert call(normalize=0) == _lib.ERR_INVALID_ARG            # a weight without the norm
    assert call(dtype=3) == _lib.ERR_INVALID_ARG and call(dtype=-1) == _lib.ERR_INVALID_ARG
    assert call(residual=FAKE) == _lib.ERR_INVALID_ARG          # nowhere to put the sum
    assert call(h=FAKE) == _lib.ERR_INVALID_ARG
    assert call(ldx=255) == _lib.ERR_INVALID_ARG                # rows overlap
    assert call(residual=FAKE, h=FAKE + 16, ldr=128) == _lib.ERR_INVALID_ARG
    assert call(residual=FAKE, h=FAKE, ldh=512) == _lib.ERR_INVALID_ARG     # in place, other stride
    assert call(residual=FAKE + 16, h=FAKE, ldh=512) == _lib.ERR_INVALID_ARG
    assert call(ldx=260) == _lib.ERR_MISALIGNED                 # 520 bytes
    assert call(dtype=_lib.F32, ldx=258) == _lib.ERR_MISALIGNED
    for k in ("x", "weight", "xq"):
        assert call(**{k: MISALIGNED}) == _lib.ERR_MISALIGNED
    assert call(amax=ODD) == _lib.ERR_MISALIGNED and call(xsum=ODD) == _lib.ERR_MISALIGNED
    assert call(residual=MISALIGNED, h=FAKE) == _lib.ERR_MISALIGNED
    assert call(residual=FAKE, h=MISALIGNED) == _lib.ERR_MISALIGNED


def test_gated_norm_quant_argument_errors(L):
    f = L.bitlinear_gated_norm_quant

    def call(**kw):
        return f(gated(**kw), None)

    assert f(None, None) == _lib.ERR_INVALID_ARG
    assert call(N=0) == _lib.OK
    assert call(K=100) == _lib.ERR_UNSUPPORTED_SHAPE
    for k in ("gate", "up", "xq", "amax"):
        assert call(**{k: 0}) == _lib.ERR_INVALID_ARG
    assert call(activation=6) == _lib.ERR_INVALID_ARG
    assert call(activation=-1, N=0) == _lib.ERR_INVALID_ARG
    assert call(dtype=7) == _lib.ERR_INVALID_ARG
    assert call(eps=0.0) == _lib.ERR_INVALID_ARG
    assert call(normalize=0) == _lib.ERR_INVALID_ARG
    assert call(ldg=200) == _lib.ERR_INVALID_ARG and call(ldu=0) == _lib.ERR_INVALID_ARG
    assert call(ldu=260) == _lib.ERR_MISALIGNED
    assert call(gate=MISALIGNED) == _lib.ERR_MISALIGNED
    assert call(up=ODD) == _lib.ERR_MISALIGNED


def test_linear_argument_errors(L):
    f = L.bitlinear_linear
    P = _lib.LinearProblem

    def call(N=4, **kw):
        return f((P * 2)(linear(), linear(**kw)), 2, N, None)

    arr = (P * 1)(linear())
    assert f(arr, 0, 4, None) == _lib.OK and f(arr, 1, 0, None) == _lib.OK
    assert f(None, 1, 4, None) == _lib.ERR_INVALID_ARG
    assert f(arr, -1, 4, None) == _lib.ERR_INVALID_ARG
    assert f(arr, 1, -1, None) == _lib.ERR_INVALID_ARG
    assert call(N=1 << 31) == _lib.ERR_UNSUPPORTED_SHAPE
    for kw in (dict(K=200), dict(K=0), dict(M=0), dict(K=131072 + 16), dict(M=1 << 40)):
        assert call(**kw) == _lib.ERR_UNSUPPORTED_SHAPE
    for k in ("packed", "alpha", "xq", "amax", "xsum", "y"):
        assert call(**{k: 0}) == _lib.ERR_INVALID_ARG
    assert call(dtype=3) == _lib.ERR_INVALID_ARG
    assert call(activation=6) == _lib.ERR_INVALID_ARG
    assert call(ldy=127) == _lib.ERR_INVALID_ARG and call(ldr=127) == _lib.ERR_INVALID_ARG
    assert call(residual=FAKE, y=FAKE, ldr=256) == _lib.ERR_INVALID_ARG
    for k in ("packed", "xq"):
        assert call(**{k: MISALIGNED}) == _lib.ERR_MISALIGNED
    for k in ("alpha", "amax", "xsum", "bias"):
        assert call(**{k: FAKE + 2}) == _lib.ERR_MISALIGNED
    assert call(y=FAKE + 2) == _lib.ERR_MISALIGNED
    assert call(residual=ODD, dtype=_lib.BF16) == _lib.ERR_MISALIGNED


def test_python_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.norm_quant(x)
    with pytest.raises(TypeError):
        api.norm_quant([1.0])
    with pytest.raises(ValueError, match="CUDA"):
        api.gated_norm_quant(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear(torch.zeros(4, 4, dtype=torch.int32), torch.ones(1),
                   torch.zeros(1, 64, dtype=torch.int8), torch.ones(1),
                   torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="activation"):
        api._activation("tanh")
    with pytest.raises(ValueError, match="activation"):
        api._activation([])
    assert api.linear_grouped([], None, None, None) == []


@pytest.mark.gpu
def test_python_refusals_on_device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    x = torch.zeros(2, 64, device="cuda")
    with pytest.raises(TypeError):
        api.norm_quant(x.double())
    with pytest.raises(TypeError):
        api.norm_quant(x, residual=x.half())
    with pytest.raises(ValueError, match="shape"):
        api.norm_quant(x, residual=x[:1])
    with pytest.raises(ValueError, match="dense"):
        api.norm_quant(x.t())
    with pytest.raises(ValueError, match="overlap"):
        api.norm_quant(x[:1].expand(2, 64))
    with pytest.raises(ValueError, match="h_out"):
        api.norm_quant(x, h_out=x)
    with pytest.raises(ValueError, match="weight"):
        api.norm_quant(x, torch.ones(64, device="cuda"), normalize=False)
    with pytest.raises(ValueError, match="64"):
        api.norm_quant(x, torch.ones(65, device="cuda"))
    with pytest.raises(ValueError, match="device"):
        api._vector_ptr(torch.ones(64, device="cuda"), 64, torch.float32, "weight",
                        torch.device("cuda", 1))
    with pytest.raises(_lib.BitLinearError):
        api.norm_quant(x[:, 1:49])                    # rows not on 16 bytes
    with pytest.raises(_lib.BitLinearError):
        api.norm_quant(x, eps=0.0)
    with pytest.raises(ValueError, match="shape"):
        api.gated_norm_quant(x, x[:, :32])
    with pytest.raises(ValueError, match="activation"):
        api.gated_norm_quant(x, x, activation="swish")
    packed, alpha = api.pack_weights(torch.randn(32, 64, device="cuda"))
    q = api.quant_act(x)
    with pytest.raises(ValueError, match="32"):
        api.linear(packed, alpha, *q, bias=torch.ones(31, device="cuda"))
    with pytest.raises(TypeError):
        api.linear(packed, alpha, *q, out_dtype=torch.int8)
    with pytest.raises(TypeError):
        api.linear(packed, alpha, *q, residual=torch.zeros(2, 32, device="cuda"),
                   out_dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        api.linear(packed, alpha, *q, out=torch.zeros(2, 31, device="cuda"))
    with pytest.raises(ValueError, match="one per layer"):
        api.linear_grouped([(packed, alpha)] * 2, *q, bias=[None])


def test_reference_quantiser_rounds_half_to_even_and_zeroes_bad_rows():
    v = np.array([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0], [1, np.nan, 2, 3], [1, np.inf, 2, 3]],
                 np.float32)
    q, a, s = ref.quantise(v)
    assert q.tolist() == [[127, 0, 2, -2], [0] * 4, [0] * 4, [0] * 4]
    assert a[0] == 127 and a[1] == 0 and np.isnan(a[2:]).all() and s.tolist() == [127, 0, 0, 0]


def test_reference_codes_follow_the_layout():
    w = torch.zeros(1, 4, dtype=torch.int32)
    w[0, 0] = 0x55555555 + 1          # weight 0: field 2 -> +1
    w[0, 1] = 0x55555555 - (1 << 26)  # word 1, bit 26 = 8*3 + 2*1: weight 16 + 4 + 3
    c = ref.codes_of(w, 64)
    assert c[0, 0] == 1 and c[0, 16 + 7] == -1 and (c[0, 1:16] == 0).all()


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets of the mirrored structures, from a C compiler."""
    import os
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = ['#include <stdio.h>', '#include "bitlinear.h"', 'int main(void){']
    for name, cls in (("bitlinear_norm", _lib.Norm), ("bitlinear_gated_norm", _lib.GatedNorm),
                      ("bitlinear_linear_problem", _lib.LinearProblem)):
        src.append('printf("%%zu\\n", sizeof(%s));' % name)
        for f, _ in cls._fields_:
            src.append('printf("%%zu\\n", offsetof(%s, %s));' % (name, f))
    src.append("return 0;}")
    (tmp_path / "t.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", inc, str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for cls in (_lib.Norm, _lib.GatedNorm, _lib.LinearProblem):
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want
