"""bitlinear_linear's activations over the whole range of their argument: far
below zero, where e^-v leaves fp32, at the infinities and at NaN.

Codes of zero make the product zero, so the bias is the activation's argument,
exactly.  Bounds, in half steps of fp32 (U = 2^-24), from the documented errors
(expf 1 unit in the last place, erff and tanhf 2, an approximate division 2; a
unit is 2 half steps):

With e = e^-|t| silu (t = v) and gelu_tanh (t = 2 sqrt(2/pi) (v + 0.044715 v^3))
are v e / (1 + e) below zero and v / (1 + e) above.
silu: 2 + 1 + 1 and the quotient, 4 approximate (16-bit outputs) or 1 + 2^-20
refined (fp32): 8, or 5.001, of |y|; the 9 and 6 of act_error.
gelu_tanh: 5 roundings of t more, at most 0.37 |v| each: below 10, or 7, of |v|;
the 11 and 7 of act_error.
Both keep |v| 2^-148 from e's last subnormal, which fp32's own last subnormal
covers up to |v| = 2 and the 2^-127 below for e subnormal (v < -87).
"""
import numpy as np
import pytest
import torch

import between64 as ref
from ternary_weight_bit_bitlinear_b200 import _lib, api, build

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = ["relu", "relu2", "silu", "gelu", "gelu_tanh"]
FAR = [-3.4e38, -1e38, -1e30, -1e19, -70000.0, -1000.0, -200.0, -150.0, -104.0, -100.0, -95.0,
       -88.8, -88.72, -88.5, -88.0, -87.5, -87.34, -87.0, -86.9, -45.0, -17.0, -9.0, -0.0, 0.0,
       1e-40, -1e-40, 9.0, 17.0, 45.0, 87.0, 88.8, 200.0, 1e19]
K = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    _lib.load()
    yield
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


def apply(values, N, name, dtype):
    """act(values) of every token, [N, M]."""
    M = values.numel()
    packed, alpha = api.pack_weights(torch.randn(M, K, device="cuda"))
    xq = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    return api.linear(packed, alpha, xq, torch.ones(N, device="cuda"),
                      torch.zeros(N, dtype=torch.int32, device="cuda"), bias=values,
                      activation=name, out_dtype=dtype)


# CUDA cores; tensor cores, whole blocks of rows and a ragged one
@pytest.mark.parametrize("N", [1, 2, 20, 70])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ACTS)
def test_whole_range(name, dtype, N):
    v = torch.cat([torch.tensor(FAR), torch.linspace(-110, 30, 2 * 317 + 1)]).cuda()
    v64 = v.double().cpu().numpy()
    want = ref.act64(v64, name)
    err = ref.act_error(v64, name, product=dtype != torch.float32)
    if dtype == torch.float32 and name == "silu":
        err = err + np.where(v64 < -88, np.abs(v64), 0) * 2.0 ** -127
    elif name in ("silu", "gelu_tanh"):
        err = (8 * ref.U * np.abs(want) if name == "silu" else 10 * ref.U * np.abs(v64)) \
            + np.abs(v64) * 2.0 ** -148
    fi = torch.finfo(dtype)
    with np.errstate(over="ignore"):
        bound = err * (1 + 2.0 ** -10)
        bound = bound + ref.half_step(dtype) * (np.abs(want) + bound) + fi.smallest_normal * fi.eps
    got = apply(v, N, name, dtype).double().cpu().numpy()
    limit = float(fi.max) * (1 + ref.half_step(dtype))        # from here on it rounds to inf
    inside = np.abs(want) + bound < limit
    assert inside.sum() > 600
    off = np.abs(got - want)[:, inside] / bound[inside]
    assert off.max() <= 1.0, (off.max(), v64[inside][off.max(0).argmax()])
    assert (got[:, np.abs(want) - bound > limit] == np.inf).all()


@pytest.mark.parametrize("N", [1, 20, 70])
@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan(dtype, N):
    """The formulas of the header at -inf, +inf and NaN, the same as
    gated_norm_quant's activations."""
    v = torch.tensor([float("-inf"), float("inf"), float("nan")] * 16, device="cuda")
    nan, inf = float("nan"), float("inf")
    want = {"relu": [0, inf, nan], "relu2": [0, inf, nan], "silu": [nan, inf, nan],
            "gelu": [nan, inf, nan], "gelu_tanh": [nan, inf, nan]}
    for name in ACTS:
        y = apply(v, N, name, dtype).float().cpu().numpy()
        assert np.array_equal(y, np.tile(np.float32(want[name] * 16), (N, 1)), equal_nan=True), name


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_16_bit_outputs_are_the_rounded_fp32_ones_almost_everywhere(name):
    """The approximate division moves a value by at most 8 (10) half steps of
    fp32, a 2^-13th (2^-12th) of a bf16 half step: it changes the rounding of
    few of them."""
    v = torch.randn(4096, device="cuda") * 3
    for N in (20, 70):
        y = apply(v, N, name, torch.float32)
        b = apply(v, N, name, torch.bfloat16)
        assert (b == y.to(torch.bfloat16)).float().mean() > 0.99
