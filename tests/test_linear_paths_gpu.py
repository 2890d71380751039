"""bitlinear_linear through every kernel it chooses from: the plan each case
takes is asked for, so that a case reaches what it is here for.

The CTA-pair kernel of long prompts (256 tokens a tile) is taken where there are
many row blocks and more than 128 tokens; its epilogue is run here with ragged
rows, odd strides, in place, all types and activations, and lists whose layers
differ.  The way out of a wait that ran out is run too, with one, two
and four pairs per tile.
"""
import numpy as np
import pytest
import torch

import between64 as ref
import test_between_gpu as between
from ternary_weight_bit_bitlinear_b200 import _lib, api, build, inputs

pytestmark = pytest.mark.gpu

DTYPES = between.DTYPES
ACTS = between.ACTS
FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    _lib.load()
    yield
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


def plan(shapes, N):
    """(tokens, pairs) of a call over layers of (M, K)."""
    arr = (_lib.LinearProblem * len(shapes))()
    for i, (M, K) in enumerate(shapes):
        arr[i] = _lib.LinearProblem(FAKE, FAKE, M, K, FAKE, FAKE, FAKE, None, None, FAKE, 0, M,
                                    _lib.F32, _lib.ACT_NONE)
    return _lib.bitlinear_linear_plan(arr, len(shapes), N)


def random_packed(M, K, seed):
    """Packed rows of random codes (K a multiple of 64), without latent weights."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    words = torch.from_numpy(np.random.RandomState(seed).randint(0, 3, (64, 16)) @
                             (4 ** np.arange(16, dtype=np.int64)))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()
    return words[torch.randint(0, 64, (M, K // 16), generator=g, device="cuda")]


def layer(M, K, N, seed):
    """(packed, alpha, xq, amax, xsum)"""
    packed, alpha = api.pack_weights(inputs.latent_weights(M, K, seed=seed, device="cuda"))
    x = inputs.activations(N, K, seed=seed + 1, device="cuda", outlier_frac=0.01)
    return (packed, alpha) + tuple(api.quant_act(x))


def columns(M, seed):
    """Rows of the weights to check in 64 bits: both ends, and some between."""
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.cat([torch.arange(0, 300), torch.randint(0, M, (600,), generator=g),
                      torch.arange(M - 600, M)]).cuda()


def check(y, p, K, pick, bias, name, residual, dtype):
    """y against the definition at the columns `pick`."""
    packed, alpha, xq, amax, _ = p
    codes = ref.codes_of(packed[pick], K)
    acc = (xq.cpu().numpy().astype(np.float64) @ codes.T.astype(np.float64)).astype(np.int64)
    between.check_linear(y[:, pick], acc, alpha, amax, None if bias is None else bias[pick], name,
                         None if residual is None else residual[:, pick], dtype)


def test_every_kernel_and_split_is_reached():
    """By the cases of this file and those that compare linear with gemm."""
    seen = {plan([(M, K)], N) for N, M, K in between.SPLITS}
    seen |= {plan([(M, K)], N) for M, K in between.LINEAR_SHAPES for N in between.TOKENS}
    seen |= {plan([(M, K)], N) for N, M, K in SPLITS}
    want = {(0, 0), (256, 1)} | {(BN, S) for BN in (32, 64, 128) for S in (1, 2, 4)}
    assert want <= seen, want - seen


# the tiles and splits that the comparison with gemm leaves out
SPLITS = [(24, 300, 512), (48, 300, 1040), (128, 300, 400), (60, 256 * 20, 16384),
          (100, 256 * 20, 16384), (24, 256 * 20, 16384), (64, 256 * 70, 8192),
          (100, 256 * 70, 8192), (100, 512, 65536), (100, 256 * 11, 16384)]


@pytest.mark.parametrize("N,M,K", SPLITS)
def test_linear_equals_gemm(N, M, K):
    p = layer(M, K, N, N + M)
    want = api.gemm(*p)
    assert torch.equal(api.linear(*p), want)
    r = between.rows(N, M, 1, torch.float16)
    y = api.linear(*p, activation="relu", residual=r)
    assert torch.equal(y, (torch.clamp_min(want, 0) + r.float()).to(torch.float16))


# ------------------------------------------------------------ the pair kernel

# whole blocks of rows, a ragged last block, an odd count; one tile of tokens
# with a single one past 128, two with a single one in the second
PAIR = [(129, 24000, 272), (257, 24013, 528), (300, 30001, 272)]


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", PAIR)
def test_pair_kernel_epilogue(N, M, K, dtype, name):
    assert plan([(M, K)], N) == (256, 1)
    p = layer(M, K, N, M)
    bias, res = torch.randn(M, device="cuda"), between.rows(N, M, 3, dtype, scale=2.0)
    pick = columns(M, N)
    for b, r in ((bias, res), (None, res), (bias, None)):
        y = api.linear(*p, bias=b, activation=name, residual=r, out_dtype=dtype)
        check(y, p, K, pick, b, name, r, dtype)
        if name in ("none", "relu", "relu2"):     # every output, to the bit
            z = api.gemm(*p) if b is None else api.gemm(*p) + b
            z = z if name == "none" else torch.clamp_min(z, 0)
            z = z * z if name == "relu2" else z
            assert torch.equal(y, (z if r is None else z + r.float()).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,pad,off", [(24000, 8, 0), (24000, 64, 32), (24013, 3, 1), (30001, 7, 0)])
def test_pair_kernel_strided_and_in_place(M, pad, off, dtype):
    """y and residual as columns of wider buffers, of any alignment."""
    N, K = 200, 272
    assert plan([(M, K)], N) == (256, 1)
    p = layer(M, K, N, M + 1)
    bias = torch.randn(M, device="cuda")
    buf = torch.full((N + 2, M + pad), 7.0, dtype=dtype, device="cuda")
    out = buf[1:N + 1, off:off + M]
    res = between.rows(N, M + pad, 4, dtype)[:, off:off + M]
    z = torch.clamp_min(api.gemm(*p) + bias, 0)
    want = (z + res.float()).to(dtype)
    y = api.linear(*p, bias=bias, activation="relu", residual=res, out=out)
    assert y.data_ptr() == out.data_ptr() and torch.equal(out, want)
    out.copy_(res)                                 # in place: the residual is the output
    api.linear(*p, bias=bias, activation="relu", residual=out, out=out)
    assert torch.equal(out, want)
    buf[1:N + 1, off:off + M] = 7.0
    assert (buf == 7.0).all()                      # nothing written around the view
    check(want, p, K, columns(M, 2), bias, "relu", res, dtype)


def test_pair_kernel_list_of_unlike_layers():
    """Layers are taken in the order of their K; each keeps its own epilogue."""
    N = 200
    shapes = [(24000, 272), (13001, 528), (40, 1040), (9000, 144), (513, 16)]
    assert plan(shapes, N) == (256, 1)
    ps = [layer(M, K, N, 31 * i) for i, (M, K) in enumerate(shapes)]
    bias = [torch.randn(M, device="cuda") if i % 2 else None for i, (M, K) in enumerate(shapes)]
    acts = ["relu2", "none", "silu", "gelu", "gelu_tanh"]
    dts = [torch.bfloat16, torch.float32, torch.float16, torch.float32, torch.bfloat16]
    res = [between.rows(N, M, i, dts[i]) if i % 3 != 1 else None
           for i, (M, K) in enumerate(shapes)]
    ys = api.linear_grouped([p[:2] for p in ps], *([p[j] for p in ps] for j in (2, 3, 4)),
                            bias=bias, activation=acts, residual=res, out_dtype=dts)
    for i, (p, y, (M, K)) in enumerate(zip(ps, ys, shapes)):
        pick = columns(M, i) if M > 1300 else torch.arange(M, device="cuda")
        check(y, p, K, pick, bias[i], acts[i], res[i], dts[i])


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_pair_kernel_far_arguments(dtype, name):
    """Codes of zero: the bias is the argument.  As the other kernels have it,
    to the bit."""
    N, M, K = 160, 24000, 64
    assert plan([(M, K)], N) == (256, 1)
    packed, alpha = random_packed(M, K, 1), torch.ones(1, device="cuda")
    v = torch.linspace(-120, 40, M, device="cuda")
    v[:8] = torch.tensor([float("-inf"), float("inf"), float("nan"), -1e38, 1e38, -0.0, -87.0,
                          -89.0])
    q = (torch.zeros(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"),
         torch.zeros(N, dtype=torch.int32, device="cuda"))
    y = api.linear(packed, alpha, *q, bias=v, activation=name, out_dtype=dtype)
    few = [t[:40] for t in q]
    want = api.linear(packed, alpha, *few, bias=v, activation=name, out_dtype=dtype)
    assert plan([(M, K)], 40)[0] in (32, 64)
    assert torch.equal(y.nan_to_num(-3.0), want[:1].nan_to_num(-3.0).expand_as(y))
    assert torch.isnan(y[:, [0, 2]]).all() and torch.isfinite(y[:, 5:]).all()


# --------------------------------------------------- waits that run out

# The limit is 2 us; a try of a wait takes a few, and the clock is looked at after
# each.  A tile's accumulators take 1024 k-blocks, 100 us, or that over the pairs;
# 40 k-blocks, 13 us, in the pair kernel, which long K does not choose.
LONG = 131072
WAITS = [(32, 1, 16, 256 * 74, LONG), (64, 1, 64, 256 * 74, LONG), (128, 1, 128, 256 * 74, LONG),
         (32, 2, 3, 256 * 20, LONG), (64, 2, 64, 256 * 20, LONG), (128, 2, 100, 256 * 20, LONG),
         (32, 4, 3, 200, LONG), (32, 4, 9, 256 * 11, LONG), (64, 4, 64, 256 * 11, LONG),
         (128, 4, 100, 256 * 11, LONG), (256, 1, 1024, 256 * 74, 5120)]


@pytest.mark.parametrize("tokens,pairs,N,M,K", WAITS)
def test_wait_limit(tokens, pairs, N, M, K):
    """The kernel winds down and returns, says so in the error word, writes
    nothing outside its output, and the same call is right again."""
    assert plan([(M, K)], N) == (tokens, pairs)
    packed, alpha = random_packed(M, K, 3), torch.ones(1, device="cuda")
    q = api.quant_act(inputs.activations(N, K, seed=4, device="cuda"))
    want = api.gemm(packed, alpha, *q)
    buf = torch.full((N + 2, M + 8), 7.0, dtype=torch.float32, device="cuda")
    out = buf[1:N + 1, 4:4 + M]
    torch.cuda.synchronize()
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK
    old = _lib.bitlinear_set_wait_limit(2000)
    try:
        api.linear(packed, alpha, *q, out=out)
        torch.cuda.synchronize()
    finally:
        _lib.bitlinear_set_wait_limit(old)
    assert _lib.bitlinear_device_error(clear=True) == _lib.ERR_DEVICE_TIMEOUT
    api.linear(packed, alpha, *q, out=out)
    assert torch.equal(out, want)
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK
    out.fill_(7.0)
    assert (buf == 7.0).all()
