"""The operators between two products -- norm_quant, gated_norm_quant, linear --
against their restatement in numpy (between64.py), at the sizes where they can
go wrong: one token, rows wider than a CTA's registers, ragged M and K, strided
views, in-place residuals, zero and non-finite rows, other streams, graphs.
"""
import numpy as np
import pytest
import torch

import between64 as ref
from ternary_weight_bit_bitlinear_b200 import _lib, api, build, inputs

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    _lib.load()
    yield
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


def f32(t):
    return t.detach().float().cpu().numpy()


def rows(N, K, seed, dtype, pad=0, scale=1.0):
    """[N, K] view of a wider buffer (16-byte aligned rows), outliers among it."""
    x = inputs.activations(N, K + pad, seed, "cuda", outlier_frac=0.02) * scale
    return x.to(dtype)[:, :K]


def weight(K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")


def check_codes(got, want):
    xq, amax, xsum = got
    q, a, s = want
    assert np.array_equal(amax.cpu().numpy(), a, equal_nan=True)
    assert np.array_equal(xq.cpu().numpy(), q)
    assert np.array_equal(xsum.cpu().numpy(), s)


# ------------------------------------------------------------------ norm_quant

# one chunk; ragged; each CTA width at its limit and just past it; wider than
# any CTA's registers; the widest; many rows
NORM_SHAPES = [(1, 16), (3, 48), (1, 2560), (2, 4096), (2, 4112), (5, 8192), (2, 8208),
               (2, 16384), (2, 16400), (2, 32768), (2, 32784), (1, 131072), (700, 1040)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", NORM_SHAPES)
def test_norm_quant(N, K, dtype):
    x, res, w = rows(N, K, K + N, dtype), rows(N, K, K + N + 1, dtype, scale=3.0), weight(K, K)
    check_codes(api.norm_quant(x, w, eps=EPS), ref.norm_rows(f32(x), w.cpu().numpy(), EPS))
    h, *got = api.norm_quant(x, w, eps=EPS, residual=res)
    assert h.dtype == dtype
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    check_codes(got, ref.norm_rows(f32(h), w.cpu().numpy(), EPS))


# each register count of the kernels at its limit and just past it, in several
# rounds of the resident CTAs (a row's padding does not reach the next row)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1008, 1024, 1040, 2032, 2048, 2064, 2544, 2560, 2576, 4080, 4096,
                               6128, 6144, 6160, 8192, 8208, 12272, 12288, 12304, 65536, 65552])
def test_norm_quant_at_each_register_count(K, dtype):
    N = 2500 if K <= 2576 else 700 if K <= 12304 else 3
    x, res, w = rows(N, K, K, dtype), rows(N, K, K + 1, dtype, scale=3.0), weight(K, K)
    x[1::7] = 0.0
    x[2::11, K - 1] = float("inf")
    pick = torch.cat([torch.arange(0, min(N, 12)), torch.arange(max(N - 12, 0), N)]).unique().cuda()
    h, *got = api.norm_quant(x, w, eps=EPS, residual=res)
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    check_codes([g[pick] for g in got], ref.norm_rows(f32(h[pick]), w.cpu().numpy(), EPS))
    # the rows in another order: every row's codes follow it
    back = torch.arange(N - 1, -1, -1, device="cuda")
    again = api.norm_quant(h[back].contiguous(), w, eps=EPS)
    for g, o in zip(got, again):
        assert torch.equal(g[back].nan_to_num(-1.0) if g.is_floating_point() else g[back],
                           o.nan_to_num(-1.0) if o.is_floating_point() else o)
    gated = api.gated_norm_quant(x, res, w, activation="relu2", eps=EPS)
    a = np.maximum(f32(x[pick]), np.float32(0))
    with np.errstate(all="ignore"):
        v = a * a * f32(res[pick])
    check_codes([g[pick] for g in gated], ref.norm_rows(v, w.cpu().numpy(), EPS))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K,pad", [(1, 144, 16), (9, 2000, 48), (4, 40000, 80)])
def test_norm_quant_strided_and_in_place(N, K, pad, dtype):
    x, res, w = rows(N, K, 5, dtype, pad), rows(N, K, 6, dtype, pad), weight(K, 7)
    want_h = (x.float() + res.float()).to(dtype)
    want = ref.norm_rows(f32(want_h), w.cpu().numpy(), EPS)
    for place in ("new", "x", "residual", "view"):
        a, b = x.clone(memory_format=torch.preserve_format), res
        buf = torch.full((N, K + pad), 7.0, dtype=dtype, device="cuda")
        if place in ("x", "residual", "view"):     # rows inside a guarded buffer
            out = buf[:, :K]
            if place == "x":
                out.copy_(x)
                a = out
            if place == "residual":
                out.copy_(res)
                b = out
        else:
            out = None
        h, *got = api.norm_quant(a, w, eps=EPS, residual=b, h_out=out)
        assert torch.equal(h, want_h)
        check_codes(got, want)
        assert (buf[:, K:] == 7.0).all()           # nothing past the rows


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_quant_without_weight_or_norm(dtype):
    x = rows(6, 2064, 11, dtype)
    check_codes(api.norm_quant(x, eps=EPS), ref.norm_rows(f32(x), None, EPS))
    got = api.norm_quant(x, normalize=False)
    check_codes(got, ref.quantise(f32(x)))
    for g, q in zip(got, api.quant_act(x.float().contiguous())):   # the quantiser's own codes
        assert torch.equal(g, q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [64, 33024])
def test_norm_quant_special_rows(K, dtype):
    x = rows(7, K, 3, dtype).contiguous()
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x[0] = 0.0
    x[1, K - 1] = float("nan")
    x[2, 3] = float("inf")
    x[3] = big                                       # squares far above fp32
    x[4] = small / 16                                # subnormal: eps decides
    x[5] = 0.0
    x[5, K - 2] = -1.0
    for eps in (1e-5, 1e-30):
        got = api.norm_quant(x, eps=eps)
        check_codes(got, ref.norm_rows(f32(x), None, eps))
    xq, amax, xsum = got
    assert torch.isnan(amax[1:3]).all() and (xq[1:3] == 0).all() and (xsum[1:3] == 0).all()
    assert amax[0] == 0 and (xq[0] == 0).all()
    assert xq[5, K - 2] == -127


def test_norm_quant_nonfinite_weight_reaches_its_rows_only_as_nan():
    x, w = rows(2, 64, 1, torch.float32).contiguous(), weight(64, 2)
    w[5] = float("inf")
    xq, amax, _ = api.norm_quant(x, w)
    assert torch.isnan(amax).all() and (xq == 0).all()


def test_norm_quant_xsum_is_optional_and_no_rows_is_a_no_op():
    x = rows(3, 256, 4, torch.float32)
    xq = torch.empty(3, 256, dtype=torch.int8, device="cuda")
    amax = torch.empty(3, device="cuda")
    a = _lib.Norm(x.data_ptr(), None, None, None, xq.data_ptr(), amax.data_ptr(), None, 3, 256,
                  256, 0, 0, EPS, _lib.F32, 1)
    assert _lib.bitlinear_norm_quant(a) == _lib.OK
    q, am, _ = ref.norm_rows(f32(x), None, EPS)
    assert np.array_equal(xq.cpu().numpy(), q) and np.array_equal(amax.cpu().numpy(), am)
    xq, amax, xsum = api.norm_quant(x[:0])
    assert xq.shape == (0, 256) and amax.numel() == 0 and xsum.numel() == 0


# ------------------------------------------------------------ gated_norm_quant

GATED_SHAPES = [(1, 16), (2, 4112), (3, 6912), (1, 28672), (2, 32784), (300, 1040)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("N,K", GATED_SHAPES)
def test_gated_exact_activations(N, K, normalize, dtype):
    """relu, relu2 and none are single fp32 operations: bit for bit."""
    gu = rows(N, 2 * K, N + K, dtype)
    g, u = gu[:, :K], gu[:, K:]
    w = weight(K, K) if normalize else None
    for name in ("none", "relu", "relu2"):
        a = f32(g)
        if name != "none":
            a = np.maximum(a, np.float32(0))
        if name == "relu2":
            a = a * a
        with np.errstate(all="ignore"):
            h = a * f32(u)
        got = api.gated_norm_quant(g, u, w, eps=EPS, activation=name, normalize=normalize)
        check_codes(got, ref.norm_rows(h, None if w is None else w.cpu().numpy(), EPS,
                                       normalize))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("N,K", [(1, 28672), (33, 1040), (1, 32784)])
def test_gated_smooth_activations(N, K, name, normalize, dtype):
    """Transcendental activations: each code within half a step of the exact
    value plus what fp32 may be off by.  In half steps (U) of the row's
    largest |h|: e = act_error / U + 1 (the product) for h; the norm adds the
    sum's share (below e), r, two products: 3; the scale 127/amax and the
    product by it 2 more, and amax its own e + 3.  A code is at most 127, so
    it moves by at most 127 U (2 e + 8)."""
    g, u = rows(N, K, K, dtype).contiguous(), rows(N, K, K + 1, dtype).contiguous()
    w = weight(K, 9) if normalize else None
    xq, amax, xsum = api.gated_norm_quant(g, u, w, eps=EPS, activation=name, normalize=normalize)
    g64, u64 = f32(g).astype(np.float64), f32(u).astype(np.float64)
    a = ref.act64(g64, name)
    h = a * u64
    herr = ref.act_error(g64, name) * np.abs(u64) + ref.U * np.abs(h)
    scale = np.ones((N, 1))
    if normalize:
        scale = 1.0 / np.sqrt((h ** 2).mean(1, keepdims=True) + EPS)
        scale = scale * w.cpu().numpy().astype(np.float64)
    v, verr = h * scale, herr * np.abs(scale)
    if normalize:
        rel = np.sqrt((herr ** 2).sum(1) / (h ** 2).sum(1))[:, None]   # of the norm itself
        verr = verr + np.abs(v) * (rel + 3 * ref.U)
    top = np.abs(v).max(1)
    terr = verr.max(1)
    assert (np.abs(amax.cpu().numpy() - top) <= terr * 1.01).all()
    want = v * (127.0 / top)[:, None]
    slack = verr * (127.0 / top)[:, None] + np.abs(want) * (terr / top)[:, None] \
        + 3 * ref.U * np.abs(want)
    q = xq.cpu().numpy().astype(np.float64)
    assert (np.abs(q - want) <= 0.5 + slack * 1.01).all()
    assert np.array_equal(xsum.cpu().numpy(), q.sum(1).astype(np.int32))


def test_gated_special_rows():
    g, u = rows(4, 96, 1, torch.float32).contiguous(), rows(4, 96, 2, torch.float32).contiguous()
    g[0] = -1.0                                     # relu leaves nothing
    g[1, 0] = float("nan")
    u[2, 95] = float("-inf")
    g[2, 95] = 1.0
    xq, amax, xsum = api.gated_norm_quant(g, u, activation="relu")
    assert amax[0] == 0 and (xq[:3] == 0).all() and (xsum[:3] == 0).all()
    assert torch.isnan(amax[1:3]).all() and torch.isfinite(amax[3])


# ---------------------------------------------------------------------- linear

def product(M, K, N, seed):
    """(packed, alpha, xq, amax, xsum, exact acc [N, M])"""
    W = inputs.latent_weights(M, K, seed=seed, device="cuda")
    packed, alpha = api.pack_weights(W)
    x = inputs.activations(N, K, seed=seed + 1, device="cuda", outlier_frac=0.01)
    xq, amax, xsum = api.quant_act(x)
    acc = xq.cpu().numpy().astype(np.int64) @ ref.codes_of(packed, K).T
    return packed, alpha, xq, amax, xsum, acc


def check_linear(y, acc, alpha, amax, bias, name, residual, dtype):
    assert y.dtype == dtype
    want, err = ref.linear64(acc, alpha.item(), amax.cpu().numpy(),
                             None if bias is None else bias.cpu().numpy(), name,
                             None if residual is None else f32(residual), dtype)
    got = y.double().cpu().numpy()
    worst = (np.abs(got - want) / err).max()
    assert worst <= 1.0, worst


# every kernel's range of tokens, both sides of each limit
TOKENS = [1, 2, 16, 17, 32, 33, 64, 65, 128, 129, 257]
LINEAR_SHAPES = [(128, 128), (1, 16), (33, 80), (260, 2000), (517, 1040)]


@pytest.mark.parametrize("M,K", LINEAR_SHAPES)
@pytest.mark.parametrize("N", TOKENS)
def test_linear_without_epilogue_is_matmul(N, M, K):
    packed, alpha, xq, amax, xsum, acc = product(M, K, N, 100 + N + M)
    y = api.linear(packed, alpha, xq, amax, xsum)
    assert torch.equal(y, api.matmul(packed, alpha, xq, amax, xsum))
    check_linear(y, acc, alpha, amax, None, None, None, torch.float32)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(1, 517, 1040), (2, 260, 2000), (16, 128, 4096), (31, 77, 528),
                                   (63, 260, 528), (100, 300, 272), (129, 264, 144),
                                   (300, 517, 272)])
def test_linear_epilogue(N, M, K, dtype, name):
    packed, alpha, xq, amax, xsum, acc = product(M, K, N, N + M + K)
    bias = torch.randn(M, device="cuda")
    res = rows(N, M, 3, dtype, scale=2.0)
    for b, r in ((bias, res), (None, res), (bias, None)):
        y = api.linear(packed, alpha, xq, amax, xsum, bias=b, activation=name, residual=r,
                       out_dtype=dtype)
        check_linear(y, acc, alpha, amax, b, name, r, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,pad,off", [(260, 4, 0), (256, 64, 32), (77, 3, 1)])
@pytest.mark.parametrize("N", [1, 9, 40, 128, 200])
def test_linear_strided_and_in_place(N, M, pad, off, dtype):
    """y and residual as columns of wider buffers, of any alignment."""
    K = 400
    packed, alpha, xq, amax, xsum, acc = product(M, K, N, N + M)
    bias = torch.randn(M, device="cuda")
    buf = torch.full((N + 2, M + pad), 7.0, dtype=dtype, device="cuda")
    out = buf[1:N + 1, off:off + M]
    res = rows(N, M + pad, 4, dtype)[:, off:off + M]
    y = api.linear(packed, alpha, xq, amax, xsum, bias=bias, activation="relu", residual=res,
                   out=out)
    assert y.data_ptr() == out.data_ptr()
    check_linear(y, acc, alpha, amax, bias, "relu", res, dtype)
    guard = buf.clone()
    guard[1:N + 1, off:off + M] = 7.0
    assert (guard == 7.0).all()                    # nothing written around the view
    out.copy_(res)                                 # in place: the residual is the output
    z = api.linear(packed, alpha, xq, amax, xsum, bias=bias, activation="relu", residual=out,
                   out=out)
    check_linear(z, acc, alpha, amax, bias, "relu", res, dtype)


@pytest.mark.parametrize("N", [1, 5, 50, 150])
def test_linear_grouped(N):
    """More layers than one launch of the GEMM takes, of different sizes."""
    shapes = [(128, 256), (40, 528), (300, 272)] * 4
    parts = [product(M, K, N, 17 * i + N) for i, (M, K) in enumerate(shapes)]
    bias = [torch.randn(M, device="cuda") if i % 2 else None for i, (M, K) in enumerate(shapes)]
    acts = [ACTS[i % len(ACTS)] for i in range(len(shapes))]
    dts = [DTYPES[i % 3] for i in range(len(shapes))]
    res = [rows(N, M, i, dts[i]) if i % 3 else None for i, (M, K) in enumerate(shapes)]
    ys = api.linear_grouped([p[:2] for p in parts], [p[2] for p in parts], [p[3] for p in parts],
                            [p[4] for p in parts], bias=bias, activation=acts, residual=res,
                            out_dtype=dts)
    for p, y, b, a, r, d in zip(parts, ys, bias, acts, res, dts):
        check_linear(y, p[5], p[1], p[3], b, a, r, d)


@pytest.mark.parametrize("N", [1, 3])
def test_linear_many_layers(N):
    """More layers than one launch of either kernel takes."""
    packed, alpha, xq, amax, xsum, acc = product(40, 64, N, 5)
    ys = api.linear_grouped([(packed, alpha)] * 70, xq, amax, xsum)
    for y in ys:
        assert torch.equal(y, ys[0])
    check_linear(ys[0], acc, alpha, amax, None, None, None, torch.float32)


def test_linear_nan_rows_stay_where_they_are():
    for N in (2, 40, 200):
        packed, alpha, xq, amax, xsum, acc = product(128, 256, N, N)
        amax = amax.clone()
        amax[1] = float("nan")
        y = api.linear(packed, alpha, xq, amax, xsum, activation="relu")
        assert torch.isnan(y[1]).all()
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_linear_no_tokens():
    packed, alpha, xq, amax, xsum, _ = product(16, 64, 1, 1)
    assert api.linear(packed, alpha, xq[:0], amax[:0], xsum[:0]).shape == (0, 16)


def test_layer_with_bias():
    W = inputs.latent_weights(96, 160, seed=8, device="cuda")
    b = torch.randn(96, device="cuda")
    plain, biased = api.TernaryLinear.from_float(W), api.TernaryLinear.from_float(W, bias=b)
    for N in (1, 6):
        x = inputs.activations(N, 160, seed=N, device="cuda")
        assert torch.equal(biased(x), plain(x) + b)
        q = api.quant_act(x)
        assert torch.equal(biased.quantized(*q, residual=x[:, :96].contiguous()),
                           plain(x) + b + x[:, :96])


# -------------------------------------------------------------- used together

class Mlp:
    """norm -> gate, up -> gate * up, norm -> down onto the residual."""

    def __init__(self, H, F, seed):
        def lin(M, K, s):
            return api.pack_weights(inputs.latent_weights(M, K, seed=s, device="cuda"))
        self.gate, self.up, self.down = lin(F, H, seed), lin(F, H, seed + 1), lin(H, F, seed + 2)
        self.w1, self.w2 = weight(H, seed), weight(F, seed + 1)

    def __call__(self, x, res, stream=None):
        h, *q = api.norm_quant(x, self.w1, eps=EPS, residual=res, stream=stream)
        g, u = api.linear_grouped([self.gate, self.up], *q, out_dtype=x.dtype, stream=stream)
        q = api.gated_norm_quant(g, u, self.w2, eps=EPS, activation="relu2", stream=stream)
        return api.linear(*self.down, *q, residual=h, out=h, stream=stream)

    def plain(self, x, res):
        """The same in numpy, fp32 step by step."""
        def lin(layer, q, amax, K):
            acc = q.astype(np.int64) @ ref.codes_of(layer[0], K).T
            s = np.float32(layer[1].item()) * (amax / np.float32(127))
            return acc.astype(np.float32) * s[:, None]
        H, F = self.w1.numel(), self.w2.numel()
        h = x + res
        q, a, _ = ref.norm_rows(h, self.w1.cpu().numpy(), EPS)
        g, u = lin(self.gate, q, a, H), lin(self.up, q, a, H)
        r = np.maximum(g, np.float32(0))
        q, a, _ = ref.norm_rows(r * r * u, self.w2.cpu().numpy(), EPS)
        return lin(self.down, q, a, F) + h


@pytest.mark.parametrize("N", [1, 7, 48, 130, 300])
def test_mlp_block(N):
    """fp32 with squared ReLU: every step is defined to the bit, so the whole
    block is."""
    H, F = 272, 720
    mlp = Mlp(H, F, 40)
    x, res = rows(N, H, 1, torch.float32), rows(N, H, 2, torch.float32)
    y = mlp(x, res)
    assert np.array_equal(y.cpu().numpy(), mlp.plain(f32(x), f32(res)))


# one token and five: CUDA cores; 40 and 150: tensor cores
@pytest.mark.parametrize("N", [1, 5, 40, 150])
def test_mlp_block_on_another_stream_and_in_a_graph(N):
    mlp = Mlp(256, 704, 50)
    x, res = rows(N, 256, 1, torch.bfloat16), rows(N, 256, 2, torch.bfloat16)
    want = mlp(x, res)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = mlp(x, res, stream=s)                # handed over by argument
        with torch.cuda.stream(s):
            again = mlp(x, res)                    # and by context
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(again, want)
    assert torch.equal(mlp(x, res, stream=s.cuda_stream), want)    # a raw handle
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mlp(x, res)
    x2, res2 = rows(N, 256, 3, torch.bfloat16), rows(N, 256, 4, torch.bfloat16)
    want2 = mlp(x2, res2)
    x.copy_(x2)
    res.copy_(res2)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want2)


# ------------------------------------------- every split and round of linear

# Tokens x rows x K chosen so that the tensor-core path runs with one, two and
# four pairs per cluster, one tile and several per cluster, a last tile of a
# single token, clusters whose later pairs finish no token, K of one stage.
SPLITS = [(9, 12800, 16384), (17, 12800, 16384), (33, 11008, 4096), (65, 11008, 4096),
          (129, 2560, 2560), (200, 6912, 2560), (3, 19000, 4112), (40, 300, 28672),
          (130, 300, 28672), (16, 40000, 1040), (96, 40000, 1040), (300, 20000, 528),
          (257, 513, 16400), (64, 8192, 8192), (512, 2560, 6912), (5, 257, 131072),
          (1000, 1040, 1040), (2048, 640, 2560)]


@pytest.mark.parametrize("N,M,K", SPLITS)
def test_linear_equals_gemm_at_every_split(N, M, K):
    """The accumulators are integers: whatever the split, the product without
    an epilogue has the bits of the library's other GEMM."""
    packed, alpha = api.pack_weights(inputs.latent_weights(M, K, seed=N + M, device="cuda"))
    q = api.quant_act(inputs.activations(N, K, seed=K, device="cuda", outlier_frac=0.01))
    want = api.gemm(packed, alpha, *q)
    for _ in range(2):                              # the second finds warm plans and caches
        assert torch.equal(api.linear(packed, alpha, *q), want)
    b, r = torch.randn(M, device="cuda"), rows(N, M, 1, torch.bfloat16)
    y = api.linear(packed, alpha, *q, bias=b, activation="relu2", residual=r)
    z = torch.clamp_min(want + b, 0)
    assert torch.equal(y, (z * z + r.float()).to(torch.bfloat16))


def test_linear_equals_gemm_on_drawn_shapes():
    import random
    rng = random.Random(7)
    for i in range(40):
        N = int(round(2 ** rng.uniform(0, 9.5)))
        M = int(round(2 ** rng.uniform(0, 13.5)))
        K = 16 * int(round(2 ** rng.uniform(0, 9.5)))
        packed, alpha = api.pack_weights(inputs.latent_weights(M, K, seed=i, device="cuda"))
        q = api.quant_act(inputs.activations(N, K, seed=i + 99, device="cuda"))
        assert torch.equal(api.linear(packed, alpha, *q), api.gemm(packed, alpha, *q)), (N, M, K)


def test_linear_extreme_sums():
    """The largest sums in magnitude: all weights +1 (or -1) against all codes
    127 and -128 at the widest K, where the kernels' shifted sums just fit."""
    K, M = 131072, 40
    for c in (2, 0):                               # code + 1
        word = sum(c << (2 * i) for i in range(16))
        packed = torch.full((M, K // 16), word - (1 << 32 if word >> 31 else 0),
                            dtype=torch.int32, device="cuda")
        alpha = torch.ones(1, device="cuda")
        for code in (127, -128):
            for N in (1, 4, 20, 70, 140):
                xq = torch.full((N, K), code, dtype=torch.int8, device="cuda")
                amax = torch.full((N,), 127.0, device="cuda")
                xsum = torch.full((N,), code * K, dtype=torch.int32, device="cuda")
                y = api.linear(packed, alpha, xq, amax, xsum)
                assert (y == float((c - 1) * code * K)).all(), (c, code, N)


@pytest.mark.parametrize("N", [3, 40, 100, 300])
def test_linear_wait_limit(N):
    """A wait that runs out: the kernel returns, the error word says so, and the
    same call with the default limit is right again.  80 row blocks of 1024
    k-blocks, so that no cluster splits K: the accumulators take 100 us and more,
    the limit is 2 us (a wait looks at the clock every eighth try)."""
    M, K = 256 * 80, 131072
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    words = torch.from_numpy(np.random.RandomState(1).randint(0, 3, (64, 16)) @
                             (4 ** np.arange(16, dtype=np.int64)))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()
    packed = words[torch.randint(0, 64, (M, K // 16), generator=g, device="cuda")]
    alpha = torch.ones(1, device="cuda")
    q = api.quant_act(inputs.activations(N, K, seed=4, device="cuda"))
    want = api.gemm(packed, alpha, *q)
    torch.cuda.synchronize()
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK
    old = _lib.bitlinear_set_wait_limit(2000)
    try:
        api.linear(packed, alpha, *q)
        torch.cuda.synchronize()
    finally:
        _lib.bitlinear_set_wait_limit(old)
    assert _lib.bitlinear_device_error(clear=True) == _lib.ERR_DEVICE_TIMEOUT
    assert torch.equal(api.linear(packed, alpha, *q), want)
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


@pytest.mark.parametrize("N,K", [(400, 2048), (3, 28672), (40, 28672), (2, 65536)])
def test_norm_wait_limit(N, K):
    """With a limit of a nanosecond the row kernels' waits may run out or not;
    they return either way, and the default limit is right again."""
    x = rows(N, K, 9, torch.bfloat16).contiguous()
    want = ref.norm_rows(f32(x), None, EPS)
    old = _lib.bitlinear_set_wait_limit(1)
    try:
        api.norm_quant(x, eps=EPS)
        api.gated_norm_quant(x, x, eps=EPS)
        torch.cuda.synchronize()
    finally:
        _lib.bitlinear_set_wait_limit(old)
    assert _lib.bitlinear_device_error(clear=True) in (_lib.OK, _lib.ERR_DEVICE_TIMEOUT)
    check_codes(api.norm_quant(x, eps=EPS), want)
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


def test_norm_rows_beyond_32_bit_offsets():
    """Row offsets past 2^31 elements: views with a large row stride."""
    K, N, ld = 1024, 3, (1 << 30) + 64                # 2 * ld elements from first to last row
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    buf = torch.empty(2 * ld + K, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((N, K), (ld, 1))
    x.copy_(rows(N, K, 5, torch.bfloat16))
    w = weight(K, 6)
    check_codes(api.norm_quant(x, w, eps=EPS), ref.norm_rows(f32(x), w.cpu().numpy(), EPS))
    h, *got = api.norm_quant(x.contiguous(), w, eps=EPS, residual=x.contiguous(), h_out=x)
    check_codes(got, ref.norm_rows(f32(h), w.cpu().numpy(), EPS))
    assert h.data_ptr() == buf.data_ptr()
    packed, alpha, xq, amax, xsum, acc = product(40, 272, N, 8)
    for n in (1, 3):
        y = api.linear(packed, alpha, xq[:n], amax[:n], xsum[:n], out=x[:n, :40],
                       residual=x[:n, 40:80])
        check_linear(y, acc[:n], alpha, amax[:n], None, None, x[:n, 40:80], torch.bfloat16)


def test_norm_many_rows():
    """More rows than resident CTAs, several of each CTA's, all types."""
    for dtype in DTYPES:
        x, res, w = rows(5000, 272, 3, dtype), rows(5000, 272, 4, dtype), weight(272, 5)
        h, *got = api.norm_quant(x, w, eps=EPS, residual=res)
        check_codes(got, ref.norm_rows(f32(h), w.cpu().numpy(), EPS))


def test_two_streams_at_once():
    """Calls on two streams share no workspace: each gives what it gives alone."""
    mlps = [Mlp(512, 1408, 60), Mlp(512, 1408, 70)]
    ins = [(rows(64, 512, i, torch.bfloat16), rows(64, 512, i + 1, torch.bfloat16))
           for i in (1, 3)]
    want = [m(*i) for m, i in zip(mlps, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in mlps]
    for _ in range(10):
        got = [m(*i, stream=s) for m, i, s in zip(mlps, ins, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


FIRST_CALL = """
import torch
from ternary_weight_bit_bitlinear_b200 import api, inputs
packed, alpha = api.pack_weights(inputs.latent_weights(512, 1024, seed=1, device="cuda"))
x = inputs.activations(40, 1024, seed=2, device="cuda")
wide = inputs.activations(40, 20480, seed=3, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = api.norm_quant(x)
    ys = [api.linear(packed, alpha, *(t[:n] for t in q)) for n in (1, 3, 40)]
    z = api.gated_norm_quant(wide, wide)
g.replay()
torch.cuda.synchronize()
for got, want in zip(q, api.norm_quant(x)):
    assert torch.equal(got, want)
for n, y in zip((1, 3, 40), ys):
    assert torch.equal(y, api.matmul(packed, alpha, *(t[:n] for t in q)))
for got, want in zip(z, api.gated_norm_quant(wide, wide)):
    assert torch.equal(got, want)
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """What a call looks up once per device (attributes, occupancy) can be
    looked up while a graph is being captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]


def test_host_threads_at_once():
    """Two host threads, each on its own stream, of sizes that make the
    once-per-device caches change hands."""
    import threading
    packed, alpha = api.pack_weights(inputs.latent_weights(640, 1024, seed=1, device="cuda"))
    xs = [rows(400, 1024, i, torch.bfloat16).contiguous() for i in (1, 2)]
    want = [api.linear(packed, alpha, *api.norm_quant(x), out_dtype=torch.bfloat16) for x in xs]
    other = [api.norm_quant(x[:, :512 * (i + 1)].contiguous()) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                y = api.linear(packed, alpha, *api.norm_quant(xs[i]), out_dtype=torch.bfloat16)
                o = api.norm_quant(xs[i][:, :512 * (i + 1)].contiguous())
                s.synchronize()
                if not torch.equal(y, want[i]) or not all(map(torch.equal, o, other[i])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad
