"""Calls that are given a stream, on the device: the memory of their codes and
workspaces stays theirs until that stream has used it (tests/test_streams_cpu.py
shows where each call allocates)."""
import pytest
import torch

from ternary_weight_bit_bitlinear_b200 import _lib, api, build, inputs

pytestmark = pytest.mark.gpu

K, M = 1024, 640
SLEEP = 20_000_000      # cycles: about 10 ms of pending work in front of a call


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    _lib.load()
    yield
    assert _lib.bitlinear_device_error(clear=True) == _lib.OK


def same_sizes(N):
    """What the current stream may allocate next: the sizes of a call's codes,
    maxima, sums and outputs, filled with a mark."""
    return [torch.full((N, K), 7, dtype=torch.int8, device="cuda"),
            torch.full((N,), 7.0, device="cuda"),
            torch.full((N,), 7, dtype=torch.int32, device="cuda"),
            torch.full((N, M), 7.0, device="cuda")]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("N", [1, 6, 200])
def test_layer_on_a_busy_stream(N, bias):
    W = inputs.latent_weights(M, K, seed=3, device="cuda")
    layer = api.TernaryLinear.from_float(W, bias=torch.randn(M, device="cuda") if bias else None)
    xs = [inputs.activations(N, K, seed=i, device="cuda") for i in range(3)]
    want = [layer(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for given in (lambda s: s, lambda s: s.cuda_stream):
        got, marks = [], []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                torch.cuda._sleep(SLEEP)
            got.append(layer(x, stream=given(s)))        # pending behind the sleep
            marks.append(same_sizes(N))                  # the current stream runs on
        torch.cuda.synchronize()
        for g, w, m in zip(got, want, marks):
            assert torch.equal(g, w)
            assert all((t == 7).all() for t in m)        # nothing wrote into them later


def test_packing_on_a_busy_stream():
    W = inputs.latent_weights(M, K, seed=4, device="cuda")
    packed, alpha = api.pack_weights(W)
    nbytes = _lib.bitlinear_pack_workspace_bytes(M, K)
    x = inputs.activations(5, K, seed=5, device="cuda")
    want = api.quant_act_per_tensor(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    p, a = api.pack_weights(W, s)
    marks = [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")]
    got = api.quant_act_per_tensor(x, s)
    nbytes = _lib.load().bitlinear_quant_act_per_tensor_workspace_bytes()
    marks.append(torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(p, packed) and torch.equal(a, alpha)
    assert all(map(torch.equal, got, want))
    assert all((t == 7).all() for t in marks)


def test_handle_of_the_default_stream():
    """0 is a stream like another: a call given it from within another stream
    allocates and runs there."""
    x = inputs.activations(6, K, seed=6, device="cuda")
    W = inputs.latent_weights(M, K, seed=7, device="cuda")
    layer = api.TernaryLinear.from_float(W, bias=torch.randn(M, device="cuda"))
    want, codes = layer(x), api.norm_quant(x)
    default, s = torch.cuda.default_stream(), torch.cuda.Stream()
    assert default.cuda_stream == 0
    torch.cuda.synchronize()
    for given in (0, default):
        torch.cuda._sleep(SLEEP)
        with torch.cuda.stream(s):
            got, again = layer(x, stream=given), api.norm_quant(x, stream=given)
            marks = same_sizes(6)                        # on s, which runs on
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(map(torch.equal, again, codes))
        assert all((t == 7).all() for t in marks)
