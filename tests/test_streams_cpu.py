"""Which stream the torch-facing calls allocate on, on the CPU.

A call that is given a stream writes its outputs, its int8 codes and its
workspace there.  Their memory has to come from that stream's pool: memory of
the current stream's pool may still be in use by work pending there when the
call writes it, and a temporary goes back to the pool when the call returns,
before its stream has run.  Here the C entry points, the device and stream
contexts and torch's allocating calls are replaced by recorders.
"""
import contextlib

import pytest
import torch

from ternary_weight_bit_bitlinear_b200 import _lib, api, build

DEV = torch.device("cpu")
CURRENT = 0x11          # the handle of the current stream


class Stream:
    cuda_stream = 0x51
    device = DEV


class Record:
    """Active streams and devices, and what was active at each allocation and
    at each call of an entry point."""

    def __init__(self):
        self.streams, self.devices = [CURRENT], []
        self.allocated, self.called, self.set_devices = [], [], []

    def current(self, device=None):
        s = Stream()
        s.cuda_stream = self.streams[-1]
        return s

    def set(self, s):      # back to the one before, or on to another
        if len(self.streams) > 1 and self.streams[-2] == s.cuda_stream:
            self.streams.pop()
        else:
            self.streams.append(s.cuda_stream)

    @contextlib.contextmanager
    def device(self, d):
        self.devices.append(torch.device(d))
        yield
        self.devices.pop()


@pytest.fixture
def record(monkeypatch):
    build.build()
    _lib.load()
    r = Record()

    def of(h):
        s = Stream()
        s.cuda_stream = h
        return s

    def external(h, device=None):          # torch takes 0 for "none given": a new stream
        return of(h or 0xE0)

    def handle(s):                         # that a call given `s` launches on
        if s is None:
            return r.streams[-1]
        return getattr(s, "cuda_stream", s)

    def noting(fn):
        def f(*a, **kw):
            r.allocated.append(r.streams[-1])
            return fn(*a, **kw)
        return f

    def entry(name):
        def f(*a):
            r.called.append((name, r.devices[-1] if r.devices else None, handle(a[-1])))
            return _lib.OK
        return f

    monkeypatch.setattr(api, "_need", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: of(0))
    monkeypatch.setattr(torch.cuda, "current_stream", r.current)
    monkeypatch.setattr(torch.cuda, "set_stream", r.set)
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: r.set_devices.append(d))
    monkeypatch.setattr(torch.cuda, "device", r.device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # never the tensors' own
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", noting(torch.Tensor.new_empty))
    for name in [n for n in dir(_lib) if n.startswith("bitlinear_") and n not in
                 ("bitlinear_pack_workspace_bytes",)]:
        monkeypatch.setattr(_lib, name, entry(name))
    lib = _lib.load()

    class Calls:      # the loaded library, its launching entry points replaced
        bitlinear_linear = staticmethod(entry("bitlinear_linear"))

        def __getattr__(self, name):
            return getattr(lib, name)
    monkeypatch.setattr(_lib, "load", lambda *a: Calls())
    monkeypatch.setattr(_lib, "raw_stream", lambda s, i: handle(s))
    return r


def layer(bias):
    packed = torch.zeros((96, api.packed_row_words(160)), dtype=torch.int32)
    return api.TernaryLinear(packed, torch.ones(1), 160, 96, torch.zeros(96) if bias else None)


def codes(N, K=160):
    return (torch.zeros((N, K), dtype=torch.int8), torch.zeros(N),
            torch.zeros(N, dtype=torch.int32))


CALLS = {
    "layer, one token": lambda s: layer(False)(torch.zeros(1, 160), stream=s),
    "layer, six tokens": lambda s: layer(False)(torch.zeros(6, 160), stream=s),
    "layer with a bias": lambda s: layer(True)(torch.zeros(6, 160), stream=s),
    "layer, its codes given": lambda s: layer(True).quantized(*codes(6), stream=s),
    "pack_weights": lambda s: api.pack_weights(torch.zeros(96, 160), s),
    "quant_act": lambda s: api.quant_act(torch.zeros(6, 160), s),
    "quant_act_grouped": lambda s: api.quant_act_grouped([torch.zeros(6, 160)] * 2, s),
    "quant_act_per_tensor": lambda s: api.quant_act_per_tensor(torch.zeros(6, 160), s),
    "gemv": lambda s: api.gemv(layer(False).packed, torch.ones(1), *codes(2), with_acc=True,
                               stream=s),
    "gemm": lambda s: api.gemm(layer(False).packed, torch.ones(1), *codes(2), stream=s),
    "gemv_quant": lambda s: api.gemv_quant(layer(False).packed, torch.ones(1),
                                           torch.zeros(2, 160), with_acc=True, stream=s),
    "gemm_grouped": lambda s: api.gemm_grouped([(layer(False).packed, torch.ones(1))] * 2,
                                               *codes(2), with_acc=True, stream=s),
    "gemv_quant_grouped": lambda s: api.gemv_quant_grouped(
        [(layer(False).packed, torch.ones(1))] * 2, torch.zeros(2, 160), with_acc=True, stream=s),
    "tl2_from_packed": lambda s: api.tl2_from_packed(layer(False).packed, 160, s),
    "gemv_tl2": lambda s: api.gemv_tl2(torch.zeros((96, api.tl2_row_bytes(160)),
                                                   dtype=torch.uint8),
                                       torch.ones(1), *codes(2)[:2], with_acc=True, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_a_call_belongs_to_its_stream(record, name):
    class Other:                                        # another library's stream
        cuda_stream = 0x99
    for given in (Stream(), 0x77, 0, Other()):          # raw handles; 0: the default stream
        record.allocated.clear()
        record.called.clear()
        CALLS[name](given)
        want = getattr(given, "cuda_stream", given)
        assert record.called and record.allocated
        assert all(s == want for s in record.allocated), (record.allocated, want)
        assert all(s == want for _, _, s in record.called), (record.called, want)
        assert record.streams == [CURRENT]              # as it was before the call
        assert set(record.set_devices) == {-1}          # and the device


@pytest.mark.parametrize("name", sorted(CALLS))
def test_without_a_stream_nothing_changes_the_current_one(record, name):
    for given in (None, CURRENT):
        record.allocated.clear()
        CALLS[name](given)
        assert record.called and record.allocated and set(record.allocated) == {CURRENT}
        assert {s for _, _, s in record.called} == {CURRENT}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_calls_launch_with_the_device_of_their_tensors_current(record, name):
    """Another device may be current: the pointers are of the tensors' own."""
    for given in (None, Stream()):
        CALLS[name](given)
    assert record.called and all(d == DEV for _, d, _ in record.called), record.called


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_stream_of_another_device_is_refused(record, name):
    given = Stream()
    given.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](given)
    assert not record.called and record.streams == [CURRENT]
