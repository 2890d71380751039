"""Torch-facing calls of the ternary BitLinear path.

Each function checks dtype, device and contiguity, allocates its outputs with
torch (device memory is torch's job here) from the pool of the stream that
writes them, and hands raw pointers to one C entry point of libbitlinear.so.
All arithmetic runs in the CUDA kernels; nothing here falls back to the CPU.
"""
import torch

from . import _lib

# Largest token count the CUDA-core GEMV handles.
GEMV_MAX_TOKENS = 16

# Smallest token count for which `matmul` and `TernaryLinear` use the
# tensor-core GEMM.  Measured on B200 on an 8B-shaped layer (7 projections,
# one grouped launch, weights not in L2): GEMV 24.6 / 30.1 / 40.8 / 54.9 /
# 104 us and GEMM 24.5 / 24.6 / 24.6 / 24.3 / 24.3 us at N = 1 / 2 / 4 / 8 /
# 16; from fp32 activations, the fused quantise+GEMV 26.8 / 38.4 us at N = 1 /
# 2.  The two tie at one token; from two on, the GEMV's per-token dp4a work
# costs more than the GEMM's whole launch.
GEMM_MIN_TOKENS = 2


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _on(device, **tensors):
    """Every given tensor (None skipped) must sit on `device`: the kernels run
    on one GPU and dereference all pointers there."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, the weights on %s: all operands must share one "
                             "device" % (name, t.device, device))


def _launch(fn, name, dev, stream, *args):
    """fn(*args, raw stream) with `dev` current, whichever device was; raises on a
    status other than OK."""
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            status = fn(*args, _lib.raw_stream(stream, dev.index))
    else:
        status = fn(*args, _lib.raw_stream(stream, dev.index))
    if status != _lib.OK:
        raise _lib.BitLinearError(status, name)


def _handle(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _as_stream(stream, device):
    """torch's object for a stream, or for the handle of one.  (0 is the default
    stream's; ExternalStream takes it for no handle and makes a new stream.)"""
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError("the stream is of %s, the tensors are on %s" % (stream.device, device))
        return stream
    handle = _handle(stream)
    if handle == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


class _OnStream:
    """`stream` (an object or a handle) as the current one of `device`: what
    torch.cuda.stream does, with less host time (a layer called for another
    stream: 35 us against 42)."""

    def __init__(self, stream, device):
        self.stream, self.device = _as_stream(stream, device), device

    def __enter__(self):
        self.current = torch.cuda.current_device()
        self.before = torch.cuda.current_stream(self.device)
        torch.cuda.set_stream(self.stream)      # makes its device current too

    def __exit__(self, *error):
        torch.cuda.set_stream(self.before)
        if self.current != self.device.index:
            torch.cuda.set_device(self.current)


def _allocate(stream, like, *shapes):
    """Uninitialised tensors beside `like`, (shape, dtype) each, that belong to
    the stream that will write them: nothing pending elsewhere still uses their
    memory, and once dropped it is not handed out again before that stream is
    done with it.  Outputs, codes and workspaces all come from here."""
    if stream is None or _handle(stream) == _lib.raw_stream(None, like.device.index):
        return [like.new_empty(s, dtype=d) for s, d in shapes]
    with _OnStream(stream, like.device):
        return [like.new_empty(s, dtype=d) for s, d in shapes]


def _outputs(stream, like, N, M, out, with_acc):
    """y (`out` where it is given) and acc (None unless asked for) of a product."""
    if out is None:
        out, = _allocate(stream, like, ((N, M), torch.float32))
    return out, (_allocate(stream, like, ((N, M), torch.int32))[0] if with_acc else None)


def _check_out(out, N, M, device, name="out"):
    """A caller-supplied output must be fp32 [N, M], contiguous, on `device`
    (the kernels write N*M floats through its pointer)."""
    if out is None:
        return
    if not isinstance(out, torch.Tensor) or tuple(out.shape) != (N, M):
        raise ValueError("%s must have shape (%d, %d), got %s"
                         % (name, N, M, tuple(getattr(out, "shape", ()))))
    _need(out, torch.float32, name)
    _on(device, **{name: out})


def _check_token_vector(t, N, dtype, name):
    """amax / xsum: one entry per token, read for every n < N."""
    _need(t, dtype, name)
    if t.numel() != N:
        raise ValueError("%s must hold N = %d entries, got %d" % (name, N, t.numel()))


def packed_row_words(K):
    """Words per packed row: K/16 rounded up to a multiple of 4 (rows end on a
    16-byte boundary; the padding fields hold code 0)."""
    return 4 * ((K + 63) // 64)


def pack_weights(W, stream=None):
    """fp32 W[M,K] -> (packed int32 [M, packed_row_words(K)] holding the uint32
    words, alpha fp32 [1])."""
    _need(W, torch.float32, "W")
    M, K = W.shape
    nbytes = _lib.bitlinear_pack_workspace_bytes(M, K)
    packed, alpha, ws = _allocate(stream, W, ((M, packed_row_words(K)), torch.int32),
                                  (1, torch.float32), (nbytes, torch.uint8))
    _launch(_lib.bitlinear_pack_weights, "bitlinear_pack_weights", W.device, stream,
            W, M, K, packed, alpha, ws, nbytes)
    return packed, alpha


def quant_act(x, stream=None, with_sum=True):
    """fp32 x[N,K] -> (xq int8 [N,K], amax fp32 [N], xsum int32 [N] or None)."""
    _need(x, torch.float32, "x")
    N, K = x.shape
    xq, amax, *xsum = _allocate(stream, x, ((N, K), torch.int8), (N, torch.float32),
                                *(((N, torch.int32),) if with_sum else ()))
    xsum = xsum[0] if with_sum else None
    _launch(_lib.bitlinear_quant_act, "bitlinear_quant_act", x.device, stream,
            x, N, K, xq, amax, xsum)
    return xq, amax, xsum


def quant_act_per_tensor(x, stream=None):
    """Per-tensor variant: one absmax over all of x; amax[n] holds it for every n."""
    _need(x, torch.float32, "x")
    N, K = x.shape
    nbytes = _lib.load().bitlinear_quant_act_per_tensor_workspace_bytes()
    xq, amax, xsum, ws = _allocate(stream, x, ((N, K), torch.int8), (N, torch.float32),
                                   (N, torch.int32), (nbytes, torch.uint8))
    _launch(_lib.bitlinear_quant_act_per_tensor, "bitlinear_quant_act_per_tensor", x.device,
            stream, x, N, K, xq, amax, xsum, ws, nbytes)
    return xq, amax, xsum


def quant_act_grouped(xs, stream=None):
    """Quantise several fp32 activation matrices in one launch; returns a list
    of (xq, amax, xsum)."""
    xs = list(xs)
    outs, entries = [], []
    for x in xs:
        _need(x, torch.float32, "x")
        if x.device != xs[0].device:
            raise ValueError("all activations of a call must share one device")
        N, K = x.shape
        o = tuple(_allocate(stream, x, ((N, K), torch.int8), (N, torch.float32),
                            (N, torch.int32)))
        outs.append(o)
        entries.append((x,) + o)
    if entries:
        _launch(_lib.bitlinear_quant_act_grouped, "bitlinear_quant_act_grouped", xs[0].device,
                stream, _lib.make_acts(entries), len(entries))
    return outs


def _matmul(fn, name, packed, alpha, xq, amax, xsum, M, with_acc, stream, out=None):
    _need(packed, torch.int32, "packed")
    _need(alpha, torch.float32, "alpha")
    _need(xq, torch.int8, "xq")
    N, K = xq.shape
    _check_token_vector(amax, N, torch.float32, "amax")
    _check_token_vector(xsum, N, torch.int32, "xsum")
    if packed.shape != (M, packed_row_words(K)):
        raise ValueError("packed must be [M, packed_row_words(K)] = [%d, %d], got %s"
                         % (M, packed_row_words(K), tuple(packed.shape)))
    dev = packed.device
    _on(dev, alpha=alpha, xq=xq, amax=amax, xsum=xsum)
    _check_out(out, N, M, dev)
    y, acc = _outputs(stream, packed, N, M, out, with_acc)
    with torch.cuda.device(dev):
        _lib.check(fn(packed, alpha, M, K, xq, amax, xsum, N, y, acc, stream), name)
    return (y, acc) if with_acc else y


def gemv(packed, alpha, xq, amax, xsum, M=None, with_acc=False, stream=None, out=None):
    """Decode GEMV (N <= 16): y[N,M] fp32 (and int32 acc if with_acc)."""
    M = packed.shape[0] if M is None else M
    return _matmul(_lib.bitlinear_gemv, "bitlinear_gemv", packed, alpha, xq, amax, xsum, M,
                   with_acc, stream, out)


def _grouped(fn, name, layers, xq, amax, xsum, with_acc, stream, outs):
    n = len(layers)
    xqs = xq if isinstance(xq, (list, tuple)) else [xq] * n
    amaxs = amax if isinstance(amax, (list, tuple)) else [amax] * n
    xsums = xsum if isinstance(xsum, (list, tuple)) else [xsum] * n
    if not (len(xqs) == len(amaxs) == len(xsums) == n) or (outs is not None and len(outs) != n):
        raise ValueError("one xq, amax, xsum (and out) per layer, or one for all")
    N = xqs[0].shape[0]
    dev = layers[0][0].device if n else None
    ys, accs, entries = [], [], []
    for i, (packed, alpha) in enumerate(layers):
        _need(packed, torch.int32, "packed")
        _need(alpha, torch.float32, "alpha")
        _need(xqs[i], torch.int8, "xq")
        _check_token_vector(amaxs[i], N, torch.float32, "amax")
        _check_token_vector(xsums[i], N, torch.int32, "xsum")
        M, K = packed.shape[0], xqs[i].shape[1]
        if xqs[i].shape[0] != N or packed.shape[1] != packed_row_words(K):
            raise ValueError("layer %d: packed [M, packed_row_words(K)] must match xq [N, K];"
                             " N shared" % i)
        _on(dev, packed=packed, alpha=alpha, xq=xqs[i], amax=amaxs[i], xsum=xsums[i])
        if outs is not None:
            _check_out(outs[i], N, M, dev, "outs[%d]" % i)
        y, acc = _outputs(stream, packed, N, M, None if outs is None else outs[i], with_acc)
        ys.append(y)
        accs.append(acc)
        entries.append((packed, alpha, M, K, xqs[i], amaxs[i], xsums[i], y, acc))
    arr = _lib.make_problems(entries)
    if n:
        with torch.cuda.device(dev):
            _lib.check(fn(arr, n, N, stream), name)
    return (ys, accs) if with_acc else ys


def gemv_grouped(layers, xq, amax, xsum, with_acc=False, stream=None, outs=None):
    """One grouped decode call over several layers sharing the token count.
    layers: list of (packed, alpha); xq/amax/xsum: one tensor for all layers or
    a list with one entry per layer (K may differ between layers).  Returns a
    list of y (and of acc)."""
    return _grouped(_lib.bitlinear_gemv_grouped, "bitlinear_gemv_grouped", layers, xq, amax,
                    xsum, with_acc, stream, outs)


def gemm_grouped(layers, xq, amax, xsum, with_acc=False, stream=None, outs=None):
    """Tensor-core GEMM over several layers in one persistent launch; same
    arguments as gemv_grouped."""
    return _grouped(_lib.bitlinear_gemm_grouped, "bitlinear_gemm_grouped", layers, xq, amax,
                    xsum, with_acc, stream, outs)


def gemm(packed, alpha, xq, amax, xsum, M=None, with_acc=False, stream=None, out=None):
    """Tensor-core GEMM (any N and M): y[N,M] fp32 (and int32 acc)."""
    M = packed.shape[0] if M is None else M
    return _matmul(_lib.bitlinear_gemm, "bitlinear_gemm", packed, alpha, xq, amax, xsum, M,
                   with_acc, stream, out)


def matmul(packed, alpha, xq, amax, xsum, M=None, with_acc=False, stream=None, out=None):
    """GEMV below GEMM_MIN_TOKENS tokens, else the tensor-core GEMM."""
    M = packed.shape[0] if M is None else M
    if xq.shape[0] < GEMM_MIN_TOKENS:
        return gemv(packed, alpha, xq, amax, xsum, M, with_acc, stream, out)
    return gemm(packed, alpha, xq, amax, xsum, M, with_acc, stream, out)


# Shared-memory bound of the fused decode kernel: tokens x K rounded up to 512.
GEMV_QUANT_MAX_BYTES = 65536


def gemv_quant_fits(N, K):
    """Whether the fused quantise+GEMV kernel takes N tokens of width K."""
    return 1 <= N <= GEMV_MAX_TOKENS and N * (-(-K // 512) * 512) <= GEMV_QUANT_MAX_BYTES


def use_fused_decode(N, K):
    """TernaryLinear's choice: the fused kernel below the GEMM crossover."""
    return N < GEMM_MIN_TOKENS and gemv_quant_fits(N, K)


def gemv_quant(packed, alpha, x, M=None, with_acc=False, stream=None, out=None):
    """Decode GEMV straight from fp32 activations x[N,K] (N <= 16): the kernel
    quantises x per token itself.  Same y (and acc) as quant_act + gemv."""
    _need(packed, torch.int32, "packed")
    _need(alpha, torch.float32, "alpha")
    _need(x, torch.float32, "x")
    M = packed.shape[0] if M is None else M
    N, K = x.shape
    if packed.shape != (M, packed_row_words(K)):
        raise ValueError("packed must be [M, packed_row_words(K)] = [%d, %d], got %s"
                         % (M, packed_row_words(K), tuple(packed.shape)))
    dev = packed.device
    _on(dev, alpha=alpha, x=x)
    _check_out(out, N, M, dev)
    y, acc = _outputs(stream, packed, N, M, out, with_acc)
    with torch.cuda.device(dev):
        _lib.check(_lib.bitlinear_gemv_quant(packed, alpha, M, K, x, N, y, acc, stream),
                   "bitlinear_gemv_quant")
    return (y, acc) if with_acc else y


def gemv_quant_grouped(layers, x, with_acc=False, stream=None, outs=None):
    """Fused decode over several layers in one launch.  layers: list of
    (packed, alpha); x: one fp32 tensor [N,K] for all layers or a list with
    one per layer.  Layers that share an input should pass the same tensor and
    be adjacent, so that the kernel quantises it once for the rows it streams.
    Returns a list of y (and of acc)."""
    n = len(layers)
    xs = x if isinstance(x, (list, tuple)) else [x] * n
    if len(xs) != n or (outs is not None and len(outs) != n):
        raise ValueError("one x (and out) per layer, or one x for all")
    N = xs[0].shape[0]
    dev = layers[0][0].device if n else None
    ys, accs, entries = [], [], []
    for i, (packed, alpha) in enumerate(layers):
        _need(packed, torch.int32, "packed")
        _need(alpha, torch.float32, "alpha")
        _need(xs[i], torch.float32, "x")
        M, K = packed.shape[0], xs[i].shape[1]
        if xs[i].shape[0] != N or packed.shape[1] != packed_row_words(K):
            raise ValueError("layer %d: packed [M, packed_row_words(K)] must match x [N, K];"
                             " N shared" % i)
        _on(dev, packed=packed, alpha=alpha, x=xs[i])
        if outs is not None:
            _check_out(outs[i], N, M, dev, "outs[%d]" % i)
        y, acc = _outputs(stream, packed, N, M, None if outs is None else outs[i], with_acc)
        ys.append(y)
        accs.append(acc)
        entries.append((packed, alpha, M, K, xs[i], y, acc))
    arr = _lib.make_fused_problems(entries)
    if n:
        with torch.cuda.device(dev):
            _lib.check(_lib.bitlinear_gemv_quant_grouped(arr, n, N, stream),
                       "bitlinear_gemv_quant_grouped")
    return (ys, accs) if with_acc else ys


def tl2_row_bytes(K):
    """Bytes of one TL2-style row (5 bits per three weights, see include/bitlinear.h)."""
    n = _lib.load().bitlinear_tl2_row_bytes(int(K))
    if n == 0:
        raise ValueError("K must be a positive multiple of 16, at most 131072")
    return n


def tl2_from_packed(packed, K, stream=None):
    """Re-encode 2-bit packed weights [M, packed_row_words(K)] as TL2-style
    rows: uint8 [M, tl2_row_bytes(K)]."""
    _need(packed, torch.int32, "packed")
    M = packed.shape[0]
    if packed.shape[1] != packed_row_words(K):
        raise ValueError("packed must be [M, packed_row_words(K)]")
    out, = _allocate(stream, packed, ((M, tl2_row_bytes(K)), torch.uint8))
    _launch(_lib.bitlinear_tl2_from_packed, "bitlinear_tl2_from_packed", packed.device, stream,
            packed, M, K, out)
    return out


def gemv_tl2(tl2, alpha, xq, amax, M=None, with_acc=False, stream=None, out=None):
    """Decode GEMV over TL2-style rows (N <= 16): same y (and acc) as gemv."""
    _need(tl2, torch.uint8, "tl2")
    _need(alpha, torch.float32, "alpha")
    _need(xq, torch.int8, "xq")
    M = tl2.shape[0] if M is None else M
    N, K = xq.shape
    _check_token_vector(amax, N, torch.float32, "amax")
    if tl2.shape != (M, tl2_row_bytes(K)):
        raise ValueError("tl2 must be [M, tl2_row_bytes(K)] = [%d, %d]" % (M, tl2_row_bytes(K)))
    dev = tl2.device
    _on(dev, alpha=alpha, xq=xq, amax=amax)
    _check_out(out, N, M, dev)
    y, acc = _outputs(stream, tl2, N, M, out, with_acc)
    with torch.cuda.device(dev):
        _lib.check(_lib.bitlinear_gemv_tl2(tl2, alpha, M, K, xq, amax, N, y, acc, stream),
                   "bitlinear_gemv_tl2")
    return (y, acc) if with_acc else y


# ------------------------------------------------ between two products

# Element types of activation matrices in norm_quant, gated_norm_quant and linear.
ACT_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}

ACTIVATIONS = {None: _lib.ACT_NONE, "none": _lib.ACT_NONE, "relu": _lib.ACT_RELU,
               "relu2": _lib.ACT_RELU2, "silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU,
               "gelu_tanh": _lib.ACT_GELU_TANH}


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError("activation must be one of %s, got %r"
                         % (sorted(k for k in ACTIVATIONS if k), name)) from None


# The calls below run between the products of a decoded token, where the host's
# time per call counts: each check first asks, in one expression, whether all is
# well, and works out what is wrong only if it is not.

def _need_rows(t, name, shape=None, dtype=None):
    """An activation matrix [N, K] of a known type whose rows are dense (the
    row stride is free).  Returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if t.dtype not in ACT_DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s"
                        % (name, dtype or "float32, bfloat16 or float16", t.dtype))
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError("%s must have shape %s, got %s"
                         % (name, shape or "[N, K]", tuple(t.shape)))
    N, K = t.shape
    ld, inner = t.stride()
    if K > 1 and inner != 1:
        raise ValueError("%s must have dense rows (stride 1 along the last dimension)" % name)
    if N <= 1:
        return K
    if ld < K:
        raise ValueError("%s: its rows overlap" % name)
    return ld


def _vector_ptr(t, n, dtype, name, device):
    """Pointer of a vector of n entries of `dtype` on `device`; None for None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n
            and t.device == device and t.is_cuda and t.is_contiguous()):
        _need(t, dtype, name)
        if t.numel() != n:
            raise ValueError("%s must hold %d entries, got %d" % (name, n, t.numel()))
        _on(device, **{name: t})
    return t.data_ptr()


def norm_quant(x, weight=None, eps=1e-5, residual=None, normalize=True, h_out=None, stream=None):
    """Root-mean-square norm, with the residual's addition in front of it, and
    the per-token int8 quantiser behind it, in one launch.

    x: [N, K] fp32, bf16 or fp16 with dense rows of any row stride (16-byte
    aligned); residual: another of its type and shape, or None; weight: fp32
    [K] or None.  Without `normalize` the rows are quantised as they are.
    Returns (xq, amax, xsum) as quant_act does, or with a residual (h, xq,
    amax, xsum) with h = x + residual in x's type, which the norm is taken of;
    h_out may be x or residual, to write it in place.  A row with NaN or inf
    gets amax NaN and codes 0.  Outputs belong to the stream that writes them.
    """
    ldx = _need_rows(x, "x")
    shape, dtype, dev = x.shape, x.dtype, x.device
    N, K = shape
    ldr = ldh = 0
    rp = hp = None
    if residual is not None:
        ldr = _need_rows(residual, "residual", shape, dtype)
        rp = residual.data_ptr()
        if residual.device != dev:
            _on(dev, residual=residual)
        if h_out is not None:
            ldh = _need_rows(h_out, "h_out", shape, dtype)
            _on(dev, h_out=h_out)
    elif h_out is not None:
        raise ValueError("h_out without a residual: x itself is what the norm is taken of")
    w = _vector_ptr(weight, K, torch.float32, "weight", dev)
    if w is not None and not normalize:
        raise ValueError("weight belongs to the norm: pass None without it")
    out = _allocate(stream, x, (shape, torch.int8), (N, torch.float32), (N, torch.int32),
                    *(((shape, dtype),) if rp is not None and h_out is None else ()))
    xq, amax, xsum = out[:3]
    if rp is not None:
        if h_out is None:
            h_out, ldh = out[3], K
        hp = h_out.data_ptr()
    a = _lib.Norm(x.data_ptr(), rp, hp, w, xq.data_ptr(), amax.data_ptr(), xsum.data_ptr(), N, K,
                  ldx, ldr, ldh, eps, ACT_DTYPES[dtype], 1 if normalize else 0)
    _launch(_lib.load().bitlinear_norm_quant, "bitlinear_norm_quant", dev, stream, a)
    return (xq, amax, xsum) if residual is None else (h_out, xq, amax, xsum)


def gated_norm_quant(gate, up, weight=None, eps=1e-5, activation="silu", normalize=True,
                     stream=None):
    """The middle of a gated MLP: act(gate) * up, the norm (unless `normalize`
    is false) and the int8 quantiser, in one launch.  gate and up: [N, K] of
    one type with dense rows of any row stride, for instance the halves of one
    [N, 2K] buffer.  Returns (xq, amax, xsum), the input of the down
    projection."""
    ldg = _need_rows(gate, "gate")
    shape, dtype, dev = gate.shape, gate.dtype, gate.device
    N, K = shape
    ldu = _need_rows(up, "up", shape, dtype)
    if up.device != dev:
        _on(dev, up=up)
    act = _activation(activation)
    w = _vector_ptr(weight, K, torch.float32, "weight", dev)
    if w is not None and not normalize:
        raise ValueError("weight belongs to the norm: pass None without it")
    xq, amax, xsum = _allocate(stream, gate, (shape, torch.int8), (N, torch.float32),
                               (N, torch.int32))
    a = _lib.GatedNorm(gate.data_ptr(), up.data_ptr(), w, xq.data_ptr(), amax.data_ptr(),
                       xsum.data_ptr(), N, K, ldg, ldu, eps, ACT_DTYPES[dtype], act,
                       1 if normalize else 0)
    _launch(_lib.load().bitlinear_gated_norm_quant, "bitlinear_gated_norm_quant", dev, stream, a)
    return xq, amax, xsum


def _codes_in(xq, amax, xsum, dev):
    """Checks quantised activations; returns (N, K, their pointers)."""
    if not (isinstance(xq, torch.Tensor) and xq.dtype is torch.int8 and xq.is_cuda
            and xq.is_contiguous() and xq.device == dev):
        _need(xq, torch.int8, "xq")
        _on(dev, xq=xq)
    N, K = xq.shape
    _need_given(amax, "amax")
    _need_given(xsum, "xsum")
    return (N, K, xq.data_ptr(), _vector_ptr(amax, N, torch.float32, "amax", dev),
            _vector_ptr(xsum, N, torch.int32, "xsum", dev))


def _need_given(t, name):
    if t is None:
        raise TypeError("%s must be a torch.Tensor" % name)


def _linear_entry(packed, alpha, dev, codes, bias, activation, residual, out_dtype, out, stream):
    """Checks one layer of a linear call; returns its entry and its output."""
    if not (isinstance(packed, torch.Tensor) and packed.dtype is torch.int32 and packed.is_cuda
            and packed.is_contiguous() and packed.device == dev):
        _need(packed, torch.int32, "packed")
        _on(dev, packed=packed)
    N, K, xq, amax, xsum = codes
    M, words = packed.shape
    if words != packed_row_words(K):
        raise ValueError("packed must be [M, packed_row_words(K)] = [%d, %d], got %s"
                         % (M, packed_row_words(K), tuple(packed.shape)))
    _need_given(alpha, "alpha")
    if out_dtype is None:
        out_dtype = (out.dtype if out is not None else
                     residual.dtype if residual is not None else torch.float32)
    code = ACT_DTYPES.get(out_dtype)
    if code is None:
        raise TypeError("out_dtype must be float32, bfloat16 or float16, got %s" % out_dtype)
    ldr, rp = 0, None
    if residual is not None:
        ldr = _need_rows(residual, "residual", (N, M), out_dtype)
        rp = residual.data_ptr()
        if residual.device != dev:
            _on(dev, residual=residual)
    if out is None:
        out, = _allocate(stream, packed, ((N, M), out_dtype))
        ldy = M
    else:
        ldy = _need_rows(out, "out", (N, M), out_dtype)
        _on(dev, out=out)
    return (packed.data_ptr(), _vector_ptr(alpha, 1, torch.float32, "alpha", dev), M, K, xq, amax,
            xsum, _vector_ptr(bias, M, torch.float32, "bias", dev), rp, out.data_ptr(), ldr, ldy,
            code, _activation(activation)), out


def linear(packed, alpha, xq, amax, xsum, bias=None, activation=None, residual=None,
           out_dtype=None, out=None, stream=None):
    """The ternary product with its epilogue, any token count:
    act(y + bias) + residual, computed in fp32 and rounded once to out_dtype
    (fp32, bf16 or fp16; by default the type of out, else of the residual,
    else fp32).  bias: fp32 [M]; residual and out: [N, M] of out_dtype with
    dense rows of any row stride; out may be the residual itself."""
    _need_given(packed, "packed")
    dev = packed.device
    codes = _codes_in(xq, amax, xsum, dev)
    entry, out = _linear_entry(packed, alpha, dev, codes, bias, activation, residual, out_dtype,
                               out, stream)
    _launch(_lib.load().bitlinear_linear, "bitlinear_linear", dev, stream,
            _lib.LinearProblem(*entry), 1, codes[0])
    return out


def linear_grouped(layers, xq, amax, xsum, bias=None, activation=None, residual=None,
                   out_dtype=None, outs=None, stream=None):
    """linear over several layers that share the token count, in one launch
    (q, k and v; gate and up).  layers: list of (packed, alpha); every other
    argument is one value for all layers or a list with one per layer.
    Returns the list of outputs."""
    n = len(layers)
    if n == 0:
        return []

    def each(v, name):
        if not isinstance(v, (list, tuple)):
            return [v] * n
        if len(v) != n:
            raise ValueError("%s: one per layer, or one for all" % name)
        return v

    if outs is not None and not isinstance(outs, (list, tuple)):
        raise ValueError("outs: one per layer")
    shared = not any(isinstance(v, (list, tuple)) for v in (xq, amax, xsum))
    dev = layers[0][0].device
    codes = _codes_in(xq, amax, xsum, dev) if shared else None
    xqs, amaxs, xsums = each(xq, "xq"), each(amax, "amax"), each(xsum, "xsum")
    biases, acts = each(bias, "bias"), each(activation, "activation")
    residuals, dtypes = each(residual, "residual"), each(out_dtype, "out_dtype")
    outs = each(outs, "outs")
    arr, ys = (_lib.LinearProblem * n)(), []
    N = xqs[0].shape[0]
    for i, (packed, alpha) in enumerate(layers):
        if not shared:
            codes = _codes_in(xqs[i], amaxs[i], xsums[i], dev)
            if codes[0] != N:
                raise ValueError("layer %d: all layers share the token count" % i)
        arr[i], y = _linear_entry(packed, alpha, dev, codes, biases[i], acts[i], residuals[i],
                                  dtypes[i], outs[i], stream)
        ys.append(y)
    _launch(_lib.load().bitlinear_linear, "bitlinear_linear", dev, stream, arr, n, N)
    return ys


class TernaryLinear:
    """A BitLinear layer: packed 2-bit ternary weights + alpha (and a bias, if
    the layer has one), applied to fp32 activations: the fused quantise+GEMV
    kernel below GEMM_MIN_TOKENS tokens, else quant_act -> tensor-core GEMM
    with the fused rescale; with a bias, quant_act -> linear.  `quantized`
    takes what norm_quant, gated_norm_quant or quant_act gave."""

    def __init__(self, packed, alpha, in_features, out_features, bias=None):
        self.packed, self.alpha, self.bias = packed, alpha, bias
        self.in_features, self.out_features = in_features, out_features

    @classmethod
    def from_float(cls, W, stream=None, bias=None):
        packed, alpha = pack_weights(W, stream)
        return cls(packed, alpha, W.shape[1], W.shape[0], bias)

    def quantized(self, xq, amax, xsum, activation=None, residual=None, out_dtype=None, out=None,
                  stream=None):
        return linear(self.packed, self.alpha, xq, amax, xsum, self.bias, activation, residual,
                      out_dtype, out, stream)

    def __call__(self, x, stream=None):
        dev = self.packed.device
        if stream is None or _handle(stream) == _lib.raw_stream(None, dev.index):
            return self._apply(x, stream)
        with _OnStream(stream, dev):       # once for all that is allocated
            return self._apply(x, stream)

    def _apply(self, x, stream):
        if self.bias is not None:
            return self.quantized(*quant_act(x, stream), stream=stream)
        if use_fused_decode(x.shape[0], x.shape[1]):
            return gemv_quant(self.packed, self.alpha, x, self.out_features, stream=stream)
        xq, amax, xsum = quant_act(x, stream)
        return matmul(self.packed, self.alpha, xq, amax, xsum, self.out_features, stream=stream)
