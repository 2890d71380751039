"""Cases for the operators between two ternary products: what they are given,
one pass through each, and what a pass cannot do without.

  norm        root-mean-square norm with the residual's addition, int8 output
              with one scale per token (input of q/k/v and of gate/up)
  gated       act(gate) * up, norm, int8 output with scales (input of down)
  linear      ternary product with bias, activation and residual applied to
              its result, stored as fp32, bf16 or fp16

With `own` false, run() computes them in elementary torch operations; with
`own` true it makes the library's calls.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
EPS = 1e-5


def listed():
    def norm(name, N, K, dtype, residual, pad=0):
        return {"name": name, "op": "norm", "N": N, "K": K, "dtype": dtype,
                "residual": residual, "pad": pad}

    def gated(name, N, K, dtype, act, normalize, joined):
        return {"name": name, "op": "gated", "N": N, "K": K, "dtype": dtype, "act": act,
                "normalize": normalize, "joined": joined}

    def linear(name, N, M, K, dtype, bias, act, residual, kv=0):
        return {"name": name, "op": "linear", "N": N, "M": M, "K": K, "dtype": dtype,
                "bias": bias, "act": act, "residual": residual, "kv": kv}

    return [
        # one decoded token of the 2B shape: the norm before q/k/v, a latency
        norm("norm 1x2560 bf16", 1, 2560, "bf16", True),
        # a small batch whose rows sit in a wider buffer, no residual
        norm("norm 77x6928 fp16 strided", 77, 6928, "fp16", False, pad=48),
        # prefill of the 70B shape on an fp32 residual stream
        norm("norm 2048x8192 fp32", 2048, 8192, "fp32", True),
        # one decoded token of the 70B shape: the input of down
        gated("gated 1x28672 bf16 silu", 1, 28672, "bf16", "silu", True, True),
        # prefill of the 7B shape, squared ReLU, gate and up as halves of one buffer
        gated("gated 512x11008 bf16 relu2", 512, 11008, "bf16", "relu2", True, True),
        # one decoded token: the output projection of the 2B shape onto the residual
        linear("linear 1x2560x2560 bf16", 1, 2560, 2560, "bf16", False, "none", True),
        # one decoded token: down of the 70B shape onto an fp32 residual
        linear("linear 1x8192x28672 fp32", 1, 8192, 28672, "fp32", False, "none", True),
        # sixteen sequences decoded together: q, k and v of the 8B shape with biases, one call
        linear("linear 16x(4096+2x1024)x4096", 16, 4096, 4096, "bf16", True, "none", False,
               kv=1024),
        # a ragged mid-size batch through an up projection with an activation
        linear("linear 93x11005x4112 fp32 silu", 93, 11005, 4112, "fp32", True, "silu", False),
        # prefill of the 7B shape: gate with squared ReLU
        linear("linear 512x11008x4096 relu2", 512, 11008, 4096, "bf16", False, "relu2", False),
        # prefill of the 70B shape: down onto the residual
        linear("linear 2048x8192x28672 bf16", 2048, 8192, 28672, "bf16", True, "none", True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "gated", "linear", "linear"))
    dtype = rng.choice(("fp32", "bf16", "fp16"))
    N = _spread(rng, 1, 2048)
    if op == "norm":
        K = 16 * _spread(rng, 64, 1792)
        while N * K > 2048 * 8192:
            N = max(1, N // 2)
        return {"op": op, "N": N, "K": K, "dtype": dtype, "residual": rng.random() < 0.6,
                "pad": rng.choice((0, 0, 16, 80))}
    if op == "gated":
        K = 16 * _spread(rng, 128, 1792)
        while N * K > 2048 * 8192:
            N = max(1, N // 2)
        return {"op": op, "N": N, "K": K, "dtype": dtype, "act": rng.choice(ACTS[1:]),
                "normalize": rng.random() < 0.7, "joined": rng.random() < 0.5}
    K = 16 * _spread(rng, 64, 1792)
    M = _spread(rng, 512, 28672)
    if rng.random() < 0.7:
        M = max(16, M // 16 * 16)
    while N * M * K > 2048 * 8192 * 28672 or M * K > 28672 * 8192:
        M = max(16, M // 2)
    kv = max(8, M // 4 // 8 * 8) if rng.random() < 0.25 else 0
    if kv and N * (M + 2 * kv) * K > 2048 * 8192 * 28672:
        kv = 0
    return {"op": op, "N": N, "M": M, "K": K, "dtype": dtype, "bias": rng.random() < 0.5,
            "act": rng.choice(("none", "none") + ACTS[1:]), "residual": rng.random() < 0.5,
            "kv": kv}


# ------------------------------------------------------------------ inputs

def _packed(M, K, g):
    """Ternary weights in the library's 2-bit rows, drawn with the zero share
    (31 %) that absmean leaves of Gaussian weights: int32 [M, 4*ceil(K/64)]."""
    rb = 16 * ((K + 63) // 64)   # bytes per row
    out = torch.zeros((M, rb // 4, 4), dtype=torch.uint8, device="cuda")   # [row, word, byte]
    for j in range(4):   # field j of byte b of word w: weight 16 w + 4 j + b
        u = torch.randint(0, 256, (M, rb // 4, 4), dtype=torch.uint8, device="cuda", generator=g)
        f = (u >= 88).to(torch.uint8) + (u >= 168).to(torch.uint8)   # code + 1
        k = (16 * torch.arange(rb // 4, device="cuda")[:, None] + 4 * j
             + torch.arange(4, device="cuda")[None, :])
        f = torch.where(k < K, f, torch.ones_like(f))   # padding fields hold code 0
        out |= f << (2 * j)
    return out.reshape(M, rb).view(torch.int32)


def _activations(N, K, g, pad=0):
    """N(0,1) rows with one channel in a hundred ten times as large."""
    x = torch.randn((N, K + pad), generator=g, device="cuda")
    c = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
    x[:, c] *= 10.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, K, T = case["N"], case["K"], TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        s["x"] = _activations(N, K, g, case["pad"]).to(T)[:, :K]
        s["res"] = (_activations(N, K, g, case["pad"]).mul_(3.0).to(T)[:, :K]
                    if case["residual"] else None)
        s["w"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        return s
    if case["op"] == "gated":
        gu = torch.randn((N, 2 * K), generator=g, device="cuda").to(T)
        s["gate"], s["up"] = gu[:, :K], gu[:, K:]
        if not case["joined"]:
            s["gate"], s["up"] = s["gate"].contiguous(), s["up"].contiguous()
        s["w"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        return s
    s["layers"], s["biases"], s["residuals"] = [], [], []
    for M in [case["M"]] + ([case["kv"]] * 2 if case["kv"] else []):
        alpha = 0.016 * (1.0 + 0.1 * torch.rand(1, generator=g, device="cuda"))
        s["layers"].append((_packed(M, K, g), alpha))
        s["biases"].append(torch.randn(M, generator=g, device="cuda") if case["bias"] else None)
        s["residuals"].append(3.0 * torch.randn((N, M), generator=g, device="cuda")
                              if case["residual"] else None)
    s["residuals"] = [None if r is None else r.to(T) for r in s["residuals"]]
    x = _activations(N, K, g)
    s["amax"] = x.abs().amax(1)
    s["xq"] = torch.round(x / s["amax"][:, None] * 127.0).to(torch.int8)
    s["xsum"] = s["xq"].sum(1, dtype=torch.int32)
    return s


# -------------------------------------------------------------- plain forms

def _act(v, name):
    if name == "none":
        return v
    if name == "relu":
        return torch.clamp_min(v, 0.0)
    if name == "relu2":
        return torch.clamp_min(v, 0.0) * torch.clamp_min(v, 0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))


def _quantise(h, w, normalize):
    """fp32 rows h -> what the int8 codes stand for, the scales' maxima and the
    code sums.  The sum of squares is a long sum whose last bits decide codes
    next to a border: 64 bits."""
    if normalize:
        ss = h.double().square().mean(1, keepdim=True)
        r = (1.0 / torch.sqrt(ss + EPS)).float()
        h = h * r * w
    amax = h.abs().amax(1, keepdim=True)
    s = torch.full_like(amax, 127.0) / amax
    q = torch.clamp(torch.round(h * s), -128.0, 127.0)
    return {"values": q * (amax / 127.0), "amax": amax[:, 0],
            "xsum": q.sum(1, dtype=torch.int32)}


def _codes(packed, K):
    """2-bit rows -> fp32 codes [M, K]."""
    k = torch.arange(16, device=packed.device)
    shift = (8 * (k % 4) + 2 * (k // 4)).to(torch.int32)
    c = ((packed[:, :, None] >> shift) & 3).reshape(packed.shape[0], -1)
    return c[:, :K].float() - 1.0


def _plain(s):
    T = TYPES[s["dtype"]]
    if s["op"] == "norm":
        h = s["x"].float()
        if s["res"] is None:
            return _quantise(h, s["w"], True)
        h = (h + s["res"].float()).to(T)
        return dict(_quantise(h.float(), s["w"], True), h=h)
    if s["op"] == "gated":
        return _quantise(_act(s["gate"].float(), s["act"]) * s["up"].float(), s["w"],
                         s["normalize"])
    ys = []
    for (packed, alpha), bias, res in zip(s["layers"], s["biases"], s["residuals"]):
        # integers below 2^24: the fp32 product is exact
        y = (s["xq"].float() @ _codes(packed, s["K"]).t()) * (alpha * (s["amax"] / 127.0))[:, None]
        if bias is not None:
            y = y + bias
        y = _act(y, s["act"])
        if res is not None:
            y = y + res.float()
        ys.append(y.to(T))
    return ys


# ------------------------------------------------------------ library calls

def _values(xq, amax, xsum):
    return {"values": xq * (amax / 127.0)[:, None], "amax": amax, "xsum": xsum}


def run(state):
    if not own:
        return _plain(state)
    from ternary_weight_bit_bitlinear_b200 import api
    s = state
    if s["op"] == "norm":
        if s["res"] is None:
            return _values(*api.norm_quant(s["x"], s["w"], eps=EPS))
        h, xq, amax, xsum = api.norm_quant(s["x"], s["w"], eps=EPS, residual=s["res"])
        return dict(_values(xq, amax, xsum), h=h)
    if s["op"] == "gated":
        return _values(*api.gated_norm_quant(s["gate"], s["up"],
                                             s["w"] if s["normalize"] else None, eps=EPS,
                                             activation=s["act"], normalize=s["normalize"]))
    if len(s["layers"]) == 1:
        packed, alpha = s["layers"][0]
        return [api.linear(packed, alpha, s["xq"], s["amax"], s["xsum"], bias=s["biases"][0],
                           activation=s["act"], residual=s["residuals"][0],
                           out_dtype=TYPES[s["dtype"]])]
    return api.linear_grouped(s["layers"], s["xq"], s["amax"], s["xsum"], bias=s["biases"],
                              activation=s["act"], residual=s["residuals"],
                              out_dtype=TYPES[s["dtype"]])


# -------------------------------------------------------------- work, exact

def work(case):
    N, K = case["N"], case["K"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        return {"bytes": N * K * e * (3 if case["residual"] else 1) + 4 * K + N * K + 8 * N,
                "flops": 8 * N * K}
    if case["op"] == "gated":
        return {"bytes": 2 * N * K * e + (4 * K if case["normalize"] else 0) + N * K + 8 * N,
                "flops": 10 * N * K}
    M = case["M"] + 2 * case["kv"]
    return {"bytes": M * K / 4 + N * K + 8 * N + (4 * M if case["bias"] else 0)
            + N * M * e * (2 if case["residual"] else 1),
            "flops": 2 * N * M * K}


def _exact_act(v, name):
    """The activations from their definitions, in 64 bits."""
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return {"none": v, "relu": v.relu(), "relu2": v.relu() ** 2}[name]


def _exact_rows(h, w, normalize, defined):
    """`defined`: the rows' values are exact, so the codes are too: they are
    defined on v, the scale and their product, each rounded once to 32 bits.
    Otherwise (a transcendental activation) codes next to a border have no
    value of their own; the maxima do."""
    once = (lambda t: t.float().double()) if defined else (lambda t: t)
    v = once(h)
    if normalize:
        r = once((v.pow(2).sum(1) / v.shape[1] + EPS).rsqrt())
        v = once(once(v * r[:, None]) * w.double())
    top = v.abs().max(1).values
    if not defined:
        return {"values": None, "amax": top, "xsum": None}
    q = once(v * once(127.0 / top)[:, None]).round().clamp(-128, 127)
    return {"values": q * top[:, None] / 127.0, "amax": top, "xsum": q.sum(1).to(torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["res"] is None:
            return _exact_rows(h, s["w"], True, True)
        h = h + s["res"].double()
        return dict(_exact_rows(h.to(TYPES[case["dtype"]]).double(), s["w"], True, True), h=h)
    if case["op"] == "gated":
        a = _exact_act(s["gate"].double(), case["act"])
        defined = case["act"] in ("relu", "relu2")
        if case["act"] == "relu2":
            a = a.float().double()
        return _exact_rows(a * s["up"].double(), s["w"], case["normalize"], defined)
    out = []
    for (packed, alpha), bias, res in zip(s["layers"], s["biases"], s["residuals"]):
        M, WP = packed.shape
        b = packed.view(torch.uint8).reshape(M, WP, 1, 4)
        fields = torch.cat([(b >> (2 * j)) & 3 for j in range(4)], 2)   # [row, word, j, byte]
        c = fields.reshape(M, WP * 16)[:, : case["K"]].double() - 1.0
        y = torch.einsum("nk,mk->nm", s["xq"].double(), c)
        y *= alpha.double() * s["amax"].double()[:, None] / 127.0
        if bias is not None:
            y += bias.double()
        y = _exact_act(y, case["act"])
        out.append(y if res is None else y + res.double())
    return out
