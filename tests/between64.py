"""The operators between two products, restated in numpy for the tests.

norm_rows and gated_rows follow the definition of include/bitlinear.h: sums
and r in 64 bits, every other step one fp32 rounding (numpy's fp32 operations
are IEEE), so codes, maxima and sums have to agree bit for bit wherever the
row's values are free of transcendental functions.  linear64 gives the exact
result in 64 bits and a bound on what fp32 may be off by.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24          # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantise(v):
    """fp32 rows -> (q int8, amax fp32, xsum int32) of the definition."""
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(1)
        bad = ~np.isfinite(v).all(1)
        s = (np.float32(127) / amax).astype(np.float32)
        t = v * s[:, None]
        t = np.where(np.isnan(t), np.float32(0), t)      # 0 * inf
        q = np.clip(np.rint(t), -128, 127)
    q[(amax == 0) | bad] = 0
    amax = np.where(bad, np.float32(np.nan), amax).astype(np.float32)
    return q.astype(np.int8), amax, q.sum(1).astype(np.int32)


def normalise(h, w, eps):
    with np.errstate(all="ignore"):
        ss = (h.astype(np.float64) ** 2).sum(1) / h.shape[1]
        r = (1.0 / np.sqrt(ss + eps)).astype(np.float32)
        v = h * r[:, None]
        return v if w is None else v * w


def norm_rows(h, w, eps, normalize=True):
    """h: fp32 [N, K], already rounded to the stored type."""
    return quantise(normalise(h, w, eps) if normalize else h)


def act64(v, name):
    """Activations in 64 bits from their definitions."""
    if name in (None, "none"):
        return v
    if name == "relu":
        return np.maximum(v, 0)
    if name == "relu2":
        return np.maximum(v, 0) ** 2
    t = torch.from_numpy(np.ascontiguousarray(v))
    if name == "silu":
        return (t * torch.sigmoid(t)).numpy()
    if name == "gelu":
        return (t * torch.special.ndtr(t)).numpy()
    return (t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))).numpy()


# What an activation evaluated in fp32 may be off by on an exact argument u,
# in half steps of fp32 (2^-24), and the largest slope it passes an argument's
# error on with.  relu: exact.  relu2: one product.  silu: expf within 2 units
# in the last place (4 half steps), 1 + e and the division one each: 6 of |y|.
# gelu: the rounded argument of erf (error |z| half a step, slope of erf at
# most 1.13: z * 1.13 e^(-z^2) < 0.5), erff within 2 units of a value at most
# 1 (4), the sum 1 + erf <= 2 (2), two products (at most 2 * 2): below 11 in
# units of |u| / 2 < 6 |u|.  gelu_tanh: its argument carries 5 roundings
# (slope: |a tanh'(a)| < 0.45, so < 2.3), tanhf within 2 units (4), the sum
# (2), two products (4): below 13 |u| / 2 < 7 |u|.
#
# Behind a product the kernels divide approximately (__fdividef, within 2 units:
# 4 half steps, instead of 1), and stop the exponential's argument at 87:
# silu  4 + 1 + 4 = 9 of |y|, plus |v| 2^-125.
# gelu_tanh as v / (1 + e^-a), a = 2 sqrt(2/pi) (v + 0.044715 v^3) with 5
# roundings: e^-a is off by 5 |a| + 4, which passes on e^-a / (1 + e^-a) of it;
# |y| |a| e^-a / (1 + e^-a) <= 0.37 |v| on either side, so 5 * 0.37 + 4 + 1 + 4
# < 11 of |v|, plus |v| 2^-125.
def act_error(u, name, product=False):
    au = np.abs(u)
    if product and name == "silu":
        return 9 * U * np.abs(act64(u, "silu")) + au * 2.0 ** -125
    if product and name == "gelu_tanh":
        return 11 * U * au
    if name in (None, "none", "relu"):
        return np.zeros_like(u)
    if name == "relu2":
        return U * np.maximum(u, 0) ** 2
    if name == "silu":
        return 6 * U * np.abs(act64(u, "silu"))
    return (6 if name == "gelu" else 7) * U * au


def act_slope(u, name):
    if name in (None, "none", "relu"):
        return np.ones_like(u)
    if name == "relu2":
        return 2 * np.maximum(u, 0) + 1e-6
    return np.full_like(u, 1.13)      # |silu'| <= 1.10, |gelu'| and |gelu_tanh'| <= 1.13


def linear64(acc, alpha, amax, bias, name, residual, dtype):
    """(exact y, bound on |y computed - exact y|) in 64 bits.
    acc: exact integers [N, M] (below 2^24: exact in fp32)."""
    p = acc.astype(np.float64) * float(alpha) * (amax.astype(np.float64) / 127.0)[:, None]
    err = 3 * U * np.abs(p)                       # amax/127, alpha *, acc *
    u = p if bias is None else p + bias.astype(np.float64)
    if bias is not None:
        err = err + U * np.abs(u)
    y = act64(u, name)
    err = err * act_slope(u, name) + act_error(u, name, product=True)
    if residual is not None:
        y = y + residual.astype(np.float64)
        err = err + U * np.abs(y)
    # first order above; the 2^-10 covers the products of errors; subnormals: one step
    tiny = float(torch.finfo(dtype).smallest_normal) * float(torch.finfo(dtype).eps)
    err = err * (1 + 2.0 ** -10)
    return y, err + half_step(dtype) * (np.abs(y) + err) + tiny


def codes_of(packed, K):
    """int64 codes [M, K] of packed 2-bit rows, by the layout's bit formula."""
    w = packed.cpu().numpy().view(np.uint32)
    k = np.arange(K)
    f = (w[:, k // 16] >> (8 * (k % 4) + 2 * ((k % 16) // 4)).astype(np.uint32)) & 3
    return f.astype(np.int64) - 1
