"""Plain fp64 numpy definitions of the dense operators (test infrastructure
only): the RMS norm with the residual's addition, the gated feed-forward
projections, the linear layer and AdamW."""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def rmsnorm_residual(x, res, w, eps):
    """(r, rstd, y) of r = x + res, y = r rstd w."""
    r = np.asarray(x, np.float64) + (0.0 if res is None else np.asarray(res, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r, rstd, r * rstd[:, None] * np.asarray(w, np.float64)


def rmsnorm_residual_bwd(dy, r, w, rstd, dres=None):
    """(dx, dw), rstd taken as it is given."""
    xhat = np.asarray(r, np.float64) * np.asarray(rstd, np.float64)[:, None]
    t = dy * np.asarray(w, np.float64)
    dx = rstd[:, None] * (t - xhat * np.mean(t * xhat, axis=1, keepdims=True))
    return dx if dres is None else dx + dres, np.sum(dy * xhat, axis=0)


def e8m0_byte(amax):
    """Byte e + 127 of the smallest e with amax <= 448 * 2^e; 0 for zero."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(amax / 448.0)), -127)
    # log2 may round across the border: settle it by the definition
    e = np.where((amax > 0) & (amax <= 448.0 * np.exp2(e - 1)), e - 1, e)
    e = np.where(amax > 448.0 * np.exp2(e), e + 1, e)
    return np.clip(e, -127, 127).astype(np.int64) + 127


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    assert kind == "none"
    return z


def act_slope(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    assert kind == "none"
    return np.ones_like(z)


def gated_ffn(x, w1, kind="silu"):
    """(h, a): a = x w1 = [gate | up], h = act(gate) * up."""
    a = np.asarray(x, np.float64) @ np.asarray(w1, np.float64)
    f = a.shape[1] // 2
    return act(a[:, :f], kind) * a[:, f:], a


def gated_ffn_bwd(dh, a, x, w1, kind="silu"):
    """(dx, dw1, da) for the kept a."""
    a, dh = np.asarray(a, np.float64), np.asarray(dh, np.float64)
    f = a.shape[1] // 2
    da = np.concatenate([dh * a[:, f:] * act_slope(a[:, :f], kind), dh * act(a[:, :f], kind)], axis=1)
    return da @ np.asarray(w1, np.float64).T, np.asarray(x, np.float64).T @ da, da


def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z): z = x w + bias, y = act(z) + residual."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, kind)
    return y if residual is None else y + np.asarray(residual, np.float64), z


def linear_bwd(dy, x, w, z=None, kind="none"):
    """(dx, dw, dbias, dz) for the kept z."""
    dz = np.asarray(dy, np.float64)
    if kind != "none":
        dz = dz * act_slope(z, kind)
    return dz @ np.asarray(w, np.float64).T, np.asarray(x, np.float64).T @ dz, dz.sum(axis=0), dz


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd, grad_scale=1.0):
    """(p, m, v) after step number t."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * wd * p - upd, m, v


def mix32(x):
    """32 mixed bits of 32: the counter mixing of the 8-bit rounding."""
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x85EBCA77)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def dither_bits(counter, seed, step):
    """The 32 bits of the counters (int64): low 16 for m, high 16 for v."""
    c = np.asarray(counter, np.uint64)
    key = mix32(np.uint64(seed) ^ mix32(np.uint64(step)))
    return mix32((c + mix32((c >> np.uint64(32)) ^ key)) & np.uint64(0xFFFFFFFF))


def e4m3_dither(x, bits16):
    """|x| (up to 448) rounded down or up to a multiple of its E4M3 step."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    with np.errstate(divide="ignore"):
        e = np.where(a > 0, np.floor(np.log2(a)), -100)
    step = np.exp2(np.maximum(e - 3, -9))
    return np.copysign(np.minimum(np.floor(a / step + np.asarray(bits16, np.float64) / 65536.0) * step, 448.0), x)
