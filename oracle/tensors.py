"""AdamW over a list of tensors with 8-bit moments, and the global gradient
norm.  TEST INFRASTRUCTURE.

The 8-bit codes are defined by their tables: the values of all 256 codes,
computed from the bit fields, and the nearest of them.  The update around them
is numpy float32, one rounding per operation, in the order written.
"""
from __future__ import annotations

import math

import numpy as np

from .numerics import AdamWConfig, adamw_scalars

BLOCK = 256
E4M3_MAX = np.float32(448.0)
ROOT_MAX = np.float32(1.9375)
TINY = np.float32(2.0) ** np.float32(-100)


def e4m3_values():
    """Code -> value: sign, 4 exponent bits (bias 7, 0 subnormal), 3 mantissa
    bits; exponent 15 with mantissa 7 is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            mag = math.nan
        out[c] = -mag if c & 128 else mag
    return out


def root_values():
    """Code -> value: (1 + (c & 15) / 16) 2^((c >> 4) - 15), code 0 -> 0."""
    return np.array([0.0] + [(1 + (c & 15) / 16) * 2.0 ** ((c >> 4) - 15) for c in range(1, 256)])


def _nearest(x, values, tie_even):
    """Index of the value nearest to each x (values ascending); a tie goes to
    the even index or to the upper one."""
    x = np.clip(np.asarray(x, np.float64), values[0], values[-1])
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    up = (dh < dl) | ((dh == dl) & ((hi % 2 == 0) if tie_even else True))
    return np.where(up, hi, lo)


def _scales(x, top):
    big = np.abs(x).max(axis=1)      # NaN where a NaN is
    with np.errstate(divide="ignore", invalid="ignore"):
        small = big < TINY
        return (np.where(small, np.float32(0), big / top).astype(np.float32),
                np.where(small, np.float32(0), top / big).astype(np.float32))


def _blocks(x):
    x = np.asarray(x, np.float32).ravel()
    pad = -len(x) % BLOCK
    return np.concatenate([x, np.zeros(pad, np.float32)]).reshape(-1, BLOCK)


def encode_m(m):
    """fp32 -> (codes, scales), nearest, ties to the even code."""
    n, x = np.asarray(m).size, _blocks(m)
    scale, up = _scales(x, E4M3_MAX)
    y = (x * up[:, None]).astype(np.float32)
    k = _nearest(np.abs(y), e4m3_values()[:127], True)
    code = np.where(np.isnan(y), 127, k + np.where(np.signbit(y), 128, 0)).astype(np.uint8)
    return code.ravel()[:n], scale


def encode_r(r):
    """fp32 roots -> (codes, scales), nearest, ties up, non-zero at least 1."""
    n, x = np.asarray(r).size, _blocks(r)
    scale, up = _scales(x, ROOT_MAX)
    with np.errstate(invalid="ignore"):
        y = (x * up[:, None]).astype(np.float32)
        k = np.maximum(_nearest(np.nan_to_num(y), root_values(), False), 1)
        code = np.where(y > 0, k, 0).astype(np.uint8)
    return code.ravel()[:n], scale


def _decode(code, scale, values):
    each = np.repeat(np.asarray(scale, np.float32), BLOCK)[:np.asarray(code).size]
    return (values.astype(np.float32)[code] * each).astype(np.float32)


def decode_m(code, scale):
    return _decode(code, scale, e4m3_values())


def decode_r(code, scale):
    return _decode(code, scale, root_values())


def adamw8(g, p, mc, ms, vc, vs, hp: AdamWConfig, t: int):
    """One step on fp32 gradients; returns (p, mc, ms, vc, vs)."""
    c = adamw_scalars(hp, t)
    m, r = decode_m(mc, ms), decode_r(vc, vs)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        p = p - c.lr_wd * p
        m = c.beta1 * m + c.omb1 * g
        r = np.sqrt(c.beta2 * (r * r) + (c.omb2 * g) * g)
        p = p - (c.step_size * m) / (r / c.sqrt_bc2 + c.eps)
    return (p, *encode_m(m), *encode_r(r))


def grad_norm(grads, max_norm, scale=1.0):
    """(norm, factor) of float64 sums."""
    norm = math.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)) / scale
    return norm, min(1.0, max_norm / (norm + 1e-6)) / scale
