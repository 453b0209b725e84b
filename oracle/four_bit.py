"""The 4-bit cache, eviction from it and the norm ahead of 8-bit products, in 64 bits.

Test infrastructure (see the package docstring). Readings: e2m1 values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
their negatives, ties to the even mantissa; 16 elements share an e4m3 scale max|x| / 6 / unit, at least
2^-9; codes are integers decided by floating point, so what decides them is computed in fp32, each
operation rounded, as ``oracle.quant`` does for e4m3."""
from __future__ import annotations

import numpy as np

from .quant import E4M3_MAX, round_to_e4m3

E2M1_MAX, BLOCK, SCALE_MIN = 6.0, 16, 2.0 ** -9
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def round_to_e2m1(x) -> np.ndarray:
    """Nearest e2m1 value (ties to the even mantissa), saturated to +-6."""
    a = np.abs(np.asarray(x, np.float64))
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.round(a / step) * step, E2M1_MAX), x)


def quantise(x, unit):
    """x [..., dim] in fp32, unit broadcast against [..., dim / 16]: (code values [..., dim], scales
    [..., dim / 16]). Blocks that are not finite have a NaN scale and codes of 0."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    unit = np.broadcast_to(np.asarray(unit, np.float32), b.shape[:-1])
    with np.errstate(invalid="ignore"):
        top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    top = np.where(bad, np.float32(0), top)
    s = round_to_e4m3(np.clip((top / np.float32(6)).astype(np.float32) / unit, SCALE_MIN, E4M3_MAX))
    whole = (s * unit).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        c = round_to_e2m1((b / whole[..., None]).astype(np.float32))
    c = np.where(bad[..., None], 0.0, c)
    return c.reshape(x.shape), np.where(bad, np.nan, s)


def values(codes, scales, unit):
    """What code values [..., dim] with scales [..., dim / 16] stand for."""
    b = np.asarray(codes, np.float64).reshape(*codes.shape[:-1], codes.shape[-1] // BLOCK, BLOCK)
    return (b * (np.asarray(scales, np.float64) * unit)[..., None]).reshape(codes.shape)


def unpack(data):
    """Code values [..., dim] of bytes [..., dim / 2], the even element in the low half."""
    d = np.asarray(data)
    n = np.stack([d & 15, d >> 4], -1).reshape(*d.shape[:-1], 2 * d.shape[-1])
    return np.where(n & 8, -1.0, 1.0) * E2M1[n & 7]


def round_to_24_bits(x) -> np.ndarray:
    """Nearest value with fp32's 24 bits (ties to even), of any exponent."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(m * 2.0 ** 24), e - 24)


def norm_rotate(x, weight, table, pos, interleaved: bool, eps: float = 1e-6) -> np.ndarray:
    """``oracle.paged.norm_rotate`` in fp32: the norm's factor rounded once, then every product
    and sum. The factor and its product with the weight are no results: they have fp32's bits and no ends."""
    y = np.asarray(x, np.float32).copy()
    if weight is not None:
        r = (1 / np.sqrt(np.mean(y.astype(np.float64) ** 2, -1, keepdims=True) + np.float64(np.float32(eps))))
        r = round_to_24_bits(round_to_24_bits(r) * np.asarray(weight, np.float32).astype(np.float64))
        y = (y * r).astype(np.float32)
    rot = 0 if table is None else table.shape[1]
    if rot:
        t = np.asarray(table, np.float32)[pos]
        c, s = t[:, None, :rot // 2], t[:, None, rot // 2:]
        i = np.arange(rot // 2)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first] = a * c - b * s
        y[..., second] = b * c + a * s
    return y


def kept(mass, keep: int, recent: int) -> np.ndarray:
    """Places, ascending, of the tokens that one head of one sequence keeps: mass [n]."""
    n = len(mass)
    if n <= keep:
        return np.arange(n)
    old = np.asarray(mass[:n - recent], np.float64)
    # largest first, NaN last, ties by the lower place
    order = np.lexsort((np.arange(len(old)), -np.where(np.isnan(old), -np.inf, old), np.isnan(old)))
    return np.sort(np.concatenate([order[:keep - recent], np.arange(n - recent, n)]))


def add_rmsnorm(x, delta, weight, eps: float):
    """(s, y): the sum and its RMS norm times the weight."""
    s = np.asarray(x, np.float64) + (0 if delta is None else np.asarray(delta, np.float64))
    return s, s * np.asarray(weight, np.float64) / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps)
