"""Attention over packed and paged sequences in 64 bits: rotary positions, per-head norms, the
8-bit block quantisation of the cache, and masked softmax products.

Test infrastructure (see the package docstring). Readings: e4m3 as in ``oracle.quant``; a
block's scale is 2^e with the least e in [-40, 40] for which the block's largest magnitude is at
most 448 * 2^e."""
from __future__ import annotations

import numpy as np

from .quant import E4M3_MAX, round_to_e4m3

E_MIN, E_MAX = -40, 40


def rope_table(positions: int, rot: int, base: float = 10000.0, factor: float = 1.0) -> np.ndarray:
    """[positions, rot] in 64 bits: cos in the first half of the columns, sin in the second."""
    inv = base ** (-2.0 * np.arange(rot // 2) / rot)
    a = np.arange(positions)[:, None] / factor * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1)


def norm_rotate(x, weight, table, pos, interleaved: bool, eps: float = 1e-6) -> np.ndarray:
    """Head rows x [n, heads, d] of tokens at positions pos [n]; table rows as rope_table's."""
    y = np.asarray(x, np.float64).copy()
    if weight is not None:
        y = y * np.asarray(weight, np.float64) / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
    rot = 0 if table is None else table.shape[1]
    if rot:
        t = np.asarray(table, np.float64)[pos]
        c, s = t[:, None, :rot // 2], t[:, None, rot // 2:]
        i = np.arange(rot // 2)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first] = a * c - b * s
        y[..., second] = b * c + a * s
    return y


def block_exponent(amax: float) -> int:
    e = E_MIN
    while e < E_MAX and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


def append_block(held, held_scale, x):
    """One (page, head) block: `held` [m, d] code values of its earlier tokens on `held_scale`,
    x [n, d] new tokens. Returns (code values [m + n, d], scale). NaN does not enter the maximum
    and stays NaN; infinities saturate."""
    x = np.asarray(x, np.float64)
    finite = np.abs(x[~np.isnan(x)])
    scale = 2.0 ** block_exponent(float(finite.max()) if finite.size else 0.0)
    if len(held):
        scale = max(scale, held_scale)
        held = np.where(np.isnan(held), np.nan, round_to_e4m3(np.nan_to_num(held) * (held_scale / scale)))
    y = np.clip(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf) / scale, -E4M3_MAX, E4M3_MAX)
    codes = np.where(np.isnan(x), np.nan, round_to_e4m3(y))
    return (np.concatenate([held, codes]) if len(held) else codes), scale


def softmax_rows(q, k, v, lim, scale: float):
    """q [n, hq, d], k, v [m, hkv, d]; row i sees keys [0, lim[i]). Returns (out, lse, a, s): a =
    sum of p |v| (what rounding of the weights is relative to), s = the largest sum of |q k| scale
    over a row's visible keys."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out = np.zeros((n, hq, d))
    a = np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    s_abs = np.zeros((n, hq))
    for h in range(hq):
        s = q[:, h] @ k[:, h // g].T * scale
        mag = np.abs(q[:, h]) @ np.abs(k[:, h // g]).T * scale
        for i in range(n):
            m = int(lim[i])
            if m <= 0:
                continue
            row = s[i, :m]
            top = row.max()
            p = np.exp(row - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ v[:m, h // g]
            a[i, h] = p @ np.abs(v[:m, h // g])
            s_abs[i, h] = mag[i, :m].max()
    return out, lse, a, s_abs


def limits(nq: int, nk: int, frame: int) -> np.ndarray:
    """Keys that each of nq queries at the end of nk positions sees, causal over frames."""
    p = np.arange(nq) + nk - nq
    return np.where(p >= 0, np.minimum(nk, (p // frame + 1) * frame), 0)
