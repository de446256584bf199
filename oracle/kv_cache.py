"""Plain 64-bit restatement of the cache operators -- TEST INFRASTRUCTURE ONLY.

Rotary positions, the 4-bit row format, appending rows to a paged cache, and
attention over chunk rows given as values.  bf16 values are passed as fp64
numbers unless a name says bits.  Pinned by ``tests/test_kv_cache_oracle.py``.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rope_frequencies", "rope_rotate", "round_bf16", "E2M1", "e4m3_values", "quantise_rows", "kv4_pack",
           "kv4_unpack", "kv4_values", "append_positions", "attention_rows"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rope_frequencies(rot_dim, base, scaling="plain", factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair (fp64)."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    i = np.arange(rot_dim // 2)
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        def at(turns):
            return rot_dim * math.log(orig_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
        r = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f * (1.0 - r) + f / factor * r
    if scaling == "by_wavelength":
        s = np.clip((orig_len * f / (2.0 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return f * s + f / factor * (1.0 - s)
    return f


def rope_rotate(x, pos, freq, half, gain=1.0):
    """x fp64 [..., H, 128] at positions pos [...]: pairs turned, not rounded."""
    n = len(freq)
    turn = np.asarray(pos, np.float64)[..., None, None] * freq
    c, s = gain * np.cos(turn), gain * np.sin(turn)
    i = np.arange(n)
    a, b = (i, i + n) if half else (2 * i, 2 * i + 1)
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def round_bf16(x):
    """fp64 -> the nearest bf16 value, ties to even (fp64; finite inputs in bf16's normal range or zero)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def e4m3_values():
    """The 127 finite e4m3 magnitudes, by code."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * 2.0 ** (e - 7.0))


def _nearest(v, table):
    """Code of the table entry nearest to v >= 0 (ties to the even code, beyond the end the last one)."""
    hi = np.clip(np.searchsorted(table, v), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(table[hi] - v), np.abs(v - table[lo])
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise_rows(x, exps):
    """x fp64 [..., 128], exps broadcast against [...]: (codes [..., 128] 0..15, scale codes [..., 8])."""
    g = (x * 2.0 ** -np.asarray(exps, np.float64)[..., None]).reshape(*x.shape[:-1], 8, 16)
    with np.errstate(invalid="ignore", divide="ignore"):
        a = np.abs(g)
        nan = np.isnan(g).any(-1)
        top = np.where(nan, 0.0, np.nan_to_num(a, nan=0.0, posinf=np.inf).max(-1))
        s8 = np.where(nan, 127, _nearest(np.minimum(top / 6.0, 448.0), e4m3_values()))
        s = np.where(nan, 1.0, np.concatenate([e4m3_values(), [1.0]])[s8])[..., None]
        q = np.where(s > 0, np.minimum(np.where(np.isnan(a), 0.0, a), 1e30) / np.where(s > 0, s, 1.0), 0.0)
    code = _nearest(np.minimum(q, 6.0), E2M1) | np.where(np.signbit(g), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


def kv4_pack(codes, scales):
    """codes [n, cs, 128], scales [n, cs, 8] -> pages uint8 [n, cs*72]."""
    n, cs, _ = codes.shape
    b = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(n, cs // 16, 1024)
    return np.concatenate([b, scales.reshape(n, cs // 16, 128)], -1).reshape(n, cs * 72).astype(np.uint8)


def kv4_unpack(pages):
    """pages uint8 [n, cs*72] -> (codes [n, cs, 128], scales [n, cs, 8])."""
    n, cs = pages.shape[0], pages.shape[1] // 72
    blk = pages.reshape(n, cs // 16, 1152)
    b, s = blk[..., :1024].reshape(n, cs, 64), blk[..., 1024:].reshape(n, cs, 8)
    return np.stack([b & 15, b >> 4], -1).reshape(n, cs, 128), s


def kv4_values(pages, exps):
    """Values fp64 [n, cs, 128] of pages, exps [n] (each page's head)."""
    codes, s8 = kv4_unpack(pages)
    table = np.concatenate([e4m3_values(), [np.nan]])
    s = np.where(s8 & 128, -1.0, 1.0) * table[s8 & 127] * (2.0 ** np.asarray(exps, np.float64))[:, None, None]
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return (v.reshape(*s.shape, 16) * s[..., None]).reshape(v.shape)


def append_positions(start, lens):
    """(request, row, position) of every row that is there."""
    return [(b, t, int(start[b]) + t) for b in range(len(start)) for t in range(int(lens[b]))]


def attention_rows(q, K, V, scale):
    """Softmax attention of one query q [128] over rows K, V [n, 128]; zeros without rows."""
    if len(K) == 0:
        return np.zeros(q.shape[-1])
    x = K @ q * scale
    w = np.exp(x - x.max())
    return (w / w.sum()) @ V
