"""Plain CPU implementations of the serving operators, in 64 bits (numpy).

Written from the definitions in ``include/gwa.h`` and sharing nothing with the
kernels: the paged cache's append and read (codes are decided in fp32, as the
definition says, so they are bit-exact), softmax attention in fp64, and the
sampling rule with real-valued masses.
"""
from __future__ import annotations

import numpy as np

GROUP = 64


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, round to nearest even (finite inputs)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rope_table(n: int, rot: int, base: float) -> np.ndarray:
    a = np.arange(n, dtype=np.float64)[:, None] * base ** (
        -np.arange(0, rot, 2, dtype=np.float64) / rot)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x: np.ndarray, table: np.ndarray, pos: np.ndarray) -> np.ndarray:
    """bf16 bits [tokens, heads, D] rotated at ``pos`` (a negative position
    turns nothing): bf16 bits."""
    rot = 2 * table.shape[1]
    if rot == 0:
        return x.copy()
    ok = pos >= 0
    cs = table[np.where(ok, pos, 0)]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    f = bf16_value(x)
    a, b = f[..., :rot // 2], f[..., rot // 2:rot]
    y = np.concatenate([a * cos - b * sin, b * cos + a * sin, f[..., rot:]], -1)
    return np.where(ok[:, None, None], bf16_round(y), x)


def quantize(x: np.ndarray, bits: int):
    """bf16 bits [..., D] -> codes uint32 [..., D], (scale, bias) bf16 bits
    [..., D/64, 2]: the affine rule, decided in fp32."""
    f = bf16_value(x).reshape(*x.shape[:-1], -1, GROUP)
    lo = (f.min(-1) + np.float32(0)).astype(np.float32)
    top = np.float32(2 ** bits - 1)
    sb = bf16_round(((f.max(-1) - lo) / top).astype(np.float32))
    s = bf16_value(sb)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint(((f - lo[..., None]) / s[..., None]).astype(np.float32))
    c = np.where(s[..., None] == 0, np.float32(0), c)
    c = np.clip(c, 0, top).astype(np.uint32)
    return c.reshape(x.shape), np.stack([sb, bf16_round(lo)], -1)


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    per = 32 // bits
    c = codes.reshape(*codes.shape[:-1], -1, per).astype(np.uint64)
    return (c << (np.arange(per, dtype=np.uint64) * np.uint64(bits))).sum(-1).astype(
        np.uint32)


def values(words: np.ndarray, par: np.ndarray, bits: int) -> np.ndarray:
    """fp64 values of packed words [..., W] and bf16 bits [..., D/64, 2]."""
    per = 32 // bits
    c = (words[..., None] >> (np.arange(per, dtype=np.uint32) * np.uint32(bits))) & np.uint32(
        2 ** bits - 1)
    G = words.shape[-1] * per // GROUP
    c = c.reshape(*words.shape[:-1], G, GROUP).astype(np.float64)
    p = bf16_value(par).astype(np.float64)
    return (p[..., 0:1] * c + p[..., 1:2]).reshape(*words.shape[:-1], G * GROUP)


def positions(q_start, kv_len, tokens: int):
    """Sequence and position of every token row (-1: of no sequence)."""
    seq = np.full(tokens, -1, dtype=np.int64)
    pos = np.full(tokens, -1, dtype=np.int64)
    for b in range(len(kv_len)):
        a, e = int(q_start[b]), int(q_start[b + 1])
        seq[a:e] = b
        pos[a:e] = np.arange(e - a) + int(kv_len[b]) - (e - a)
    return seq, pos


def attention(q, k, v, q_start, kv_len, scale: float, causal: bool):
    """fp64 [tokens, Hq, D]: q fp64 [tokens, Hq, D]; k, v lists (one a
    sequence) of fp64 [len, heads, D].  Rows of no sequence stay NaN."""
    T, Hq, D = q.shape
    out = np.full((T, Hq, D), np.nan)
    for b in range(len(kv_len)):
        a, e, n = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if e == a:
            continue
        rep = Hq // k[b].shape[1]
        for i in range(e - a):
            seen = n if not causal else n - (e - a) + i + 1
            seen = max(0, min(seen, n))
            for h in range(Hq):
                if seen == 0:
                    out[a + i, h] = 0.0
                    continue
                x = scale * (k[b][:seen, h // rep] @ q[a + i, h])
                p = np.exp(x - x.max())
                out[a + i, h] = (p / p.sum()) @ v[b][:seen, h // rep]
    return out


def sample_order(x: np.ndarray) -> np.ndarray:
    """Indices by logit, largest first, equal ones by index (NaN as -inf)."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    return np.argsort(-x, kind="stable")


def sample_masses(x: np.ndarray, T: float) -> np.ndarray:
    """Real masses relative to the largest logit's."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    m = x.max()
    if m == np.inf:
        return (x == np.inf).astype(np.float64)
    if T == np.inf:
        return (x > -np.inf).astype(np.float64)
    with np.errstate(over="ignore"):
        return np.exp((x - m) / T)
