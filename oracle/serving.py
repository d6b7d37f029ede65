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


def attention_window(q, k, v, q_start, kv_len, scale: float, window: int, sinks: int):
    """As ``attention`` with the causal mask, where a token at position p sees
    key t if t > p - window or t < sinks."""
    T, Hq, D = q.shape
    out = np.full((T, Hq, D), np.nan)
    for b in range(len(kv_len)):
        a, e, n = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if e == a:
            continue
        rep = Hq // k[b].shape[1]
        t = np.arange(n)
        for i in range(e - a):
            p = n - (e - a) + i
            see = (t <= p) & ((t > p - window) | (t < sinks))
            if not see.any():
                out[a + i] = 0.0
                continue
            ks, vs = k[b][see], v[b][see]  # [keys, heads, D]
            qs = q[a + i].reshape(-1, rep, D)
            x = scale * np.einsum("hrd,thd->hrt", qs, ks)
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[a + i] = np.einsum("hrt,thd->hrd", w, vs).reshape(Hq, D)
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


def lora(x, base, a, b, ids, scale=None, ranks=None):
    """fp64 outputs [M, N]: base [M, N] plus scale B (A x) of each token's
    adapter; a [adapters, sections, rank, K], b [adapters, N, rank], the
    sections of N given by ``base``'s list of arrays."""
    n = [t.shape[1] for t in base]
    out = [t.copy() for t in base]
    for m, e in enumerate(ids):
        if not 0 <= e < a.shape[0]:
            continue
        r = a.shape[2] if ranks is None else min(max(int(ranks[e]), 0), a.shape[2])
        at = 0
        for s, size in enumerate(n):
            t = a[e, s, :r] @ x[m]
            out[s][m] += (1.0 if scale is None else float(scale[e])) * (b[e, at:at + size, :r] @ t)
            at += size
    return out


def kept_shares(x: np.ndarray, T: float, k: int, p: float, mp: float, count=None):
    """Shares fp64 [V] of what the sampling rule keeps of a row, with real
    masses (``count``: the first so many of the order instead); zeros for a
    row without a finite logit."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    out = np.zeros(len(x))
    if x.max() == -np.inf:
        return out
    order = sample_order(x)
    if not T > 0:
        out[order[0]] = 1.0
        return out
    w = sample_masses(x, T)
    if count is None:
        count = int(k) if 0 < k < len(x) else len(x)
        if p < 1:
            ws = w[order[:count]]
            count = max(1, int((np.cumsum(ws) - ws < p * ws.sum()).sum()))
        if mp > 0:
            count = min(count, max(1, int((w[order[:count]] >= min(mp, 1.0)).sum())))
    keep = order[:count]
    out[keep] = w[keep] / w[keep].sum()
    return out


def verify(ps, qs, drafts, us, u_draw):
    """A sequence's tokens and how many drafts stand: ps the shares of its
    rows, qs of its drafts' rows (None: certain), one fewer."""
    fell = len(drafts)
    for j, d in enumerate(drafts):
        q = qs[j][d] if qs is not None else 1.0
        if not us[j] * q < ps[j][d]:
            fell = j
            break
    rest = ps[fell].copy()
    if fell < len(drafts):
        if qs is None:
            rest[drafts[fell]] = 0.0
        else:
            rest = np.maximum(rest - qs[fell], 0.0)
        if rest.sum() == 0:
            rest = ps[fell].copy()
    c = np.cumsum(rest)
    drawn = int(np.searchsorted(c, u_draw * c[-1], side="right")) if c[-1] > 0 else -1
    return list(drafts[:fell]) + [drawn], fell
