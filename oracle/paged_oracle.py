"""fp64 reference of the paged-cache operators: rotary positions, attention of new tokens over
pages, the weight each key gathers, eviction. Loops and plain numpy, from the definitions."""
from __future__ import annotations

import math

import numpy as np

D = 128


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, low=1.0, high=4.0,
                     original_len=0):
    """(angle per position of each pair, magnitude)."""
    n = rot_dim // 2
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(n)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        turns = original_len * f / (2 * math.pi)
        w = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return f * (w + (1 - w) / factor), 1.0
    if scaling == "yarn":
        # the (real) pair index that turns `t` times over the original length
        index = lambda t: rot_dim * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
        a, z = max(0.0, math.floor(index(high))), min(rot_dim - 1.0, math.ceil(index(low)))
        z = max(z, a + 0.001)
        w = np.clip(1.0 - (np.arange(n) - a) / (z - a), 0.0, 1.0)
        return f * (w + (1 - w) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, positions, freq, magnitude, interleaved=False, transpose=False):
    """x [..., H, 128], positions [...]: the first 2 len(freq) dims rotated."""
    x = np.asarray(x, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[..., None, None] * freq
    c, s = magnitude * np.cos(ang), magnitude * np.sin(ang)
    if transpose:
        s = -s
    n = len(freq)
    y = x.copy()
    ia = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def gather(pool, table, b, g, n):
    """Tokens [0, n) of sequence b, KV head g: [n, 128] fp64."""
    page = pool.shape[2]
    j = np.arange(n)
    return np.asarray(pool[table[b, j // page], g, j % page], dtype=np.float64)


def attend(q, K, V, table, q_start, kv_len, window=0, scale=None):
    """Per row (token, query head): out, out with |V|, lse, the largest sum |q k| of a score (a
    bound for rounding errors), and per (sequence, KV head) the weights [B, Hkv, max kv_len].
    Rows outside every sequence are NaN."""
    q = np.asarray(q, dtype=np.float64)
    total, Hq = q.shape[:2]
    Hkv = K.shape[1]
    G = Hq // Hkv
    B = len(kv_len)
    scale = 1 / math.sqrt(D) if not scale else scale
    out, out_abs = (np.full((total, Hq, D), np.nan) for _ in range(2))
    lse, size = (np.full((total, Hq), np.nan) for _ in range(2))
    weights = np.zeros((B, Hkv, max([0, *kv_len])))
    for b in range(B):
        lo, hi, kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        n = hi - lo
        if n == 0:
            continue
        p = kv - n + np.arange(n)[:, None]
        j = np.arange(kv)[None]
        seen = (j <= p) & ((j > p - window) if window else True)
        used = seen.any(0)
        for g in range(Hkv):
            k, v = gather(K, table, b, g, kv), gather(V, table, b, g, kv)
            k[~used], v[~used] = 0.0, 0.0
            for h in range(g * G, g * G + G):
                x = q[lo:hi, h]
                s = np.where(seen, scale * (x @ k.T), -np.inf)
                m = s.max(1, initial=-np.inf)
                e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
                total_e = e.sum(1)
                with np.errstate(divide="ignore"):
                    lse[lo:hi, h] = m + np.log(total_e)
                e /= np.where(total_e > 0, total_e, 1.0)[:, None]
                out[lo:hi, h], out_abs[lo:hi, h] = e @ v, e @ np.abs(v)
                size[lo:hi, h] = np.where(seen, scale * (np.abs(x) @ np.abs(k).T), 0.0).max(1, initial=0.0)
                weights[b, g, :kv] += e.sum(0)
    return out, out_abs, lse, size, weights


def evict_index(weights, kv_len, keep, sink, recent):
    """Kept cache indices [B, Hkv, keep], ascending, -1 behind the last."""
    B, Hkv, _ = weights.shape
    index = np.full((B, Hkv, keep), -1, dtype=np.int32)
    for b in range(B):
        kv = int(kv_len[b])
        m = min(kv, keep)
        for g in range(Hkv):
            def rank(j):
                w = float(weights[b, g, j])
                held = j < sink or j >= kv - recent
                return (0 if held else 1, math.isnan(w), 0.0 if math.isnan(w) or held else -w, j)
            index[b, g, :m] = sorted(sorted(range(kv), key=rank)[:m])
    return index
