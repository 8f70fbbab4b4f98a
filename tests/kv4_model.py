"""Plain numpy models, in 64 bits, of the 4-bit K/V format, of attention over it and of
eviction by attention weight -- TEST INFRASTRUCTURE ONLY, written from the definitions in
include/pagedkv.h and sharing no code with the library.

Pools are numpy arrays [num_blocks, num_kv_heads, block_size, row]; a 4-bit row is
head_dim * 5 / 8 bytes.
"""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32
LARGEST = 65408.0


def quantise(x) -> np.ndarray:
    """[..., D] values (exact in float64) -> uint8 [..., 5 D / 8], group by group."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    flat = x.reshape(-1, d)
    out = np.zeros((flat.shape[0], d * 5 // 8), dtype=np.uint8)
    pairs = np.zeros((flat.shape[0], d // GROUP, 2), dtype=np.float16)
    codes = np.zeros(flat.shape, dtype=np.uint8)
    for g in range(d // GROUP):
        v = flat[:, g * GROUP:(g + 1) * GROUP]
        bad = ~np.isfinite(v).all(1)
        v = np.clip(np.where(bad[:, None], 0.0, v), -LARGEST, LARGEST)
        lo = (v.min(1) + 0.0).astype(np.float16)
        spread = v.max(1).astype(np.float32) - lo.astype(np.float32)       # one fp32 rounding
        step = (np.maximum(spread, np.float32(0)) / np.float32(15)).astype(np.float16)
        up = (v.astype(np.float32) - lo.astype(np.float32)[:, None]).astype(np.float64)
        wide = np.where(step == 0, 1, step).astype(np.float64)[:, None]
        # fp64's quotient of a 24-bit by an 11-bit number is never rounded onto a tie
        c = np.clip(np.rint(up / wide), 0, 15)
        c[step == 0] = 0
        c[bad] = 0
        codes[:, g * GROUP:(g + 1) * GROUP] = c
        pairs[:, g, 0] = np.where(bad, np.float16(np.nan), step)
        pairs[:, g, 1] = np.where(bad, np.float16(np.nan), lo)
    out[:, :d // 2] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    bits = pairs.view(np.uint16).copy()
    bits[np.isnan(pairs)] = 0x7E00
    out[:, d // 2:] = bits.reshape(flat.shape[0], d // 16).view(np.uint8)
    return out.reshape(*x.shape[:-1], d * 5 // 8)


def widen(rows) -> np.ndarray:
    """uint8 [..., 5 D / 8] -> the float64 values (fp16 numbers) the rows stand for."""
    rows = np.ascontiguousarray(rows)
    d = rows.shape[-1] * 8 // 5
    flat = rows.reshape(-1, rows.shape[-1])
    codes = np.empty((flat.shape[0], d))
    codes[:, 0::2] = flat[:, :d // 2] & 15
    codes[:, 1::2] = flat[:, :d // 2] >> 4
    pairs = np.ascontiguousarray(flat[:, d // 2:]).view(np.float16).astype(np.float64).reshape(flat.shape[0], -1, 2)
    step, lo = (np.repeat(pairs[:, :, i], GROUP, axis=1) for i in (0, 1))
    return (lo + codes * step).astype(np.float16).astype(np.float64).reshape(*rows.shape[:-1], d)


def values(pool: torch.Tensor) -> np.ndarray:
    """float64 values of a CPU pool of any type."""
    return widen(pool.numpy()) if pool.dtype == torch.uint8 else pool.double().numpy()


def rows_of(pool: np.ndarray, table, n: int) -> np.ndarray:
    """[heads, n, D]: the first n rows of a sequence through its block table."""
    bs = pool.shape[2]
    idx = np.arange(n)
    blocks = np.asarray(table)[idx // bs].astype(np.int64)
    return pool[blocks, :, idx % bs].transpose(1, 0, 2)


def probabilities(q, k, scale) -> np.ndarray:
    """[heads, group, n] softmax of scale * q . k; q [heads * group, D], k [heads, n, D]."""
    x = np.matmul(q.reshape(k.shape[0], -1, k.shape[2]), k.transpose(0, 2, 1)) * scale
    if x.shape[-1] == 0:
        return x
    with np.errstate(invalid="ignore"):
        e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def decode(q, k_pool, v_pool, tables, lens, scale) -> np.ndarray:
    out = np.zeros(q.shape)
    for s, n in enumerate(np.asarray(lens).tolist()):
        if n:
            p = probabilities(q[s], rows_of(k_pool, tables[s], n), scale)
            out[s] = np.matmul(p, rows_of(v_pool, tables[s], n)).reshape(out[s].shape)
    return out


def weights(q, k_pool, tables, lens, scale, before, tracked, after) -> np.ndarray:
    """`after` with rows j < n replaced by (before where j < tracked, else 0) + summed probabilities."""
    after = np.array(after, dtype=np.float64)
    for s, n in enumerate(np.asarray(lens).tolist()):
        if n:
            p = probabilities(q[s], rows_of(k_pool, tables[s], n), scale).sum(1)
            t = n if tracked is None else min(n, int(tracked[s]))
            after[s, :, :n] = p
            after[s, :, :t] += np.asarray(before, dtype=np.float64)[s, :, :t]
    return after


def kept_rows(w, n: int, keep: int, recent: int) -> list:
    """Ascending rows kept of n with weights w: the last `recent` and the heaviest others."""
    k = min(n, keep)
    r = min(k, recent)
    light = [(-(-np.inf if np.isnan(x) else x), j) for j, x in enumerate(np.asarray(w[:n - r], dtype=np.float64))]
    return sorted([j for _, j in sorted(light)[:k - r]] + list(range(n - r, n)))
