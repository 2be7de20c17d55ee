"""Rotary positions, draft trees and moved rows of a paged KV cache, from their definitions
(fp64, whole numbers), row by row."""
from __future__ import annotations

import numpy as np

from . import numerics as nm
from .attention import cache_rows

__all__ = ["rope", "rope_ragged_paged", "kv_read_ragged_paged", "kv_keep_ragged_paged", "release_ragged_paged",
           "attention_tree_ragged_paged", "tree_mask"]

_TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288")


def rope(x, position: int, inv_freq, interleaved: bool, amplitude: float):
    """One token's heads [H, D] (fp64) turned: pair i by position * inv_freq[i]. The angle is reduced
    in 64 bits of significand, which hold the product of 31 and 24."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    angle = np.longdouble(position) * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    angle = (angle - np.rint(angle / _TWO_PI) * _TWO_PI).astype(np.float64)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = float(np.float32(amplitude)) * np.cos(angle), float(np.float32(amplitude)) * np.sin(angle)
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def rope_ragged_paged(q_bits, k_bits, v_bits, row_offsets, cache_lengths, page_table, page_size: int, inv_freq,
                      positions=None, interleaved: bool = False, amplitude: float = 1.0):
    """(q, k, v, page, slot): exact turned queries and keys and the values [T', H, D] of the rows that
    sequences cover, and where in a plane each row's key and value go. q_bits, or k_bits and v_bits,
    may be None."""
    T = int(row_offsets[-1])
    page, slot, where = np.zeros(T, np.int64), np.zeros(T, np.int64), np.zeros(T, np.int64)
    for b in range(len(row_offsets) - 1):
        for r in range(int(row_offsets[b]), int(row_offsets[b + 1])):
            p = int(cache_lengths[b]) + r - int(row_offsets[b])
            page[r], slot[r] = int(page_table[b, p // page_size]) if k_bits is not None else 0, p % page_size
            where[r] = p if positions is None else int(positions[r])
    def turned(bits):
        if bits is None:
            return None
        x = nm.decode_bf16(bits[:T])
        with np.errstate(invalid="ignore"):
            return np.stack([rope(x[r], where[r], inv_freq, interleaved, amplitude) for r in range(T)]) if T else x
    return turned(q_bits), turned(k_bits), None if v_bits is None else nm.decode_bf16(v_bits[:T]), page, slot


def kv_read_ragged_paged(row_offsets, first_positions, blocks, page_table, layer: int, scales=None, G: int = 0):
    """Keys and values [2, T', Hkv, D] (fp64) of the ranges."""
    out = []
    for plane in (0, 1):
        rows = [np.zeros((0,) + blocks.shape[4:])]
        for b in range(len(row_offsets) - 1):
            n = int(row_offsets[b + 1]) - int(row_offsets[b])
            first = 0 if first_positions is None else int(first_positions[b])
            S = blocks.shape[3]
            pos = np.arange(first, first + n)
            page, slot = page_table[b][pos // S].astype(np.int64), pos % S
            raw = blocks[layer, plane, page, slot]
            rows.append(nm.decode_bf16(raw) if scales is None else
                        nm.decode_e4m3(raw) * np.repeat(scales[layer, plane, page, slot].astype(np.float64), G, axis=-1))
        out.append(np.concatenate(rows))
    return np.stack(out)


def kv_keep_ragged_paged(path, kept, blocks, cache_lengths, page_table, scales=None):
    """(blocks, scales) after the moves, one row after the other."""
    blocks = blocks.copy()
    scales = None if scales is None else scales.copy()
    S = blocks.shape[3]
    for b in range(len(kept)):
        c = int(cache_lengths[b])
        for i in range(min(int(kept[b]), path.shape[1])):
            if path[b, i] <= i:
                continue
            of, to = c + int(path[b, i]), c + i
            for t in (blocks, scales):
                if t is not None:
                    t[:, :, page_table[b, to // S], to % S] = t[:, :, page_table[b, of // S], of % S]
    return blocks, scales


def release_ragged_paged(free_pages, page_table, held, kept, free_count: int, page_size: int):
    """(free_pages, result); free_pages is None where the status in result[1] is not 0."""
    W = page_table.shape[1]
    back, status = [], 0
    for b in range(len(held)):
        h, k = int(held[b]), int(kept[b])
        first, last = -(-k // page_size), -(-h // page_size)
        if last > first and h > W * page_size:
            status |= 2
        back += [int(page_table[b, i]) if i < W else -1 for i in range(first, min(last, W + 1))] if last - first < 10**6 else []
        if last - first >= 10**6:
            status |= 1
    if free_count + len(back) > len(free_pages):
        status |= 1
    if status:
        return None, (int(free_count), status)
    out = free_pages.copy()
    out[free_count:free_count + len(back)] = back[::-1]
    return out, (free_count + len(back), 0)


def tree_mask(parents, words: int):
    """Rows of the mask, u32 [n, words], of one sequence's tree: a token's ancestors and itself.
    parents[j] < j, or -1 for a root."""
    seen = []
    for j, p in enumerate(parents):
        seen.append(1 << j | (seen[p] if p >= 0 else 0))
    return np.array([[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in seen], np.uint32).reshape(len(seen), words)


def attention_tree_ragged_paged(q_bits, row_offsets, mask, blocks, cache_lengths, page_table, layer: int, scale: float,
                                window: int = 0, scales=None, G: int = 0):
    """Returns (out, spread, size) as attention_ragged_paged does; rows that see nothing are zeros."""
    T, Hq, D = q_bits.shape
    Hkv = blocks.shape[4]
    q = nm.decode_bf16(q_bits)
    out, spread, size = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(len(row_offsets) - 1):
            r0, n, c = int(row_offsets[b]), int(row_offsets[b + 1]) - int(row_offsets[b]), int(cache_lengths[b])
            if n == 0:
                continue
            k = cache_rows(blocks, page_table[b], c + n, layer, 0, scales, G)
            v = cache_rows(blocks, page_table[b], c + n, layer, 1, scales, G)
            for r in range(r0, r0 + n):
                drafted = [i for i in range(min(n, 32 * mask.shape[1])) if int(mask[r, i // 32]) >> i % 32 & 1]
                first = max(0, c - max(window - len(drafted), 0)) if window else 0
                see = np.concatenate([np.arange(first, c), c + np.array(drafted, np.int64)]).astype(np.int64)
                for h in range(Hq):
                    g = h // (Hq // Hkv)
                    kk, vv = k[see, g], v[see, g]
                    if len(see) == 0:
                        out[r, h] = spread[r, h] = size[r, h] = 0
                        continue
                    s = scale * (kk @ q[r, h])
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[r, h] = w @ vv
                    spread[r, h] = w @ np.abs(vv)
                    size[r, h] = (scale * (np.abs(kk) @ np.abs(q[r, h]))).max()
    return out, spread, size
