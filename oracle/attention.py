"""Attention over a paged KV cache, and the cache's tables, from their definitions (fp64,
whole numbers), sequence by sequence and head by head."""
from __future__ import annotations

import numpy as np

from . import numerics as nm

__all__ = ["attention_ragged_paged", "cache_rows", "tables_ragged_paged"]


def cache_rows(blocks, page_table_row, length: int, layer: int, plane: int, scales=None, G: int = 0):
    """Values [length, Hkv, D] (fp64) of one sequence's positions 0 .. length - 1: blocks are
    bf16 bit patterns, or e4m3 codes (uint8) with f32 scales."""
    S = blocks.shape[3]
    pos = np.arange(length)
    page, slot = page_table_row[pos // S].astype(np.int64), pos % S
    raw = blocks[layer, plane, page, slot]
    if scales is None:
        return nm.decode_bf16(raw)
    return nm.decode_e4m3(raw) * np.repeat(scales[layer, plane, page, slot].astype(np.float64), G, axis=-1)


def attention_ragged_paged(q_bits, row_offsets, blocks, cache_lengths, page_table, layer: int, scale: float,
                           causal: bool = True, window: int = 0, scales=None, G: int = 0):
    """Returns (out, spread, size): the exact output [T, Hq, D] (NaN in rows that no sequence
    covers), the same weighted mean of |v| in place of v, and for each (row, head) the
    largest scale * sum |q| |k| over the visible positions."""
    T, Hq, D = q_bits.shape
    Hkv = blocks.shape[4]
    q = nm.decode_bf16(q_bits)
    out = np.full((T, Hq, D), np.nan)
    spread = np.full((T, Hq, D), np.nan)
    size = np.full((T, Hq), np.nan)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(len(row_offsets) - 1):
            r0, n, c = int(row_offsets[b]), int(row_offsets[b + 1]) - int(row_offsets[b]), int(cache_lengths[b])
            if n == 0:
                continue
            k = cache_rows(blocks, page_table[b], c + n, layer, 0, scales, G)
            v = cache_rows(blocks, page_table[b], c + n, layer, 1, scales, G)
            for j in range(n):
                last = c + j if causal else c + n - 1
                first = max(0, last - window + 1) if window else 0
                for h in range(Hq):
                    g = h // (Hq // Hkv)
                    kk, vv = k[first:last + 1, g], v[first:last + 1, g]
                    s = scale * (kk @ q[r0 + j, h])
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[r0 + j, h] = w @ vv
                    spread[r0 + j, h] = w @ np.abs(vv)
                    size[r0 + j, h] = (scale * (np.abs(kk) @ np.abs(q[r0 + j, h]))).max()
    return out, spread, size


def tables_ragged_paged(page_table, cache_lengths, new_lengths, free_pages, free_count: int, page_size: int,
                        slots: int | None):
    """(offsets, page_table, slot_map, result); offsets, page_table and slot_map are None where
    the status in result[1] is not 0. `slots`: elements of the slot map, None without one."""
    B, W = page_table.shape
    left, status = int(free_count), 0
    table, offs, slot = page_table.copy(), [0], []
    short = free_count > len(free_pages)
    for b in range(B):
        c, n = int(cache_lengths[b]), int(new_lengths[b])
        offs.append(offs[-1] + n)
        if n == 0:
            continue
        held, need = -(-c // page_size), -(-(c + n) // page_size)
        if need > W:
            status |= 2
        for i in range(held, need):
            left -= 1
            if left < 0 or short:
                short = True
            elif need <= W:
                table[b, i] = free_pages[left]
        if need <= W:
            slot += [int(table[b, p // page_size]) * page_size + p % page_size for p in range(c, c + n)]
    if short:
        status |= 1
    if offs[-1] > (2**31 - 1 if slots is None else slots):
        status |= 4
    if status:
        return None, None, None, (int(free_count), status)
    return np.array(offs), table, np.array(slot, dtype=np.int64), (left, 0)
