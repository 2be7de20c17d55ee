"""Which form of the attention kernels a call takes, worked out from its sizes as the library's
launcher does, so that a test can say that its case is of the form that it means to test."""
import numpy as np

ROWS_TARGET = 512          # shares of the kernel for few rows, at most
WIDE_BLOCKS = 8            # blocks per wave from which a workgroup takes several heads
TILE_TARGET, TILE_CHUNK, TILE_STEP = 512, 256, 64


def new_lengths(d):
    return np.diff(d.row_offsets.astype(np.int64))


def kernel(d, cus):
    """'rows1', 'rows2' (16 or 32 rows per tile) or 'tile'."""
    batch, hkv = len(d.cache_lengths), d.blocks.shape[4]
    rows = d.q.shape[0] * (d.q.shape[1] // hkv)
    if rows <= 16 * batch:
        return "rows1"
    few = rows <= 32 * batch and (4 * batch * hkv > cus or (d.gran and d.q.shape[2] > 128))
    return "rows2" if few else "tile"


def heads_per_workgroup(d, cus, window=0):
    """Of the kernel for few rows: 1, or 2 or 4 where there is much to read."""
    form = kernel(d, cus)
    assert form != "tile"
    hkv, D = d.blocks.shape[4], d.q.shape[2]
    group = d.q.shape[1] // hkv
    mt = int(form[-1])
    dp = 64 if D <= 64 else 128 if D <= 128 else 256
    waves = 2 if dp == 256 else 4
    block = 2 * dp * (1 if d.gran else 2) * 16                       # a block's keys, or values, in LDS
    runs = dp // d.gran if d.gran else 1
    lds = waves * 2 * 2 * block + 4 * (waves if d.gran else 1) * 2 * runs * 64 + 4096 + 4 * waves * (32 * mt + 1)
    target = min(cus * max(1, min(163840 // (lds + 128), 8 // waves)), ROWS_TARGET)
    heads = waves
    while hkv % heads:
        heads //= 2
    groups = hkv // heads
    new = new_lengths(d)
    length = new + d.cache_lengths.astype(np.int64)
    if window:
        length = np.minimum(length, window + (16 * mt - 1) // group + 1 + 32)
    units = int((-(-new * group // (16 * mt)) * -(-length // 32)).sum())
    return heads if units * groups >= WIDE_BLOCKS * max(target, groups) else 1


def tile_cuts(d, window=0):
    """Of the kernel for many rows: the chunk, and how many chunks each sequence's tiles get."""
    hkv = d.blocks.shape[4]
    group = d.q.shape[1] // hkv
    target = max(TILE_TARGET, 1 << (hkv - 1).bit_length())
    new = new_lengths(d)
    span = new + d.cache_lengths.astype(np.int64)
    if window:
        span = np.minimum(span, window + 127 // group + 1 + TILE_STEP)
    tiles = -(-new * group // 128)
    chunk = max(-(-int((tiles * span).sum()) * hkv // target), TILE_CHUNK)
    chunk = -(-chunk // TILE_STEP) * TILE_STEP
    return chunk, np.where(tiles > 0, -(-span // chunk), 0)
