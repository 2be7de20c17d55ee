"""kv_read_ragged_paged and kv_keep_ragged_paged on the GPU: moved rows are equal to the oracle's, and
values read back to code * scale rounded once."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import Guarded, bf16v, dev16, dev32, devf32, host16, say

pytestmark = pytest.mark.gpu


def cache(d):
    return torch.from_numpy(d.blocks).cuda() if d.gran else dev16(d.blocks, torch.bfloat16)


def bits(t, gran):
    torch.cuda.synchronize()
    return t.cpu().numpy() if gran else host16(t)


def read(lib, d, counts, first, kind=torch.bfloat16, planes=(True, True), spare=3, stream=None):
    """k and v, with the rows that no sequence covers still 7."""
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.uint32)
    shape = (int(offs[-1]) + spare, *d.blocks.shape[4:])
    out = [torch.full(shape, 7.0, dtype=kind, device="cuda") if p else None for p in planes]
    torch.cuda.synchronize()
    lib.kv_read_ragged_paged(*out, dev32(offs), None if first is None else dev32(np.asarray(first, np.uint32)), cache(d),
                             dev32(d.page_table), d.layer_idx, kv_scales=devf32(d.scales) if d.gran else None,
                             quantization_granularity=d.gran, stream=stream)
    torch.cuda.synchronize()
    return offs, out


def check_read(lib, d, counts, first, **how):
    say(f"[read] cache {d.blocks.shape} gran {d.gran} rows {sum(counts)} {how}")
    offs, out = read(lib, d, counts, first, **how)
    want = oracle.kv_read_ragged_paged(offs, first, d.blocks, d.page_table, d.layer_idx, d.scales, d.gran)
    n = int(offs[-1])
    for plane, t in enumerate(out):
        if t is None:
            continue
        assert (t[n:] == 7).all(), "rows behind the last sequence changed"
        x = want[plane].astype(np.float32)      # exact for bf16; a code times its scale has 4 + 24 bits: one rounding
        if t.dtype == torch.float32:
            assert np.array_equal(t[:n].cpu().numpy(), x)
        else:   # rounded to fp32, then to bf16: as the formula says
            assert np.array_equal(host16(t[:n]), synth.bf16_bits(x.astype(np.float64)))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,dim,gran", [(1, 8, 0), (2, 64, 0), (3, 72, 0), (8, 128, 0), (1, 256, 0), (1, 32, 32), (3, 32, 32), (2, 64, 64),
                                          (8, 128, 32), (8, 128, 128), (5, 96, 32), (1, 256, 64)])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_read(lib, gpu, hkv, dim, gran, kind, page):
    new, hist = [3, 1, 1, 20, 2], [40, 5, 40, 61, 130]
    d = synth.attention_inputs(1, new, hist, hq=hkv, hkv=hkv, d=dim, page=page, gran=gran)
    check_read(lib, d, [30, 0, 1, 81, 2], [13, 0, 40, 0, 130], kind=kind)


@pytest.mark.parametrize("gran", [0, 32])
def test_read_from_the_start_and_one_plane(lib, gpu, gran):
    d = synth.attention_inputs(2, [1, 1, 1], [30, 7, 400], hq=2, hkv=2, d=64, gran=gran)
    check_read(lib, d, [31, 8, 401], None)
    for planes in ((True, False), (False, True)):
        check_read(lib, d, [5, 0, 300], [20, 0, 70], planes=planes)


@pytest.mark.parametrize("batch", [1, 64, 65, 700, 4100])
def test_read_of_many_sequences(lib, gpu, batch):
    rng = np.random.default_rng(batch)
    d = synth.attention_inputs(3, np.ones(batch, int), rng.integers(0, 12, batch), hq=1, hkv=1, d=32, gran=32, page=4)
    counts = np.minimum(rng.integers(0, 6, batch) * rng.integers(0, 2, batch), d.cache_lengths.astype(int) + 1)
    counts[-1] = 1
    check_read(lib, d, counts.tolist(), (d.cache_lengths.astype(int) + 1 - counts).tolist())


def test_read_behind_many_empty_sequences(lib, gpu):
    d = synth.attention_inputs(4, [1] * 300, [20] * 300, hq=1, hkv=1, d=16, page=8)
    counts = [0] * 300
    counts[0], counts[280] = 3, 19
    check_read(lib, d, counts, [2] * 300)


def test_read_keeps_every_bit_of_a_bf16_cache(lib, gpu):
    """NaN with its payload, infinities, subnormal numbers and -0."""
    d = synth.attention_inputs(5, [1], [40], hq=1, hkv=1, d=64)
    rng = np.random.default_rng(0)
    held = d.blocks[d.layer_idx] != 0xFFFF
    d.blocks[d.layer_idx] = np.where(held, rng.integers(0, 1 << 16, d.blocks[0].shape), 0xFFFF).astype(np.uint16)
    offs, out = read(lib, d, [41], None)
    for plane in (0, 1):
        pos = np.arange(41)
        raw = d.blocks[d.layer_idx, plane, d.page_table[0, pos // 16], pos % 16]
        assert np.array_equal(host16(out[plane])[:41], raw)


def test_read_on_another_stream_and_replayed(lib, gpu):
    d = synth.attention_inputs(6, [1, 1], [50, 90], hq=2, hkv=2, d=64, gran=64)
    check_read(lib, d, [20, 60], [1, 30], stream=torch.cuda.Stream())
    blocks, scales, table = cache(d), devf32(d.scales), dev32(d.page_table)
    offs, first = dev32(np.array([0, 20, 50], np.int32)), dev32(np.array([0, 0], np.int32))
    k, v = (torch.zeros(50, 2, 64, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kv_read_ragged_paged(k, v, offs, first, blocks, table, d.layer_idx, kv_scales=scales, quantization_granularity=64)
        first.add_(7)
    for turn in range(3):
        k.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        want = oracle.kv_read_ragged_paged([0, 20, 50], [7 * turn] * 2, d.blocks, d.page_table, d.layer_idx, d.scales, 64)
        assert np.array_equal(k.cpu().numpy(), want[0].astype(np.float32)) and np.array_equal(v.cpu().numpy(), want[1].astype(np.float32))
        _ = (torch.ones(1000, device="cuda") * 2).sum().item()


def drafts(seed, drafted, hist, hkv, dim, gran, page, layers):
    """A cache whose every byte differs, in all layers."""
    d = synth.attention_inputs(seed, drafted, hist, hq=hkv, hkv=hkv, d=dim, gran=gran, page=page, layers=layers)
    rng = np.random.default_rng(seed)
    d.blocks[:] = rng.integers(0, 256 if gran else 65536, d.blocks.shape).astype(d.blocks.dtype)
    if gran:
        d.scales[:] = rng.random(d.scales.shape)
    return d


def keep(lib, d, path, kept, stream=None):
    blocks, scales = cache(d), devf32(d.scales) if d.gran else None
    torch.cuda.synchronize()
    lib.kv_keep_ragged_paged(dev32(np.asarray(path, np.int32)), dev32(np.asarray(kept, np.int32)), blocks, dev32(d.cache_lengths),
                             dev32(d.page_table), kv_scales=scales, quantization_granularity=d.gran, stream=stream)
    torch.cuda.synchronize()
    return bits(blocks, d.gran), None if scales is None else scales.cpu().numpy()


def check_keep(lib, d, path, kept, stream=None):
    path, kept = np.asarray(path, np.int32), np.asarray(kept, np.uint32)
    say(f"[keep] cache {d.blocks.shape} gran {d.gran} path {path.shape} kept {kept[:6].tolist()}")
    got, got_s = keep(lib, d, path, kept, stream)
    want, want_s = oracle.kv_keep_ragged_paged(path, kept, d.blocks, d.cache_lengths, d.page_table, d.scales)
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {got.size} elements differ"
    assert not d.gran or np.array_equal(got_s, want_s)


def paths(rng, drafted, width):
    """Random increasing paths; entries from the kept ones on are wild."""
    out, kept = np.full((len(drafted), width), -(1 << 30), np.int32), []
    out[:, ::2] = 1 << 30
    for b, n in enumerate(drafted):
        m = int(rng.integers(0, min(n, width) + 1))
        out[b, :m] = np.sort(rng.choice(n, m, replace=False))
        kept.append(m)
    return out, kept


@pytest.mark.parametrize("hkv,dim,gran", [(1, 8, 0), (2, 64, 0), (3, 72, 0), (8, 128, 0), (1, 32, 32), (3, 32, 32), (2, 96, 32), (8, 128, 128),
                                          (1, 256, 64)])
@pytest.mark.parametrize("page", [1, 16, 48])
@pytest.mark.parametrize("layers", [1, 5])
def test_keep(lib, gpu, hkv, dim, gran, page, layers):
    rng = np.random.default_rng(dim + page)
    drafted = [20, 1, 0, 8, 33, 13]
    d = drafts(7, drafted, [5, 40, 3, 0, 61, 15], hkv, dim, gran, page, layers)
    check_keep(lib, d, *paths(rng, drafted, 12))


def test_keep_of_long_paths(lib, gpu):
    """More moves than are found, or read, at a time: rows that are read lie behind those written."""
    n = 300
    d = drafts(8, [n, n, n, n], [5, 0, 17, 30], 1, 16, 0, 16, 2)
    every = np.arange(n)
    path = np.zeros((4, 200), np.int32)
    path[0] = every[100:300]
    path[1] = every[1:201]
    path[2, :150] = every[::2]
    path[3] = np.concatenate([every[:70], every[75:145], every[240:300]])
    check_keep(lib, d, path, [200, 200, 150, 200])


def test_keep_nothing_and_everything(lib, gpu):
    d = drafts(9, [4, 4, 4], [3, 3, 3], 2, 32, 32, 16, 3)
    check_keep(lib, d, [[1, 2, 3], [0, 1, 2], [0, 2, 3]], [0, 3, 1])
    check_keep(lib, d, [[1, 2, 3], [0, 1, 3], [0, 2, 3]], [3, 9, 0xFFFFFFFF])      # more than the path has count as its length


def test_keep_of_many_sequences(lib, gpu):
    rng = np.random.default_rng(10)
    drafted = rng.integers(0, 9, 700)
    d = drafts(10, drafted, rng.integers(0, 20, 700), 1, 8, 0, 8, 2)
    check_keep(lib, d, *paths(rng, drafted, 8))


def test_keep_on_another_stream_and_replayed(lib, gpu):
    rng = np.random.default_rng(11)
    drafted = [20, 30]
    d = drafts(11, drafted, [5, 9], 2, 64, 64, 16, 2)
    path, kept = paths(rng, drafted, 9)
    check_keep(lib, d, path, kept, stream=torch.cuda.Stream())
    blocks, scales = cache(d), devf32(d.scales)
    table, lengths, p, m = dev32(d.page_table), dev32(d.cache_lengths), dev32(path), dev32(np.array([3, 5], np.int32))
    p.copy_(dev32(np.array([[0, 2, 4, 6, 8, 10, 12, 14, 15], [1, 2, 3, 5, 6, 8, 11, 12, 13]], np.int32)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kv_keep_ragged_paged(p, m, blocks, lengths, table, kv_scales=scales, quantization_granularity=64)
        lengths.add_(1)
    want, want_s, at = d.blocks, d.scales, d.cache_lengths.copy()
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        want, want_s = oracle.kv_keep_ragged_paged(p.cpu().numpy(), [3, 5], want, at, d.page_table, want_s)
        at = at + 1
        assert np.array_equal(blocks.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), want_s)
        _ = (torch.ones(1000, device="cuda") * 2).sum().item()


def test_rows_past_32_bit_offsets(lib, gpu):
    """Planes of more than 4 GB, the pages in use at their ends."""
    d = drafts(12, [9, 6], [5, 0], 8, 128, 0, 128, 1)
    used, pages = d.blocks.shape[2], (5 << 30) // (128 * 8 * 128 * 2)
    blocks = torch.empty((1, 2, pages, 128, 8, 128), dtype=torch.bfloat16, device="cuda")
    blocks[:, :, pages - used:] = cache(d)
    table = d.page_table.astype(np.int64)
    table[table != 0xFFFFFFFF] += pages - used
    table = dev32(table.astype(np.uint32))
    path = np.array([[0, 3, 8], [1, 2, 5]], np.int32)
    lib.kv_keep_ragged_paged(dev32(path), dev32(np.array([3, 3], np.int32)), blocks, dev32(d.cache_lengths), table)
    want, _ = oracle.kv_keep_ragged_paged(path, [3, 3], d.blocks, d.cache_lengths, d.page_table)
    assert np.array_equal(host16(blocks[:, :, pages - used:]), want)
    k, v = (torch.zeros(20, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv_read_ragged_paged(k, v, dev32(np.array([0, 14, 20], np.int32)), None, blocks, table, 0)
    for plane, t in ((0, k), (1, v)):
        rows = [want[0, plane, d.page_table[b, p // 128], p % 128] for b, n in ((0, 14), (1, 6)) for p in range(n)]
        assert np.array_equal(host16(t), np.stack(rows))


def test_refusals_with_device_tensors(lib, gpu):
    d = drafts(13, [4], [3], 2, 64, 0, 16, 2)
    blocks, table, lengths = cache(d), dev32(d.page_table), dev32(d.cache_lengths)
    path, kept = dev32(np.array([[1, 3]], np.int32)), dev32(np.array([2], np.int32))
    k = torch.full((4, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    offs = dev32(np.array([0, 4], np.int32))
    with pytest.raises(lib.QgError):
        lib.kv_keep_ragged_paged(path.long(), kept, blocks, lengths, table)
    with pytest.raises(ValueError):
        lib.kv_keep_ragged_paged(path, kept, blocks, lengths[:0], table)
    with pytest.raises(ValueError):
        lib.kv_keep_ragged_paged(path.cpu(), kept, blocks, lengths, table)
    with pytest.raises(lib.QgError):
        lib.kv_read_ragged_paged(k, k.float(), offs, None, blocks, table, 1)
    with pytest.raises(ValueError):
        lib.kv_read_ragged_paged(k.transpose(0, 1), None, offs, None, blocks, table, 1)
    with pytest.raises(lib.QgError):
        lib.kv_read_ragged_paged(k, None, offs, None, blocks, table, 2)
    assert np.array_equal(host16(blocks), d.blocks) and (k == 7).all()


@pytest.mark.parametrize("hkv,dim,gran", [(1, 8, 0), (1, 32, 32), (1, 128, 0), (2, 128, 128), (4, 72, 0), (16, 256, 0), (16, 256, 64), (3, 1024, 0)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_read_in_workgroups_of_few_and_of_many_rows(lib, gpu, hkv, dim, gran, kind):
    """Up to 64 rows of a workgroup, of as many sequences (with empty ones between), or of one."""
    rng = np.random.default_rng(3)
    new = np.where(rng.random(2000) < 0.5, rng.integers(0, 40, 2000), 0) if hkv * dim <= 512 else rng.integers(0, 4, 120)
    for counts in (new, np.array([int(new.sum()), 0, 1])):
        history = rng.integers(0, 30, len(counts))
        d = synth.attention_inputs(21, counts, history, hq=hkv, hkv=hkv, d=dim, page=16, gran=gran, layers=1)
        check_read(lib, d, counts, rng.integers(0, history + 1), kind=kind)
