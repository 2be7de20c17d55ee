"""attention_ragged_paged on the GPU against the 64-bit oracle.

Tolerance, per element, with A = sum_i w_i |v_i| (w: the exact softmax weights), N visible
positions, D head dims and Z = the largest scale * sum |q| |k|:
  * each probability (times its value scale) is rounded to bf16 once: 2^-8 of A;
  * the output is rounded to bf16 once: 2^-8 |out|;
  * a score is a sum of D exact products in fp32, D * 2^-23 Z at most (each addition off by
    at most one unit in the last place, whatever way the matrix instruction rounds), plus
    three fp32 roundings of values up to Z (scales, base-2 exponent, its maximum) in this
    score and in the maximum's: a weight is off by (2 D + 8) 2^-23 Z;
  * exp2 and the sums over N positions add (N + 16) 2^-23 of A, the rescalings by a new
    maximum (one per 32 positions, two roundings each) stay inside it;
  * all of it twice, since the weights' sum in the denominator has the same error.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import Guarded, bf16v, dev16, dev32, devf32, host16, say

pytestmark = pytest.mark.gpu


def place(d):
    return dict(q=dev16(d.q, torch.bfloat16), offs=dev32(d.row_offsets),
                blocks=torch.from_numpy(d.blocks).cuda() if d.gran else dev16(d.blocks, torch.bfloat16),
                lengths=dev32(d.cache_lengths), table=dev32(d.page_table),
                scales=devf32(d.scales) if d.gran else None)


def workspace(lib, d):
    hq, hd = d.q.shape[1:]
    n = lib.attention_ragged_paged_workspace(d.q.shape[0], len(d.cache_lengths), hq, d.blocks.shape[4], hd)
    return torch.full((n,), float("nan"), device="cuda")   # its content has no meaning


def call(lib, d, dev, out, ws, scale, causal=True, window=0, stream=None):
    lib.attention_ragged_paged(out, dev["q"], dev["offs"], dev["blocks"], dev["lengths"], dev["table"], d.layer_idx,
                               scale, ws, causal=causal, window=window, kv_scales=dev["scales"],
                               quantization_granularity=d.gran, stream=stream)


def run(lib, d, scale, causal=True, window=0):
    out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
    call(lib, d, place(d), out.view, workspace(lib, d), scale, causal, window)
    assert out.bands_intact(), "bytes around the output changed"
    return host16(out.view)


def exact(d, scale, causal=True, window=0):
    return oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table, d.layer_idx, scale,
                                         causal, window, d.scales, d.gran)


def tolerance(d, ref):
    out, spread, size = ref
    n = int((d.cache_lengths.astype(np.int64) + np.diff(d.row_offsets.astype(np.int64))).max())
    D = d.q.shape[2]
    small = 2 * ((2 * D + 8) * size[..., None] + n + 16) * 2.0**-23
    return 2.0**-8 * (spread + np.abs(out)) * (1 + 2.0**-7) + spread * small


def compare(d, got, ref, what=""):
    out, _, _ = ref
    rows = int(d.row_offsets[-1])
    assert (got[rows:] == 0x7FC1).all(), "rows behind the last sequence changed"
    g, o = bf16v(got[:rows]), out[:rows]
    bad = np.isnan(o) != np.isnan(g)
    assert not bad.any(), f"{what}: NaN at {np.argwhere(bad)[:4].tolist()} on one side only"
    fine = np.isfinite(o)
    assert np.array_equal(g[~fine & ~np.isnan(o)], o[~fine & ~np.isnan(o)]), what
    tol = tolerance(d, ref)[:rows]
    err = np.abs(np.where(fine, g, 0) - np.where(fine, o, 0))
    over = fine & (err > tol)
    if over.any():
        i = tuple(np.argwhere(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.size} off, first at {i}: {g[i]} for {o[i]}, tolerance {tol[i]}")
    return float((err[fine] / np.maximum(tol[fine], 1e-300)).max(initial=0.0))


def check(lib, d, scale=None, causal=True, window=0, what=""):
    scale = d.q.shape[2] ** -0.5 if scale is None else scale
    say(f"[attention] {what} q {d.q.shape} lengths {d.cache_lengths[:6].tolist()} cache {d.blocks.shape} gran {d.gran} "
        f"causal {causal} window {window}")
    got = run(lib, d, scale, causal, window)
    used = compare(d, got, exact(d, scale, causal, window), what)
    say(f"[attention]   worst element at {used:.2f} of its tolerance")
    return got


# few rows per sequence, and many: one kernel for each
RAGGED = ([3, 0, 1, 7, 2], [0, 5, 40, 61, 130])
CHUNKS = ([70, 0, 33, 1, 129], [0, 5, 40, 61, 130])


@pytest.mark.parametrize("gran,dim", [(0, 8), (0, 64), (0, 72), (0, 96), (0, 128), (0, 136), (0, 256), (32, 32), (32, 64),
                                      (64, 64), (32, 96), (32, 128), (64, 128), (128, 128), (64, 192), (32, 256), (64, 256),
                                      (128, 256)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("lengths", [RAGGED, CHUNKS], ids=["few", "chunks"])
def test_head_dims_and_scale_runs(lib, gpu, gran, dim, hq, hkv, lengths):
    check(lib, synth.attention_inputs(11, *lengths, hq=hq, hkv=hkv, d=dim, gran=gran, spare_rows=3))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (7, 1), (6, 2), (10, 2), (16, 1), (17, 1), (32, 2), (40, 1), (130, 1)])
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("lengths", [RAGGED, CHUNKS], ids=["few", "chunks"])
def test_head_groups(lib, gpu, hq, hkv, gran, lengths):
    check(lib, synth.attention_inputs(12, *lengths, hq=hq, hkv=hkv, d=64, gran=gran))


@pytest.mark.parametrize("page", [1, 3, 16, 48, 128])
@pytest.mark.parametrize("gran", [0, 32])
def test_pages(lib, gpu, page, gran):
    check(lib, synth.attention_inputs(13, [1, 5, 0, 33, 1], [0, 300, 7, 64, 129], hq=4, hkv=2, d=64, page=page, gran=gran))


@pytest.mark.parametrize("new,history", [([1], [0]), ([1], [31]), ([1], [32]), ([1], [63]), ([1], [64]), ([1], [1000]),
                                         ([1] * 5, [0, 1, 2, 63, 500]), ([64], [0]), ([65], [0]), ([200], [0]), ([31, 33], [1, 700]),
                                         ([0, 0, 2], [0, 9, 9]), ([2, 0, 0], [5, 1, 0]), ([300, 1, 1], [0, 900, 20])])
@pytest.mark.parametrize("gran", [0, 128])
def test_lengths(lib, gpu, new, history, gran):
    check(lib, synth.attention_inputs(14, new, history, hq=4, hkv=1, d=128, gran=gran, spare_rows=1))


@pytest.mark.parametrize("batch", [63, 64, 65, 200, 300, 600])
@pytest.mark.parametrize("hq,hkv,dim", [(4, 2, 64), (9, 3, 64), (2, 1, 256), (40, 1, 64)])
def test_batches(lib, gpu, batch, hq, hkv, dim):
    """From one sequence per lane to several per thread, in both kernels (40 rows per token: the
    one for chunks)."""
    rng = np.random.default_rng(batch)
    check(lib, synth.attention_inputs(15, rng.integers(0, 3, batch), rng.integers(0, 90, batch), hq=hq, hkv=hkv, d=dim))


def test_a_page_table_far_wider_than_the_sequences(lib, gpu):
    """Work is counted by what the table has room for where only that is known on the host."""
    d = synth.attention_inputs(36, [1, 2, 1], [90, 700, 3], hq=8, hkv=4, d=64, page=16)
    wide = np.full((3, 1 << 20), 0xFFFFFFFF, np.uint32)
    wide[:, :d.page_table.shape[1]] = d.page_table
    check(lib, dataclasses.replace(d, page_table=wide))
    d = synth.attention_inputs(37, [100, 2, 70], [90, 700, 3], hq=8, hkv=4, d=64, page=16)
    wide = np.full((3, 1 << 20), 0xFFFFFFFF, np.uint32)
    wide[:, :d.page_table.shape[1]] = d.page_table
    check(lib, dataclasses.replace(d, page_table=wide), window=50)


def test_the_widest_window_is_none(lib, gpu):
    for new in ([2, 1], [100, 1]):
        d = synth.attention_inputs(38, new, [300, 40], hq=4, hkv=2, d=64)
        assert np.array_equal(run(lib, d, 0.125, True, 2**31 - 1), run(lib, d, 0.125))


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 5000])
@pytest.mark.parametrize("gran", [0, 64])
def test_windows(lib, gpu, window, gran):
    check(lib, synth.attention_inputs(16, [1, 40, 3, 90], [400, 130, 0, 33], hq=4, hkv=2, d=64, gran=gran), window=window)


@pytest.mark.parametrize("gran", [0, 32])
def test_not_causal(lib, gpu, gran):
    check(lib, synth.attention_inputs(17, [1, 40, 3, 90], [400, 130, 0, 33], hq=4, hkv=2, d=64, gran=gran), causal=False)


@pytest.mark.parametrize("gran", [0, 128])
def test_long_history_is_split(lib, gpu, gran):
    check(lib, synth.attention_inputs(18, [1, 2, 1], [9000, 40, 2500], hq=4, hkv=1, d=128, page=64, gran=gran, layers=1))
    check(lib, synth.attention_inputs(19, [40], [5000], hq=4, hkv=1, d=128, page=64, gran=gran, layers=1))
    check(lib, synth.attention_inputs(19, [2, 90, 0, 1], [2000, 5000, 3, 40], hq=4, hkv=1, d=64, page=1, gran=gran and 64,
                                      layers=1))
    check(lib, synth.attention_inputs(19, [3, 2, 0, 1], [2000, 5000, 3, 40], hq=4, hkv=1, d=64, page=1, gran=gran and 64,
                                      layers=1), window=1500)


@pytest.mark.parametrize("scale", [1e-6, 1.0, 30.0])
@pytest.mark.parametrize("new", [[5, 3], [5, 150]], ids=["few", "chunks"])
def test_scales(lib, gpu, scale, new):
    """From nearly even weights to a single one."""
    check(lib, synth.attention_inputs(20, new, [90, 20], hq=4, hkv=2, d=64), scale=scale)


@pytest.mark.parametrize("new", [[2], [100]], ids=["few", "chunks"])
@pytest.mark.parametrize("order", [1, -1])
def test_scores_that_grow_along_the_sequence(lib, gpu, new, order):
    """The running maximum moves at every block (or never after the first)."""
    d = synth.attention_inputs(34, new, [900], hq=4, hkv=2, d=64)
    n = 900 + new[0]
    page, slot = d.page_table[0, np.arange(n) // 16], np.arange(n) % 16
    size = np.linspace(0.0, 40.0, n)[::order]
    k = np.zeros((n, 2, 64))
    k[:, :, 0] = size[:, None]
    d.blocks[1, 0, page, slot] = synth.bf16_bits(k)
    d.q[:] = synth.bf16_bits(np.broadcast_to(np.eye(64)[0], d.q.shape))
    check(lib, d, scale=1.0)


def test_constant_values_come_back(lib, gpu):
    """v = 1 everywhere: the weights' sum over itself. Numerator and denominator see the same
    weights, but for the numerator's roundings to bf16."""
    d = synth.attention_inputs(21, [4, 1], [100, 700], hq=4, hkv=2, d=64)
    d.blocks[1, 1][d.blocks[1, 1] != 0xFFFF] = 0x3F80
    check(lib, d)


def test_page_table_entries_of_an_evicted_prefix_are_not_read(lib, gpu):
    """With a window, pages before every visible position may be gone."""
    d = synth.attention_inputs(22, [3, 1], [500, 300], hq=4, hkv=2, d=64, page=16)
    ref = exact(d, 0.125, True, 50)
    d.page_table[0, :(500 - 49) // 16] = 0xFFFFFFFF
    d.page_table[1, :(300 - 49) // 16] = 0xFFFFFFFF
    compare(d, run(lib, d, 0.125, True, 50), ref)


@pytest.mark.parametrize("gran", [0, 32])
@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("new", [[40, 2, 1], [150, 2, 1]], ids=["few", "chunks"])
def test_what_a_row_must_not_see_does_not_reach_it(lib, gpu, gran, plane, bad, window, new):
    """One position of a chunk holds infinities or NaN: the tokens before it (and, with a
    window, far behind it) are as without it, and those that see it are as the formula says."""
    if gran and bad != "nan" and plane == 0:
        pytest.skip("e4m3 has no infinities; an infinite key scale is the NaN case of the scores")
    d = synth.attention_inputs(23, new, [70, 3, 60], hq=4, hkv=2, d=64, page=16, gran=gran)
    at = 70 + 17
    page, slot = d.page_table[0, at // 16], at % 16
    value = float(bad)
    if gran and bad == "nan":
        d.blocks[1, plane, page, slot, :, 5] = 0x7F
    elif gran:
        d.scales[1, plane, page, slot, :, 0] = value
    else:
        d.blocks[1, plane, page, slot, :, 5] = synth.bf16_bits(np.array([value]))[0]
    got = run(lib, d, 0.125, True, window)
    ref = exact(d, 0.125, True, window)
    if plane == 0 and bad != "nan":
        # a score of +infinity has no softmax; one of -infinity is a weight of zero
        rows = np.isfinite(ref[0]).all(axis=(1, 2))
        sees = np.zeros(len(d.q), bool)
        sees[17:new[0]] = True
        if window:
            sees[17 + window:new[0]] = False
        assert rows[~sees].all()
        g = bf16v(got)
        assert (np.abs(g - ref[0]) <= tolerance(d, ref))[~sees].all()
        return
    compare(d, got, ref)
    before = bf16v(got)[:17]
    assert np.isfinite(before).all()


@pytest.mark.parametrize("new", [[6, 3], [160, 3]], ids=["few", "chunks"])
def test_a_bad_query_reaches_its_own_row_only(lib, gpu, new):
    d = synth.attention_inputs(24, new, [40, 9], hq=4, hkv=2, d=64)
    d.q[2, 1, 3] = 0x7FC0
    got, ref = run(lib, d, 0.125), exact(d, 0.125)
    g = bf16v(got)
    assert np.isnan(g[2, 1]).all()
    keep = np.ones(g.shape[:2], bool)
    keep[2, 1] = False
    assert (np.abs(g - ref[0]) <= tolerance(d, ref))[keep].all()


def test_same_bits_twice_and_on_another_stream(lib, gpu):
    for gran in (0, 64):
        d = synth.attention_inputs(25, [1, 70, 2], [3000, 200, 15], hq=8, hkv=2, d=128, gran=gran, page=32)
        first = run(lib, d, 0.1)
        assert np.array_equal(first, run(lib, d, 0.1))
        dev, out, ws = place(d), torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda"), workspace(lib, d)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call(lib, d, dev, out, ws, 0.1)
        s.synchronize()
        assert np.array_equal(host16(out), first)
        out.zero_()
        torch.cuda.synchronize()
        call(lib, d, dev, out, ws, 0.1, stream=s)
        s.synchronize()
        assert np.array_equal(host16(out), first)


def test_two_calls_at_once(lib, gpu):
    """Two streams, a workspace each."""
    ds = [synth.attention_inputs(s, [1, 2], [4000, 900], hq=8, hkv=2, d=128, page=32) for s in (26, 27)]
    want = [run(lib, d, 0.1) for d in ds]
    parts = [(d, place(d), torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda"), workspace(lib, d), torch.cuda.Stream())
             for d in ds]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, dev, out, ws, s in parts:
            call(lib, d, dev, out, ws, 0.1, stream=s)
    torch.cuda.synchronize()
    for (d, _, out, _, _), w in zip(parts, want):
        assert np.array_equal(host16(out), w)


def test_two_graphs_share_a_workspace(lib, gpu):
    """Replayed in turn, with lengths that change between the replays."""
    ds = [synth.attention_inputs(28, [1, 1, 1], [2000, 900, 3], hq=8, hkv=2, d=128, page=32),
          synth.attention_inputs(29, [30, 1], [1500, 40], hq=8, hkv=2, d=128, page=32, gran=64)]
    n = max(workspace(lib, d).numel() for d in ds)
    ws = torch.full((n,), float("nan"), device="cuda")
    parts = [(d, place(d), torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda")) for d in ds]
    for d, dev, out in parts:
        call(lib, d, dev, out, ws, 0.1)
    torch.cuda.synchronize()
    graphs = []
    for d, dev, out in parts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(lib, d, dev, out, ws, 0.1)
        graphs.append(g)
    for turn in range(4):
        for k, (d, dev, out) in enumerate(parts):
            less = dataclasses.replace(d, cache_lengths=np.maximum(d.cache_lengths.astype(np.int64) - 97 * turn, 0).astype(np.uint32))
            dev["lengths"].copy_(dev32(less.cache_lengths))
            out.fill_(7)
            torch.cuda.synchronize()
            graphs[k].replay()
            torch.cuda.synchronize()
            replayed = host16(out)
            assert np.array_equal(replayed, run(lib, less, 0.1)), (turn, k)
            compare(less, replayed, exact(less, 0.1))


def test_cache_past_32_bit_offsets(lib, gpu):
    """A plane of 6 GB: the pages in use lie behind byte 2^32 of each plane (and element 2^31)."""
    for gran, dtype in ((0, torch.bfloat16), (128, torch.uint8)):
        d = synth.attention_inputs(30, [1, 20], [700, 90], hq=8, hkv=8, d=128, page=128, gran=gran, layers=1)
        page_bytes = 128 * 8 * 128 * (1 if gran else 2)
        pages = (6 << 30) // page_bytes
        used = d.blocks.shape[2]
        blocks = torch.empty((1, 2, pages, 128, 8, 128), dtype=dtype, device="cuda")
        dev = place(d)
        blocks[:, :, pages - used:] = dev["blocks"]
        dev["blocks"] = blocks
        if gran:
            scales = torch.empty((1, 2, pages, 128, 8, 1), device="cuda")
            scales[:, :, pages - used:] = dev["scales"]
            dev["scales"] = scales
        table = d.page_table.astype(np.int64)
        table[table != 0xFFFFFFFF] += pages - used
        dev["table"] = dev32(table.astype(np.uint32))
        out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
        call(lib, d, dev, out.view, workspace(lib, d), 0.1)
        compare(d, host16(out.view), exact(d, 0.1))
        del blocks, dev


def test_refusals_with_device_tensors(lib, gpu):
    d = synth.attention_inputs(31, [1], [5], hq=2, hkv=1, d=64)
    dev, ws = place(d), workspace(lib, d)
    out = torch.full(d.q.shape, 3.0, dtype=torch.bfloat16, device="cuda")

    def bad(error, **over):
        a = dict(out=out, q=dev["q"], offs=dev["offs"], blocks=dev["blocks"], lengths=dev["lengths"], table=dev["table"],
                 layer=1, scale=0.1, ws=ws)
        a.update(over)
        with pytest.raises(error):
            lib.attention_ragged_paged(*a.values())

    bad(ValueError, lengths=dev["lengths"].long())
    bad(ValueError, table=dev["table"][:, ::2])
    bad(ValueError, table=dev["table"][0])
    bad(ValueError, q=torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")[..., ::2])
    bad(ValueError, lengths=dev["lengths"].cpu())
    bad(lib.QgError, q=dev["q"].half())
    bad(lib.QgError, layer=2)
    if ws.numel():
        bad(lib.QgError, ws=ws[:4])
    assert lib.attention_ragged_paged(out, dev["q"], dev["offs"], dev["blocks"], dev["lengths"], dev["table"], 2, 0.1, ws,
                                      raise_on_error=False) == lib.QG.ERR_INVALID_ARG
    assert (out == 3).all()


@pytest.mark.parametrize("gran", [0, 64])
def test_a_serving_run(lib, gpu, gran):
    """As a program uses them: prompts, then single tokens; each step builds its tables, projects
    keys and values into the pages and attends over them. Against the oracles of the three."""
    rng = np.random.default_rng(32)
    hkv, hd, hq, Kh, page, pages, W = 2, 64, 4, 128, 16, 40, 10
    k = synth.kproj_inputs(seed=33, Kh=Kh, n_kv_heads=hkv, head_dim=hd, lens=[1], max_len=16, page_size=page, num_pages=pages,
                           num_layers=1, layer_idx=0, planes=2, max_pages=1, cache="fp8" if gran else "bf16", qgran=gran or 128)
    blocks_h, scales_h = k.blocks.copy(), None if k.scales is None else k.scales.copy()
    blocks = torch.from_numpy(blocks_h.copy()).cuda() if gran else dev16(blocks_h, torch.bfloat16)
    scales = devf32(scales_h) if gran else None
    from gpu_util import dev8
    weight, wscale = dev8(k.weight), devf32(k.weight_scale)
    free_h = rng.permutation(pages).astype(np.uint32)
    B = 3
    table_h, count = np.zeros((B, W), np.uint32), pages
    table, free = dev32(table_h), dev32(free_h)
    counts = [dev32(np.array([pages, 0], np.int32)), dev32(np.zeros(2, np.int32))]
    cached_h = np.zeros(B, np.uint32)
    cached = dev32(cached_h)
    for step, new in enumerate(([37, 1, 20], [1, 1, 1], [1, 0, 1], [4, 1, 30], [1, 1, 1])):
        T = sum(new)
        offs, slots = dev32(np.zeros(B + 1, np.int32)), dev32(np.zeros(T, np.int32))
        lib.tables_ragged_paged(offs, slots, table, counts[(step + 1) % 2], cached, dev32(np.array(new, np.int32)), free,
                                counts[step % 2][:1], page)
        hid = synth.bf16_bits(rng.standard_normal((T, Kh)))
        isc = rng.uniform(0.5, 2.0, (T, 1)).astype(np.float32)
        lib.kv_matmul_ragged_paged_scale(dev16(hid, torch.bfloat16), offs, weight, devf32(isc), wscale, blocks, cached, table,
                                         0, kv_scales=scales, quantization_granularity=gran)
        qb = synth.bf16_bits(rng.standard_normal((T, hq, hd)))
        qd = dev16(qb, torch.bfloat16)
        out = torch.zeros_like(qd)
        ws = torch.empty(lib.attention_ragged_paged_workspace(T, B, hq, hkv, hd), device="cuda")
        lib.attention_ragged_paged(out, qd, offs, blocks, cached, table, 0, hd ** -0.5, ws, kv_scales=scales,
                                   quantization_granularity=gran)
        cached.add_(dev32(np.array(new, np.int32)))
        torch.cuda.synchronize()
        # tables and cache rows as their oracles have them, attention over the cache as it is
        offs_h, table_h, slots_h, (count, status) = oracle.tables_ragged_paged(table_h, cached_h, new, free_h, count, page, T)
        assert status == 0 and counts[(step + 1) % 2].cpu().tolist() == [count, 0]
        assert np.array_equal(table.cpu().numpy().view(np.uint32), table_h)
        assert np.array_equal(slots.cpu().numpy(), slots_h)
        now = blocks.cpu().numpy() if gran else host16(blocks)
        now_s = scales.cpu().numpy() if gran else None
        row = now[0, 0].reshape(pages * page, hkv * hd)[slots_h]
        want = oracle.kproj_exact(hid, k.weight, isc, k.weight_scale)[:, :hkv * hd]
        if gran:
            row = oracle.decode_e4m3(row) * np.repeat(now_s[0, 0].reshape(pages * page, -1)[slots_h].astype(np.float64), gran, 1)
        assert (np.abs((row if gran else bf16v(row)) - want) <= (0.07 if gran else 1e-2) * (np.abs(want) + 1)).all()
        d = synth.AttentionInputs(q=qb, row_offsets=offs_h.astype(np.uint32), blocks=now, cache_lengths=cached_h, page_table=table_h,
                                  layer_idx=0, scales=now_s, gran=gran)
        compare(d, host16(out), exact(d, hd ** -0.5), f"step {step}")
        cached_h = cached_h + np.array(new, np.uint32)


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("history", [1531, 1563, 1595])
def test_a_window_that_starts_anywhere_in_a_block(lib, gpu, page, history):
    """The first position seen, and the parts that the work is cut into, at every place of 32 and
    64: no part may consist of positions (and pages) before it."""
    d = synth.attention_inputs(35, [1, 2, 1], [history, history + 7, history + 20], hq=4, hkv=1, d=64, page=page, layers=1)
    ref = exact(d, 0.125, True, 1500)
    for b in range(3):
        d.page_table[b, :(int(d.cache_lengths[b]) - 1499) // page] = 0xFFFFFFFF
    compare(d, run(lib, d, 0.125, True, 1500), ref)


def _drafts(batch, most, group):
    """New tokens of `batch` sequences whose rows per key/value head are 17 to 32 on average:
    the two row tiles of the kernel for few rows, which takes them where sequences are many."""
    new = [most, 0, 1] + [24 // group] * (batch - 3)
    assert 16 * batch < sum(new) * group <= 32 * batch
    return new


@pytest.mark.parametrize("gran,dim", [(0, 40), (0, 64), (0, 128), (0, 256), (32, 64), (64, 64), (32, 128), (64, 128), (128, 128),
                                      (32, 192), (32, 256), (64, 256), (128, 256)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("batch", [33, 70])
def test_drafts_of_many_sequences(lib, gpu, gran, dim, window, batch):
    rng = np.random.default_rng(dim + gran)
    d = synth.attention_inputs(38, _drafts(batch, 9, 4), rng.integers(0, 300, batch), hq=8, hkv=2, d=dim, gran=gran, spare_rows=2)
    check(lib, d, window=window)


@pytest.mark.parametrize("batch,hkv", [(4, 16), (5, 16), (8, 8), (9, 8), (65, 1), (64, 1)])
@pytest.mark.parametrize("gran,dim", [(0, 64), (64, 256)])
def test_drafts_at_the_change_of_kernels(lib, gpu, batch, hkv, gran, dim):
    check(lib, synth.attention_inputs(39, _drafts(batch, 20, 4), [200 + 7 * i for i in range(batch)], hq=4 * hkv, hkv=hkv, d=dim,
                                      gran=gran))


@pytest.mark.parametrize("gran,dim", [(0, 64), (0, 128), (0, 256), (32, 64), (32, 256), (128, 128)])
@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("window", [0, 9])
def test_nan_among_drafts_of_many_sequences(lib, gpu, gran, dim, plane, window):
    d = synth.attention_inputs(40, _drafts(34, 40, 4), [70] + [5 + 2 * i for i in range(33)], hq=8, hkv=2, d=dim, page=16, gran=gran)
    at = 70 + 17
    page, slot = d.page_table[0, at // 16], at % 16
    d.blocks[1, plane, page, slot, :, 5] = 0x7F if gran else 0x7FC0
    ref = exact(d, 0.125, True, window)
    got = run(lib, d, 0.125, True, window)
    compare(d, got, ref)
    assert np.isfinite(bf16v(got)[:17]).all() and np.isfinite(bf16v(got)[40:]).all()
