"""attention_tree_ragged_paged on the GPU against the 64-bit oracle, to the tolerance of
attention_ragged_paged (derived in test_gpu_attention.py; the arithmetic is the same)."""
import numpy as np
import pytest
import torch

import oracle
import synth
import attention_shapes
from gpu_util import Guarded, bf16v, dev16, dev32, host16, say
from test_gpu_attention import compare, place, workspace
from test_gpu_attention_extremes import cus, huge_values, put

pytestmark = pytest.mark.gpu


def kernel(d, cus):
    """The kernel that a call takes, as attention_shapes.kernel says it of the other calls: trees on
    bf16 caches take the one for many rows from 17 rows per sequence and head on."""
    form = attention_shapes.kernel(d, cus)
    return "tile" if form == "rows2" and not d.gran else form


def tree_rows(d, words, seed=0, kind="tree"):
    """Rows of the mask for the new tokens of d: trees, chains, or any bits at all (some rows none,
    bits behind the last token set). Rows that no sequence covers are all ones."""
    rng = np.random.default_rng(seed)
    rows = np.full((len(d.q), words), 0xFFFFFFFF, np.uint32)
    for b in range(len(d.cache_lengths)):
        r0, r1 = int(d.row_offsets[b]), int(d.row_offsets[b + 1])
        n = r1 - r0
        if kind == "any":
            rows[r0:r1] = rng.integers(0, 1 << 32, (n, words), dtype=np.uint64).astype(np.uint32)
            rows[r0:r1][rng.random(n) < 0.2] = 0
        elif n:
            parents = [j - 1 if kind == "chain" else int(rng.integers(-1, j)) if j else -1 for j in range(n)]
            rows[r0:r1] = oracle.tree_mask(parents, words)
    return rows


def call(lib, d, mask, dev, out, ws, scale, window=0, stream=None):
    lib.attention_tree_ragged_paged(out, dev["q"], dev["offs"], dev["mask"] if "mask" in dev else dev32(mask), dev["blocks"],
                                    dev["lengths"], dev["table"], d.layer_idx, scale, ws, window=window, kv_scales=dev["scales"],
                                    quantization_granularity=d.gran, stream=stream)


def run(lib, d, mask, scale, window=0):
    out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
    call(lib, d, mask, place(d), out.view, workspace(lib, d), scale, window)
    assert out.bands_intact(), "bytes around the output changed"
    return host16(out.view)


def exact(d, mask, scale, window=0):
    return oracle.attention_tree_ragged_paged(d.q, d.row_offsets, mask, d.blocks, d.cache_lengths, d.page_table, d.layer_idx, scale,
                                              window, d.scales, d.gran)


def check(lib, d, mask, window=0, what="", scale=None):
    scale = d.q.shape[2] ** -0.5 if scale is None else scale
    say(f"[tree] {what} {kernel(d, cus())} q {d.q.shape} words {mask.shape[1]} lengths {d.cache_lengths[:6].tolist()} cache {d.blocks.shape} "
        f"gran {d.gran} window {window}")
    got = run(lib, d, mask, scale, window)
    used = compare(d, got, exact(d, mask, scale, window), what)
    say(f"[tree]   worst element at {used:.2f} of its tolerance")
    return got


FEW = ([3, 0, 1, 7, 2], [0, 5, 40, 61, 130])
MANY = ([70, 0, 33, 1, 129], [0, 5, 40, 61, 130])


@pytest.mark.parametrize("gran,dim", [(0, 8), (0, 64), (0, 72), (0, 128), (0, 256), (32, 32), (32, 64), (64, 64), (32, 96), (32, 128),
                                      (64, 128), (128, 128), (64, 192), (32, 256), (64, 256), (128, 256)])
@pytest.mark.parametrize("lengths", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("window", [0, 30])
def test_head_dims_and_scale_runs(lib, gpu, gran, dim, lengths, window):
    d = synth.attention_inputs(1, *lengths, hq=8, hkv=2, d=dim, gran=gran, spare_rows=3)
    check(lib, d, tree_rows(d, 5), window)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (7, 1), (6, 2), (17, 1), (32, 2), (130, 1)])
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("lengths", [FEW, MANY], ids=["few", "many"])
def test_head_groups(lib, gpu, hq, hkv, gran, lengths):
    d = synth.attention_inputs(2, *lengths, hq=hq, hkv=hkv, d=64, gran=gran)
    check(lib, d, tree_rows(d, 5, 1))


@pytest.mark.parametrize("page", [1, 3, 16, 48, 128])
@pytest.mark.parametrize("gran", [0, 32])
@pytest.mark.parametrize("lengths", [([1, 5, 0, 6, 1], [0, 300, 7, 64, 129]), ([40, 90, 0, 33, 1], [0, 300, 7, 64, 129])], ids=["few", "many"])
def test_pages(lib, gpu, page, gran, lengths):
    d = synth.attention_inputs(3, *lengths, hq=4, hkv=2, d=64, page=page, gran=gran)
    check(lib, d, tree_rows(d, 3, 2))
    check(lib, d, tree_rows(d, 3, 3, "any"), window=50)


@pytest.mark.parametrize("history", [0, 1, 31, 32, 33, 63, 64, 65, 95, 100, 127, 2000, 2017])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 130])
def test_trees_at_every_place_of_a_block(lib, gpu, history, n):
    """The words' bits meet the blocks' positions at all offsets; with any bits, rows may be empty."""
    d = synth.attention_inputs(4, [n, 1, n], [history, history, 0], hq=2, hkv=1, d=64)
    words = -(-n // 32)
    check(lib, d, tree_rows(d, words, n, "tree"))
    got = check(lib, d, tree_rows(d, words, n, "any"))
    check(lib, d, tree_rows(d, words + 2, n, "any"), window=history // 2 + 1)
    assert np.isfinite(bf16v(got)).all()


@pytest.mark.parametrize("gran,dim", [(0, 64), (0, 128), (64, 64), (32, 128), (0, 256), (128, 256)])
@pytest.mark.parametrize("lengths", [FEW, MANY], ids=["few", "many"])
def test_rows_that_see_nothing_are_zero(lib, gpu, gran, dim, lengths):
    """Without history and without bits: zeros, beside rows that see one token. No word is named of
    sequences longer than the mask."""
    new, _ = lengths
    d = synth.attention_inputs(5, new, [0] * len(new), hq=8, hkv=2, d=dim, gran=gran, spare_rows=2)
    mask = np.zeros((len(d.q), 1), np.uint32)
    mask[1::3, 0] = 1
    got = check(lib, d, mask)
    n = int(d.row_offsets[-1])
    empty = np.zeros(n, bool)
    empty[np.arange(n) % 3 != 1] = True
    assert (got[:n][empty] == 0).all()
    # values that are infinite or NaN change nothing of that
    for b in range(len(new)):
        if new[b]:
            put(type("One", (), dict(d.__dict__, page_table=d.page_table[b:b + 1]))(), 1, 0, float("nan"))
    again = run(lib, d, mask, 0.125)
    assert (again[:n][empty] == 0).all() and not np.isfinite(bf16v(again[:n][~empty])).all()


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("lengths", [FEW, MANY], ids=["few", "many"])
def test_masks_shorter_than_the_sequence(lib, gpu, gran, lengths):
    """Tokens that the words have no bit for are seen by nobody."""
    d = synth.attention_inputs(6, *lengths, hq=4, hkv=2, d=64, gran=gran)
    for words in (1, 2):
        check(lib, d, tree_rows(d, words, 4, "any"))
        check(lib, d, tree_rows(d, words, 4, "any"), window=35)


@pytest.mark.parametrize("window", [1, 2, 5, 31, 32, 33, 64, 100, 2**31 - 1])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("lengths", [([3, 0, 1, 7, 2], [0, 5, 400, 61, 230]), ([70, 0, 33, 1, 129], [0, 5, 400, 61, 230])], ids=["few", "many"])
def test_windows(lib, gpu, window, page, lengths):
    """Pages of the history that no token sees do not exist."""
    d = synth.attention_inputs(7, *lengths, hq=4, hkv=1, d=64, page=page)
    mask = tree_rows(d, 5, 5)
    ref = exact(d, mask, 0.125, window)
    for b in range(len(d.cache_lengths)):
        d.page_table[b, :max(0, int(d.cache_lengths[b]) - window) // page] = 0xFFFFFFFF
    compare(d, run(lib, d, mask, 0.125, window), ref)


def test_a_chain_gives_what_the_causal_attention_gives(lib, gpu):
    """To the tolerance of the causal oracle, and near the causal kernel (which cuts the work otherwise)."""
    for lengths in (FEW, MANY, ([64] * 6, [3000, 100, 0, 7, 999, 64])):
        for gran in (0, 64):
            d = synth.attention_inputs(8, *lengths, hq=8, hkv=2, d=64, gran=gran)
            a = run(lib, d, tree_rows(d, 5, 0, "chain"), 0.125)
            out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
            dev = place(d)
            lib.attention_ragged_paged(out.view, dev["q"], dev["offs"], dev["blocks"], dev["lengths"], dev["table"], d.layer_idx, 0.125,
                                       workspace(lib, d), kv_scales=dev["scales"], quantization_granularity=gran)
            compare(d, a, oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table, d.layer_idx, 0.125,
                                                        True, 0, d.scales, gran))
            assert np.abs(bf16v(a) - bf16v(host16(out.view))).max() <= 2.0**-6 * np.abs(bf16v(a)).max()


FORMS = {
    "rows1": ([4, 2, 1], [70, 3, 60], 4, 2),
    "rows1 cut": ([4, 2, 1], [3000, 3, 60], 4, 2),
    "rows2": ([40, 0, 1] + [6] * 31, [70] + [5 + 2 * i for i in range(33)], 8, 2),
    "rows2 cut": ([40, 0, 1] + [6] * 31, [3000] + [5 + 2 * i for i in range(33)], 8, 2),
    "tile": ([150, 2, 1], [70, 3, 60], 4, 2),
    "tile cut": ([150, 2, 1], [3000, 3, 60], 4, 2),
}


def form_case(seed, form, dim, gran):
    new, hist, hq, hkv = FORMS[form]
    d = synth.attention_inputs(seed, new, hist, hq=hq, hkv=hkv, d=dim, gran=gran)
    assert attention_shapes.kernel(d, cus()) == form.split()[0]
    say(f"[tree] {form} head {dim} gran {gran}")
    return d


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,gran", [(64, 0), (64, 32), (128, 128), (256, 0), (256, 64)])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("plane", [0, 1])
def test_what_a_row_does_not_see_changes_no_bit_of_it(lib, gpu, form, dim, gran, window, plane):
    """Infinities and NaN in the key or value of one drafted token, and of one position of the history
    that a window hides from some; their scales in an e4m3 cache."""
    d = form_case(9, form, dim, gran)
    n, c = int(d.row_offsets[1]), int(d.cache_lengths[0])
    mask = tree_rows(d, 5, 6)
    at = 1 if n < 10 else 17
    sees = (mask[:, at // 32] >> np.uint32(at % 32) & 1).astype(bool)
    sees[n:] = False
    assert sees[:n].any() and not sees[:n].all()
    clean = run(lib, d, mask, 0.125, window)
    places = [(c + at, sees)]
    if window:
        seen = np.array([sum(bin(int(w)).count("1") for w in row) for row in mask])
        near = np.arange(len(mask)) < n
        places.append((c - window + 1, near & (seen <= 1)))
    for pos, visible in places:
        for value in (float("nan"), float("inf")):
            held = d.blocks.copy(), None if d.scales is None else d.scales.copy()
            put(d, plane, pos, value)
            got = run(lib, d, mask, 0.125, window)
            assert np.array_equal(got[~visible], clean[~visible]), f"{int((got != clean)[~visible].sum())} elements changed by {value}"
            if plane == 1:
                assert not np.isfinite(bf16v(got)[visible]).all()
                compare(d, got, exact(d, mask, 0.125, window), form)
            d.blocks[:] = held[0]
            if gran:
                d.scales[:] = held[1]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("growing", [False, True])
def test_sums_of_large_values_do_not_leave_the_type(lib, gpu, form, gran, growing):
    d = form_case(10, form, 128, gran)
    huge_values(d, growing)
    mask, scale = tree_rows(d, 5, 7), 1.0 if growing else 0.125
    ref = exact(d, mask, scale)
    assert np.isfinite(ref[0]).all() and np.abs(ref[0]).max() > 2.0**124
    compare(d, run(lib, d, mask, scale), ref, form)


def test_stale_slots_and_other_layers_do_not_matter(lib, gpu):
    """All that no sequence holds is NaN, as are the other layers (the inputs are made so); bits behind
    the last token name stale slots."""
    d = synth.attention_inputs(11, [5, 40], [3, 70], hq=4, hkv=2, d=64, layers=3)
    mask = tree_rows(d, 4, 8)
    mask[:5, 0] |= 0xFFFFFFE0
    mask[:, 2:] = 0xFFFFFFFF
    assert np.isfinite(bf16v(check(lib, d, mask))).all()


def test_the_same_bits_every_time_and_in_any_batch(lib, gpu):
    """Also with another call of the same workspace in between."""
    d = synth.attention_inputs(12, [64] * 5, [3000, 10, 500, 0, 77], hq=8, hkv=2, d=64)
    mask = tree_rows(d, 2, 9)
    first = run(lib, d, mask, 0.125)
    assert all(np.array_equal(run(lib, d, mask, 0.125), first) for _ in range(3))


def test_stream_and_replays(lib, gpu):
    """Captured with a history that grows and a mask that changes between replays; two graphs share a
    workspace in turn."""
    d = synth.attention_inputs(13, [13, 1, 0, 20], [40, 300, 7, 0], hq=4, hkv=2, d=64, layers=1)
    S = d.blocks.shape[3]   # room to grow: every page is there
    rng = np.random.default_rng(1)
    pages = 4 * 30
    d.blocks = synth.bf16_bits(rng.standard_normal((1, 2, pages, S, 2, 64)))
    d.page_table = rng.permutation(pages).reshape(4, 30).astype(np.uint32)
    s = torch.cuda.Stream()
    mask = tree_rows(d, 1, 10)
    dev = {**place(d), "mask": dev32(mask)}
    ws, out = workspace(lib, d), [torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    call(lib, d, mask, dev, out[0], ws, 0.125, stream=s)
    s.synchronize()
    compare(d, host16(out[0]), exact(d, mask, 0.125))
    graphs = []
    for turn in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(lib, d, mask, dev, out[turn], ws, 0.125, window=turn * 50)
        graphs.append(g)
    for turn in range(4):
        d.cache_lengths = d.cache_lengths + np.uint32(9)
        mask = tree_rows(d, 1, 20 + turn)
        dev["lengths"].copy_(dev32(d.cache_lengths))
        dev["mask"].copy_(dev32(mask))
        for o in out:
            o.fill_(0)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for k in range(2):
            compare(d, host16(out[k]), exact(d, mask, 0.125, k * 50))
        _ = (torch.ones(1000, device="cuda") * 2).sum().item()   # the program's own work in between


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(lib, gpu, seed):
    rng = np.random.default_rng(1000 + seed)
    gran = int(rng.choice([0, 0, 32, 64, 128]))
    dim = int(gran * rng.integers(1, 256 // gran + 1)) if gran else int(8 * rng.integers(1, 33))
    hkv = int(rng.integers(1, 5))
    batch = int(rng.choice([1, 2, 5, 40, 70]))
    most = int(rng.choice([2, 9, 40, 140])) if batch < 40 else int(rng.choice([2, 9, 30]))
    new = rng.integers(0, most, batch)
    new[0] = max(new[0], 1)
    d = synth.attention_inputs(seed, new, rng.integers(0, int(rng.choice([3, 70, 900])), batch), hq=hkv * int(rng.integers(1, 6)), hkv=hkv,
                               d=dim, page=int(rng.choice([1, 8, 16, 20, 64])), gran=gran, spare_rows=int(rng.integers(0, 3)))
    words = max(1, -(-int(new.max()) // 32) + int(rng.integers(-1, 3)))
    kind = "any" if rng.random() < 0.5 or words * 32 < new.max() else "tree"
    check(lib, d, tree_rows(d, words, seed, kind), window=int(rng.choice([0, 0, 1, 20, 300])), what=f"seed {seed}")


def test_refusals_with_device_tensors(lib, gpu):
    d = synth.attention_inputs(14, [2], [5], hq=2, hkv=1, d=64)
    dev, ws = place(d), workspace(lib, d)
    out = torch.full(d.q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    mask = dev32(np.ones((2, 1), np.int32))

    def bad(error, **over):
        a = dict(out=out, q=dev["q"], offs=dev["offs"], mask=mask, blocks=dev["blocks"], lengths=dev["lengths"], table=dev["table"],
                 layer=1, scale=0.1, ws=ws)
        a.update(over)
        with pytest.raises(error):
            lib.attention_tree_ragged_paged(*a.values())

    bad(lib.QgError, mask=mask.long())
    bad(lib.QgError, mask=mask[:1])
    bad(lib.QgError, mask=mask[:, :0].contiguous())
    bad(ValueError, mask=mask.cpu())
    bad(ValueError, mask=torch.zeros(2, 4, dtype=torch.int32, device="cuda")[:, ::2])
    bad(lib.QgError, ws=ws[:4])
    bad(lib.QgError, layer=2)
    bad(ValueError, lengths=dev["lengths"].long())
    assert (out == 3).all()
