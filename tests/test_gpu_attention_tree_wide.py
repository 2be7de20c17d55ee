"""attention_tree_ragged_paged where a sequence and key/value head has more than 128 rows on the average:
tiles of 256 rows (heads above 64 up to 128, pages a multiple of 16). And for every form: calls at once on
two streams, and a cache past 32-bit offsets."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import Guarded, bf16v, dev32, host16
from test_gpu_attention import compare, place, workspace
from test_gpu_attention_extremes import huge_values, put
from test_gpu_attention_tree import call, check, exact, run, tree_rows

pytestmark = pytest.mark.gpu

HEADS = [(72, 0), (128, 0), (96, 32), (128, 32), (128, 64), (128, 128)]
WHOLE, CUT = ([150, 2, 100], [70, 3, 60]), ([150, 0, 100], [3000, 30, 60])


def wide(seed, lengths, dim, gran, **kw):
    d = synth.attention_inputs(seed, *lengths, **{"hq": 8, "hkv": 2, "d": dim, "gran": gran, **kw})
    assert len(d.q) * d.q.shape[1] // d.blocks.shape[4] > 128 * len(d.cache_lengths)
    return d


@pytest.mark.parametrize("dim,gran", HEADS)
@pytest.mark.parametrize("lengths", [WHOLE, CUT, ([64] * 5, [0, 1, 64, 700, 127]), ([33], [31]), ([300, 1], [5, 2000])],
                         ids=["whole", "cut", "64 each", "one", "long"])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_matches_the_oracle(lib, gpu, dim, gran, lengths, window):
    d = wide(1, lengths, dim, gran)
    check(lib, d, tree_rows(d, 10, 2), window)
    check(lib, d, tree_rows(d, 3, 3, "any"), window)


@pytest.mark.parametrize("hq,hkv", [(5, 1), (17, 1), (300, 1), (12, 3), (40, 8)])
@pytest.mark.parametrize("page", [16, 48, 112])
@pytest.mark.parametrize("gran", [0, 64])
def test_groups_and_pages(lib, gpu, hq, hkv, page, gran):
    d = wide(2, ([40, 90, 0, 70], [0, 300, 7, 129]), 128, gran, hq=hq, hkv=hkv, page=page)
    check(lib, d, tree_rows(d, 3, 4))


@pytest.mark.parametrize("dim,gran", HEADS)
@pytest.mark.parametrize("lengths", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("plane", [0, 1])
def test_what_a_row_does_not_see_changes_no_bit_of_it(lib, gpu, dim, gran, lengths, plane):
    d = wide(3, lengths, dim, gran)
    n, c = int(d.row_offsets[1]), int(d.cache_lengths[0])
    mask = tree_rows(d, 5, 6)
    sees = (mask[:, 0] >> np.uint32(17) & 1).astype(bool)
    sees[n:] = False
    assert sees[:n].any() and not sees[:n].all()
    clean = run(lib, d, mask, 0.125)
    for value in (float("nan"), float("inf")):
        held = d.blocks.copy(), None if d.scales is None else d.scales.copy()
        put(d, plane, c + 17, value)
        got = run(lib, d, mask, 0.125)
        assert np.array_equal(got[~sees], clean[~sees]), f"{int((got != clean)[~sees].sum())} elements changed by {value}"
        if plane == 1:
            assert not np.isfinite(bf16v(got)[sees]).all()
            compare(d, got, exact(d, mask, 0.125))
        d.blocks[:] = held[0]
        if gran:
            d.scales[:] = held[1]


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("lengths", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("growing", [False, True])
def test_sums_of_large_values_do_not_leave_the_type(lib, gpu, gran, lengths, growing):
    d = wide(4, lengths, 128, gran)
    huge_values(d, growing)
    mask, scale = tree_rows(d, 5, 7), 1.0 if growing else 0.125
    ref = exact(d, mask, scale)
    assert np.isfinite(ref[0]).all() and np.abs(ref[0]).max() > 2.0**124
    compare(d, run(lib, d, mask, scale), ref)


@pytest.mark.parametrize("gran", [0, 128])
def test_rows_that_see_nothing_are_zero(lib, gpu, gran):
    d = wide(5, ([100, 130, 60], [0, 0, 40]), 128, gran)
    mask = tree_rows(d, 5, 8)
    empty = np.random.default_rng(1).random(230) < 0.4
    empty[:70] = True   # more than a wave's 32 rows of a tile
    mask[:230][empty] = 0
    got = check(lib, d, mask)
    assert not got[:230][empty].any() and (got[:230][~empty] != 0).any()


FORMS = {"few": ([3, 1, 6], [700, 0, 90], 128), "many": ([40, 9], [700, 90], 64), "wide": ([90, 70], [700, 90], 128)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
def test_cache_past_32_bit_offsets(lib, gpu, form, gran):
    """A plane of 6 GB: the pages in use lie behind byte 2^32 of each plane (and element 2^31)."""
    new, history, dim = FORMS[form]
    d = synth.attention_inputs(6, new, history, hq=8, hkv=2, d=dim, page=128, gran=gran, layers=1)
    used, shape = d.blocks.shape[2], d.blocks.shape
    pages = (6 << 30) // (128 * 2 * dim * (1 if gran else 2))
    mask = tree_rows(d, 3, 9)
    dev = {**place(d), "mask": dev32(mask)}
    blocks = torch.empty((1, 2, pages, *shape[3:]), dtype=dev["blocks"].dtype, device="cuda")
    blocks[:, :, pages - used:] = dev["blocks"]
    dev["blocks"] = blocks
    if gran:
        scales = torch.empty((1, 2, pages, *d.scales.shape[3:]), device="cuda")
        scales[:, :, pages - used:] = dev["scales"]
        dev["scales"] = scales
    table = d.page_table.astype(np.int64)
    table[table != 0xFFFFFFFF] += pages - used
    dev["table"] = dev32(table.astype(np.uint32))
    out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
    call(lib, d, mask, dev, out.view, workspace(lib, d), 0.1)
    compare(d, host16(out.view), exact(d, mask, 0.1))


@pytest.mark.parametrize("form", FORMS)
def test_calls_at_once_on_two_streams(lib, gpu, form):
    """Each with a workspace of its own, over one cache."""
    new, history, dim = FORMS[form]
    d = synth.attention_inputs(7, new, [30 * h + 5 for h in history], hq=8, hkv=2, d=dim)
    masks = [tree_rows(d, 3, 10 + k) for k in range(2)]
    devs = [{**place(d), "mask": dev32(m)} for m in masks]
    alone = [run(lib, d, m, 0.1) for m in masks]
    outs = [torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda") for _ in masks]
    spaces, streams = [workspace(lib, d) for _ in masks], [torch.cuda.Stream() for _ in masks]
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            call(lib, d, masks[k], devs[k], outs[k], spaces[k], 0.1, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert np.array_equal(host16(outs[k]), alone[k])
