"""attention_tree_ragged_paged reads no page that no token sees: not those before the first position of the
history that some token's window leaves, nor those behind the last drafted token that some token names. Their
page table entries are far out of range here. Tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import bf16v, say
from test_gpu_attention import compare
from test_gpu_attention_extremes import put
from test_gpu_attention_tree import exact, run, tree_rows

pytestmark = pytest.mark.gpu


def seen_ranges(d, mask, window):
    """Of each sequence: first position that some token sees, and the one behind the last."""
    ranges = []
    for b in range(len(d.cache_lengths)):
        r0, n, c = int(d.row_offsets[b]), int(d.row_offsets[b + 1] - d.row_offsets[b]), int(d.cache_lengths[b])
        first, end = c, c
        for r in range(r0, r0 + n):
            named = [i for i in range(min(n, 32 * mask.shape[1])) if int(mask[r, i // 32]) >> i % 32 & 1]
            first = min(first, max(0, c - max(window - len(named), 0)) if window else 0)
            end = max([end] + [c + i + 1 for i in named])
        ranges.append((first, end))
    return ranges


def hide(d, mask, window):
    """Entries of pages that hold no position of a range, in a table that is as wide as before."""
    page = d.blocks.shape[3]
    for b, (first, end) in enumerate(seen_ranges(d, mask, window)):
        used = range(first // page, -(-end // page) if end > first else first // page)
        for e in range(d.page_table.shape[1]):
            if e not in used:
                d.page_table[b, e] = 0xFFFFFFFF


def masks(d, words, kind):
    if kind in ("tree", "any"):
        return tree_rows(d, words, 3, kind)
    rows = np.zeros((len(d.q), words), np.uint32)
    for b in range(len(d.cache_lengths)):
        r0, r1 = int(d.row_offsets[b]), int(d.row_offsets[b + 1])
        n = min(r1 - r0, 2)
        if kind == "padded" and n:   # a tree of two tokens at most; the other rows name none
            rows[r0:r0 + n] = oracle.tree_mask([-1, 0][:n], words)
    return rows


CASES = {
    "few": ([3, 0, 1, 7, 2], [0, 5, 400, 61, 230], 4, 2, 64),
    "few cut": ([4, 2, 1], [3000, 3, 60], 4, 2, 128),
    "many": ([70, 0, 33, 1, 129], [0, 5, 400, 61, 230], 4, 2, 64),
    "many cut": ([150, 2, 1], [3000, 3, 60], 4, 2, 128),
    "wide": ([150, 0, 100], [70, 3, 1000], 8, 2, 128),
    "heads of 256": ([40, 1], [300, 70], 4, 1, 256),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("page", [1, 16, 20])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_pages_that_no_token_sees_do_not_exist(lib, gpu, case, gran, page, window):
    new, hist, hq, hkv, dim = CASES[case]
    for kind in ("tree", "any", "padded", "none"):
        d = synth.attention_inputs(30, new, hist, hq=hq, hkv=hkv, d=dim, page=page, gran=gran)
        mask = masks(d, 5, kind)
        ref = exact(d, mask, 0.125, window)
        hide(d, mask, window)
        say(f"[tree pages] {case} gran {gran} page {page} window {window} {kind}")
        got = run(lib, d, mask, 0.125, window)
        compare(d, got, ref)
        if kind == "none":   # a sequence without history sees nothing at all: no page is read
            empty = np.repeat(np.asarray(hist) == 0, new)
            assert not got[:len(empty)][empty].any()


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("window", [0, 33])
def test_nor_by_the_pass_for_values_that_are_not_finite(lib, gpu, case, gran, window):
    """A NaN among the values that some rows see: they are computed again, over the same pages."""
    new, hist, hq, hkv, dim = CASES[case]
    d = synth.attention_inputs(31, new, hist, hq=hq, hkv=hkv, d=dim, page=16, gran=gran)
    mask = masks(d, 5, "padded")
    put(d, 1, hist[0], float("nan"))
    ref = exact(d, mask, 0.125, window)
    hide(d, mask, window)
    say(f"[tree pages] {case} gran {gran} window {window}, NaN")
    got = run(lib, d, mask, 0.125, window)
    compare(d, got, ref)
    assert not np.isfinite(bf16v(got[:int(d.row_offsets[1])])).all()
