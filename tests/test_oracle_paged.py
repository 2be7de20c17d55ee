"""Pins of the oracles of rotary positions, draft trees and moved rows: values worked out by hand,
closed forms, and agreement with the oracles that they extend."""
import numpy as np
import pytest

import oracle
import synth


def test_rope_by_hand():
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    f = np.array([np.pi / 2, np.pi], np.float32)   # a quarter and half a turn per position
    got = oracle.rope(x, 1, f, False, 2.0)
    assert np.allclose(got, [[-6, -4, 2, -8, 5]], atol=1e-6)           # (1, 3) -> (-3, 1), (2, 4) -> (-2, -4)
    got = oracle.rope(x, 1, f, True, 1.0)
    assert np.allclose(got, [[-2, 1, -3, -4, 5]], atol=1e-6)
    assert np.array_equal(oracle.rope(x, 0, f, True, 1.0), x)
    assert np.array_equal(oracle.rope(x, 9, np.zeros(0, np.float32), False, 3.0), x)


def test_rope_depends_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 16))
    f = (1e4 ** (-np.arange(8) / 8)).astype(np.float32)
    for interleaved in (False, True):
        dots = [float((oracle.rope(q, p + 7, f, interleaved, 1) * oracle.rope(k, p, f, interleaved, 1)).sum())
                for p in (0, 3, 1000, 2**31 - 8, -(2**31))]
        assert np.allclose(dots, dots[0], rtol=1e-9)
        assert not np.allclose(dots[0], (q * k).sum())


def test_rope_of_far_positions_is_exact():
    """2^30 steps of 2 pi / 2^30, as nearly as fp32 says it: the angle is the product, unrounded."""
    f = np.float32(2 * np.pi / 2**30)
    turned = oracle.rope(np.array([[1.0, 0.0]]), 2**30, [f], True, 1.0)
    off = float(f) * 2**30 - 2 * np.pi           # exact in fp64
    assert np.allclose(turned, [[np.cos(off), np.sin(off)]], atol=1e-12)


def test_rope_goes_where_tokens_go():
    offs, lens = np.array([0, 2, 2, 3], np.uint32), np.array([3, 9, 0], np.uint32)
    table = np.array([[5, 6], [9, 9], [2, 9]])
    x = synth.bf16_bits(np.ones((3, 1, 8)))
    q, k, v, page, slot = oracle.rope_ragged_paged(x, x, x, offs, lens, table, 4, np.float32([np.pi / 2]), interleaved=True)
    assert page.tolist() == [5, 6, 2] and slot.tolist() == [3, 0, 0]
    # positions 3, 4, 0: three quarters of a turn, a whole one, none
    assert np.allclose(q[:, 0, :2], [[1, -1], [1, 1], [1, 1]], atol=1e-5)
    q, *_ = oracle.rope_ragged_paged(x, None, None, offs, lens, table, 4, np.float32([np.pi / 2]), [1, 2, 3], True)
    assert np.allclose(q[:, 0, :2], [[-1, 1], [-1, -1], [1, -1]], atol=1e-5)


def test_tree_mask_by_hand():
    assert oracle.tree_mask([-1, 0, 0, 1, -1], 1).ravel().tolist() == [1, 3, 5, 11, 16]
    m = oracle.tree_mask([-1] + list(range(39)), 2)
    assert m[39].tolist() == [0xFFFFFFFF, 0xFF] and m[3].tolist() == [15, 0]


@pytest.mark.parametrize("window", [0, 1, 5, 30])
def test_a_chain_is_causal_attention(window):
    """Where each token's parent is the one before it, the tree's attention is the causal one (with a
    window: as long as that is no shorter than the chain, whose tokens count first)."""
    new, hist = [5, 1, 0, 3], [20, 0, 3, 7]
    d = synth.attention_inputs(1, new, hist, hq=4, hkv=2, d=16)
    mask = np.concatenate([oracle.tree_mask([j - 1 for j in range(n)], 2) for n in new])
    if window == 1:
        mask = np.concatenate([np.array([[1 << j, 0] for j in range(n)], np.uint32).reshape(n, 2) for n in new])
    a = oracle.attention_tree_ragged_paged(d.q, d.row_offsets, mask, d.blocks, d.cache_lengths, d.page_table, 1, 0.3, window)
    b = oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table, 1, 0.3, True, window)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12)


def test_full_masks_are_attention_without_order():
    new, hist = [40, 3], [0, 9]
    d = synth.attention_inputs(2, new, hist, hq=2, hkv=2, d=16, gran=0)
    mask = np.full((43, 2), 0xFFFFFFFF, np.uint32)
    a = oracle.attention_tree_ragged_paged(d.q, d.row_offsets, mask, d.blocks, d.cache_lengths, d.page_table, 1, 0.3)
    b = oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table, 1, 0.3, False)
    assert all(np.allclose(x, y, rtol=1e-12) for x, y in zip(a, b))


def test_a_row_that_sees_nothing_is_zero():
    d = synth.attention_inputs(3, [2], [0], hq=1, hkv=1, d=8)
    out, _, _ = oracle.attention_tree_ragged_paged(d.q, d.row_offsets, np.array([[4], [2]], np.uint32), d.blocks, d.cache_lengths,
                                                   d.page_table, 1, 1.0)
    assert (out[0] == 0).all()                                        # (bit 2 is behind the last token)
    v = oracle.cache_rows(d.blocks, d.page_table[0], 2, 1, 1)
    assert np.allclose(out[1, 0], v[1, 0])


def test_a_window_counts_drafted_tokens_first():
    d = synth.attention_inputs(4, [3], [6], hq=1, hkv=1, d=8)
    d.q[:] = 0                                                        # equal weights: the mean of what is seen
    mask = oracle.tree_mask([-1, 0, 0], 1)
    v = oracle.cache_rows(d.blocks, d.page_table[0], 9, 1, 1)[:, 0]
    for window, seen in ((1, [[6], [6, 7], [6, 8]]), (3, [[4, 5, 6], [5, 6, 7], [5, 6, 8]]),
                         (90, [[0, 1, 2, 3, 4, 5, 6], [0, 1, 2, 3, 4, 5, 6, 7], [0, 1, 2, 3, 4, 5, 6, 8]])):
        out, _, _ = oracle.attention_tree_ragged_paged(d.q, d.row_offsets, mask, d.blocks, d.cache_lengths, d.page_table, 1, 1.0, window)
        for r in range(3):
            assert np.allclose(out[r, 0], v[seen[r]].mean(0))


def test_keep_by_hand():
    blocks = np.arange(8, dtype=np.uint16).reshape(1, 1, 2, 4, 1, 1).repeat(2, 1)
    table = np.array([[1, 0]])
    got, _ = oracle.kv_keep_ragged_paged(np.array([[0, 2, 5]]), [3], blocks, [1], table)
    # positions 0 .. 7 hold 4 5 6 7 0 1 2 3; drafted 0 2 5 are positions 1 3 6
    assert got[0, 0, :, :, 0, 0].tolist() == [[0, 1, 2, 3], [4, 5, 7, 2]]
    got, _ = oracle.kv_keep_ragged_paged(np.array([[1, 2, 3]]), [2], blocks, [1], table)
    assert got[0, 0, :, :, 0, 0].tolist() == [[0, 1, 2, 3], [4, 6, 7, 7]]
    got, _ = oracle.kv_keep_ragged_paged(np.array([[0, 1, 2]]), [9], blocks, [1], table)
    assert np.array_equal(got, blocks)


def test_released_pages_are_handed_out_in_the_same_order():
    rng = np.random.default_rng(5)
    page, B, W = 4, 6, 12
    cached, new = rng.integers(0, 20, B), rng.integers(0, 25, B)
    free = rng.permutation(100).astype(np.uint32)
    table = np.full((B, W), 999, np.uint32)
    _, table, _, (left, status) = oracle.tables_ragged_paged(table, np.zeros(B, int), cached, free, 100, page, None)
    _, full, slots, (less, status2) = oracle.tables_ragged_paged(table, cached, new, free, left, page, None)
    assert status == status2 == 0 and less < left
    back, (count, status) = oracle.release_ragged_paged(free, full, cached + new, cached, less, page)
    assert status == 0 and count == left and np.array_equal(back[:count], free[:count])
    _, again, slots2, _ = oracle.tables_ragged_paged(full, cached, new, back, count, page, None)
    assert np.array_equal(again, full) and np.array_equal(slots, slots2)


def test_release_by_hand():
    table = np.array([[7, 8, 9], [4, 5, 6]], np.uint32)
    free = np.array([1, 2, 0, 0, 0, 0], np.uint32)
    got, result = oracle.release_ragged_paged(free, table, [9, 12], [4, 5], 2, 4)
    assert got.tolist() == [1, 2, 6, 9, 8, 0] and result == (5, 0)
    assert oracle.release_ragged_paged(free, table, [9, 12], [4, 0], 2, 4)[1] == (2, 1)     # five pages, room for four
    assert oracle.release_ragged_paged(free, table, [13, 1], [4, 1], 2, 4)[1] == (2, 2)
    assert oracle.release_ragged_paged(free, table, [13, 1], [13, 5], 2, 4)[1] == (2, 0)


def test_read_by_hand():
    d = synth.attention_inputs(6, [1, 1], [30, 17], hq=1, hkv=2, d=32, gran=32)
    got = oracle.kv_read_ragged_paged([0, 3, 3], [15, 0], d.blocks, d.page_table, 1, d.scales, 32)
    assert got.shape == (2, 3, 2, 32)
    for plane in (0, 1):
        assert np.array_equal(got[plane], oracle.cache_rows(d.blocks, d.page_table[0], 31, 1, plane, d.scales, 32)[15:18])
