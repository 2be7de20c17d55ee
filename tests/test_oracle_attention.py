"""Pins of the attention and tables oracles: worked examples by hand, closed forms and a
brute force that shares nothing with them."""
import math

import numpy as np
import pytest

import oracle
import synth
from oracle import numerics as nm


def test_one_visible_position_gives_its_value():
    d = synth.attention_inputs(1, [1, 1], [0, 0], hq=4, hkv=2, d=8, page=3)
    out, spread, _ = oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table,
                                                   d.layer_idx, 0.5)
    for b in range(2):
        v = nm.decode_bf16(d.blocks[1, 1, d.page_table[b, 0], 0])
        assert np.array_equal(out[b], v[[0, 0, 1, 1]])
        assert np.array_equal(spread[b], np.abs(v[[0, 0, 1, 1]]))


def test_worked_example():
    """Two positions with scores ln 3 and 0: weights 3/4 and 1/4."""
    d = synth.attention_inputs(2, [1], [1], hq=1, hkv=1, d=8, page=2, layers=1)
    k = np.zeros((2, 8))
    k[0, 0] = 1
    v = np.zeros((2, 8))
    v[:, 1] = [8, -4]
    page = d.page_table[0, 0]
    d.blocks[0, 0, page, :2, 0] = synth.bf16_bits(k)
    d.blocks[0, 1, page, :2, 0] = synth.bf16_bits(v)
    d.q[0, 0] = synth.bf16_bits(np.eye(8)[0])
    out, spread, size = oracle.attention_ragged_paged(d.q, d.row_offsets, d.blocks, d.cache_lengths, d.page_table, 0,
                                                      math.log(3.0))
    assert np.allclose(out[0, 0], [0, 5, 0, 0, 0, 0, 0, 0], atol=1e-14)
    assert np.allclose(spread[0, 0, 1], 7, atol=1e-14)
    assert np.isclose(size[0, 0], math.log(3.0))


def brute(d, scale, causal, window):
    """Scalar loops over python floats."""
    T, Hq, D = d.q.shape
    Hkv, S = d.blocks.shape[4], d.blocks.shape[3]
    q = nm.decode_bf16(d.q)
    out = np.full((T, Hq, D), np.nan)

    def value(plane, b, pos, g, e):
        page, slot = int(d.page_table[b, pos // S]), pos % S
        x = d.blocks[d.layer_idx, plane, page, slot, g, e]
        if d.scales is None:
            return float(nm.decode_bf16(np.array([x]))[0])
        return float(nm.decode_e4m3(np.array([x]))[0]) * float(d.scales[d.layer_idx, plane, page, slot, g, e // d.gran])

    for b in range(len(d.cache_lengths)):
        for row in range(int(d.row_offsets[b]), int(d.row_offsets[b + 1])):
            p = int(d.cache_lengths[b]) + row - int(d.row_offsets[b])
            total = int(d.cache_lengths[b]) + int(d.row_offsets[b + 1]) - int(d.row_offsets[b])
            seen = [i for i in range(total) if (not causal or i <= p) and (not window or i > p - window)]
            for h in range(Hq):
                g = h * Hkv // Hq
                s = [scale * math.fsum(q[row, h, e] * value(0, b, i, g, e) for e in range(D)) for i in seen]
                w = [math.exp(x - max(s)) for x in s]
                for e in range(D):
                    out[row, h, e] = math.fsum(wi * value(1, b, i, g, e) for wi, i in zip(w, seen)) / math.fsum(w)
    return out


@pytest.mark.parametrize("gran,d,causal,window", [(0, 8, True, 0), (0, 16, False, 0), (0, 8, True, 3), (32, 64, True, 0),
                                                   (64, 64, True, 2)])
def test_brute_force(gran, d, causal, window):
    x = synth.attention_inputs(3, [2, 0, 3, 1], [3, 4, 0, 6], hq=4, hkv=2, d=d, page=3, gran=gran)
    out, _, _ = oracle.attention_ragged_paged(x.q, x.row_offsets, x.blocks, x.cache_lengths, x.page_table, x.layer_idx,
                                              0.3, causal, window, x.scales, x.gran)
    assert np.allclose(out, brute(x, 0.3, causal, window), rtol=1e-12, atol=1e-12)


def test_window_of_one_is_the_own_value_and_a_wide_one_is_none():
    x = synth.attention_inputs(4, [5], [7], hq=2, hkv=1, d=8, page=4)
    a = (x.q, x.row_offsets, x.blocks, x.cache_lengths, x.page_table, x.layer_idx, 0.3, True)
    v = oracle.cache_rows(x.blocks, x.page_table[0], 12, 1, 1)
    assert np.array_equal(oracle.attention_ragged_paged(*a, 1)[0][:, 0], v[7:, 0])
    assert np.array_equal(oracle.attention_ragged_paged(*a, 12)[0], oracle.attention_ragged_paged(*a, 0)[0])


def test_mutations_are_seen():
    """What the oracle must not ignore: the history, the page order, the group of heads."""
    x = synth.attention_inputs(5, [2, 2], [9, 3], hq=4, hkv=2, d=8, page=4)
    a = [x.q, x.row_offsets, x.blocks, x.cache_lengths, x.page_table, x.layer_idx, 0.3]
    ref = oracle.attention_ragged_paged(*a)[0]
    short = list(a)
    short[3] = x.cache_lengths - 1
    assert not np.allclose(oracle.attention_ragged_paged(*short)[0], ref)
    swapped = list(a)
    swapped[4] = x.page_table.copy()
    swapped[4][0, :2] = x.page_table[0, 1::-1]
    assert np.allclose(oracle.attention_ragged_paged(*swapped)[0][0], ref[0])   # all its positions seen: order is free
    swapped[4] = x.page_table.copy()
    swapped[4][0, :3] = x.page_table[0, 2::-1]
    swapped[2] = np.where(x.blocks == 0xFFFF, 0, x.blocks).astype(np.uint16)
    assert not np.allclose(oracle.attention_ragged_paged(*swapped)[0][0], ref[0])
    heads = list(a)
    heads[0] = x.q[:, [0, 2, 1, 3]]
    assert not np.allclose(oracle.attention_ragged_paged(*heads)[0][:, [0, 2, 1, 3]], ref)


def test_tables_worked_example():
    """Pages of 4: sequence 0 holds 5 tokens in pages (7, 2) and adds 4: one new page; 1 adds
    nothing; 2 starts with 5 tokens: two new pages; 3 fills its page and needs none."""
    table = np.array([[7, 2, 99, 99], [3, 99, 99, 99], [99, 99, 99, 99], [6, 99, 99, 99]], dtype=np.uint32)
    offs, t, slots, result = oracle.tables_ragged_paged(table, [5, 2, 0, 3], [4, 0, 5, 1], [11, 12, 13, 14, 15], 4, 4, 10)
    assert offs.tolist() == [0, 4, 4, 9, 10]
    assert t.tolist() == [[7, 2, 14, 99], [3, 99, 99, 99], [13, 12, 99, 99], [6, 99, 99, 99]]
    assert slots.tolist() == [9, 10, 11, 56, 52, 53, 54, 55, 48, 27]
    assert result == (1, 0)
    assert oracle.tables_ragged_paged(table, [5, 2, 0, 3], [4, 0, 5, 1], [11, 12, 13, 14, 15], 2, 4, 9)[3] == (2, 5)
    assert oracle.tables_ragged_paged(table, [5, 2, 0, 3], [4, 0, 17, 1], [11] * 20, 20, 4, 99)[3] == (20, 2)
    assert oracle.tables_ragged_paged(table, [5, 2, 0, 3], [4, 0, 5, 1], [11, 12], 4, 4, 10)[3] == (4, 1)
