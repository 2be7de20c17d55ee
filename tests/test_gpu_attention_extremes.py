"""attention_ragged_paged where numbers are extreme: what a row does not see must not change a
bit of it, and large finite values and scores must give the formula's finite results."""
import numpy as np
import pytest
import torch

import synth
from attention_shapes import kernel, tile_cuts
from gpu_util import bf16v, say
from test_gpu_attention import _drafts, compare, exact, run

pytestmark = pytest.mark.gpu


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def history(batch, first):
    return [first] + [5 + 2 * i for i in range(batch - 1)]


# name: new tokens, history, query heads, key/value heads; sequence 0 is the one looked at
FORMS = {
    "rows1": ([4, 2, 1], [70, 3, 60], 4, 2),
    "rows1 cut": ([4, 2, 1], [3000, 3, 60], 4, 2),
    "rows2": (_drafts(34, 40, 4), history(34, 70), 8, 2),
    "rows2 cut": (_drafts(34, 40, 4), history(34, 3000), 8, 2),
    "tile": ([150, 2, 1], [70, 3, 60], 4, 2),
    "tile cut": ([150, 2, 1], [3000, 3, 60], 4, 2),
}


def case(seed, form, dim, gran):
    new, hist, hq, hkv = FORMS[form]
    d = synth.attention_inputs(seed, new, hist, hq=hq, hkv=hkv, d=dim, gran=gran)
    assert kernel(d, cus()) == form.split()[0]
    if form == "tile cut":
        assert tile_cuts(d)[1][0] > 1
    say(f"[extremes] {form} q {d.q.shape} head {dim} gran {gran}")
    return d


def put(d, plane, pos, value):
    """One element of every head at one position of sequence 0."""
    page, slot = d.page_table[0, pos // 16], pos % 16
    if not d.gran:
        d.blocks[d.layer_idx, plane, page, slot, :, 5] = synth.bf16_bits(np.array([value]))[0]
    elif np.isnan(value):
        d.blocks[d.layer_idx, plane, page, slot, :, 5] = 0x7F
    else:
        d.scales[d.layer_idx, plane, page, slot, :, 0] = value


def blind(d, at, window):
    """Rows that do not see position `at` of sequence 0."""
    rows = np.ones(len(d.q), bool)
    first = at - int(d.cache_lengths[0])
    new = int(d.row_offsets[1])
    rows[first:min(new, first + window) if window else new] = False
    return rows


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,gran", [(64, 0), (64, 32), (128, 128), (256, 0), (256, 64)])
@pytest.mark.parametrize("window", [0, 2])
def test_a_value_that_a_row_does_not_see_changes_no_bit_of_it(lib, gpu, form, dim, gran, window):
    """Infinities and NaN in one position's values, or in their scales."""
    if form.startswith("rows2") and window:
        window = 20   # (its first sequence has 40 new tokens)
    d = case(50, form, dim, gran)
    at = int(d.cache_lengths[0]) + (2 if form.startswith("rows1") else 17)
    clean = run(lib, d, 0.125, True, window)
    hidden = blind(d, at, window)
    for value in (float("nan"), float("inf")):
        put(d, 1, at, value)
        got = run(lib, d, 0.125, True, window)
        assert not np.isfinite(bf16v(got)[~hidden]).all()
        compare(d, got, exact(d, 0.125, True, window), form)
        assert np.array_equal(got[hidden], clean[hidden]), f"{int((got != clean)[hidden].sum())} elements changed by {value}"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,gran", [(64, 0), (64, 32), (128, 128), (256, 0), (256, 64)])
@pytest.mark.parametrize("window", [0, 2])
def test_a_key_that_a_row_does_not_see_changes_no_bit_of_it(lib, gpu, form, dim, gran, window):
    """One position's keys are such that the rows which see it get the largest of their scores
    there, an infinite one, or NaN; the rows that do not share their waves with those."""
    if form.startswith("rows2") and window:
        window = 20
    d = case(51, form, dim, gran)
    at = int(d.cache_lengths[0]) + (2 if form.startswith("rows1") else 17)
    clean = run(lib, d, 0.125, True, window)
    hidden = blind(d, at, window)
    page, slot = d.page_table[0, at // 16], at % 16
    for value in (float("nan"), float("inf"), None):
        if value is None:
            # eight times the length of the others, and so of its scores
            if gran:
                d.blocks[1, 0, page, slot] = 0x70
                d.scales[1, 0, page, slot] = 0.0625
            else:
                d.blocks[1, 0, page, slot] = synth.bf16_bits(np.random.default_rng(3).standard_normal((d.blocks.shape[4], dim)) * 8)
        else:
            put(d, 0, at, value)
        got = run(lib, d, 0.125, True, window)
        assert np.array_equal(got[hidden], clean[hidden]), f"{int((got != clean)[hidden].sum())} elements changed by {value}"


def huge_values(d, growing):
    """Values of 2^125 to 2^126 in the first 64 dims, about 1 in the others; the sign depends on the
    head and dim alone, so that the weighted mean is as large. growing: scores that grow along
    the sequences, so that weights exceed 1 against the reference that rows keep."""
    rng = np.random.default_rng(7)
    L, _, P, S, hkv, D = d.blocks.shape
    sign = np.where(rng.random((hkv, D)) < 0.5, -1.0, 1.0)
    size = rng.uniform(0.5, 1.0, (P, S, hkv, D))
    big = np.arange(D) < 64
    held = (d.blocks[1, 1] != 0xFFFF) if not d.gran else (d.blocks[1, 1] != 0x7F)
    if d.gran:
        codes = synth.e4m3_codes(sign * size * 448)
        d.blocks[1, 1] = np.where(held, codes, 0x7F)
        runs = np.where(big.reshape(-1, d.gran)[:, 0], 2.0**126, 1.0) / 448
        d.scales[1, 1] = np.where(np.isnan(d.scales[1, 1]), np.nan, runs).astype(np.float32)
    else:
        d.blocks[1, 1] = np.where(held, synth.bf16_bits(sign * size * np.where(big, 2.0**126, 1.0)), 0xFFFF)
    if growing:
        for b in range(len(d.cache_lengths)):
            n = int(d.cache_lengths[b]) + int(d.row_offsets[b + 1]) - int(d.row_offsets[b])
            at = np.arange(n)
            k = np.zeros((n, hkv, D))
            k[:, :, 0] = np.linspace(0.0, 30.0, n)[:, None]
            if d.gran:
                d.blocks[1, 0, d.page_table[b, at // S], at % S] = synth.e4m3_codes(k * 8)
                d.scales[1, 0, d.page_table[b, at // S], at % S] = 0.125
            else:
                d.blocks[1, 0, d.page_table[b, at // S], at % S] = synth.bf16_bits(k)
        d.q[:] = synth.bf16_bits(np.broadcast_to(np.eye(D)[0], d.q.shape))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("dim", [128, 256])
def test_sums_of_large_values_do_not_leave_the_type(lib, gpu, form, gran, growing, dim):
    """The weighted mean of finite values is finite, however many they are."""
    d = case(52, form, dim, gran)
    huge_values(d, growing)
    scale = 1.0 if growing else 0.125
    ref = exact(d, scale)
    assert np.isfinite(ref[0]).all() and np.abs(ref[0]).max() > 2.0**125
    say(f"[extremes]   worst element at {compare(d, run(lib, d, scale), ref, form):.2f} of its tolerance")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_large_values_beside_an_infinite_one(lib, gpu, form, gran, bad):
    """Rows that see it and rows that do not, all of which have sums that are too large as they are."""
    d = case(54, form, 128, gran)
    huge_values(d, False)
    clean = run(lib, d, 0.125)
    at = int(d.cache_lengths[0]) + (2 if form.startswith("rows1") else 17)
    put(d, 1, at, float(bad))
    got, hidden = run(lib, d, 0.125), blind(d, at, 0)
    compare(d, got, exact(d, 0.125), form)
    assert np.isfinite(bf16v(got)[hidden]).all() and np.array_equal(got[hidden], clean[hidden])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("order", ["first", "last"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_an_infinite_value_counts_however_small_its_weight(lib, gpu, form, gran, order, bad):
    """A position whose weight is e^-200 of the others', less than fp32 holds: before all scores that
    are so much larger (the row's sums are rescaled, in a block, between waves or between parts),
    or behind them."""
    d = case(55, form, 128, gran)
    S = d.blocks.shape[3]
    n = int(d.cache_lengths[0]) + int(d.row_offsets[1])
    at = np.arange(n)
    small = int(d.cache_lengths[0]) // 2 if order == "first" else 0   # positions with a score of 0
    k = np.zeros((n, d.blocks.shape[4], 128))
    k[small:, :, 0] = 200.0
    spot = small // 3 if order == "first" else int(d.cache_lengths[0]) - 2
    k[spot] = 0.0
    page = d.page_table[0, at // S]
    if gran:
        d.blocks[1, 0, page, at % S] = synth.e4m3_codes(k)
        d.scales[1, 0, page, at % S] = 1.0
    else:
        d.blocks[1, 0, page, at % S] = synth.bf16_bits(k)
    d.q[:int(d.row_offsets[1])] = synth.bf16_bits(np.broadcast_to(np.eye(128)[0], d.q[:int(d.row_offsets[1])].shape))
    put(d, 1, spot, float(bad))
    ref = exact(d, 1.0)
    assert not np.isfinite(ref[0][0]).all()
    compare(d, run(lib, d, 1.0), ref, form)

@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dim", [128, 256])
def test_scores_far_beyond_one(lib, gpu, form, gran, sign, dim):
    """Scores of 2^40 and more, exact in fp32 (one product of two short numbers each), so far apart
    that all weight is on the largest, or even on those that share it: their mean comes out.

    The weights are 1 or 0, so what is rounded is the sum over equal ones (N + 1 roundings of 2^-24
    of the mean of |v|, as the division) and the result to bf16 (2^-8); with an e4m3 cache also
    the weight times its value's scale, to bf16 in the kernel for many rows: at most 2^-8 of each
    |v|, so 2^-8 of their mean, which the result's rounding then sees (a factor 1 + 2^-8)."""
    d = case(53, form, dim, gran)
    rng = np.random.default_rng(8)
    d.q[:] = synth.bf16_bits(np.broadcast_to(sign * np.eye(dim)[0] * 2.0**20, d.q.shape))
    keys = d.blocks[1, 0]
    k = np.zeros(keys.shape)
    k[..., 0] = 1 + rng.integers(0, 8, keys.shape[:-1]) / 8
    if gran:
        held = keys != 0x7F
        d.blocks[1, 0] = np.where(held, synth.e4m3_codes(k), 0x7F)
        d.scales[1, 0] = np.where(np.isnan(d.scales[1, 0]), np.nan, 2.0**20).astype(np.float32)
    else:
        d.blocks[1, 0] = np.where(keys != 0xFFFF, synth.bf16_bits(k * 2.0**20), 0xFFFF)
    out, spread, _ = exact(d, 1.0)
    n = int((d.cache_lengths.astype(np.int64) + np.diff(d.row_offsets.astype(np.int64))).max())
    got = bf16v(run(lib, d, 1.0))
    err = np.abs(got - out)
    tol = 2.0**-8 * np.abs(out) + (n + 4) * 2.0**-23 * spread
    if gran:
        tol += 2.0**-8 * (1 + 2.0**-8) * spread
    good = bool((err <= tol).all())
    assert good, (int(np.isnan(got).sum()), float(np.nanmax(err)))
