"""attention_ragged_paged in the forms that its sizes choose between: workgroups that take several
heads, many sequences with cut tiles, and counting tests that see every single position."""
import dataclasses

import numpy as np
import pytest
import torch

import synth
from attention_shapes import heads_per_workgroup, kernel, new_lengths, tile_cuts
from gpu_util import bf16v, say
from test_gpu_attention import check, compare, exact, run, tolerance

pytestmark = pytest.mark.gpu


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def lengths(seed, batch, new, history, long=()):
    """new, history: (lowest, highest); a few empty sequences; long: (sequence, history)."""
    rng = np.random.default_rng(seed)
    n = rng.integers(new[0], new[1] + 1, batch)
    n[rng.integers(0, batch, batch // 20)] = 0
    h = rng.integers(history[0], history[1] + 1, batch)
    for b, x in long:
        n[b], h[b] = max(n[b], 1), x
    return n, h


# form, heads per workgroup, head dim, gran, query heads, key/value heads, batch, new, history, page, window
WIDE = [
    ("rows1", 4, 128, 0, 16, 8, 260, (1, 1), (90, 200), 16, 0),
    ("rows1", 4, 128, 0, 8, 8, 260, (1, 1), (90, 200), 12, 0),
    ("rows1", 4, 64, 0, 8, 4, 700, (1, 1), (150, 280), 16, 0),
    ("rows1", 4, 64, 32, 8, 4, 700, (1, 1), (150, 280), 1, 0),
    ("rows1", 4, 128, 128, 8, 8, 330, (1, 1), (170, 260), 32, 0),
    ("rows1", 2, 64, 64, 6, 2, 700, (1, 1), (150, 280), 48, 0),
    ("rows1", 2, 256, 0, 4, 2, 330, (1, 1), (170, 300), 16, 0),
    ("rows1", 2, 256, 64, 4, 2, 660, (1, 1), (170, 300), 16, 0),
    ("rows2", 4, 128, 0, 16, 4, 330, (5, 11), (150, 300), 16, 0),
    ("rows2", 4, 64, 32, 16, 4, 700, (5, 11), (100, 280), 16, 0),
    ("rows2", 2, 64, 0, 8, 2, 700, (5, 11), (100, 280), 20, 0),
    ("rows2", 2, 256, 128, 8, 2, 660, (5, 11), (150, 300), 16, 0),
    ("rows1", 4, 64, 0, 8, 4, 900, (1, 1), (200, 400), 16, 150),
    ("rows2", 2, 64, 64, 8, 2, 900, (5, 11), (200, 400), 16, 150),
]


def wide_case(seed, form, heads, dim, gran, hq, hkv, batch, new, history, page, window):
    d = synth.attention_inputs(seed, *lengths(seed, batch, new, history, long=((batch // 2, 1500),)), hq=hq, hkv=hkv, d=dim,
                               page=page, gran=gran, layers=1)
    assert kernel(d, cus()) == form
    assert heads_per_workgroup(d, cus(), window) == heads
    return d


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(str(x) for x in c[:4]) + f"-p{c[9]}-w{c[10]}")
def test_workgroups_that_take_several_heads(lib, gpu, case):
    d = wide_case(60, *case)
    check(lib, d, window=case[10])


@pytest.mark.parametrize("case", [WIDE[2], WIDE[7], WIDE[9], WIDE[10]], ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_nan_where_workgroups_take_several_heads(lib, gpu, case):
    """In the values of the last position of some sequences: seen by their last token alone."""
    d = wide_case(61, *case)
    clean = run(lib, d, 0.125)
    new = new_lengths(d)
    seen = np.zeros(len(d.q), bool)
    for b in range(0, len(new), 7):
        if new[b]:
            at = int(d.cache_lengths[b]) + int(new[b]) - 1
            page = case[9]
            d.blocks[0, 1, d.page_table[b, at // page], at % page, :, 3] = 0x7F if d.gran else 0x7FC0
            seen[int(d.row_offsets[b + 1]) - 1] = True
    got = run(lib, d, 0.125)
    compare(d, got, exact(d, 0.125))
    assert np.array_equal(got[~seen], clean[~seen]) and np.isnan(bf16v(got)[seen][..., 3]).all()


@pytest.mark.parametrize("batch", [65, 200, 257, 600])
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("window", [0, 700])
def test_many_sequences_of_which_some_are_cut(lib, gpu, batch, gran, window):
    """The kernel for many rows where a workgroup looks its item up with all its threads."""
    long = [(0, 1900), (63, 2000), (64, 1500), (batch - 1, 1700)] + [(b, 1800) for b in (127, 128, 255, 256, 511, 512) if b < batch]
    d = synth.attention_inputs(62, *lengths(62, batch, (2, 6), (0, 90), long), hq=32, hkv=2, d=64, gran=gran, layers=1)
    assert kernel(d, cus()) == "tile"
    parts = tile_cuts(d, window)[1]
    assert (parts > 1).sum() >= 3 and (parts == 1).any() and (parts == 0).any()
    check(lib, d, window=window)


# ---------------------------------------------------------------------------
# counting: with q = 0 every weight is 1, and with the value N (the number of
# positions that a row sees) in head dim p mod D of position p, 0 elsewhere, the output
# is the number of positions of each residue. N is a bf16, the products and their sums
# are whole numbers below 2^24 and a count is at most 256, a bf16 too, so the result has
# to be equal: N * fl(1 / N) is off by 2^-23 at most, which the rounding to bf16 takes back.
# ---------------------------------------------------------------------------

def counting(d, seen_by_seq):
    """Puts the values; seen_by_seq: N of each sequence."""
    D, S = d.q.shape[2], d.blocks.shape[3]
    d.q[:] = 0
    for b, n in enumerate(seen_by_seq):
        total = int(d.cache_lengths[b]) + int(new_lengths(d)[b])
        assert n < 256 or n % (1 << (int(n).bit_length() - 8)) == 0, "N is a bf16"
        at = np.arange(total)
        page, slot = d.page_table[b, at // S], at % S
        if d.gran:
            d.blocks[d.layer_idx, 1, page, slot] = 0
            d.blocks[d.layer_idx, 1, page, slot, :, at % D] = 0x38   # one
            d.scales[d.layer_idx, 1, page, slot] = n
        else:
            d.blocks[d.layer_idx, 1, page, slot] = 0
            d.blocks[d.layer_idx, 1, page, slot, :, at % D] = synth.bf16_bits(np.array([float(n)]))[0]


def counts(d, causal, window):
    D = d.q.shape[2]
    out = np.zeros((int(d.row_offsets[-1]), D))
    for b, n in enumerate(new_lengths(d)):
        c = int(d.cache_lengths[b])
        for j in range(int(n)):
            last = c + j if causal else c + int(n) - 1
            first = max(0, last - window + 1) if window else 0
            out[int(d.row_offsets[b]) + j] = np.bincount(np.arange(first, last + 1) % D, minlength=D)
    return out


def check_counts(lib, d, causal=True, window=0):
    say(f"[counting] q {d.q.shape} lengths {d.cache_lengths[:6].tolist()} cache {d.blocks.shape} gran {d.gran} causal {causal} "
        f"window {window} {kernel(d, cus())}")
    got = bf16v(run(lib, d, 1.0, causal, window))
    want = counts(d, causal, window)[:, None]
    assert want.max() <= 256
    bad = (got != want).nonzero()
    assert len(bad[0]) == 0, f"{len(bad[0])} counts off, first at {[int(x[0]) for x in bad]}: {got[tuple(x[0] for x in bad)]}"


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("page", [1, 16, 48, 100, 128])
@pytest.mark.parametrize("hkv", [1, 4])
def test_every_position_counts_once_single_tokens(lib, gpu, gran, page, hkv):
    total = [9216, 33, 4096, 1, 5056, 255, 64, 2144]
    d = synth.attention_inputs(63, [1] * 8, [n - 1 for n in total], hq=2 * hkv, hkv=hkv, d=64, page=page, gran=gran, layers=1)
    assert kernel(d, cus()) == "rows1"
    counting(d, total)
    check_counts(lib, d)


@pytest.mark.parametrize("gran,dim", [(0, 128), (32, 64), (128, 128), (64, 256)])
def test_every_position_counts_once_many_single_tokens(lib, gpu, gran, dim):
    """Shares that hold several sequences, several heads per workgroup."""
    rng = np.random.default_rng(64)
    total = rng.integers(130, 256, 700)
    total[5::50] = rng.integers(1, 40, 14)
    total[::9] = 2 * rng.integers(128, 256, len(total[::9]))
    total[350] = 4096
    d = synth.attention_inputs(64, [1] * 700, total - 1, hq=4, hkv=4, d=dim, page=16, gran=gran, layers=1)
    assert kernel(d, cus()) == "rows1" and heads_per_workgroup(d, cus()) > 1
    counting(d, total)
    check_counts(lib, d)


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("page", [1, 16, 48])
@pytest.mark.parametrize("new,total,hq", [([90, 33, 150], [9216, 512, 160], 4), ([40, 128, 1], [5056, 4096, 2144], 2),
                                          ([3, 2, 4], [9216, 2144, 512], 4)], ids=["chunks", "cut chunks", "drafts"])
def test_every_position_counts_once_not_causal(lib, gpu, gran, page, new, total, hq):
    d = synth.attention_inputs(65, new, np.array(total) - np.array(new), hq=hq, hkv=2, d=64, page=page, gran=gran, layers=1)
    assert kernel(d, cus()) == ("rows1" if max(new) < 10 else "tile")
    if new[0] == 40:
        assert tile_cuts(d)[1].max() > 1
    counting(d, total)
    check_counts(lib, d, causal=False)


@pytest.mark.parametrize("gran", [0, 64])
def test_every_position_counts_once_two_row_tiles(lib, gpu, gran):
    """Drafts of many sequences, all positions seen."""
    rng = np.random.default_rng(66)
    new = rng.integers(5, 8, 70)
    new[3] = 40
    total = 2 * rng.integers(64, 250, 70)
    total[3], total[20] = 5056, 9216
    d = synth.attention_inputs(66, new, total - new, hq=8, hkv=2, d=64, gran=gran, layers=1)
    assert kernel(d, cus()) == "rows2"
    counting(d, total)
    check_counts(lib, d, causal=False)


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("window", [31, 32, 33, 96, 1504])
@pytest.mark.parametrize("new", [[1, 2, 1], [150, 3, 66]], ids=["few", "chunks"])
def test_every_position_counts_once_in_a_window(lib, gpu, gran, page, window, new):
    for shift in (0, 17):
        d = synth.attention_inputs(67, new, np.array([window - 1, window + 40 + shift, 4000 + shift]), hq=4, hkv=2, d=64, page=page,
                                   gran=gran, layers=1)
        counting(d, [window] * 3)
        check_counts(lib, d, True, window)


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("new,history", [([600], [0]), ([300], [700]), ([5], [900]), ([129, 1, 40], [500, 64, 127])])
def test_every_position_counts_once_causal(lib, gpu, gran, page, new, history):
    """Rows that see different numbers of positions: values of one, so that the output is a count
    over N, at most about 20 / N: one position more or less is 5 % of it or all, the rounding
    to bf16 2^-8 (the division and the sum's rounding 2^-22)."""
    d = synth.attention_inputs(68, new, history, hq=2, hkv=1, d=64, page=page, gran=gran, layers=1)
    counting(d, [1] * len(new))
    want = counts(d, True, 0)
    assert want.max() <= 20
    got = bf16v(run(lib, d, 1.0))
    want = (want / want.sum(1, keepdims=True))[:, None]
    assert (np.abs(got - want) <= (2.0**-8 + 2.0**-20) * want).all()


# ---------------------------------------------------------------------------
# the probabilities of the kernel for few rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("form,new,history,hq,hkv", [
    ("rows1", [3, 0, 1, 7, 2], [0, 5, 40, 61, 130], 2, 2), ("rows1", [1, 2, 1], [9000, 40, 2500], 4, 1),
    ("rows1", [1] * 70, list(range(300, 370)), 8, 8), ("rows2", [9, 0, 1] + [6] * 67, list(range(200, 270)), 8, 2)])
@pytest.mark.parametrize("dim,gran", [(64, 0), (128, 0), (256, 0), (64, 32), (128, 128), (256, 64)])
def test_few_rows_lose_nothing_to_the_probabilities(lib, gpu, form, new, history, hq, hkv, dim, gran):
    """That kernel takes a probability (times its value's scale) as two bf16, value and
    remainder: the remainder is exact in fp32 and at most 2^-8 of the probability, its own rounding
    2^-8 of that, so 2^-16 of the weighted mean of |v| takes the place of 2^-8 in the bound."""
    d = synth.attention_inputs(69, new, history, hq=hq, hkv=hkv, d=dim, gran=gran, layers=1)
    assert kernel(d, cus()) == form
    ref = exact(d, dim ** -0.5)
    out, spread, _ = ref
    tol = tolerance(d, ref) - 2.0**-8 * (1 + 2.0**-7) * spread + 2.0**-16 * spread
    err = np.abs(bf16v(run(lib, d, dim ** -0.5)) - out)
    used = float((err / tol).max())
    say(f"[forms] {form} head {dim} gran {gran}: worst element at {used:.2f} of its tolerance")
    assert used <= 1


# ---------------------------------------------------------------------------
# batches that a server sends
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [3, 90])
@pytest.mark.parametrize("history", [0, 700])
def test_a_batch_without_new_tokens_leaves_everything(lib, gpu, rows, history):
    """A buffer of rows, none of which belongs to a sequence."""
    d = synth.attention_inputs(70, [0, 0, 0], [history, 5, 0], hq=4, hkv=2, d=64, spare_rows=rows, layers=1)
    assert kernel(d, cus()) == ("rows1" if rows == 3 else "tile")
    assert (run(lib, d, 0.125) == 0x7FC1).all()


@pytest.mark.parametrize("new,spare", [([1, 0, 2, 0, 1], 0), ([90, 0, 2, 0, 1], 0), ([1, 0, 2, 0, 1], 200)])
@pytest.mark.parametrize("batch", [5, 100])
@pytest.mark.parametrize("length", [0x7FFFFFFF, 0x80000000, 0xFFFFFFFF])
def test_sequences_without_new_tokens_may_have_any_length(lib, gpu, new, spare, batch, length):
    """A slot of the batch that nobody uses: its length and pages are what they were."""
    new = new + [0] * (batch - 5)
    d = synth.attention_inputs(71, new, [300, 9, 40, 3, 0] + [7] * (batch - 5), hq=4, hkv=2, d=64, spare_rows=spare, layers=1)
    ref = exact(d, 0.125)
    lengths, table = d.cache_lengths.copy(), d.page_table.copy()
    lengths[np.array(new) == 0] = length
    table[np.array(new) == 0] = 0xFFFFFFFF
    d = dataclasses.replace(d, cache_lengths=lengths, page_table=table)
    got = run(lib, d, 0.125)
    tol = tolerance(dataclasses.replace(d, cache_lengths=np.where(np.array(new) == 0, 0, lengths)), ref)
    rows = int(d.row_offsets[-1])
    assert (got[rows:] == 0x7FC1).all()
    assert (np.abs(bf16v(got) - ref[0]) <= tol)[:rows].all()


@pytest.mark.parametrize("new", [[1, 2, 1], [70, 2, 40]], ids=["few", "chunks"])
def test_sequences_that_share_their_first_pages(lib, gpu, new):
    d = synth.attention_inputs(72, new, [200, 210, 190], hq=4, hkv=2, d=64, layers=1)
    d.page_table[1, :11] = d.page_table[0, :11]
    d.page_table[2, :11] = d.page_table[0, :11]
    check(lib, d)


def test_tables_and_codes_in_their_own_types(lib, gpu):
    """uint32 tables and float8_e4m3fn blocks give what int32 and uint8 ones do."""
    d = synth.attention_inputs(73, [1, 2], [300, 40], hq=4, hkv=2, d=64, gran=32, layers=1)
    from test_gpu_attention import call, place, workspace
    dev, out = place(d), torch.zeros(d.q.shape, dtype=torch.bfloat16, device="cuda")
    for k in ("offs", "lengths", "table"):
        dev[k] = dev[k].view(torch.uint32)
    dev["blocks"] = dev["blocks"].view(torch.float8_e4m3fn)
    call(lib, d, dev, out, workspace(lib, d), 0.125)
    torch.cuda.synchronize()
    assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), run(lib, d, 0.125))
