"""The projections into an e4m3 cache where a token's hidden row is NaN, and with it whole runs of keys and
values: their codes are NaN's, whose product with any scale is NaN. Other tokens are as without it."""
import numpy as np
import pytest

import oracle
from gpu_util import say
from test_gpu_kv_cache import kv_inputs, run_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("qgran", [32, 64, 128])
@pytest.mark.parametrize("hidden,nan", [("bf16", 0x7FC0), ("fp8", 0x7F)])
@pytest.mark.parametrize("lens", [(5, 17, 3), (300, 400)])
def test_hidden_rows_of_nan(lib, gpu, planes, qgran, hidden, nan, lens):
    k = kv_inputs(50, lens, planes=planes, cache="fp8", qgran=qgran, hidden=hidden)
    say(f"[kproj NaN] {hidden} hidden, planes {planes} G {qgran} tokens {lens}")
    rows = [3, 8, sum(lens) - 1]
    k.hidden[rows] = 0
    codes, scales = run_gpu(lib, k)
    k.hidden[rows] = nan
    with_nan, nan_scales = run_gpu(lib, k)
    _, page, slot = oracle.token_slots(k.row_offsets, k.cache_lengths, k.page_table, k.blocks.shape[3])
    there = np.zeros(k.blocks.shape[:4], bool)
    there[k.layer_idx, :planes, page[rows], slot[rows]] = True
    assert np.array_equal(with_nan[~there], codes[~there]) and np.array_equal(nan_scales[~there], scales[~there])
    assert not (codes[there] & 0x7F).any()
    assert (with_nan[there] & 0x7F == 0x7F).all(), "values of a NaN row are numbers"
