"""attention_tree_ragged_paged on bf16 caches with up to 32 rows per sequence and key/value head on the
average: the weights enter the product with the values as two bf16 numbers, value and remainder.

Tolerance: that of test_gpu_attention.py but for its first item. A weight is off by 2^-8 of itself as one
bf16 number; what that loses is off by 2^-8 of itself as another: 2^-16 of A."""
import numpy as np
import pytest

import synth
from gpu_util import bf16v, say
from test_gpu_attention_extremes import put
from test_gpu_attention_tree import exact, run, tree_rows

pytestmark = pytest.mark.gpu


def narrow_tolerance(d, ref):
    out, spread, size = ref
    n = int((d.cache_lengths.astype(np.int64) + np.diff(d.row_offsets.astype(np.int64))).max())
    small = 2 * ((2 * d.q.shape[2] + 8) * size[..., None] + n + 16) * 2.0**-23
    return 2.0**-8 * np.abs(out) * (1 + 2.0**-7) + spread * (2.0**-16 + small)


@pytest.mark.parametrize("dim", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("new", [[2, 3, 1, 4, 2], [5, 7, 6, 1, 8], [8] * 5], ids=["up to 16", "up to 32", "32"])
@pytest.mark.parametrize("cut", [False, True])
def test_weights_keep_their_remainders(lib, gpu, dim, page, new, cut):
    d = synth.attention_inputs(70, new, [900 if cut else 9, 0, 5, 30, 2], hq=8, hkv=2, d=dim, page=page)
    assert len(d.q) * 4 <= 32 * len(new)
    mask, scale = tree_rows(d, 1, 3), 1.0 / dim   # small scores: what fp32 loses in them is nothing beside 2^-8
    ref = exact(d, mask, scale)
    say(f"[tree weights] head {dim} page {page} new {new} lengths {d.cache_lengths.tolist()}")
    got = bf16v(run(lib, d, mask, scale))
    over = np.abs(got - ref[0]) > narrow_tolerance(d, ref)
    assert not over.any(), f"{int(over.sum())} of {over.size} elements off by more than two bf16 numbers allow"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16])
def test_so_does_the_pass_for_values_that_are_not_finite(lib, gpu, dim, page):
    """Rows that do not see a NaN keep every bit where others of their tile do."""
    d = synth.attention_inputs(71, [8, 6], [40, 3], hq=8, hkv=2, d=dim, page=page)
    mask = tree_rows(d, 1, 4)
    sees = (mask[:, 0] >> np.uint32(3) & 1).astype(bool)
    sees[8:] = False
    clean = run(lib, d, mask, 0.125)
    put(d, 1, 43, float("nan"))
    got = run(lib, d, mask, 0.125)
    assert sees.any() and np.isnan(bf16v(got)[sees]).any() and np.array_equal(got[~sees], clean[~sees])
