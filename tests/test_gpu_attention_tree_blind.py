"""attention_tree_ragged_paged: a row that sees nothing becomes zeros; one that sees positions whose scores
are all -infinity has no softmax, as in attention_ragged_paged, and becomes NaN. The oracle is the formula's;
tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest

import synth
from gpu_util import bf16v, say
from test_gpu_attention import compare
from test_gpu_attention_tree import exact, run

pytestmark = pytest.mark.gpu

# new tokens, history, query heads, key/value heads, head dim: every kernel, tiles whole and cut
CASES = {
    "few": ([4, 1, 2], [0, 3, 60], 4, 2, 64),
    "few cut": ([4, 1, 2], [2000, 3, 60], 4, 2, 64),
    "many": ([70, 3], [0, 40], 4, 2, 64),
    "many cut": ([70, 3], [2000, 40], 4, 2, 64),
    "wide": ([90, 70], [0, 40], 8, 2, 128),
    "wide cut": ([90, 70], [2000, 40], 8, 2, 128),
    "heads of 256": ([40, 1], [300, 7], 4, 1, 256),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("gran", [0, 64])
def test_scores_of_minus_infinity(lib, gpu, case, gran):
    """The keys of the first sequence's history and of its first drafted token give -infinity for queries
    that are positive in element 5, +infinity (and NaN) for the others."""
    new, hist, hq, hkv, dim = CASES[case]
    d = synth.attention_inputs(60, new, hist, hq=hq, hkv=hkv, d=dim, gran=gran)
    n, c, G = new[0], hist[0], gran
    d.q[:n, :, 5] = synth.bf16_bits(np.abs(bf16v(d.q[:n, :, 5])) + 1.0)
    d.q[1:n:4, :, 5] ^= 0x8000
    pos = np.arange(c + 1)
    page, slot = d.page_table[0, pos // 16], pos % 16
    if not gran:
        d.blocks[d.layer_idx, 0, page, slot, :, 5] = 0xFF80
    else:   # a run of -1 times an infinite scale, and queries of one sign in it
        d.blocks[d.layer_idx, 0, page, slot, :, :G] = 0xB8
        d.scales[d.layer_idx, 0, page, slot, :, 0] = np.inf
        d.q[:n, :, :G] = synth.bf16_bits(np.where(np.arange(n)[:, None, None] % 4 == 1, -1.0, 1.0) + np.zeros((n, hq, G)))
    mask = np.zeros((len(d.q), 4), np.uint32)
    r = np.arange(len(d.q))
    mask[r % 4 == 0, 0] = 1                 # the first token only
    mask[r % 4 == 1, 0] = 1
    mask[r % 4 == 2, 0] = 1 | (1 << 2)      # and one of finite scores
    say(f"[tree blind] {case} gran {gran}")
    ref = exact(d, mask, 0.125)
    got = run(lib, d, mask, 0.125)
    compare(d, got, ref)
    g = bf16v(got[:n])
    assert np.isnan(g[0::4]).all(), "a row whose scores are all -infinity"
    assert np.isnan(g[1::4]).all()
    # all weight on one token: rounded to bf16 (2^-8) where it is multiplied by a scale, and so is the result
    assert (np.abs(g[2::4] - ref[0][:n][2::4]) <= 2.0**-7 * np.abs(ref[0][:n][2::4])).all()
    assert (g[3::4] == 0).all() if c == 0 else np.isnan(g[3::4]).all()
