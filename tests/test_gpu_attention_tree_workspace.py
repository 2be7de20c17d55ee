"""attention_tree_ragged_paged with a workspace that holds what another call left there: records and parts of
other tiles, of another kernel's sizes. The bits are those of a call with a workspace of its own, which starts
as NaN."""
import itertools

import pytest
import torch

import synth
from gpu_util import Guarded, dev32, host16, say
from test_gpu_attention import place, workspace
from test_gpu_attention_extremes import cus
from test_gpu_attention_tree import call, run, tree_rows

pytestmark = pytest.mark.gpu

# new tokens, history, query heads, key/value heads, head dim, run of a scale; all with tiles that are cut
CALLS = {
    "16 rows": ([4, 2, 1], [3000, 3, 60], 4, 2, 64, 0),
    "32 rows, e4m3": ([6] * 40, [3000] + [5 + 2 * i for i in range(39)], 8, 2, 128, 64),
    "32 rows, bf16": ([6] * 8, [3000] + [5 + 2 * i for i in range(7)], 8, 2, 64, 0),
    "tiles of 128": ([30, 2, 9], [3000, 300, 60], 4, 1, 256, 0),
    "tiles of 128, e4m3": ([40, 2, 9], [3000, 300, 60], 4, 2, 64, 32),
    "tiles of 256": ([150, 0, 100], [3000, 30, 60], 8, 2, 128, 128),
}


def form(d):
    """Rows of a tile, as the launcher chooses them."""
    batch, hkv, D = len(d.cache_lengths), d.blocks.shape[4], d.q.shape[2]
    rows = len(d.q) * (d.q.shape[1] // hkv)
    if rows <= 16 * batch:
        return 16
    if d.gran and rows <= 32 * batch and (4 * batch * hkv > cus() or D > 128):
        return 32
    return 256 if rows > 128 * batch and 64 < D <= 128 and d.blocks.shape[3] % 16 == 0 else 128


def test_the_calls_are_of_every_form(lib, gpu):
    assert [form(synth.attention_inputs(1, *c[:2], hq=c[2], hkv=c[3], d=c[4], gran=c[5])) for c in CALLS.values()] == [16, 32, 128, 128, 128, 256]


@pytest.mark.parametrize("a,b", list(itertools.permutations(CALLS, 2)))
def test_what_another_call_left_does_not_matter(lib, gpu, a, b):
    say(f"[tree workspace] {a}, {b}, {a}")
    made = []
    for seed, name in ((80, a), (81, b)):
        new, hist, hq, hkv, dim, gran = CALLS[name]
        d = synth.attention_inputs(seed, new, hist, hq=hq, hkv=hkv, d=dim, gran=gran)
        made.append((d, tree_rows(d, 5, seed), dict(place(d))))
    alone = [run(lib, d, mask, 0.125) for d, mask, _ in made]
    ws = torch.full((max(workspace(lib, d).numel() for d, _, _ in made),), float("nan"), device="cuda")
    for k in (0, 1, 0, 0, 1):
        d, mask, dev = made[k]
        out = Guarded(d.q.shape, torch.bfloat16, 0x7FC1)
        call(lib, d, mask, {**dev, "mask": dev32(mask)}, out.view, ws, 0.125)
        assert (host16(out.view) == alone[k]).all() and out.bands_intact(), f"call {k} differs"
