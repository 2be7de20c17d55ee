"""Seeded random-shape parity sweep of the paged cache's tables and attention against their
oracles: what the sweep over the products' entry points is for those. Every head layout, cache,
scale run, page, window and mask of a wide range, ragged lengths from none on."""
import numpy as np
import pytest

import synth
import test_gpu_attention as ta
import test_gpu_tables as tt
from gpu_util import say

pytestmark = pytest.mark.gpu


def spread(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.49)))))


def attention_case(lib, rng, i):
    kind = rng.random()
    batch = spread(rng, 1, 90 if kind < 0.6 else 6)
    most = spread(rng, 1, 9 if kind < 0.6 else 200)
    new = rng.integers(0, most + 1, batch)
    new[int(rng.integers(0, batch))] = most
    top = spread(rng, 1, 1200 if batch < 10 else 250)
    history = rng.integers(0, top + 1, batch)
    gran = int(rng.choice([0, 0, 32, 64, 128]))
    dim = gran * int(rng.integers(1, 256 // gran + 1)) if gran else 8 * int(rng.integers(1, 33))
    hkv = int(rng.choice([1, 1, 2, 3, 4, 8])) if dim <= 128 else int(rng.choice([1, 2]))
    group = int(rng.choice([1, 2, 3, 4, 5, 8]))
    causal = bool(rng.random() < 0.8)
    window = spread(rng, 1, 600) if causal and rng.random() < 0.35 else 0
    d = synth.attention_inputs(7000 + i, new, history, hq=hkv * group, hkv=hkv, d=dim, page=int(rng.choice([1, 2, 7, 8, 16, 32, 48, 100, 128])),
                               gran=gran, layers=int(rng.integers(1, 3)), spare_rows=int(rng.integers(0, 4)))
    ta.check(lib, d, causal=causal, window=window, what=f"random {i}")


def tables_case(lib, rng, i):
    batch, page = spread(rng, 1, 4000), int(rng.choice([1, 3, 16, 48, 100, 256]))
    new = rng.integers(0, spread(rng, 1, 200) + 1, batch) * (rng.random(batch) < rng.random())
    c = tt.case(8000 + i, new, rng.integers(0, spread(rng, 1, 3000) + 1, batch), page, slack=int(rng.integers(0, 50)),
                spare=int(rng.integers(0, 4)), spare_slots=int(rng.integers(0, 9)))
    say(f"[random {i}] tables batch {batch} page {page} tokens {int(new.sum())}")
    tt.check(c, tt.run(lib, c, with_slots=bool(rng.random() < 0.8)))


@pytest.mark.parametrize("seed", range(4))
def test_random_shapes(gpu, lib, seed):
    rng = np.random.default_rng(300 + seed)
    for j in range(30):
        i = 30 * seed + j
        if rng.random() < 0.25:
            tables_case(lib, rng, i)
        else:
            attention_case(lib, rng, i)
