"""release_ragged_paged on the GPU: whole numbers, equal to the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev32, say

pytestmark = pytest.mark.gpu


def case(seed, held, kept, page, below=5, above=7, spare=2):
    rng = np.random.default_rng(seed)
    held, kept = np.asarray(held, np.int64), np.asarray(kept, np.int64)
    back = int(np.maximum(-(-held // page) - -(-kept // page), 0).sum())
    wide = int((-(-held // page)).max(initial=0)) + spare
    return dict(table=rng.permutation(len(held) * wide).reshape(len(held), wide).astype(np.uint32), held=held.astype(np.uint32),
                kept=kept.astype(np.uint32), free=rng.integers(0, 1 << 30, below + back + above).astype(np.uint32), count=below, page=page)


def run(lib, c, stream=None):
    dev = dict(free=dev32(c["free"]), result=dev32(np.full(2, -3, np.int32)), table=dev32(c["table"]), held=dev32(c["held"]),
               kept=dev32(c["kept"]), count=dev32(np.array([c["count"]], np.int32)))
    torch.cuda.synchronize()
    lib.release_ragged_paged(*dev.values(), c["page"], stream=stream)
    torch.cuda.synchronize()
    return dev


def host(t):
    return t.cpu().numpy().view(np.uint32)


def check(c, dev):
    want, result = oracle.release_ragged_paged(c["free"], c["table"], c["held"], c["kept"], c["count"], c["page"])
    assert tuple(host(dev["result"]).tolist()) == result
    assert np.array_equal(host(dev["free"]), c["free"] if want is None else want)
    assert np.array_equal(host(dev["table"]), c["table"])


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 256, 257, 1000, 8192])
@pytest.mark.parametrize("page", [1, 3, 16, 128])
def test_matches_the_oracle(lib, gpu, batch, page):
    rng = np.random.default_rng(batch * 10 + page)
    held = rng.integers(0, 90, batch)
    kept = np.where(rng.random(batch) < 0.3, 0, held - rng.integers(-3, 40, batch)).clip(0)
    say(f"[release] batch {batch} page {page}")
    c = case(1, held, kept, page)
    check(c, run(lib, c))


@pytest.mark.parametrize("held,kept", [([0], [0]), ([5], [5]), ([1], [0]), ([16], [16]), ([17], [16]), ([17], [17]), ([33, 0, 5], [16, 0, 9]),
                                       ([100000, 3], [1, 3])])
def test_lengths(lib, gpu, held, kept):
    c = case(2, held, kept, 16)
    check(c, run(lib, c))
    c = case(2, held, kept, 16, below=0, above=0)
    check(c, run(lib, c))


def test_what_cannot_be_done_is_refused_whole(lib, gpu):
    c = case(3, [40, 9, 30], [3, 9, 0], 16, above=0)
    for over, status in (({"count": c["count"] + 1}, 1), ({"count": len(c["free"]) + 1}, 1), ({"count": 0xFFFFFFFF}, 1),
                         ({"table": c["table"][:, :2].copy()}, 2), ({"table": c["table"][:, :2].copy(), "count": 99}, 3)):
        x = {**c, **over}
        dev = run(lib, {**x, "count": np.uint32(x["count"]).view(np.int32)})
        assert host(dev["result"]).tolist() == [x["count"], status]
        assert np.array_equal(host(dev["free"]), c["free"])
    # lengths past 31 bits
    x = {**c, "held": np.array([0xFFFFFFFF, 0, 0x80000000], np.uint32), "kept": np.array([0, 0, 0], np.uint32), "page": 1}
    assert host(run(lib, x)["result"]).tolist() == [c["count"], 3]
    # a sequence that releases nothing may have any length
    x = {**c, "held": np.array([40, 0xFFFFFFF1, 0x80000000], np.uint32), "kept": np.array([3, 0xFFFFFFF0 + 15, 0xFFFFFFFF], np.uint32)}
    check(x, run(lib, x))


def test_it_undoes_the_tables(lib, gpu):
    """Captured: a step's tables, then its pages back. Every replay finds the stack as it was and hands
    out the same pages."""
    rng = np.random.default_rng(4)
    B, W, page = 40, 12, 4
    cached, new = rng.integers(0, 20, B), rng.integers(0, 20, B)
    held = -(-cached // page)
    ids = rng.permutation(600).astype(np.uint32)
    table_h = np.full((B, W), 0xABABABAB, np.uint32)
    at = 0
    for b in range(B):
        table_h[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free_h = ids[at:]
    table, free = dev32(table_h), dev32(free_h)
    lens, add = dev32(cached.astype(np.int32)), dev32(new.astype(np.int32))
    both = lens + add
    offs, slots = dev32(np.zeros(B + 1, np.int32)), dev32(np.zeros(int(new.sum()), np.int32))
    pair = [dev32(np.array([len(free_h), 0], np.int32)), dev32(np.zeros(2, np.int32))]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.tables_ragged_paged(offs, slots, table, pair[1], lens, add, free, pair[0][:1], page)
        lib.release_ragged_paged(free, pair[0], table, both, lens, pair[1][:1], page)
    want = oracle.tables_ragged_paged(table_h, cached, new, free_h, len(free_h), page, int(new.sum()))
    for _ in range(3):
        slots.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert host(pair[1]).tolist() == list(want[3]) and host(pair[0]).tolist() == [len(free_h), 0]
        assert np.array_equal(host(free), free_h) and np.array_equal(host(table), want[1])
        assert np.array_equal(slots.cpu().numpy(), want[2])
        _ = (torch.ones(1000, device="cuda") * 2).sum().item()


def test_another_stream(lib, gpu):
    c = case(5, [40, 9, 30], [3, 9, 0], 16)
    check(c, run(lib, c, stream=torch.cuda.Stream()))
