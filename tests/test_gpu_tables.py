"""tables_ragged_paged on the GPU: whole numbers, equal to the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev32, say

pytestmark = pytest.mark.gpu


def case(seed, new, cached, page, slack=5, spare=3, spare_slots=7):
    """Distinct page ids in the sequences' own entries and on the free stack."""
    rng = np.random.default_rng(seed)
    new, cached = np.asarray(new, np.int64), np.asarray(cached, np.int64)
    held, need = -(-cached // page), -(-(cached + new) // page)
    fresh = int(np.where(new > 0, need - held, 0).sum())
    ids = rng.permutation(int(held.sum()) + fresh + slack).astype(np.uint32)
    table = np.full((len(new), int(max(need.max(initial=0), held.max(initial=0))) + spare), 0xABABABAB, np.uint32)
    at = 0
    for b in range(len(new)):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return dict(table=table, cached=cached.astype(np.uint32), new=new.astype(np.uint32), free=ids[at:],
                count=len(ids) - at, page=page, slots=int(new.sum()) + spare_slots)


def run(lib, c, stream=None, with_slots=True):
    dev = dict(offsets=dev32(np.full(len(c["new"]) + 1, -7, np.int32)),
               slots=dev32(np.full(c["slots"], -9, np.int32)) if with_slots else None,
               table=dev32(c["table"]), result=dev32(np.full(2, -3, np.int32)), cached=dev32(c["cached"]),
               fresh=dev32(c["new"]), free=dev32(c["free"]), count=dev32(np.array([c["count"]], np.int32)))
    torch.cuda.synchronize()
    lib.tables_ragged_paged(*dev.values(), c["page"], stream=stream)
    torch.cuda.synchronize()
    return dev


def host(t):
    return t.cpu().numpy().view(np.uint32)


def check(c, dev):
    offs, table, slots, result = oracle.tables_ragged_paged(c["table"], c["cached"], c["new"], c["free"], c["count"],
                                                            c["page"], c["slots"] if dev["slots"] is not None else None)
    assert tuple(host(dev["result"]).tolist()) == result
    if result[1]:
        assert (dev["offsets"].cpu() == -7).all() and np.array_equal(host(dev["table"]), c["table"])
        assert dev["slots"] is None or (dev["slots"].cpu() == -9).all()
        return
    assert np.array_equal(host(dev["offsets"]), offs)
    assert np.array_equal(host(dev["table"]), table)
    if dev["slots"] is not None:
        got = dev["slots"].cpu().numpy()
        assert np.array_equal(got[:len(slots)], slots)
        assert (got[len(slots):] == -9).all()


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 1000, 1024, 1025, 8192])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_matches_the_oracle(lib, gpu, batch, page):
    rng = np.random.default_rng(batch * 100 + page)
    new = rng.integers(0, 9, batch) * rng.integers(0, 2, batch)
    new[-1] = 3
    c = case(1, new, rng.integers(0, 70, batch), page)
    say(f"[tables] batch {batch} page {page} tokens {new.sum()}")
    check(c, run(lib, c))


@pytest.mark.parametrize("new,cached,page", [([1], [0], 128), ([0], [5], 16), ([0, 0, 0], [0, 3, 9], 4), ([5000], [77], 16),
                                              ([0, 300, 0, 1, 0], [9, 0, 0, 31, 2], 32), ([9000, 1], [0, 4], 128)])
def test_lengths(lib, gpu, new, cached, page):
    c = case(2, new, cached, page)
    check(c, run(lib, c))
    check(c, run(lib, c, with_slots=False))


def test_many_tokens_use_many_workgroups(lib, gpu):
    rng = np.random.default_rng(3)
    c = case(3, rng.integers(0, 2000, 300), rng.integers(0, 5000, 300), 16)
    check(c, run(lib, c))


def test_what_cannot_be_built_is_refused_whole(lib, gpu):
    c = case(4, [5, 0, 40], [3, 9, 30], 16, slack=0)
    for over, status in (({"count": c["count"] - 1}, 1), ({"count": len(c["free"]) + 1}, 1), ({"slots": 44}, 4),
                         ({"table": c["table"][:, :4].copy()}, 2), ({"count": 0, "slots": 0}, 5)):
        x = {**c, **over}
        dev = run(lib, x)
        assert host(dev["result"])[1] == status
        check(x, dev)
    # lengths whose sum passes 32 bits
    x = {**c, "new": np.array([0xFFFFFFFF, 1, 0xFFFFFFFF], np.uint32)}
    dev = run(lib, x)
    assert host(dev["result"]).tolist() == [c["count"], 7]
    # a sequence without new tokens may have any length
    x = {**c, "cached": np.array([3, 0xFFFFFFF0, 30], np.uint32)}
    check(x, run(lib, x))


def test_an_empty_stack_suffices_where_no_page_is_needed(lib, gpu):
    c = case(5, [1, 1], [3, 14], 16, slack=0)
    c["free"], c["count"] = np.zeros(0, np.uint32), 0
    check(c, run(lib, c))


def test_other_stream_and_replays(lib, gpu):
    """A captured step whose count goes back and forth between two buffers: every replay is
    the step after the one before."""
    rng = np.random.default_rng(6)
    s = torch.cuda.Stream()
    c = case(6, rng.integers(1, 4, 40), rng.integers(0, 50, 40), 4, slack=600, spare=40)
    with torch.cuda.stream(s):
        check(c, run(lib, c))
    dev = run(lib, c)
    pair = [dev32(np.array([c["count"], 0], np.int32)), dev32(np.zeros(2, np.int32))]

    def step(a, b):
        lib.tables_ragged_paged(dev["offsets"], dev["slots"], dev["table"], b, dev["cached"], dev["fresh"], dev["free"],
                                a[:1], c["page"])
        dev["cached"].add_(dev["fresh"])

    dev["table"].copy_(dev32(c["table"]))
    dev["cached"].copy_(dev32(c["cached"]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(pair[0], pair[1])
        step(pair[1], pair[0])
    table, cached, count = c["table"], c["cached"].astype(np.int64), c["count"]
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        for _ in range(2):
            offs, table, slots, (count, status) = oracle.tables_ragged_paged(table, cached, c["new"], c["free"], count,
                                                                             c["page"], c["slots"])
            assert status == 0
            cached = cached + c["new"]
        assert np.array_equal(host(dev["table"]), table)
        assert np.array_equal(dev["slots"].cpu().numpy()[:len(slots)], slots)
        assert host(pair[0]).tolist() == [count, 0]
        _ = (torch.ones(1000, device="cuda") * 2).sum().item()   # the program's own work in between


def test_a_captured_step_that_no_longer_fits_leaves_the_tables(lib, gpu):
    """Replayed until the stack is empty: from there on every replay says so and writes nothing else."""
    c = case(7, [5, 3], [0, 9], 4, slack=4, spare=40)
    dev = run(lib, c)
    pair = [dev32(np.array([c["count"], 0], np.int32)), dev32(np.zeros(2, np.int32))]
    dev["table"].copy_(dev32(c["table"]))
    dev["cached"].copy_(dev32(c["cached"]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.tables_ragged_paged(dev["offsets"], dev["slots"], dev["table"], pair[1], dev["cached"], dev["fresh"], dev["free"],
                                pair[0][:1], c["page"])
        pair[0].copy_(pair[1])
        dev["cached"].add_(dev["fresh"])
    table, cached, count, kept = c["table"], c["cached"].astype(np.int64), c["count"], None
    for turn in range(8):
        g.replay()
        torch.cuda.synchronize()
        offs, built, slots, (count, status) = oracle.tables_ragged_paged(table, cached, c["new"], c["free"], count, c["page"],
                                                                         c["slots"])
        cached = cached + c["new"]
        assert host(pair[0]).tolist() == [count, status]
        if status == 0:
            table, kept = built, (offs, slots)
        assert np.array_equal(host(dev["table"]), table)
        assert np.array_equal(host(dev["offsets"]), kept[0]) and np.array_equal(dev["slots"].cpu().numpy()[:len(kept[1])], kept[1])
    assert status == 1 and turn == 7
