"""rope_ragged_paged on the GPU against the 64-bit oracle.

Tolerances, per element of a pair (x, y) with A = |amplitude|, u = 2^-24 (an fp32 rounding is off by
at most u of the value):
  * the part of a turn is rounded to fp32 (at most 2^-26 of a turn, 1.6 u of a radian); sine and cosine
    are good to 4 u, the amplitude's product adds one u, the two products and their sum three: in
    all less than 10 u A (|x| + |y|);
  * a bf16 result is rounded once: 2^-8 of it;
  * e4m3: the run's scale is amax / 448 of values that are off by the first item, and rounded (u);
    the code is that of x / s with two more roundings, off by half a step: 2^-4 of it, or half of the
    smallest step, 2^-10. In units of x: s * max(2^-4 |x / s|, 2^-10), plus the first item and four u of
    x. A code is one of two neighbours where x / s lies that near to a middle.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import Guarded, bf16v, dev16, dev32, devf32, host16, say

pytestmark = pytest.mark.gpu
U = 2.0**-24
SENTINEL = 0x7FC1


class Case:
    def __init__(self, seed, new, cached, hq=4, hkv=2, d=64, page=16, gran=0, rot=None, layers=2, fused=True, positions=None,
                 spare=3, amplitude=1.0, interleaved=False, freq=None):
        rng = np.random.default_rng(seed)
        self.new, self.cached = np.asarray(new, np.int64), np.asarray(cached, np.int64)
        self.offs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.uint32)
        self.T = int(self.offs[-1]) + spare
        self.hq, self.hkv, self.d, self.page, self.gran, self.layers = hq, hkv, d, page, gran, layers
        rot = d if rot is None else rot
        self.freq = (1e4 ** (-np.arange(rot // 2) / max(rot // 2, 1)) if freq is None else np.asarray(freq)).astype(np.float32)
        self.interleaved, self.amplitude, self.positions, self.fused = interleaved, amplitude, positions, fused
        self.rows = synth.bf16_bits(rng.standard_normal((self.T, hq + 2 * hkv, d)))
        first, need = self.cached // page, -(-(self.cached + self.new) // page)
        held = np.maximum(need - first, 0)
        self.pages = int(held.sum()) + 2
        ids = rng.permutation(self.pages)
        self.table = np.full((len(new), max(int(need.max(initial=0)), 1) + 1), 0xFFFFFFFF, np.uint32)
        at = 0
        for b in range(len(new)):   # only pages that tokens land in; all other ids are far out of range
            self.table[b, first[b]:need[b]] = ids[at:at + held[b]]
            at += held[b]

    @property
    def q(self):
        return self.rows[:, :self.hq]

    @property
    def k(self):
        return self.rows[:, self.hq:self.hq + self.hkv]

    @property
    def v(self):
        return self.rows[:, self.hq + self.hkv:]

    def place(self):
        rows = dev16(self.rows, torch.bfloat16)
        parts = list(rows.split([self.hq, self.hkv, self.hkv], 1))
        if not self.fused:
            parts = [p.contiguous() for p in parts]
        shape = (self.layers, 2, self.pages, self.page, self.hkv, self.d)
        if self.gran:
            blocks = torch.full(shape, 0x7E, dtype=torch.uint8, device="cuda")
            scales = torch.full((*shape[:5], self.d // self.gran), -1.0, device="cuda")
        else:
            blocks, scales = torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16), None
        return dict(q=parts[0], k=parts[1], v=parts[2], blocks=blocks, scales=scales, offs=dev32(self.offs),
                    lengths=dev32(self.cached.astype(np.uint32)), table=dev32(self.table), freq=devf32(self.freq),
                    positions=None if self.positions is None else dev32(np.asarray(self.positions, np.int32)))


def call(lib, c, dev, q_out, with_q=True, with_kv=True, stream=None):
    lib.rope_ragged_paged(q_out if with_q else None, dev["q"] if with_q else None, dev["k"] if with_kv else None,
                          dev["v"] if with_kv else None, dev["offs"], dev["blocks"], dev["lengths"], dev["table"], c.layers - 1,
                          dev["freq"], positions=dev["positions"], interleaved=c.interleaved, amplitude=c.amplitude,
                          kv_scales=dev["scales"], quantization_granularity=c.gran, stream=stream)


def partner(c, bits):
    """|x| + |y| of each element's pair; |x| where nothing is turned."""
    x = np.abs(bf16v(bits))
    y, half = x.copy(), len(c.freq)
    if c.interleaved:
        y[..., 0:2 * half:2] = y[..., 1:2 * half:2] = x[..., 0:2 * half:2] + x[..., 1:2 * half:2]
    else:
        y[..., :half] = y[..., half:2 * half] = x[..., :half] + x[..., half:2 * half]
    return y


def close(got, want, tol, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN on one side only"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    err = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)), 0)
    over = err > np.where(fine, tol, 0)
    if over.any():
        i = tuple(np.argwhere(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.size} off, first at {i}: {got[i]} for {want[i]}, tolerance {tol[i]}")
    return float((err[fine] / np.maximum(tol[fine], 1e-300)).max(initial=0.0))


def verify(c, dev, q_bits, with_q=True, with_kv=True):
    """The queries' bits and the cache on the device against the oracle."""
    n = int(c.offs[-1])
    q, k, v, page, slot = oracle.rope_ragged_paged(c.q, c.k, c.v, c.offs, c.cached, c.table, c.page, c.freq, c.positions,
                                                   c.interleaved, c.amplitude)
    A = abs(float(np.float32(c.amplitude)))
    A = max(A, 1.0) if len(c.freq) * 2 < c.d else A
    used = []
    if with_q:
        assert (q_bits[n:] == SENTINEL).all(), "rows behind the last sequence changed"
        rot = 10 * U * A * partner(c, c.q[:n])
        used.append(close(bf16v(q_bits[:n]), q, 2.0**-8 * (np.abs(q) + rot) + rot + 2.0**-134, "queries"))
    layer = c.layers - 1
    blocks = dev["blocks"].cpu().numpy() if c.gran else host16(dev["blocks"])
    touched = np.zeros(blocks.shape[:4], bool)
    if with_kv:
        touched[layer][:, page, slot] = True
    assert (blocks[~touched] == (0x7E if c.gran else SENTINEL)).all(), "cache rows of no token changed"
    scales = dev["scales"].cpu().numpy() if c.gran else None
    if c.gran:
        assert (scales[~touched] == -1).all(), "scales of no token changed"
    if not with_kv:
        return used
    for plane, want, bits, what in ((0, k, c.k[:n], "keys"), (1, v, c.v[:n], "values")):
        got = blocks[layer, plane, page, slot]
        rot = 10 * U * A * partner(c, bits) if plane == 0 else np.zeros_like(want)
        if not c.gran:
            if plane == 1:
                assert np.array_equal(got, bits) or np.isnan(want).any(), "values changed"
                close(bf16v(got), want, np.zeros_like(want), what)
            else:
                used.append(close(bf16v(got), want, 2.0**-8 * (np.abs(want) + rot) + rot + 2.0**-134, what))
            continue
        runs = lambda x: x.reshape(n, c.hkv, c.d // c.gran, c.gran)   # noqa: E731
        s = scales[layer, plane, page, slot].astype(np.float64)
        amax = np.nanmax(np.abs(np.where(np.isnan(runs(want)), 0, runs(want))), -1)
        off = runs(rot).max(-1)
        used.append(close(s, amax / 448, (off * (1 + U) + U * amax) / 448 + 2.0**-149, what + "' scales"))
        codes = oracle.decode_e4m3(runs(got))
        sk = s[..., None]
        with np.errstate(invalid="ignore", divide="ignore"):
            step = np.maximum(2.0**-4 * np.abs(runs(want)), 2.0**-10 * sk)
            value = np.where(sk > 0, codes * sk, codes)
        used.append(close(value, runs(want), step + runs(rot) * (1 + 2.0**-4) + 4 * U * np.abs(runs(want)), what))
    return used


def check(lib, c, what="", **parts):
    say(f"[rope] {what} T {c.T} heads {c.hq}/{c.hkv} d {c.d} turned {2 * len(c.freq)} {'side' if c.interleaved else 'apart'} "
        f"gran {c.gran} page {c.page} cached {c.cached[:5].tolist()}")
    dev = c.place()
    out = Guarded((c.T, c.hq, c.d), torch.bfloat16, SENTINEL)
    call(lib, c, dev, out.view, **parts)
    bits = host16(out.view)
    assert out.bands_intact()
    if not parts.get("with_q", True):
        assert (bits == SENTINEL).all()
    used = verify(c, dev, bits, **parts)
    say(f"[rope]   worst elements at {['%.2f' % u for u in used]} of their tolerances")
    return dev, bits


NEW, CACHED = [3, 0, 1, 20, 2], [0, 5, 40, 61, 130]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,gran", [(8, 0), (64, 0), (72, 0), (80, 0), (128, 0), (136, 0), (256, 0), (1024, 0), (32, 32), (64, 32), (64, 64),
                                    (96, 32), (128, 32), (128, 64), (128, 128), (192, 64), (256, 128), (384, 128), (1024, 128)])
def test_head_dims(lib, gpu, d, gran, interleaved):
    check(lib, Case(1, NEW, CACHED, d=d, gran=gran, interleaved=interleaved, amplitude=1.25))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("gran", [0, 32])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 20, 30, 32, 48, 62, 94, 96])
def test_parts_of_a_head(lib, gpu, rot, gran, interleaved):
    check(lib, Case(2, NEW, CACHED, d=96, rot=rot, gran=gran, interleaved=interleaved, amplitude=0.5))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (7, 1), (40, 5), (128, 1), (3, 3)])
@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("fused", [True, False])
def test_heads(lib, gpu, hq, hkv, gran, fused):
    check(lib, Case(3, NEW, CACHED, hq=hq, hkv=hkv, gran=gran, fused=fused))


@pytest.mark.parametrize("page", [1, 3, 16, 48, 128])
@pytest.mark.parametrize("gran", [0, 64])
def test_pages(lib, gpu, page, gran):
    check(lib, Case(4, [1, 30, 0, 7], [17, 300, 3, 0], page=page, gran=gran))


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 129, 1000, 4097])
def test_many_sequences(lib, gpu, batch):
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 3, batch) * rng.integers(0, 2, batch)
    new[-1] = 2
    check(lib, Case(5, new, rng.integers(0, 100, batch), hq=2, hkv=1, d=32, gran=32))


@pytest.mark.parametrize("gran,interleaved,rot", [(0, False, 64), (0, True, 64), (32, False, 64), (32, True, 64), (32, False, 20), (0, False, 20)])
def test_many_tokens_use_workgroups_of_several(lib, gpu, gran, interleaved, rot):
    new = [1500, 0, 1, 3, 2800, 2]
    assert sum(new) >= 16 * 256
    check(lib, Case(6, new, [100, 2, 7, 0, 31, 5], hq=2, hkv=1, gran=gran, interleaved=interleaved, rot=rot, spare=2))


def test_far_positions_are_as_exact_as_near_ones(lib, gpu):
    """Up to 2^31 - 1 and below 0, with frequencies of 24 bits near one."""
    pos = [0, 1, 2**31 - 1, 2**31 - 2, -(2**31), -5, 2**24 + 1, 10**9 + 7, 999983, 123456789]
    freq = 1 - np.arange(1, 33) * 2.0**-24
    for interleaved in (False, True):
        check(lib, Case(7, [10], [3], positions=pos + [1, 2, 3], interleaved=interleaved, freq=freq))


def test_positions_of_a_tree(lib, gpu):
    """Several tokens share a depth; they are written to slots of their own."""
    check(lib, Case(8, [6, 4], [50, 0], positions=[50, 51, 51, 52, 52, 53, 0, 1, 1, 1, 0, 0, 0], gran=64))


def test_queries_or_keys_alone(lib, gpu):
    for gran in (0, 64):
        c = Case(9, NEW, CACHED, gran=gran)
        check(lib, c, with_kv=False)
        check(lib, c, with_q=False)


@pytest.mark.parametrize("gran", [0, 64])
def test_zeros_infinities_and_nan(lib, gpu, gran):
    """A run of zeros has scale 0 and codes 0. A NaN makes its pair NaN and leaves the rest of its run
    alone. (What an infinity does to its run's other codes follows from the scale, an infinity.)"""
    c = Case(10, NEW, CACHED, gran=gran, rot=32)
    c.rows[0] = 0
    c.rows[1, :, :40] = 0x8000
    c.rows[5, :, 50] = 0x7FC0
    c.rows[7, :, 3] = 0x7FC0
    check(lib, c)
    if not gran:
        c.rows[9, :, 60] = 0x7F80
        c.rows[9, :, 61] = 0xFF80
        check(lib, c)
        return
    c.rows[9, c.hq:, 60] = 0x7F80
    dev = c.place()
    out = torch.zeros(c.T, c.hq, c.d, dtype=torch.bfloat16, device="cuda")
    call(lib, c, dev, out)
    p = int(c.cached[3]) + 9 - int(c.offs[3])
    page, slot = int(c.table[3, p // c.page]), p % c.page
    assert torch.isinf(dev["scales"][-1, :, page, slot]).all()
    codes = dev["blocks"][-1, :, page, slot].cpu().numpy()
    assert (codes[..., 60] & 0x7F == 0x7F).all() and (np.delete(codes, 60, -1) & 0x7F == 0).all()


@pytest.mark.parametrize("size", [2.0**-126, 2.0**-130, 2.0**-120, 2.0**120, 3e38])
def test_sizes_at_the_ends_of_the_range(lib, gpu, size):
    """Scales down to the smallest subnormal number: a code stays within 448."""
    for gran in (0, 64):
        c = Case(11, NEW, CACHED, gran=gran, rot=0)
        c.rows = synth.bf16_bits(np.clip(bf16v(c.rows), -1, 1) * size)
        dev = c.place()
        out = Guarded((c.T, c.hq, c.d), torch.bfloat16, SENTINEL)
        call(lib, c, dev, out.view)
        if not gran:
            verify(c, dev, host16(out.view))
            continue
        n = int(c.offs[-1])
        _, k, v, page, slot = oracle.rope_ragged_paged(c.q, c.k, c.v, c.offs, c.cached, c.table, c.page, c.freq)
        for plane, want in ((0, k), (1, v)):
            s = dev["scales"][-1, plane].cpu().numpy()[page, slot].astype(np.float64)
            amax = np.abs(want).reshape(n, c.hkv, 1, 64).max(-1)
            assert (np.abs(s - amax / 448) <= U * amax / 448 + 2.0**-150).all()
            codes = oracle.decode_e4m3(dev["blocks"][-1, plane].cpu().numpy()[page, slot]).reshape(n, c.hkv, 1, 64)
            assert np.isfinite(codes).all()
            x = np.divide(want.reshape(codes.shape), s[..., None], out=np.zeros(codes.shape), where=s[..., None] > 0)
            x = np.clip(x, -448, 448)
            assert (np.abs(codes - x) <= np.maximum(2.0**-4 * np.abs(x), 2.0**-10) * (1 + 4 * U)).all()


def test_what_is_read_back_is_what_the_attention_reads(lib, gpu):
    """The written cache, through kv_read_ragged_paged: codes times scales, exactly."""
    c = Case(12, NEW, CACHED, gran=32)
    dev, _ = check(lib, c)
    n = int(c.offs[-1])
    k, v = (torch.zeros(n, c.hkv, c.d, device="cuda") for _ in range(2))
    lib.kv_read_ragged_paged(k, v, dev["offs"], dev["lengths"], dev["blocks"], dev["table"], 1, kv_scales=dev["scales"],
                             quantization_granularity=32)
    _, kx, vx, page, slot = oracle.rope_ragged_paged(c.q, c.k, c.v, c.offs, c.cached, c.table, c.page, c.freq)
    for plane, t, x in ((0, k, kx), (1, v, vx)):
        codes = oracle.decode_e4m3(dev["blocks"][1, plane].cpu().numpy()[page, slot])
        want = (codes * np.repeat(dev["scales"][1, plane].cpu().numpy()[page, slot].astype(np.float64), 32, -1)).astype(np.float32)
        assert np.array_equal(t.cpu().numpy(), want)
        assert np.abs(want - x).max() < 0.07 * np.abs(x).max()


def test_stream_and_replays(lib, gpu):
    """Captured with lengths that move on between replays; each against the oracle."""
    for gran in (0, 64):
        c = Case(13, [3, 0, 1, 5], [0, 5, 40, 61], gran=gran)
        c.table = np.random.default_rng(0).permutation(64).reshape(4, 16).astype(np.uint32)
        c.pages = 64
        s = torch.cuda.Stream()
        dev = c.place()
        out = torch.full((c.T, c.hq, c.d), 0, dtype=torch.int16, device="cuda").fill_(SENTINEL).view(torch.bfloat16)
        torch.cuda.synchronize()
        call(lib, c, dev, out, stream=s)
        s.synchronize()
        verify(c, dev, host16(out))
        clean = c.place()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(lib, c, dev, out)
            dev["lengths"].add_(1)
        for _ in range(3):
            out.view(torch.int16).fill_(SENTINEL)
            dev["blocks"].copy_(clean["blocks"])
            if gran:
                dev["scales"].copy_(clean["scales"])
            g.replay()
            torch.cuda.synchronize()
            verify(c, dev, host16(out))
            c.cached = c.cached + 1
            _ = (torch.ones(1000, device="cuda") * 2).sum().item()   # the program's own work in between


def test_cache_past_32_bit_offsets(lib, gpu):
    """A plane of more than 4 GB: the page written lies behind byte 2^32 and element 2^31."""
    c = Case(14, [2, 3], [5, 0], hq=2, hkv=8, d=128, page=128, layers=1)
    used = c.pages
    pages = (5 << 30) // (128 * 8 * 128 * 2)
    dev = c.place()
    small = dev["blocks"]
    dev["blocks"] = torch.empty((1, 2, pages, 128, 8, 128), dtype=torch.bfloat16, device="cuda")
    dev["blocks"][:, :, pages - used:] = small
    table = c.table.astype(np.int64)
    table[table != 0xFFFFFFFF] += pages - used
    dev["table"] = dev32(table.astype(np.uint32))
    out = Guarded((c.T, c.hq, c.d), torch.bfloat16, SENTINEL)
    call(lib, c, dev, out.view)
    dev["blocks"] = dev["blocks"][:, :, pages - used:].contiguous()
    verify(c, dev, host16(out.view))


def test_refusals_with_device_tensors(lib, gpu):
    c = Case(15, [2], [5])
    dev = c.place()
    out = torch.zeros(c.T, c.hq, c.d, dtype=torch.bfloat16, device="cuda")
    before = host16(dev["blocks"]).copy()
    for over in ({"q": dev["q"].half()}, {"k": dev["k"][:1].expand(c.T, -1, -1)}, {"freq": dev["freq"].double()},
                 {"freq": torch.zeros(40, device="cuda")}, {"positions": dev32(np.zeros(c.T, np.int32)).long()}):
        with pytest.raises(lib.QgError):
            call(lib, c, {**dev, **over}, out)
    for over in ({"q": dev["q"].transpose(0, 1)}, {"v": dev["v"].cpu()}, {"lengths": dev["lengths"].long()}):
        with pytest.raises(ValueError):
            call(lib, c, {**dev, **over}, out)
    assert (out == 0).all() and np.array_equal(host16(dev["blocks"]), before)


@pytest.mark.parametrize("heads,d,gran", [((1, 1), 32, 0), ((1, 1), 32, 32), ((3, 1), 64, 64), ((2, 2), 256, 128), ((20, 2), 128, 0), ((44, 2), 128, 64),
                                          ((1, 1), 1024, 0), ((5, 1), 72, 0)])
@pytest.mark.parametrize("rot", [None, 0, 20])
@pytest.mark.parametrize("kind", ["short", "empty", "long"])
def test_workgroups_of_many_tokens(lib, gpu, heads, d, gran, rot, kind):
    """Few heads: a workgroup has up to 16 tokens, of as many sequences (with empty ones between), or of one."""
    rng = np.random.default_rng(9)
    if kind == "long":
        new = [9000, 0, 7001, 1]
    else:
        new = rng.integers(0, 9, 5000) if kind == "short" else np.where(rng.random(8000) < 0.3, rng.integers(1, 15, 8000), 0)
    cut = 5 if heads[0] >= 20 or d == 1024 else 1   # of a few MB of rows
    new = np.asarray(new)[::cut] if kind != "long" else [n // cut for n in new]
    check(lib, Case(10, new, rng.integers(0, 50, len(new)), hq=heads[0], hkv=heads[1], d=d, gran=gran, rot=rot, layers=1, spare=5))
