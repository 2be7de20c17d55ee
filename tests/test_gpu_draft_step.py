"""Speculative decoding as a program runs it: each step builds its tables, turns queries and keys and
writes the drafted tokens into the pages, attends over their trees, moves the accepted path together,
gives back the pages it does not need and goes on from there. Against the oracles of each."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import bf16v, dev16, dev32, devf32, host16, say
from test_gpu_attention import compare
from test_gpu_rope import U, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gran", [0, 64])
@pytest.mark.parametrize("group,most", [(2, 7), (4, 40)], ids=["few rows", "many rows"])
def test_steps(lib, gpu, gran, group, most):
    rng = np.random.default_rng(1)
    B, hkv, hd, page, pages, W, layers = 3, 2, 64, 16, 60, 14, 2
    hq, words = group * hkv, -(-most // 32)
    shape = (layers, 2, pages, page, hkv, hd)
    blocks = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if gran else dev16(np.full(shape, 0xFFFF, np.uint16), torch.bfloat16)
    scales = torch.full((*shape[:5], 1), float("nan"), device="cuda") if gran else None
    how = dict(kv_scales=scales, quantization_granularity=gran)
    freq_h = (1e4 ** (-np.arange(16) / 16)).astype(np.float32)
    free_h = rng.permutation(pages).astype(np.uint32)
    table_h, count = np.full((B, W), 0xFFFFFFFF, np.uint32), pages
    table, free, freq = dev32(table_h), dev32(free_h), devf32(freq_h)
    counts = [dev32(np.array([pages, 0], np.int32)) for _ in range(3)]
    cached_h = np.zeros(B, np.int64)
    cache = lambda: (blocks.cpu().numpy() if gran else host16(blocks)), (lambda: scales.cpu().numpy() if gran else None)   # noqa: E731
    for step in range(7):
        # prompts first (as chains), then trees; a sequence that has nothing drafted; one that ends and starts anew
        if step == 4:
            held_h, cached_h = cached_h.copy(), np.array([cached_h[0], 0, cached_h[2]])
            lib.release_ragged_paged(free, counts[1], table, dev32(held_h.astype(np.int32)), dev32(cached_h.astype(np.int32)), counts[0][:1], page)
            counts[0].copy_(counts[1])
            free_h, (count, status) = oracle.release_ragged_paged(free_h, table_h, held_h, cached_h, count, page)
            assert status == 0 and counts[0].cpu().tolist() == [count, 0]
        new = [35, 3, 20] if step == 0 else [int(rng.integers(1, most)), 0 if step == 2 else most, int(rng.integers(1, most))]
        T = sum(new)
        cached, lens = dev32(cached_h.astype(np.int32)), dev32(np.array(new, np.int32))
        offs, slots = dev32(np.zeros(B + 1, np.int32)), dev32(np.zeros(T, np.int32))
        lib.tables_ragged_paged(offs, slots, table, counts[1], cached, lens, free, counts[0][:1], page)
        offs_h, table_h, slots_h, (count, status) = oracle.tables_ragged_paged(table_h, cached_h, new, free_h, count, page, T)
        assert status == 0 and counts[1].cpu().tolist() == [count, 0]
        assert np.array_equal(table.cpu().numpy().view(np.uint32), table_h) and np.array_equal(slots.cpu().numpy(), slots_h)

        parents = [[j - 1 if step == 0 or rng.random() < 0.3 else int(rng.integers(0, j)) if j else -1 for j in range(n)] for n in new]
        depth = []
        for tree in parents:
            own = []
            for p in tree:
                own.append(own[p] + 1 if p >= 0 else 0)
            depth.append(own)
        positions = np.concatenate([cached_h[b] + np.array(depth[b], np.int64) for b in range(B)]).astype(np.int32)
        mask_h = np.concatenate([oracle.tree_mask(t, max(words, 2)) for t in parents])
        rows = synth.bf16_bits(rng.standard_normal((T, hq + 2 * hkv, hd)))
        qkv = dev16(rows, torch.bfloat16)
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        turned = torch.zeros(T, hq, hd, dtype=torch.bfloat16, device="cuda")
        out, mask, where = torch.zeros_like(turned), dev32(mask_h), dev32(positions)
        ws = torch.empty(lib.attention_ragged_paged_workspace(T, B, hq, hkv, hd), device="cuda")
        for layer in range(layers):
            lib.rope_ragged_paged(turned, q, k, v, offs, blocks, cached, table, layer, freq, positions=where, **how)
            lib.attention_tree_ragged_paged(out, turned, offs, mask, blocks, cached, table, layer, hd ** -0.5, ws, **how)
        torch.cuda.synchronize()
        now, now_s = cache[0](), cache[1]()
        qx, kx, vx, pg, sl = oracle.rope_ragged_paged(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], offs_h, cached_h, table_h,
                                                      page, freq_h, positions)
        close(bf16v(host16(turned)), qx, 2.0**-8 * np.abs(qx) + 40 * U * 2, "queries")   # (|x| + |y| is below 12: 10 U of it)
        for plane, x in ((0, kx), (1, vx)):
            got = now[layers - 1, plane, pg, sl]
            got = oracle.decode_e4m3(got) * now_s[layers - 1, plane, pg, sl] if gran else bf16v(got)
            assert (np.abs(got - x) <= (2.0**-4 if gran else 2.0**-8) * np.abs(x) + 2.0**-9 * np.abs(x).max() / 4 * bool(gran) + 120 * U).all()
        d = synth.AttentionInputs(q=host16(turned), row_offsets=offs_h.astype(np.uint32), blocks=now, cache_lengths=cached_h.astype(np.uint32),
                                  page_table=table_h, layer_idx=layers - 1, scales=now_s, gran=gran)
        compare(d, host16(out), oracle.attention_tree_ragged_paged(d.q, d.row_offsets, mask_h, now, d.cache_lengths, table_h, layers - 1,
                                                                   hd ** -0.5, 0, now_s, gran), f"step {step}")

        path_h, kept_h = np.zeros((B, most + 35), np.int32), np.zeros(B, np.int64)
        for b, tree in enumerate(parents):
            at, path = (len(tree) - 1 if step == 0 else int(rng.integers(len(tree)))) if tree else -1, []
            while at >= 0:
                path.append(at)
                at = tree[at]
            path_h[b, :len(path)] = path[::-1]
            kept_h[b] = len(path)
        lib.kv_keep_ragged_paged(dev32(path_h), dev32(kept_h.astype(np.int32)), blocks, cached, table, **how)
        lib.release_ragged_paged(free, counts[2], table, cached + lens, cached + dev32(kept_h.astype(np.int32)), counts[1][:1], page)
        torch.cuda.synchronize()
        want, want_s = oracle.kv_keep_ragged_paged(path_h, kept_h, now, cached_h, table_h, now_s)
        assert np.array_equal(cache[0](), want) and (not gran or np.array_equal(cache[1](), want_s, equal_nan=True))
        free_h, (count, status) = oracle.release_ragged_paged(free_h, table_h, cached_h + np.array(new), cached_h + kept_h, count, page)
        assert status == 0 and counts[2].cpu().tolist() == [count, 0] and np.array_equal(free.cpu().numpy().view(np.uint32), free_h)
        counts[0].copy_(counts[2])
        cached_h = cached_h + kept_h
        held = [int(table_h[b, i]) for b in range(B) for i in range(-(-int(cached_h[b]) // page))]
        assert sorted(held + free_h[:count].tolist()) == list(range(pages)), "a page is lost or held twice"

        # what the kept tokens left, read back
        n = int(cached_h.sum())
        back = [torch.zeros(n, hkv, hd, device="cuda") for _ in range(2)]
        starts = np.concatenate([[0], np.cumsum(cached_h)])
        lib.kv_read_ragged_paged(*back, dev32(starts.astype(np.int32)), None, blocks, table, layers - 1, **how)
        rows_x = oracle.kv_read_ragged_paged(starts, None, want, table_h, layers - 1, want_s, gran)
        for plane in (0, 1):
            assert np.array_equal(back[plane].cpu().numpy(), rows_x[plane].astype(np.float32))
        say(f"[steps] {step} new {new} kept {kept_h.tolist()} cached {cached_h.tolist()} pages left {count}")
