"""CPU checks of the paged-cache entry points at the limits of their arguments: what cannot be
served is refused before the GPU is touched. No call here reaches a kernel launch."""
import math

import pytest
import torch

import grouped_gemm_qgemm_amd as q
from grouped_gemm_qgemm_amd import QG
from test_abi import Buf
from test_abi_paged import attn_call, kv_of, lib, ref


def test_a_scale_whose_base_2_form_is_infinite_is_refused(lib):
    bb = Buf()
    assert attn_call(lib, bb, scale=3.0e38) == QG.ERR_INVALID_ARG
    assert attn_call(lib, bb, scale=2.0**128 / 1.4426950408889634 * (1 + 1e-6)) == QG.ERR_INVALID_ARG
    assert attn_call(lib, bb, scale=2.0**127, out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK
    assert attn_call(lib, bb, scale=math.ldexp(1.0, -149), out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK


WIDE = (2**31, 2**32, 2**32 + 5, -2**31 - 1, -2**32)


def test_whole_numbers_that_do_not_fit_are_refused_not_cut(monkeypatch):
    """A window of 2^32 is not one of 0, a page of 2^32 + 16 slots not one of 16, layer 2^32 not
    layer 0: the binding refuses them before the library is called."""
    def reached(*a, **k):
        raise AssertionError("the library was called")

    class Library:
        def __getattr__(self, name):
            return reached
    monkeypatch.setattr(q, "load", lambda: Library())
    monkeypatch.setattr(q, "_device_of", lambda tensors: None)
    monkeypatch.setattr(q, "_launch", reached)
    monkeypatch.setattr(q, "_stream", lambda stream: None)
    t = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(1, 2, 1, 16, 1, 64, dtype=torch.bfloat16)

    def attention(layer=0, window=0):
        q.attention_ragged_paged(x, x, t[:2], blocks, t[:1], t[:1].view(1, 1), layer, 1.0, torch.zeros(4), window=window)

    def tables(page):
        q.tables_ragged_paged(torch.zeros(5, dtype=torch.int32), None, torch.zeros(4, 2, dtype=torch.int32),
                              torch.zeros(2, dtype=torch.int32), t, t, t, t[:1], page)

    def project(fn, layer):
        fn(x[0], t[:2], x[0], x[0], x[0], blocks, t[:1], t[:1].view(1, 1), layer)

    for v in WIDE:
        for call in (lambda: attention(window=v), lambda: tables(v)):
            with pytest.raises(ValueError):
                call()
    for v in (2**32, 2**32 + 1, -2**32):
        for call in (lambda: attention(layer=v), lambda: project(q.k_matmul_ragged_paged_scale, v),
                     lambda: project(q.kv_matmul_ragged_paged_scale, v)):
            with pytest.raises(ValueError):
                call()
    for call in (attention, lambda: tables(16), lambda: project(q.k_matmul_ragged_paged_scale, 0), lambda: attention(layer=-1)):
        with pytest.raises(AssertionError):
            call()


def test_more_workgroups_than_a_launch_takes_are_refused(lib):
    """A launch has less than 2^32 threads. 2^20 sequences on 16 heads with 33 rows each on average
    may need more than 2^24 workgroups of 256; one token on 2^22 heads 2^25."""
    bb = Buf()

    def call(T, B, heads, dim, max_pages):
        t = [bb.t((1, 1, dim), QG.BF16), bb.t((1, 1, dim), QG.BF16), bb.t((1,), QG.U32), bb.t((1,), QG.F32)]
        for x in t[:2]:   # (only looked at, not allocated)
            x.shape[0], x.shape[1] = T, heads
        t[2].shape[0] = B + 1
        t[3].shape[0] = 1 << 45
        kv = kv_of(bb, Hkv=1, D=dim, gran=0, maxp=max_pages)
        kv.blocks.shape[4] = heads
        return lib.attention_ragged_paged(ref(t[0]), ref(t[1]), ref(t[2]), ref(kv), 0, 0.125, 1, 0, ref(t[3]), None)

    assert call(33 << 20, 1 << 20, 16, 64, 64) == QG.ERR_UNSUPPORTED
    assert call(1, 1, 1 << 22, 8, 64) == QG.ERR_UNSUPPORTED
