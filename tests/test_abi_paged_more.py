"""CPU checks of rope_ragged_paged, kv_read_ragged_paged, kv_keep_ragged_paged,
release_ragged_paged and attention_tree_ragged_paged: refusals before the GPU is touched. No call
here reaches a kernel launch."""
import ctypes
import math

import pytest
import torch

import grouped_gemm_qgemm_amd as q
from grouped_gemm_qgemm_amd import QG
from test_abi import Buf
from test_abi_paged import kv_of, lib, ref
from test_abi_paged_limits import WIDE

RELEASE = ("free", "result", "table", "held", "kept", "count")


def release(lib, bb, B=4, W=8, F=20, page_size=16, **over):
    a = dict(free=bb.t((F,), QG.U32), result=bb.t((2,), QG.U32), table=bb.t((B, W), QG.U32), held=bb.t((B,), QG.U32),
             kept=bb.t((B,), QG.U32), count=bb.t((1,), QG.U32))
    a.update(over)
    return lib.release_ragged_paged(*[ref(a[k]) for k in RELEASE], page_size, None)


def test_release_rejections(lib):
    bb = Buf()
    for k in RELEASE:
        assert release(lib, bb, **{k: None}) == QG.ERR_NULL, k
        assert release(lib, bb, **{k: bb.t((4, 4, 4), QG.U32)}) == QG.ERR_RANK, k
        shape = {"free": (20,), "result": (2,), "table": (4, 8), "count": (1,)}.get(k, (4,))
        assert release(lib, bb, **{k: bb.t(shape, QG.I32)}) == QG.ERR_DTYPE, k
        assert release(lib, bb, **{k: bb.t(shape, QG.U32, misalign=True)}) == QG.ERR_ALIGN, k
        if k != "free":
            assert release(lib, bb, **{k: bb.t(tuple(s + 1 if i == 0 else s for i, s in enumerate(shape)), QG.U32)}) == QG.ERR_SHAPE, k
    assert release(lib, bb, page_size=0) == QG.ERR_INVALID_ARG
    assert release(lib, bb, page_size=-4) == QG.ERR_INVALID_ARG
    assert release(lib, bb, page_size=2**31 - 1) == QG.ERR_UNSUPPORTED
    assert release(lib, bb, B=8193) == QG.ERR_UNSUPPORTED
    assert release(lib, bb, B=0) == QG.OK


ROPE = ("q_out", "q", "k", "v", "strides", "offs", "kv", "freq", "pos")


def rope(lib, bb, T=3, Hq=4, Hkv=2, D=64, R=64, B=2, layer=0, interleaved=0, amplitude=1.0, **over):
    a = dict(q_out=bb.t((T, Hq, D), QG.BF16), q=bb.t((T, Hq, D), QG.BF16), k=bb.t((T, Hkv, D), QG.BF16),
             v=bb.t((T, Hkv, D), QG.BF16), strides=None, offs=bb.t((B + 1,), QG.U32), kv=kv_of(bb, Hkv=Hkv, D=D, gran=32 if D % 32 == 0 else 0),
             freq=bb.t((R // 2,), QG.F32), pos=bb.t((T,), QG.I32))
    a.update(over)
    strides = (ctypes.c_int64 * 3)(*a["strides"]) if a["strides"] else None
    args = [strides if k == "strides" else ref(a[k]) for k in ROPE]
    return lib.rope_ragged_paged(*args[:7], layer, *args[7:], interleaved, amplitude, None)


def test_rope_rejections(lib):
    bb = Buf()

    def call(**over):
        return rope(lib, bb, **over)

    for k in ("q_out", "q", "k", "v", "offs", "kv", "freq"):   # queries, or keys and values, go together
        assert call(**{k: None}) == QG.ERR_NULL, k
    assert call(q=None, q_out=None, k=None, v=None) == QG.ERR_NULL
    shapes = {"q_out": (3, 4, 64), "q": (3, 4, 64), "k": (3, 2, 64), "v": (3, 2, 64)}
    for k, shape in shapes.items():
        assert call(**{k: bb.t((3, 128), QG.BF16)}) == QG.ERR_RANK, k
        assert call(**{k: bb.t(shape, QG.F32)}) == QG.ERR_DTYPE, k
        assert call(**{k: bb.t(shape, QG.F16)}) == QG.ERR_DTYPE, k
        assert call(**{k: bb.t(shape, QG.BF16, misalign=True)}) == QG.ERR_ALIGN, k
        for i in range(3):
            other = tuple(s + 8 if j == i else s for j, s in enumerate(shape))
            if (k, i) != ("q", 0):   # (T is q's)
                assert call(**{k: bb.t(other, QG.BF16)}) == QG.ERR_SHAPE, (k, i)
    assert call(offs=bb.t((0,), QG.U32)) == QG.ERR_SHAPE
    assert call(offs=bb.t((3,), QG.F32)) == QG.ERR_DTYPE
    assert call(freq=bb.t((32,), QG.BF16)) == QG.ERR_DTYPE
    assert call(freq=bb.t((33,), QG.F32)) == QG.ERR_SHAPE
    assert call(freq=bb.t((4, 8), QG.F32)) == QG.ERR_RANK
    assert call(pos=bb.t((3,), QG.U32)) == QG.ERR_DTYPE
    assert call(pos=bb.t((4,), QG.I32)) == QG.ERR_SHAPE
    assert call(layer=2) == QG.ERR_INVALID_ARG
    for a in (math.inf, math.nan):
        assert call(amplitude=a) == QG.ERR_INVALID_ARG
    assert call(strides=(255, 128, 128)) == QG.ERR_SHAPE
    assert call(strides=(256, 120, 128)) == QG.ERR_SHAPE
    assert call(strides=(256, 128, 0)) == QG.ERR_SHAPE
    assert call(strides=(260, 128, 128)) == QG.ERR_ALIGN
    assert call(strides=(512, 512, 516)) == QG.ERR_ALIGN
    assert call(D=60, R=0) == QG.ERR_ALIGN
    assert call(D=1032, R=0) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, planes=1)) == QG.ERR_SHAPE
    assert call(kv=kv_of(bb, maxp=0)) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, P=0)) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, lengths=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, pages=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, maxp=2**31)) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, fp8=True, gran=16)) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, fp8=True, scales=bb.t((2, 2, 4, 16, 2, 1), QG.F32))) == QG.ERR_SHAPE


def big(bb, shape, dtype):
    """A descriptor of a tensor whose memory is not touched."""
    t = bb.t((1,), dtype)
    t.rank = len(shape)
    for i, s in enumerate(shape):
        t.shape[i] = s
    return t


def test_more_tokens_than_a_launch_has_threads_for_are_refused(lib):
    bb = Buf()
    T = 2**25 + 1
    assert rope(lib, bb, T=1, q_out=big(bb, (T, 4, 64), QG.BF16), q=big(bb, (T, 4, 64), QG.BF16), k=big(bb, (T, 2, 64), QG.BF16),
                v=big(bb, (T, 2, 64), QG.BF16), pos=big(bb, (T,), QG.I32)) == QG.ERR_UNSUPPORTED
    assert read(lib, bb, k=big(bb, (T, 2, 64), QG.BF16), v=None) == QG.ERR_UNSUPPORTED
    B = 2**23 + 1
    assert keep(lib, bb, path=big(bb, (B, 1), QG.I32), kept=big(bb, (B,), QG.U32)) == QG.ERR_UNSUPPORTED


def test_rope_empty_problems_are_noops(lib):
    bb = Buf()
    assert rope(lib, bb, T=0) == QG.OK
    assert rope(lib, bb, B=0) == QG.OK
    assert rope(lib, bb, Hq=0, q_out=bb.t((3, 0, 64), QG.BF16), q=bb.t((3, 0, 64), QG.BF16), k=None, v=None) == QG.OK


def read(lib, bb, T=5, Hkv=2, D=64, B=2, layer=0, **over):
    a = dict(k=bb.t((T, Hkv, D), QG.BF16), v=bb.t((T, Hkv, D), QG.BF16), offs=bb.t((B + 1,), QG.U32), first=bb.t((B,), QG.U32),
             kv=kv_of(bb, Hkv=Hkv, D=D, lengths=0))
    a.update(over)
    return lib.kv_read_ragged_paged(*[ref(a[k]) for k in ("k", "v", "offs", "first", "kv")], layer, None)


def test_read_rejections(lib):
    bb = Buf()

    def call(**over):
        return read(lib, bb, **over)

    assert call(k=None, v=None) == QG.ERR_NULL
    assert call(offs=None) == QG.ERR_NULL
    assert call(kv=None) == QG.ERR_NULL
    for k in ("k", "v"):
        assert call(**{k: bb.t((5, 128), QG.BF16)}) == QG.ERR_RANK
        assert call(**{k: bb.t((5, 2, 64), QG.F16)}) == QG.ERR_DTYPE
        assert call(**{k: bb.t((5, 2, 64), QG.F32)}) == QG.ERR_DTYPE          # one type for both
        assert call(**{k: bb.t((5, 2, 64), QG.BF16, misalign=True)}) == QG.ERR_ALIGN
        assert call(**{k: bb.t((5, 3, 64), QG.BF16)}) == QG.ERR_SHAPE
        assert call(**{k: bb.t((5, 2, 72), QG.BF16)}) == QG.ERR_SHAPE
    assert call(v=bb.t((6, 2, 64), QG.BF16)) == QG.ERR_SHAPE
    assert call(offs=bb.t((0,), QG.U32)) == QG.ERR_SHAPE
    assert call(offs=bb.t((3,), QG.I32)) == QG.ERR_DTYPE
    assert call(first=bb.t((3,), QG.U32)) == QG.ERR_SHAPE
    assert call(first=bb.t((2,), QG.I32)) == QG.ERR_DTYPE
    assert call(layer=2) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, pages=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, maxp=0)) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, fp8=True, gran=128)) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, planes=3)) == QG.ERR_SHAPE
    assert call(D=60, kv=kv_of(bb, D=60, gran=0)) == QG.ERR_ALIGN
    assert call(T=0) == QG.OK
    assert call(B=0) == QG.OK


def keep(lib, bb, B=2, M=4, **over):
    a = dict(path=bb.t((B, M), QG.I32), kept=bb.t((B,), QG.U32), kv=kv_of(bb))
    a.update(over)
    return lib.kv_keep_ragged_paged(*[ref(a[k]) for k in ("path", "kept", "kv")], None)


def test_keep_rejections(lib):
    bb = Buf()

    def call(**over):
        return keep(lib, bb, **over)

    for k in ("path", "kept", "kv"):
        assert call(**{k: None}) == QG.ERR_NULL
    assert call(path=bb.t((8,), QG.I32)) == QG.ERR_RANK
    assert call(path=bb.t((2, 4), QG.U32)) == QG.ERR_DTYPE
    assert call(path=bb.t((3, 4), QG.I32)) == QG.ERR_SHAPE
    assert call(path=bb.t((2, 4), QG.I32, misalign=True)) == QG.ERR_ALIGN
    assert call(kept=bb.t((2,), QG.I32)) == QG.ERR_DTYPE
    assert call(kv=kv_of(bb, lengths=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, pages=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, S=0)) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, planes=1)) == QG.ERR_SHAPE
    assert call(kv=kv_of(bb, maxp=2**31)) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, fp8=True, gran=48)) == QG.ERR_UNSUPPORTED
    assert call(B=0) == QG.OK
    assert call(M=0) == QG.OK
    assert call(kv=kv_of(bb, L=0)) == QG.OK


def tree(lib, bb, T=3, W=1, mask=None, out=(3, 4, 64), q_=(3, 4, 64), offs=(3,), kv=None, layer=0, scale=0.125, window=0, none=None):
    ws = bb.t((8,), QG.F32)
    ws.shape[0] = 1 << 40   # the size is checked, the memory is not touched
    t = {"out": bb.t(out, QG.BF16), "q": bb.t(q_, QG.BF16), "offs": bb.t(offs, QG.U32),
         "mask": mask if mask is not None else bb.t((T, W), QG.U32), "kv": kv if kv is not None else kv_of(bb), "ws": ws}
    if none:
        t[none] = None
    return lib.attention_tree_ragged_paged(*[ref(t[k]) for k in ("out", "q", "offs", "mask", "kv")], layer, scale, window,
                                           ref(t["ws"]), None)


def test_tree_rejections(lib):
    bb = Buf()

    def call(**over):
        return tree(lib, bb, **over)

    for n in ("out", "q", "offs", "mask", "kv", "ws"):
        assert call(none=n) == QG.ERR_NULL, n
    assert call(mask=bb.t((3,), QG.U32)) == QG.ERR_RANK
    assert call(mask=bb.t((3, 1), QG.I32)) == QG.ERR_DTYPE
    assert call(mask=bb.t((4, 1), QG.U32)) == QG.ERR_SHAPE
    assert call(mask=bb.t((3, 0), QG.U32)) == QG.ERR_SHAPE
    assert call(mask=bb.t((3, 1), QG.U32, misalign=True)) == QG.ERR_ALIGN
    assert call(mask=big(bb, (3, 2**24 + 1), QG.U32)) == QG.ERR_UNSUPPORTED
    assert call(out=(3, 3, 64), q_=(3, 3, 64)) == QG.ERR_SHAPE
    assert call(out=(3, 4, 264), q_=(3, 4, 264), kv=kv_of(bb, D=264, gran=0)) == QG.ERR_UNSUPPORTED
    assert call(layer=2) == QG.ERR_INVALID_ARG
    for s in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert call(scale=s) == QG.ERR_INVALID_ARG, s
    assert call(window=-1) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, pages=0)) == QG.ERR_NULL
    assert call(T=0, out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK
    assert call(offs=(1,)) == QG.OK


def test_whole_numbers_that_do_not_fit_are_refused_not_cut(monkeypatch):
    def reached(*a, **k):
        raise AssertionError("the library was called")

    class Library:
        def __getattr__(self, name):
            return reached
    monkeypatch.setattr(q, "load", lambda: Library())
    monkeypatch.setattr(q, "_device_of", lambda tensors: None)
    monkeypatch.setattr(q, "_launch", reached)
    t = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(1, 2, 1, 16, 1, 64, dtype=torch.bfloat16)
    f = torch.zeros(32)
    for v in WIDE:
        with pytest.raises(ValueError):
            q.release_ragged_paged(t, t[:2], t.view(4, 1), t, t, t[:1], v)
        if v != 2**31:
            with pytest.raises(ValueError):
                q.rope_ragged_paged(x, x, x, x, t[:2], blocks, t[:1], t[:1].view(1, 1), v, f)
            with pytest.raises(ValueError):
                q.kv_read_ragged_paged(x, x, t[:2], None, blocks, t[:1].view(1, 1), v)
            with pytest.raises(ValueError):
                q.attention_tree_ragged_paged(x, x, t[:2], t[:1].view(1, 1), blocks, t[:1], t[:1].view(1, 1), v, 1.0, f)
        with pytest.raises(ValueError):
            q.attention_tree_ragged_paged(x, x, t[:2], t[:1].view(1, 1), blocks, t[:1], t[:1].view(1, 1), 0, 1.0, f, window=v)


def test_binding_refuses_what_a_descriptor_cannot_say():
    t = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (x.transpose(0, 1), x[:, ::2], x[:, :, ::2]):
        with pytest.raises(ValueError):
            q._rows_record(bad)
    assert q._rows_record(torch.zeros(3, 6, 64)[:, 1:3])[1] == 6 * 64
    assert q._rows_record(torch.zeros(1, 6, 64)[:, 1:3])[1] == 2 * 64
    assert q._rows_record(torch.zeros(1, 2, 64).expand(3, 2, 64))[1] == 0      # which the library refuses
    blocks = torch.zeros(1, 2, 1, 16, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):     # host tensors
        q.rope_ragged_paged(x, x, x, x, t[:2], blocks, t[:1], t[:1].view(1, 1), 0, torch.zeros(32))
    with pytest.raises(ValueError):     # the table of two sequences for one
        q._cache_record(blocks, t[:1], t.view(2, 2), None, 0, 1)
    with pytest.raises(ValueError):
        q._cache_record(blocks, t[:2], t[:1].view(1, 1), None, 0, 1)
    with pytest.raises(ValueError):
        q._cache_record(blocks, t[:1].long(), t[:1].view(1, 1), None, 0, 1)


def test_more_rows_than_a_launch_has(lib):
    bb = Buf()

    def rows(n, shape, dtype):
        t = bb.t(shape, dtype)
        t.shape[0] = n   # the size is checked, the memory is not touched
        return t

    n = 2**24 + 1
    assert rope(lib, bb, q_out=rows(n, (1, 4, 64), QG.BF16), q=rows(n, (1, 4, 64), QG.BF16), k=rows(n, (1, 2, 64), QG.BF16),
                v=rows(n, (1, 2, 64), QG.BF16), pos=rows(n, (1,), QG.I32)) == QG.ERR_UNSUPPORTED
    assert read(lib, bb, k=rows(n, (1, 2, 64), QG.BF16), v=rows(n, (1, 2, 64), QG.BF16)) == QG.ERR_UNSUPPORTED
    n = 2**22 + 1
    assert keep(lib, bb, path=rows(n, (1, 4), QG.I32), kept=rows(n, (1,), QG.U32)) == QG.ERR_UNSUPPORTED


def test_outputs_over_inputs_are_refused(lib):
    """A program that turns its queries in place, or has a step's result overwrite the count it reads."""
    bb = Buf()

    def rows(t, first, shape):
        """[T, H, D] from element `first` of the buffer of t on."""
        r = bb.t((1,), QG.BF16)
        r.data, r.rank = t.data + 2 * first, 3
        for i, s in enumerate(shape):
            r.shape[i] = s
        return r

    fused = bb.t((5 * 8 * 64,), QG.BF16)
    q, k, v = rows(fused, 0, (3, 4, 64)), rows(fused, 4 * 64, (3, 2, 64)), rows(fused, 6 * 64, (3, 2, 64))
    no = QG.ERR_INVALID_ARG
    parts = dict(q=q, k=k, v=v, strides=(512, 512, 512))
    assert rope(lib, bb, q_out=q, **parts) == no
    assert rope(lib, bb, q_out=rows(fused, 512 * 3 - 64 - 8, (3, 4, 64)), **parts) == no   # v's last row
    q = bb.t((3, 4, 64), QG.BF16)
    assert rope(lib, bb, q=q, q_out=q) == no
    assert rope(lib, bb, q=q, q_out=q, k=None, v=None) == no
    assert rope(lib, bb, q_out=rows(fused, 0, (3, 4, 64)), k=rows(fused, 3 * 256 - 8, (3, 2, 64))) == no
    result = bb.t((2,), QG.U32)
    count = bb.t((1,), QG.U32)
    count.data = result.data
    assert release(lib, bb, result=result, count=count) == no
