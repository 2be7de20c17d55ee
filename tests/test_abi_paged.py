"""CPU checks of the paged-cache entry points: refusals before the GPU is touched. No
call here reaches a kernel launch."""
import ctypes
import math

import pytest
import torch

import grouped_gemm_qgemm_amd as q
from grouped_gemm_qgemm_amd import QG, QgPagedKV
from test_abi import Buf


@pytest.fixture(scope="module")
def lib():
    return q.load()


def ref(t):
    return ctypes.byref(t) if t is not None else None


TABLES = ("offsets", "slots", "table", "result", "cached", "fresh", "free", "count")


def tables_args(bb, B=4, W=8, F=20, T=16):
    return dict(offsets=bb.t((B + 1,), QG.U32), slots=bb.t((T,), QG.I32), table=bb.t((B, W), QG.U32),
                result=bb.t((2,), QG.U32), cached=bb.t((B,), QG.U32), fresh=bb.t((B,), QG.U32),
                free=bb.t((F,), QG.U32), count=bb.t((1,), QG.U32))


def tables_call(lib, a, page_size=16):
    return lib.tables_ragged_paged(*[ref(a[k]) for k in TABLES], page_size, None)


def test_tables_rejections(lib):
    bb = Buf()

    def with_(page_size=16, **over):
        return tables_call(lib, {**tables_args(bb), **over}, page_size)

    for k in TABLES:
        if k != "slots":
            assert with_(**{k: None}) == QG.ERR_NULL, k
        assert with_(**{k: bb.t((4, 4, 4), QG.U32)}) == QG.ERR_RANK, k
        shape = {"offsets": (5,), "slots": (16,), "table": (4, 8), "result": (2,), "free": (20,), "count": (1,)}.get(k, (4,))
        assert with_(**{k: bb.t(shape, QG.F32)}) == QG.ERR_DTYPE, k
        good = QG.I32 if k == "slots" else QG.U32
        assert with_(**{k: bb.t(shape, good, misalign=True)}) == QG.ERR_ALIGN, k
        if k not in ("slots", "free"):
            assert with_(**{k: bb.t(tuple(s + 1 if i == 0 else s for i, s in enumerate(shape)), good)}) == QG.ERR_SHAPE, k
    assert with_(page_size=0) == QG.ERR_INVALID_ARG
    assert with_(page_size=-1) == QG.ERR_INVALID_ARG
    assert with_(page_size=2**31 - 1) == QG.ERR_UNSUPPORTED        # W * S past 31 bits
    B = 8193
    assert with_(offsets=bb.t((B + 1,), QG.U32), table=bb.t((B, 1), QG.U32), cached=bb.t((B,), QG.U32),
                 fresh=bb.t((B,), QG.U32)) == QG.ERR_UNSUPPORTED


def test_tables_without_sequences_is_a_noop(lib):
    assert tables_call(lib, tables_args(Buf(), B=0)) == QG.OK


def kv_of(bb, L=2, P=4, S=16, Hkv=2, D=64, fp8=False, gran=32, planes=2, lengths=1, pages=1, maxp=2, scales=None):
    kv = QgPagedKV()
    kv.blocks = bb.t((L, planes, P, S, Hkv, D), QG.FP8_E4M3 if fp8 else QG.BF16)
    kv.cache_lengths = bb.t((8,), QG.U32).data if lengths else None
    kv.page_table = bb.t((8,), QG.U32).data if pages else None
    kv.max_pages_per_seq = maxp
    kv.scales = scales if scales is not None else bb.t((L, 2, P, S, Hkv, D // gran if gran else 1), QG.F32)
    kv.quantization_granularity = gran
    return kv


def attn_call(lib, bb, out=(3, 4, 64), q_=(3, 4, 64), offs=(3,), kv=None, layer=0, scale=0.125, causal=1, window=0,
              ws=None, odt=QG.BF16, qdt=QG.BF16, mis=None, none=None):
    t = {"out": bb.t(out, odt, mis == "out"), "q": bb.t(q_, qdt, mis == "q"), "offs": bb.t(offs, QG.U32, mis == "offs"),
         "ws": ws if ws is not None else bb.t((1 << 16,), QG.F32, mis == "ws")}
    if ws is None:   # the size is checked, the memory is not touched
        t["ws"].shape[0] = 1 << 40
    kv = kv if kv is not None else kv_of(bb)
    return lib.attention_ragged_paged(None if none == "out" else ref(t["out"]), None if none == "q" else ref(t["q"]),
                                      None if none == "offs" else ref(t["offs"]), None if none == "kv" else ref(kv),
                                      layer, scale, causal, window, None if none == "ws" else ref(t["ws"]), None)


def test_attention_rejections(lib):
    bb = Buf()

    def call(**over):
        return attn_call(lib, bb, **over)

    for n in ("out", "q", "offs", "kv", "ws"):
        assert call(none=n) == QG.ERR_NULL, n
        if n != "kv":
            assert call(mis=n) == QG.ERR_ALIGN, n
    assert call(out=(3, 256)) == QG.ERR_RANK
    assert call(q_=(3, 256)) == QG.ERR_RANK
    assert call(offs=(3, 1)) == QG.ERR_RANK
    assert call(odt=QG.F16) == QG.ERR_DTYPE
    assert call(qdt=QG.F16) == QG.ERR_DTYPE
    assert call(out=(4, 4, 64)) == QG.ERR_SHAPE
    assert call(out=(3, 2, 64)) == QG.ERR_SHAPE
    assert call(out=(3, 4, 32), q_=(3, 4, 32)) == QG.ERR_SHAPE           # not the cache's head dim
    assert call(out=(3, 3, 64), q_=(3, 3, 64)) == QG.ERR_SHAPE           # 3 query heads on 2
    assert call(offs=(0,)) == QG.ERR_SHAPE
    assert call(kv=kv_of(bb, planes=1)) == QG.ERR_SHAPE
    assert call(out=(3, 4, 60), q_=(3, 4, 60), kv=kv_of(bb, D=60, gran=0)) == QG.ERR_ALIGN
    assert call(out=(3, 4, 264), q_=(3, 4, 264), kv=kv_of(bb, D=264, gran=0)) == QG.ERR_UNSUPPORTED
    assert call(layer=2) == QG.ERR_INVALID_ARG
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == QG.ERR_INVALID_ARG, s
    assert call(window=-1) == QG.ERR_INVALID_ARG
    assert call(window=5, causal=0) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, maxp=0)) == QG.ERR_INVALID_ARG
    assert call(kv=kv_of(bb, lengths=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, pages=0)) == QG.ERR_NULL
    assert call(kv=kv_of(bb, maxp=2**31)) == QG.ERR_UNSUPPORTED
    # quantized cache
    assert call(kv=kv_of(bb, fp8=True, gran=16)) == QG.ERR_UNSUPPORTED
    assert call(kv=kv_of(bb, fp8=True, gran=128)) == QG.ERR_UNSUPPORTED  # does not divide 64
    assert call(kv=kv_of(bb, fp8=True, scales=bb.t((2, 2, 4, 16, 2), QG.F32))) == QG.ERR_RANK
    assert call(kv=kv_of(bb, fp8=True, scales=bb.t((2, 2, 4, 16, 2, 2), QG.BF16))) == QG.ERR_DTYPE
    assert call(kv=kv_of(bb, fp8=True, scales=bb.t((2, 2, 4, 16, 2, 1), QG.F32))) == QG.ERR_SHAPE
    assert call(kv=kv_of(bb, fp8=True, scales=bb.t((2, 2, 5, 16, 2, 2), QG.F32))) == QG.ERR_SHAPE


def test_attention_workspace(lib):
    bb = Buf()
    need = q.attention_ragged_paged_workspace(3, 2, 4, 2, 64)
    assert need >= 0
    if need:
        assert attn_call(lib, bb, ws=bb.t((8,), QG.F32)) == QG.ERR_SHAPE
    assert q.attention_ragged_paged_workspace(0, 2, 4, 2, 64) == 0
    assert q.attention_ragged_paged_workspace(3, 0, 4, 2, 64) == 0


def test_attention_empty_problem_is_a_noop(lib):
    bb = Buf()
    assert attn_call(lib, bb, out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK
    assert attn_call(lib, bb, offs=(1,)) == QG.OK
    assert attn_call(lib, bb, out=(3, 0, 64), q_=(3, 0, 64)) == QG.OK


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.tables_ragged_paged(torch.zeros(5, dtype=torch.int32), None, torch.zeros(4, 2, dtype=torch.int32),
                              torch.zeros(2, dtype=torch.int32), t, t, t, t[:1], 16)
    with pytest.raises(ValueError):
        x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
        q.attention_ragged_paged(x, x, t[:2], torch.zeros(1, 2, 1, 16, 1, 64, dtype=torch.bfloat16), t[:1],
                                 t[:1].view(1, 1), 0, 1.0, torch.zeros(4))
