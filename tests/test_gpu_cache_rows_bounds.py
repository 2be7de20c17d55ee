"""kv_read_ragged_paged writes nothing behind its outputs, whatever the last offset says."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import dev32, devf32, say
from test_gpu_cache_rows import cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gran", [0, 32])
@pytest.mark.parametrize("T", [1, 2001, 9001])
@pytest.mark.parametrize("planes", [(True, True), (False, True)])
def test_rows_behind_the_outputs(lib, gpu, T, gran, planes):
    """The last workgroup of several rows reaches past T: its other rows belong to a sequence, but to no output."""
    more = 200
    d = synth.attention_inputs(20, [1, 1], [30, T + more], hq=1, hkv=1, d=32, gran=gran)
    offs = np.array([0, min(T, 20), T + more], np.uint32)
    bufs = [torch.full((T + more, 1, 32), 7.0, device="cuda") if p else None for p in planes]
    say(f"[read] T {T} offsets {offs.tolist()} gran {gran} planes {planes}")
    lib.kv_read_ragged_paged(*[None if b is None else b[:T] for b in bufs], dev32(offs), None, cache(d), dev32(d.page_table), d.layer_idx,
                             kv_scales=devf32(d.scales) if gran else None, quantization_granularity=gran)
    torch.cuda.synchronize()
    want = oracle.kv_read_ragged_paged(offs, None, d.blocks, d.page_table, d.layer_idx, d.scales, gran)
    for plane, b in enumerate(bufs):
        if b is not None:
            assert (b[T:] == 7).all(), "rows behind the output changed"
            assert np.array_equal(b[:T].cpu().numpy(), want[plane][:T].astype(np.float32))
