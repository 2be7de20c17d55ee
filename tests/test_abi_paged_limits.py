"""CPU checks of the paged-cache entry points at the limits of their arguments: what cannot be
served is refused before the GPU is touched. No call here reaches a kernel launch."""
import math

import pytest
import torch

import grouped_gemm_qgemm_amd as q
from grouped_gemm_qgemm_amd import QG
from test_abi import Buf
from test_abi_paged import attn_call, lib


def test_a_scale_whose_base_2_form_is_infinite_is_refused(lib):
    bb = Buf()
    assert attn_call(lib, bb, scale=3.0e38) == QG.ERR_INVALID_ARG
    assert attn_call(lib, bb, scale=2.0**128 / 1.4426950408889634 * (1 + 1e-6)) == QG.ERR_INVALID_ARG
    assert attn_call(lib, bb, scale=2.0**127, out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK
    assert attn_call(lib, bb, scale=math.ldexp(1.0, -149), out=(0, 4, 64), q_=(0, 4, 64)) == QG.OK
