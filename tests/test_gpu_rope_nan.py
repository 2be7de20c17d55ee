"""rope_ragged_paged into an e4m3 cache where a whole run of a scale is NaN: its codes are NaN's, whose
product with any scale is NaN. Zeros beside a NaN stay zeros. (The comparison of test_gpu_rope.py: NaN on
both sides or on neither.)"""
import pytest

from test_gpu_rope import CACHED, NEW, Case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gran,d", [(32, 64), (64, 64), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_runs_of_nan(lib, gpu, gran, d, interleaved):
    c = Case(40, NEW, CACHED, gran=gran, d=d, rot=32, interleaved=interleaved)
    c.rows[2, c.hq:] = 0x7FC0               # a whole token's keys and values
    c.rows[5, c.hq:, :gran] = 0xFFFF        # a run of them, the sign bit set
    c.rows[7, c.hq:] = 0                    # zeros but for one NaN behind the turned elements
    c.rows[7, c.hq:, 40] = 0x7FC0
    check(lib, c)
