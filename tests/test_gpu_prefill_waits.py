"""Waits of the tensor-core grouped GEMM that run out: its warps leave
together, no copy outlives its block, and the next call gives what the one
before gave."""
import numpy as np
import pytest

from streamed_quantized_expert_b200 import build, ops
from tests.test_gpu_prefill_tc import _case, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


@pytest.mark.parametrize("bits", [(4, 4), (3, 6), (16, 16)])
def test_limits_around_a_tile(orc, bits):
    s, x, ids, w = _case(orc, 8, 2, 384, 256, 64, *bits, 600, R=8, seed=sum(bits))
    want = _check(orc, s, x, ids, w, 600, ntok=4)
    reported = []
    for limit in (1, 300, 2000, 5000, 12000, 50000):
        try:
            ops.moe_set_wait_limit_cycles(limit)
            for _ in range(3):
                reported.append(s.gpu(x, ids, w, 600, sorted_x=True)[1])
        finally:
            ops.moe_set_wait_limit_cycles(0)
        y, err = s.gpu(x, ids, w, 600, sorted_x=True)
        assert err == 0 and np.array_equal(y, want)
    assert set(reported) <= {0, ops.DEV_ERR_TIMEOUT}
