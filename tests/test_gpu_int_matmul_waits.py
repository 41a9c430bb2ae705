"""Waits of the integer product that run out: the warps that store leave
together, the call returns, and the next one is right."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from tests.test_gpu_int_matmul import check, dev, inputs, run

pytestmark = pytest.mark.gpu

# K split over a cluster, 64- and 256-token tiles of one CTA, pairs of CTAs
SIZES = [(40, 300, 2064), (100, 9602, 1040), (129, 19000, 2064), (700, 7001, 4112)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


@pytest.mark.parametrize("T,N,K", SIZES)
def test_limits_around_a_tile(T, N, K):
    """Limits from a few hundred cycles to the length of some tiles, so that the
    roles give up at different points: only MOE_DEV_ERR_TIMEOUT is reported,
    and whatever a call reported, the next one with the default limit is right."""
    a = inputs(7, T, N, K, True, True)
    b = [dev(x) for x in a]
    y, err = torch.empty((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for limit in (300, 2000, 5000, 12000, 50000):
        try:
            ops.moe_set_wait_limit_cycles(limit)
            for _ in range(4):
                ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, b[4], b[5], y, ops.MOE_F32, err)
            torch.cuda.synchronize()
        finally:
            ops.moe_set_wait_limit_cycles(0)
        assert int(err.item()) in (0, ops.DEV_ERR_TIMEOUT)
        check(run(*a, True), *a, True)


@pytest.mark.parametrize("T,N,K", SIZES)
def test_the_shortest_limit_runs_out(T, N, K):
    """A limit of one cycle is shorter than a copy takes: every kernel reports
    MOE_DEV_ERR_TIMEOUT, also where the default limit returns right after it."""
    a = inputs(9, T, N, K, True, True)
    b = [dev(x) for x in a]
    y, err = torch.empty((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        ops.moe_set_wait_limit_cycles(1)
        ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, b[4], b[5], y, ops.MOE_F32, err)
        torch.cuda.synchronize()
    finally:
        ops.moe_set_wait_limit_cycles(0)
    assert int(err.item()) == ops.DEV_ERR_TIMEOUT
    check(run(*a, True), *a, True)
