"""moe_int_matmul against a plain implementation in 64 bits.

The integer sum is exact.  In half steps u = 2^-24 of fp32: the sum's
conversion, two products of scales and their product with it are off by 4 u of
the product; adding gives 1 u of the result; bf16 adds 2^-8 of the result."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from streamed_quantized_expert_b200.synth import bf16_bits_to_f32
from tests import _ref64 as ref

pytestmark = pytest.mark.gpu
GUARD = 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def inputs(seed, T, N, K, add, row_w, extreme=False):
    r = np.random.default_rng(seed)
    lim = (-128, 128) if extreme else (-127, 128)
    xq, wq = r.integers(*lim, (T, K), dtype=np.int8), r.integers(*lim, (N, K), dtype=np.int8)
    xs, ws = (r.random(T) + 0.1).astype(np.float32), (r.random(N) * 0.01).astype(np.float32)
    return (xq, xs, wq, ws, r.standard_normal((T, N)).astype(np.float32) if add else None,
            r.standard_normal(T).astype(np.float32) if row_w else None)


def run(xq, xs, wq, ws, add, row_w, f32, in_place=False, stream=None):
    (T, K), N = xq.shape, wq.shape[0]
    y = torch.full((T * N + GUARD,), 77, dtype=torch.float32 if f32 else torch.int16, device="cuda")
    ad = dev(add)
    if in_place:
        y[:T * N] = ad.reshape(-1)
        ad = y
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (dev(xq), dev(xs), T, dev(wq), dev(ws), N, K, ad, dev(row_w), y, ops.MOE_F32 if f32 else ops.MOE_BF16, err)
    torch.cuda.synchronize()
    ops.moe_int_matmul(*a, stream)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    h = y.cpu().numpy()
    assert (h[T * N:] == 77).all()  # nothing behind the last row
    h = h[:T * N].reshape(T, N)
    return h if f32 else bf16_bits_to_f32(h.view(np.uint16))


def check(got, xq, xs, wq, ws, add, row_w, f32):
    y, prod = ref.int_matmul(xq, xs, wq, ws, add, row_w)
    tol = 4 * ref.U32 * np.abs(prod) + (1.01 * ref.U32 + (0 if f32 else 1.01 * ref.UBF)) * np.abs(y)
    assert np.all(np.abs(got - y) <= tol + 1e-40)


SIZES = [  # T, N, K: one token to long chunks, odd sizes on both sides of the kernels' tiles
    (1, 1, 16), (1, 16, 16), (1, 7, 48), (1, 128, 2048), (1, 333, 8192), (2, 64, 64), (3, 130, 176), (5, 1000, 512),
    (8, 256, 1024), (9, 129, 128), (15, 40, 80), (16, 512, 2048), (17, 511, 2064), (31, 96, 272), (32, 1536, 768),
    (33, 257, 144), (48, 5003, 256), (63, 64, 4096), (64, 2048, 512), (65, 100, 128), (100, 384, 8192),
    (127, 127, 1280), (128, 128, 128), (129, 130, 400), (200, 1025, 640), (255, 48, 32), (256, 256, 4096),
    (257, 640, 368), (300, 31, 65536), (513, 1100, 1024), (700, 2049, 528), (2048, 384, 256), (4100, 300, 160),
    (257, 12801, 1040), (1100, 9000, 272), (2304, 4500, 16),
]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_against_64_bits(T, N, K):
    for add, row_w, f32 in ((False, False, False), (True, True, True)):
        a = inputs(T + N + K, T, N, K, add, row_w)
        check(run(*a, f32), *a, f32)


@pytest.mark.parametrize("T", [1, 6, 24, 90, 300])
def test_options_in_place_and_extreme_codes(T):
    N, K = 200, 1008
    for add, row_w, f32, in_place in ((True, False, True, True), (True, True, True, True), (True, False, False, False),
                                      (False, True, False, False), (False, False, True, False)):
        a = inputs(T, T, N, K, add, row_w, extreme=True)
        check(run(*a, f32, in_place), *a, f32)
    K = 65536  # the largest sum: 65536 x 128 x 128 = 2^30
    a = (np.full((T, K), -128, np.int8), np.ones(T, np.float32), np.full((9, K), -128, np.int8),
         np.ones(9, np.float32), None, None)
    assert (run(*a, True) == 2.0 ** 30).all()


@pytest.mark.parametrize("T", [1, 20, 150, 600])
def test_nan_scale_stays_in_its_row(T):
    """A token whose scale is NaN (its row held an infinity) gives NaN, the others their values."""
    a = inputs(3, T, 70, 256, False, False)
    a[1][T // 2] = np.nan
    got = run(*a, True)
    assert np.isnan(got[T // 2]).all()
    keep = np.arange(T) != T // 2
    check(got[keep], a[0][keep], a[1][keep], *a[2:], True)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_streams_and_graph(T):
    """Two calls at once on two streams, and a captured call replayed on new inputs."""
    N, K = 640, 1024
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    A, B = inputs(1, T, N, K, True, False), inputs(2, T, N, K, True, False)
    bufs = []
    for a in (A, B):
        bufs.append([dev(x) for x in a] + [torch.zeros((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                                             device="cuda")])
    torch.cuda.synchronize()
    for _ in range(10):
        for st, b in ((s1, bufs[0]), (s2, bufs[1])):
            ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, b[4], None, b[6], ops.MOE_F32, b[7], st)
    torch.cuda.synchronize()
    for a, b in ((A, bufs[0]), (B, bufs[1])):
        check(b[6].cpu().numpy(), *a, True)
    b = bufs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s1):
        ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, b[4], None, b[6], ops.MOE_F32, b[7], s1)
    for seed in range(5, 8):
        a = inputs(seed, T, N, K, True, False)
        for i in range(5):
            b[i].copy_(dev(a[i]))
        g.replay()
        torch.cuda.synchronize()
        check(b[6].cpu().numpy(), *a, True)
    assert int(b[7].item()) == 0


def test_pointers_into_larger_buffers():
    """Rows of a larger tensor that start 16-byte aligned, outputs at an odd row (4-byte and 2-byte aligned)."""
    T, N, K = 20, 37, 96
    a = inputs(8, T, N, K, False, False)
    big = torch.zeros((T + 5, K), dtype=torch.int8, device="cuda")
    big[3:3 + T] = dev(a[0])
    for f32, dt in ((True, torch.float32), (False, torch.int16)):
        y = torch.full((T + 2, N), 77, dtype=dt, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.moe_int_matmul(big[3:], dev(a[1]), T, dev(a[2]), dev(a[3]), N, K, None, None, y[1:],
                           ops.MOE_F32 if f32 else ops.MOE_BF16, err)
        torch.cuda.synchronize()
        h = y.cpu().numpy()
        assert (h[0] == 77).all() and (h[T + 1] == 77).all()
        h = h[1:T + 1]
        check(h if f32 else bf16_bits_to_f32(np.ascontiguousarray(h).view(np.uint16)), *a, f32)


@pytest.mark.parametrize("T,N,K", [
    (40, 9602, 1040), (100, 2306, 1040), (41, 2309, 2064), (250, 300, 4112),       # 64-token tiles; K whole, in 2, 4 and 8
    (100, 9602, 1040), (513, 4099, 1040), (129, 19000, 2064), (700, 7001, 4112),  # 128 and 256 tokens, pairs of SMs
    (1025, 4102, 2064)])
def test_every_tile(T, N, K):
    """Sizes at which each tile and split is chosen, with every kind of output
    (even and odd N: paired and single bf16 stores)."""
    for add, row_w, f32, in_place in ((False, False, False, False), (True, True, True, True), (True, False, False, False)):
        a = inputs(T + N, T, N, K, add, row_w, extreme=True)
        check(run(*a, f32, in_place), *a, f32)


@pytest.mark.parametrize("T,N,K", [(129, 19000, 2064), (40, 2306, 2064)])
def test_two_calls_at_once(T, N, K):
    """The tiles that fill an SM's shared memory and tensor memory, on two streams."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [inputs(s, T, N, K, False, False) for s in range(2)]
    bufs = [[dev(x) for x in a[:4]] + [torch.zeros((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
            for a in sets]
    torch.cuda.synchronize()
    for _ in range(8):
        for st, b in zip(streams, bufs):
            ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, None, None, b[4], ops.MOE_F32, b[5], st)
    torch.cuda.synchronize()
    for a, b in zip(sets, bufs):
        check(b[4].cpu().numpy(), *a, True)
        assert int(b[5].item()) == 0


@pytest.mark.parametrize("T,N,K", [(40, 300, 2064), (100, 9602, 1040), (513, 4099, 1040), (700, 7001, 4112)])
def test_waits_that_may_run_out(T, N, K):
    """With the shortest limit a wait runs out or does not, as the copies
    land: the call returns, reports no error but MOE_DEV_ERR_TIMEOUT, and the
    next call with the default limit is right."""
    a = inputs(4, T, N, K, False, False)
    b = [dev(x) for x in a[:4]]
    y, err = torch.empty((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        ops.moe_set_wait_limit_cycles(1)
        for _ in range(3):
            ops.moe_int_matmul(b[0], b[1], T, b[2], b[3], N, K, None, None, y, ops.MOE_F32, err)
        torch.cuda.synchronize()
    finally:
        ops.moe_set_wait_limit_cycles(0)
    assert int(err.item()) in (0, ops.DEV_ERR_TIMEOUT)
    check(run(*a, True), *a, True)
