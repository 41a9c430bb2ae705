"""One IntExpert used by two streams, or by two captured graphs, at once: each
call's gate, up and codes are its own."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from streamed_quantized_expert_b200.runtime import IntExpert

pytestmark = pytest.mark.gpu
H, WIDE, T, REPEAT = 512, 2048, 1024, 20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def tokens(seed):
    r = np.random.default_rng(seed)
    q = torch.from_numpy(r.integers(-127, 128, (T, H), dtype=np.int8)).cuda()
    return q, torch.from_numpy((0.5 + r.random(T)).astype(np.float32) / 127).cuda()


@pytest.fixture
def expert():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = lambda *s: 0.05 * torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return IntExpert(w(2 * WIDE, H), w(H, WIDE), T)


def alone(expert, x):
    """The call by itself."""
    y, err = torch.zeros((T, H), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    expert.add(*x, T, y, err)
    torch.cuda.synchronize()
    return y


def test_two_streams(expert):
    xs = [tokens(s) for s in (1, 2)]
    want = [alone(expert, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ys = [torch.zeros((REPEAT, T, H), device="cuda") for _ in xs]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(REPEAT):
        for x, y, s in zip(xs, ys, streams):
            expert.add(*x, T, y[i], err, None, s)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for y, w in zip(ys, want):
        assert all(torch.equal(v, w) for v in y)


def test_two_graphs(expert):
    xs = [tokens(s) for s in (3, 4)]
    want = [alone(expert, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ys, graphs = [torch.zeros((REPEAT, T, H), device="cuda") for _ in xs], []
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # both on torch's stream for captures
            for i in range(REPEAT):
                expert.add(*x, T, y[i], err, None, torch.cuda.current_stream())
        graphs.append(g)
    own = alone(expert, xs[0])  # a call between the captures and their replays
    for _ in range(3):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for y, w in zip(ys, want):
            assert all(torch.equal(v, w) for v in y)
    assert torch.equal(own, want[0])
