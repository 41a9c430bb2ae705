"""What the operators around the routed experts give for a row does not depend
on the other rows or on how many there are: a call over T rows equals, bit for
bit, the calls over parts of them (other tiles, splits and kernels)."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def parts(T, sizes):
    at = 0
    for n in sizes:
        yield at, min(n, T - at)
        at += n
        if at >= T:
            return


@pytest.mark.parametrize("N,K,f32", [(4100, 2064, False), (1537, 8192, True), (9603, 1040, True)])
def test_product(N, K, f32):
    T, g = 1400, gen(N)
    xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws, rw = (torch.rand(n, generator=g, device="cuda") + 0.01 for n in (T, N, T))
    add = torch.randn((T, N), generator=g, device="cuda")
    dt = torch.float32 if f32 else torch.bfloat16

    def run(at, n):
        y = torch.empty((n, N), dtype=dt, device="cuda")
        ops.moe_int_matmul(xq[at:], xs[at:], n, wq, ws, N, K, add[at:], rw[at:], y,
                           ops.MOE_F32 if f32 else ops.MOE_BF16, None)
        return y

    whole = run(0, T)
    for at, n in parts(T, (1, 7, 13, 20, 32, 60, 100, 130, 200, 300, 600)):
        assert torch.equal(run(at, n), whole[at:at + n]), (at, n)


@pytest.mark.parametrize("H", [136, 768, 4096, 8200, 16400])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows(H, dt):
    T, g = 500, gen(H)
    kind = ops.MOE_F32 if dt == torch.float32 else ops.MOE_BF16
    h = torch.randn((T, H), generator=g, device="cuda").to(dt)
    delta = torch.randn((T, H), generator=g, device="cuda")
    gamma = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)

    def run(at, n):
        ho, x = torch.empty((n, H), dtype=dt, device="cuda"), torch.empty((n, H), dtype=torch.bfloat16, device="cuda")
        q, s = torch.empty((n, H), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        ops.moe_add_norm_quant(h[at:], kind, delta[at:], ops.MOE_F32, gamma, 1e-6, n, H, ho, x, q, s)
        q2, s2 = torch.empty((n, H // 2 // 8 * 8), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        out = [ho, x, q, s]
        if H // 2 % 8 == 0:
            ops.moe_swiglu_quant(h[at:], kind, n, H // 2, q2, s2)
            out += [q2, s2]
        return out

    whole = run(0, T)
    for at, n in parts(T, (1, 2, 9, 150, 400)):
        assert all(torch.equal(a, b[at:at + n]) for a, b in zip(run(at, n), whole)), (at, n)


@pytest.mark.parametrize("score,bias,G", [("softmax", False, 1), ("softmax", True, 8), ("sigmoid", True, 8)])
def test_routing(score, bias, G):
    T, E, k, g = 3000, 256, 8, gen(G)
    logits = torch.randn((T, E), generator=g, device="cuda")
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    cfg, d = ops.route_config(score, G, max(1, G // 2), 2 if G > 1 else 1, False, 2.5), ops.desc(E, k, 64, 32, 32, 4)

    def run(at, n):
        ids, w = torch.empty((n, k), dtype=torch.int32, device="cuda"), torch.empty((n, k), device="cuda")
        ops.moe_route_grouped(logits[at:], n, d, cfg, b, 0.0, None, 0, None, ids, w)
        return ids, w

    whole = run(0, T)
    for at, n in parts(T, (1, 3, 60, 700, 2236)):
        assert all(torch.equal(x, y[at:at + n]) for x, y in zip(run(at, n), whole)), (at, n)
