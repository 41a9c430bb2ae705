"""The operators around the routed experts at sizes whose offsets pass 32
bits: sampled rows against the 64-bit implementations, the tolerances of
their own tests."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from tests import _ref64 as ref

pytestmark = pytest.mark.gpu
U = ref.U32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()
    yield
    torch.cuda.empty_cache()


def sample(T):
    return torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")


def host(t):
    return t.float().cpu().numpy()


def test_rows_of_more_than_2_to_the_32_values():
    T, H = 270000, 16008  # 4.3e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    h[:] = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
    h *= (1 + torch.arange(T, device="cuda") % 7).to(torch.bfloat16).unsqueeze(1)
    gamma = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    x, q = torch.empty_like(h), torch.empty((T, H), dtype=torch.int8, device="cuda")
    s = torch.empty(T, device="cuda")
    ops.moe_add_norm_quant(h, ops.MOE_BF16, None, ops.MOE_BF16, gamma, 1e-6, T, H, None, x, q, s)
    at = sample(T)
    _, rx, p, r = ref.add_norm(host(h[at]), False, None, host(gamma), 1e-6)
    rq, a, _ = ref.codes(p)
    assert np.array_equal(q[at].cpu().numpy(), rq)
    assert np.all(np.abs(host(s[at]) - a * r / 127) <= (H / 512 + 16) * U * a * r / 127)
    assert np.all(np.abs(host(x[at]) - rx) <= (ref.UBF + (H / 512 + 16) * U) * np.abs(rx))
    # the same buffer as rows [gate | up] of half the width
    half = H // 2 // 8 * 8
    ops.moe_swiglu_quant(h, ops.MOE_BF16, T, half, q, s)
    q2 = q.reshape(-1)[:T * half].reshape(T, half)
    rows = h.reshape(-1)[:T * 2 * half].reshape(T, 2 * half)
    _, a, t = ref.codes(ref.swiglu(host(rows[at])))
    assert np.all(np.abs(q2[at].cpu().numpy() - t) <= 0.5 + 1.2e-4)
    assert np.all(np.abs(host(s[at]) - a / 127) <= 8 * U * a / 127)


@pytest.mark.parametrize("N,K", [(131008, 32), (9, 65536)])
def test_product_with_more_than_2_to_the_32_values(N, K):
    T = 40000 if N > 9 else 70000  # outputs, or codes, past 4.3e9
    g = torch.Generator(device="cuda").manual_seed(2)
    xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.moe_int_matmul(xq, xs, T, wq, ws, N, K, None, None, y, ops.MOE_BF16, err)
    at = sample(T)
    want, prod = ref.int_matmul(xq[at].cpu().numpy(), host(xs[at]), wq.cpu().numpy(), host(ws))
    assert np.all(np.abs(host(y[at]) - want) <= 4 * U * np.abs(prod) + 1.01 * ref.UBF * np.abs(want))
    assert int(err.item()) == 0


def test_routing_of_more_than_2_to_the_32_logits():
    T, E, k = 4200000, 1024, 3  # 17 GB of logits
    cfg = ops.route_config("sigmoid", 8, 4, 2, True, 2.5)
    d = ops.desc(E, k, 64, 32, 32, 4)
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty((T, E), device="cuda")
    for c in range(0, T, 100000):
        logits[c:c + 100000].normal_(generator=g)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ops.moe_route_grouped(logits, T, d, cfg, bias, 0.0, None, 0, None, ids, w)
    at = sample(T)
    rid, rw, _ = ref.route(host(logits[at]), k, True, host(bias), 8, 4, 2, True, 2.5)
    assert np.array_equal(ids[at].cpu().numpy(), rid)
    assert np.all(np.abs(host(w[at]) - rw) <= 16 * U * rw)
