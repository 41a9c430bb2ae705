"""moe_quantize_channels, moe_add_norm_quant and moe_swiglu_quant against
plain implementations in 64 bits.

Tolerances, in half steps u = 2^-24 of fp32:
* codes of plain rows and of the norm are defined by exact arithmetic on fp32
  numbers: equal;
* scale of plain rows: one division, 1 u;
* the norm's r: the sum of H squares passes at most H / 256 + 16 roundings on
  the way of any one term, half of which reach r, then the quotient by H, eps,
  rsqrt (2 steps, 4 u): (H / 512 + 14) u; its scale 2 u more, its x 2 u and the
  rounding to bf16, 2^-8;
* SwiGLU: exp is off by 2 steps (4 u), 1 + e, the quotient and the product 1 u
  each: 7 u for v, 8 u for the scale; 127 v / a is off by at most 127 x 15 u,
  below 1.2e-4, which is how much further than 1/2 a code may be from it."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from streamed_quantized_expert_b200.synth import bf16_bits_to_f32, to_bf16_bits
from tests import _ref64 as ref

pytestmark = pytest.mark.gpu
U = ref.U32
GUARD = 2  # rows behind the last, which stay as they were


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def dev(a, f32=True):
    """fp32 values (already rounded to their type) on the device in that type."""
    if a is None:
        return None
    a = np.ascontiguousarray(a, np.float32)
    return torch.from_numpy(a).cuda() if f32 else torch.from_numpy(to_bf16_bits(a).view(np.int16)).cuda()


def host(t):
    a = t.cpu().numpy()
    return bf16_bits_to_f32(a.view(np.uint16)) if a.dtype == np.int16 else a


def out(T, H, dt):
    return torch.full((T + GUARD, H), 77, dtype=dt, device="cuda")


def cut(t, T):
    a = t.cpu().numpy()
    assert (a[T:] == 77).all()
    return host(t[:T])


def draw(seed, T, H, f32, std=1.0):
    return ref.round_to(std * np.random.default_rng(seed).standard_normal((T, H)).astype(np.float32), f32)


def close(got, want, u):
    want = np.asarray(want, np.float64)
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got))
    assert np.all(np.abs(got - want)[~nan] <= u * np.abs(want)[~nan] + 1.5e-45)


def quantize(w, f32, stream=None):
    T, H = w.shape
    q, s = out(T, H, torch.int8), out(T, 1, torch.float32)
    x = dev(w, f32)
    torch.cuda.synchronize()
    ops.moe_quantize_channels(x, ops.MOE_F32 if f32 else ops.MOE_BF16, T, H, q, s, stream)
    torch.cuda.synchronize()
    return cut(q, T), cut(s, T)[:, 0]


SIZES = [(1, 8), (1, 2048), (3, 16), (5, 248), (2, 2040), (2, 2056), (7, 4096), (300, 64), (3, 8200), (2, 16384),
         (2, 16392), (1, 65536), (129, 1024)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", SIZES)
def test_quantize(T, H, f32):
    w = draw(T + H, T, H, f32, 0.02)
    q, s = quantize(w, f32)
    rq, a, _ = ref.codes(w)
    assert np.array_equal(q, rq)
    close(s, a / 127.0, U)


@pytest.mark.parametrize("f32", [False, True])
def test_quantize_special_rows(f32):
    H = 264
    w = draw(1, 12, H, f32)
    w[0] = 0.0
    w[1, 5] = np.inf
    w[2, H - 1] = np.nan
    w[3] = 0.0
    w[3, 7] = -3.0                                        # one value: code -127
    w[4] = np.where(np.arange(H) % 2 == 0, 127.0, 0.5)    # ties: 0.5 goes to 0
    w[5] = np.where(np.arange(H) % 3 == 0, -127.0, 1.5)   # 1.5 goes to 2
    w[6] = ref.round_to(w[6] * np.float32(2.0 ** -126), f32)  # subnormal numbers
    w[7] = ref.round_to(w[7] * np.float32(2.0 ** 125), f32)
    w[8] = 0.0
    w[8, 0] = 2.0 ** -133                                 # a scale that fp32 hardly holds
    w[9] = -1.0
    w[10] = np.finfo(np.float32).min if f32 else -3.3895314e38
    q, s = quantize(w, f32)
    rq, a, _ = ref.codes(w)
    assert np.array_equal(q, rq)
    assert np.isnan(s[1]) and np.isnan(s[2]) and (q[1:3] == 0).all() and s[0] == 0.0
    ok = ~np.isnan(a)
    assert np.all(np.abs(s[ok] - a[ok] / 127.0) <= U * a[ok] / 127.0 + 0.75e-45)


def test_codes_at_ties():
    """Quotients that are ties, or next to one: rows 127 k + {-1, 0, 1} steps
    around every half code."""
    half = np.arange(-126.5, 127.0, 1.0).astype(np.float32)
    p = np.concatenate([half, np.nextafter(half, np.float32(-999)), np.nextafter(half, np.float32(999))])
    for a in (127.0, 254.0, 127.0 * 3, 100.0, 0.0127, 33.3):
        w = (p * np.float32(a / 127.0)).astype(np.float32)
        w = np.concatenate([w, np.full(8 + (-len(w)) % 8, a, np.float32)])[None]
        q, _ = quantize(w, True)
        assert np.array_equal(q, ref.codes(w)[0]), a


def norm(h, hf, delta, df, gamma, eps=1e-6, in_place=False, want_x=True, want_q=True, want_h=True, stream=None):
    T, H = h.shape
    hd, dd, gd = dev(h, hf), dev(delta, df), dev(gamma, False)
    ht = torch.float32 if hf else torch.int16
    if in_place:
        ho = torch.cat([hd, torch.full((GUARD, H), 77, dtype=ht, device="cuda")])
        hd = ho
    else:
        ho = out(T, H, ht) if want_h else None
    x = out(T, H, torch.int16) if want_x else None
    q, s = (out(T, H, torch.int8), out(T, 1, torch.float32)) if want_q else (None, None)
    torch.cuda.synchronize()
    ops.moe_add_norm_quant(hd, ops.MOE_F32 if hf else ops.MOE_BF16, dd, ops.MOE_F32 if df else ops.MOE_BF16, gd, eps,
                           T, H, ho, x, q, s, stream)
    torch.cuda.synchronize()
    return (None if ho is None else cut(ho, T), None if x is None else cut(x, T), None if q is None else cut(q, T),
            None if s is None else cut(s, T)[:, 0])


def check_norm(h, hf, delta, df, gamma, got, eps=1e-6):
    H = h.shape[1]
    rh, rx, p, r = ref.add_norm(h, hf, delta, gamma, eps)
    rq, a, _ = ref.codes(p)
    ho, x, q, s = got
    ur = (H / 512 + 14) * U
    if ho is not None:
        assert np.array_equal(ho, rh, equal_nan=True)
    if x is not None:
        close(x, rx, ref.UBF + ur + 2 * U)
    if q is not None:
        assert np.array_equal(q, rq)
        close(s, a * r / 127.0, ur + 2 * U)


@pytest.mark.parametrize("hf", [False, True])
@pytest.mark.parametrize("df", [None, False, True])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm(T, H, hf, df):
    h, gamma = draw(H, T, H, hf), ref.round_to(1.0 + 0.2 * draw(H + 1, 1, H, True)[0], False)
    delta = None if df is None else draw(H + 2, T, H, df, 0.5)
    check_norm(h, hf, delta, df, gamma, norm(h, hf, delta, df, gamma))


@pytest.mark.parametrize("hf", [False, True])
@pytest.mark.parametrize("H", [64, 4096, 16392])
def test_norm_outputs_in_place_and_left_out(hf, H):
    T = 3
    h, gamma, delta = draw(5, T, H, hf), ref.round_to(draw(6, 1, H, True)[0], False), draw(7, T, H, True)
    check_norm(h, hf, delta, True, gamma, norm(h, hf, delta, True, gamma, in_place=True))
    check_norm(h, hf, delta, True, gamma, norm(h, hf, delta, True, gamma, want_h=False))
    check_norm(h, hf, delta, True, gamma, norm(h, hf, delta, True, gamma, want_x=False))
    check_norm(h, hf, delta, True, gamma, norm(h, hf, delta, True, gamma, want_q=False))
    check_norm(h, hf, None, None, gamma, norm(h, hf, None, None, gamma, in_place=True))


@pytest.mark.parametrize("hf", [False, True])
def test_norm_special_rows(hf):
    H = 520
    h, gamma = draw(1, 8, H, hf), ref.round_to(1.0 + draw(2, 1, H, True)[0], False)
    gamma[3] = 0.0
    h[0] = 0.0
    h[1, 4] = np.nan
    h[2, 5] = -np.inf
    h[3] = ref.round_to(h[3] * np.float32(1e17), hf)
    h[4] = ref.round_to(h[4] * np.float32(1e-25), hf)   # eps decides
    h[5] = 0.0
    h[5, 3] = 2.0                                        # the one value meets gamma 0
    h[6, 100] = 2.0 ** 30
    with np.errstate(all="ignore"):
        ho, x, q, s = norm(h, hf, None, None, gamma)
        rh, rx, p, r = ref.add_norm(h, hf, None, gamma, 1e-6)
    rq, a, _ = ref.codes(p)
    assert np.array_equal(q, rq) and np.array_equal(ho, rh, equal_nan=True)
    assert s[0] == 0 and s[5] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and (q[[0, 1, 2, 5]] == 0).all()
    fine = [0, 3, 4, 5, 6, 7]
    close(x[fine], rx[fine], ref.UBF + 18 * U)
    close(s[fine], (a * r / 127.0)[fine], 18 * U)
    assert np.isnan(x[1]).all()


def swiglu(gu, f32, stream=None):
    T, I = gu.shape[0], gu.shape[1] // 2
    q, s = out(T, I, torch.int8), out(T, 1, torch.float32)
    x = dev(gu, f32)
    torch.cuda.synchronize()
    ops.moe_swiglu_quant(x, ops.MOE_F32 if f32 else ops.MOE_BF16, T, I, q, s, stream)
    torch.cuda.synchronize()
    return cut(q, T), cut(s, T)[:, 0]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,I", SIZES)
def test_swiglu(T, I, f32):
    gu = draw(T * 3 + I, T, 2 * I, f32, 2.0)
    q, s = swiglu(gu, f32)
    _, a, t = ref.codes(ref.swiglu(gu))
    assert np.all(np.abs(q - t) <= 0.5 + 1.2e-4)
    close(s, a / 127.0, 8 * U)


def test_swiglu_special_rows():
    I = 136
    gu = draw(3, 6, 2 * I, True)
    gu[0] = 0.0
    gu[1, 3] = np.nan
    gu[2, I + 7] = np.inf
    gu[3, :I] = -200.0       # silu underflows to 0 (or below any code)
    gu[3, 0] = 1.0
    gu[4, :I] = 200.0        # silu is the identity
    gu[5, 4] = -np.inf
    q, s = swiglu(gu, True)
    _, a, t = ref.codes(ref.swiglu(gu[[0, 3, 4]]))
    assert np.all(np.abs(q[[0, 3, 4]] - t) <= 0.5 + 1.2e-4)
    close(s[[0, 3, 4]], a / 127.0, 8 * U)
    assert np.isnan(s[[1, 2, 5]]).all() and (q[[1, 2, 5]] == 0).all()


def test_repeatable_on_another_stream_and_in_a_graph():
    T, H = 40, 1040
    h, gamma, delta = draw(1, T, H, False), ref.round_to(1 + 0.1 * draw(2, 1, H, True)[0], False), draw(3, T, H, True)
    side = torch.cuda.Stream()
    a = norm(h, False, delta, True, gamma)
    b = norm(h, False, delta, True, gamma, stream=side)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    hd, dd, gd = dev(h, False), dev(delta), dev(gamma, False)
    x = torch.zeros((T, H), dtype=torch.int16, device="cuda")
    q, s = torch.zeros((T, H), dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
    q2, s2 = torch.zeros((T, H // 2), dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        ops.moe_add_norm_quant(hd, ops.MOE_BF16, dd, ops.MOE_F32, gd, 1e-6, T, H, None, x, q, s, side)
        ops.moe_swiglu_quant(x, ops.MOE_BF16, T, H // 2, q2, s2, side)  # reads what the norm has just written
    for seed in range(3):
        h = draw(10 + seed, T, H, False)
        hd.copy_(dev(h, False))
        g.replay()
        torch.cuda.synchronize()
        check_norm(h, False, delta, True, gamma, (None, host(x), q.cpu().numpy(), s.cpu().numpy()))
        _, a2, t2 = ref.codes(ref.swiglu(host(x)))
        assert np.all(np.abs(q2.cpu().numpy() - t2) <= 0.5 + 1.2e-4)
