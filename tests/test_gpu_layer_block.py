"""A layer around its routed experts, as it is used: Streamer.block (residual
sum and norm, router, grouped routing, sort, installs and the routed experts,
the always-on expert in 8-bit integers), each stage's output checked against
the 64-bit implementation of that stage on the GPU's own inputs to it; the
native decode driver with a layer's own routing; and a fully resident block
captured into a graph and replayed on new inputs."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops, synth
from streamed_quantized_expert_b200.runtime import IntExpert, LayerSpec, Streamer
from streamed_quantized_expert_b200.synth import bf16_bits_to_f32, to_bf16_bits
from tests import _ref64 as ref
from tests._bank import assert_close, oracle_bank

pytestmark = pytest.mark.gpu
E, K, H, I, G = 64, 6, 256, 128, 32  # I, G: the routed experts' width and quantisation group
WIDE = 192                           # the always-on expert's width
TOL = 2e-2                           # the routed experts' tolerance


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def bf16(a):
    return torch.from_numpy(to_bf16_bits(a).view(np.int16)).cuda().view(torch.bfloat16)


def host(t):
    return t.float().cpu().numpy()


def layers(orc, n, resident, seed=0, always=True, ns=0):
    r = np.random.default_rng(seed)
    bank = oracle_bank(orc, E, H, I, G, 4, 4, seed=3)
    pinned = torch.from_numpy(bank).pin_memory()
    specs, weights = [], []
    for l in range(n):
        wg, wd = (0.05 * r.standard_normal((2 * WIDE, H))).astype(np.float32), (0.05 * r.standard_normal((H, WIDE))).astype(np.float32)
        bias = (0.1 * r.standard_normal(E)).astype(np.float32)
        gamma = ref.round_to((1 + 0.1 * r.standard_normal(H)).astype(np.float32), False)
        router = synth.router_weights(seed, l, E, H)
        weights.append((wg, wd, bias, gamma, router))
        specs.append(LayerSpec(
            ops.desc(E, K, H, I, G, 4, 4), pinned, list(range(E)), shared=torch.from_numpy(bank[:ns]) if ns else None,
            route=ops.route_config("sigmoid", 8, 4, 2, True, 2.5), route_bias=torch.from_numpy(bias).cuda(),
            norm=bf16(gamma), router=torch.from_numpy(router.view(np.int16)).cuda().view(torch.bfloat16),
            always=IntExpert(torch.from_numpy(wg).cuda(), torch.from_numpy(wd).cuda(), 256) if always else None))
    st = Streamer(specs, resident, max_tokens=256, n_shared=ns)
    for l in range(n):
        st.place(l, list(range(resident)))
    torch.cuda.synchronize()
    return st, weights, [bank[e] for e in range(E)]


def check_block(orc, st, l, weights, slots, h0, delta, h, T, L, table, y, row_w=None, ns=0):
    """Every stage of the block that has just run, from the GPU's own inputs to it."""
    wg, wd, bias, gamma, router = weights[l]
    spec = st.layers[l]
    # the norm
    rh, rx, p, r = ref.add_norm(h0, False, delta, gamma, 1e-6)
    assert np.array_equal(host(h[:T]), rh)
    x = host(st.x[:T])
    assert np.all(np.abs(x - rx) <= (ref.UBF + 18 * ref.U32) * np.abs(rx))
    logits = st.logits[:T].cpu().numpy()
    want = x.astype(np.float64) @ bf16_bits_to_f32(router).astype(np.float64).T
    assert np.all(np.abs(logits - want) <= 64 * ref.U32 * (np.abs(x) @ np.abs(bf16_bits_to_f32(router)).T))
    # the routing
    ids, w, _ = ref.route(logits, K, True, bias, 8, 4, 2, True, 2.5, L, table)
    got = st.ids[:T].cpu().numpy()
    assert np.array_equal(got[:, :K], ids)
    wk = st.w[:T].cpu().numpy()
    assert np.all(np.abs(wk[:, :K] - w) <= 16 * ref.U32 * np.abs(w))
    if ns:
        assert np.array_equal(got[:, K:], np.tile(np.arange(E, E + ns), (T, 1)))
        w = np.concatenate([w, np.ones((T, ns))], axis=1)
    # the routed experts
    total = orc.expert_ffn(to_bf16_bits(x), H, I, G, 4, 4, got, w, slots + slots[:ns])
    if spec.always is not None:
        ex = spec.always
        xq, xs = st.xq[:T].cpu().numpy(), st.x_scale[:T].cpu().numpy()
        rq, a, _ = ref.codes(p)
        assert np.array_equal(xq, rq) and np.all(np.abs(xs - a * r / 127) <= 20 * ref.U32 * xs)
        for q, s, wt in ((ex.gu_q, ex.gu_s, wg), (ex.down_q, ex.down_s, wd)):
            cq, ca, _ = ref.codes(wt)
            assert np.array_equal(q.cpu().numpy(), cq) and np.all(np.abs(s.cpu().numpy() - ca / 127) <= ref.U32 * ca / 127)
        gu, _ = ref.int_matmul(xq, xs, ex.gu_q.cpu().numpy(), ex.gu_s.cpu().numpy())
        got_gu = host(ex.gu[:T])
        assert np.all(np.abs(got_gu - gu) <= (ref.UBF + 5 * ref.U32) * np.abs(gu) + 1e-30)
        hq = ex.hq[:T].cpu().numpy()
        _, _, t = ref.codes(ref.swiglu(got_gu))
        assert np.all(np.abs(hq - t) <= 0.5 + 1.2e-4)
        out, _ = ref.int_matmul(hq, ex.hs[:T].cpu().numpy(), ex.down_q.cpu().numpy(), ex.down_s.cpu().numpy(), None, row_w)
        total = total + out
    assert_close(y.cpu().numpy(), total, TOL)
    return total


@pytest.mark.parametrize("T,L", [(1, 0.0), (1, 0.125), (5, 0.125), (40, 0.0), (200, 0.0)])
def test_blocks_with_installs(orc, T, L):
    """Two layers of a third resident experts, over three steps: the second
    block's delta is the first one's output."""
    st, weights, slots = layers(orc, 2, 48 if T > 8 else 24)
    r = np.random.default_rng(T)
    row_w = r.random(T).astype(np.float32)
    for step in range(3):
        h0 = ref.round_to(r.standard_normal((T, H)).astype(np.float32), False)
        h, delta, rd = bf16(h0), None, None
        for l in range(2):
            table = st.table_dev[l].cpu().numpy()
            rw = row_w if l else None
            y = torch.empty((T, H), device="cuda")
            st.block(l, h, delta, T, L, row_w=None if rw is None else torch.from_numpy(rw).cuda(), y=y)
            torch.cuda.synchronize()
            check_block(orc, st, l, weights, slots, h0, rd, h, T, L, table, y, rw)
            h0, delta, rd = host(h), y, y.cpu().numpy()
    assert st.check_dev_err() == 0 and st.installs > 0


def test_block_with_shared_experts_and_without_the_always_on_one(orc):
    st, weights, slots = layers(orc, 1, 24, always=False, ns=2)
    r = np.random.default_rng(3)
    for T in (1, 7, 100):
        h0 = ref.round_to(r.standard_normal((T, H)).astype(np.float32), False)
        rd = r.standard_normal((T, H)).astype(np.float32)
        h = bf16(h0)
        if T > 64:
            st2, weights2, _ = layers(orc, 1, 64, always=False, ns=2)
        else:
            st2, weights2 = st, weights
        y = st2.block(0, h, torch.from_numpy(rd).cuda(), T)
        torch.cuda.synchronize()
        check_block(orc, st2, 0, weights2, slots, h0, rd, h, T, 0.0, None, y, ns=2)
        assert st2.check_dev_err() == 0


def test_driver_equals_the_calls_one_by_one(orc):
    """moe_decode_layer with a layer's own routing and bias: what the separate calls give, bit for bit."""
    for T in (1, 6):
        sa, _, _ = layers(orc, 1, 24, seed=5, always=False)
        sb, _, _ = layers(orc, 1, 24, seed=5, always=False)
        for step in range(4):
            x = torch.from_numpy(synth.activations(5, step, T, H).view(np.int16)).cuda()
            lg = torch.from_numpy(synth.router_logits(5, step, T, E)).cuda()
            ya = sa.decode_layer(0, x, lg, T, 0.125).clone()
            yb = sb.decode_layer_steps(0, x, lg, T, 0.125).clone()
            torch.cuda.synchronize()
            assert torch.equal(sa.ids[:T], sb.ids[:T]) and torch.equal(sa.w[:T], sb.w[:T])
            assert torch.equal(sa.table_dev, sb.table_dev) and sa.installs == sb.installs
            assert_close(ya.cpu().numpy(), yb.cpu().numpy(), 1e-5)  # resident experts are summed first by the driver
        assert sa.installs > 0


def test_prefetch_guesses_route_like_their_layer(orc):
    """moe_decode_layer_ahead: a guessed layer's experts come from its own routing."""
    st, weights, _ = layers(orc, 2, 24, always=False)
    x = torch.from_numpy(synth.activations(1, 0, 1, H).view(np.int16)).cuda()
    l0, l1 = synth.router_logits(1, 0, 1, E), synth.router_logits(1, 1, 1, E)
    st.decode_layer_ahead(0, x, torch.from_numpy(l0).cuda(), 1, 0.0, [(1, torch.from_numpy(l1).cuda())])
    torch.cuda.synchronize()
    assert np.array_equal(st.g_ids[:K].cpu().numpy(), ref.route(l1, K, True, weights[1][2], 8, 4, 2)[0][0])
    assert st.check_dev_err() == 0


@pytest.mark.parametrize("T", [1, 20])
def test_resident_block_in_a_graph(orc, T):
    st, weights, slots = layers(orc, 2, E)
    side = torch.cuda.Stream()
    st.stream = side
    r = np.random.default_rng(T)
    h, y0, y1 = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, H), device="cuda"), \
        torch.zeros((T, H), device="cuda")
    delta = torch.zeros((T, H), device="cuda")
    st.block(0, h, delta, T, y=y0)  # allocates the block's buffers outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        st.block(0, h, delta, T, y=y0)
        st.block(1, h, y0, T, y=y1)
    for step in range(3):
        h0 = ref.round_to(r.standard_normal((T, H)).astype(np.float32), False)
        d0 = r.standard_normal((T, H)).astype(np.float32)
        h.copy_(bf16(h0))
        delta.copy_(torch.from_numpy(d0))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        h1 = ref.round_to(h0 + d0, False)
        check_block(orc, st, 1, weights, slots, h1, y0.cpu().numpy(), h, T, 0.0, None, y1)
    assert st.check_dev_err() == 0


def test_block_refuses_too_many_tokens(orc):
    st, _, _ = layers(orc, 1, 24)
    h = torch.zeros((300, H), dtype=torch.bfloat16, device="cuda")
    for T in (0, 257):
        with pytest.raises(ops.MoeError) as ei:
            st.block(0, h, None, T)
        assert ei.value.status == ops.MOE_ERR_CAPACITY
    for bad in (h.to(torch.float16), h.t(), h[:2]):  # a type the library lacks, not dense, too few rows
        with pytest.raises(ops.MoeError) as ei:
            st.block(0, bad, None, 3)
        assert ei.value.status == ops.MOE_ERR_INVALID
    with pytest.raises(ops.MoeError) as ei:
        st.layers[0].always.add(h, h, 257, h, None)
    assert ei.value.status == ops.MOE_ERR_CAPACITY


def test_a_refused_block_leaves_h_as_it_was(orc):
    """What a block could not run, or would read past, is refused before h takes delta."""
    st, _, _ = layers(orc, 1, 24)
    spec = st.layers[0]
    h = torch.ones((256, H), dtype=torch.bfloat16, device="cuda")
    delta = torch.ones((256, H), device="cuda")
    good = spec.always, spec.norm, spec.router
    small = IntExpert(torch.ones((64, H), device="cuda"), torch.ones((H, 32), device="cuda"), 2)
    narrow = IntExpert(torch.ones((64, H // 2), device="cuda"), torch.ones((H // 2, 32), device="cuda"), 256)

    def refused(status, T=3, spec_values=good, **kw):
        spec.always, spec.norm, spec.router = spec_values
        try:
            with pytest.raises(ops.MoeError) as ei:
                st.block(0, h, delta, T, **kw)
        finally:
            spec.always, spec.norm, spec.router = good
        assert ei.value.status == status
        torch.cuda.synchronize()
        assert (h == 1).all()

    refused(ops.MOE_ERR_CAPACITY, spec_values=(small, *good[1:]))
    refused(ops.MOE_ERR_INVALID, spec_values=(narrow, *good[1:]))
    refused(ops.MOE_ERR_INVALID, T=65, prefill=False)
    for norm in (None, good[1][:8], good[1].float(), good[1].cpu()):
        refused(ops.MOE_ERR_INVALID, spec_values=(good[0], norm, good[2]))
    for router in (None, good[2][:-1], good[2].t(), good[2].float()):
        refused(ops.MOE_ERR_INVALID, spec_values=(good[0], good[1], router))
    w = torch.ones(8, device="cuda")
    for row_w in (w[:2], w[::2], w.double(), w.cpu()):
        refused(ops.MOE_ERR_INVALID, row_w=row_w)
    for y in (torch.empty((2, H), device="cuda"), h[:3], torch.empty((3, H))):
        refused(ops.MOE_ERR_INVALID, y=y)


def test_a_bias_needs_a_routing_that_reads_it(orc):
    st, _, _ = layers(orc, 1, 24)
    spec = st.layers[0]
    for change in (dict(route=None), dict(route_bias=spec.route_bias[:-1]), dict(route_bias=spec.route_bias.double())):
        with pytest.raises(AssertionError):
            Streamer([LayerSpec(**{**spec.__dict__, **change})], 24, max_tokens=8)
