"""What Streamer.block refuses leaves h (and y) as it was, so that the caller can correct
the call and make it again: arguments that only a later stage would refuse."""
import gc
import weakref

import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from streamed_quantized_expert_b200.runtime import IntExpert, LayerSpec, Streamer
from tests.test_gpu_layer_block import H, layers

pytestmark = pytest.mark.gpu
INV, UNS = ops.MOE_ERR_INVALID, ops.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


class Block:
    """A Streamer of one layer and a call of its block that is to be refused."""

    def __init__(self, orc, max_tokens=256):
        self.st, _, _ = layers(orc, 1, 24)
        if max_tokens != self.st.max_tokens:
            self.st = Streamer(self.st.layers, 24, max_tokens=max_tokens)
        self.spec = self.st.layers[0]

    def refused(self, status, T=3, **kw):
        h = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
        y = torch.full((T, H), 7.0, device="cuda")
        delta = torch.ones((T, H), device="cuda")
        torch.cuda.synchronize()
        with pytest.raises(ops.MoeError) as ei:
            self.st.block(0, h, delta, T, **{"y": y, **kw})
        torch.cuda.synchronize()
        assert ei.value.status == status
        assert (h == 1).all() and (y == 7).all()


@pytest.fixture
def block(orc):
    return Block(orc)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("L", [-0.5, float("nan"), float("inf"), 2e30, 1e300])
def test_substitution_strength(block, T, L):
    block.refused(INV, T=T, L=L)


@pytest.mark.parametrize("T,prefill", [(1, False), (3, False), (70, True)])
@pytest.mark.parametrize("status,change", [
    (INV, dict(n_groups=7)), (INV, dict(n_groups=32, top_groups=2)), (INV, dict(score=5)), (INV, dict(group_top=3)),
    (INV, dict(scale=float("nan"))), (UNS, dict(n_groups=64, top_groups=64, group_top=1))])
def test_route_config(orc, block, status, change, T, prefill):
    """Groups that do not divide 64 experts, 6 of 4 kept ones, and so on: refused
    when the Streamer is made, and by a block whose layer was changed afterwards."""
    good = block.spec.route
    bad = ops.RouteConfig(good.score, good.n_groups, good.top_groups, good.group_top, good.renormalise, good.scale)
    for name, v in change.items():
        setattr(bad, name, v)
    with pytest.raises(ops.MoeError) as ei:
        Streamer([LayerSpec(**{**block.spec.__dict__, "route": bad})], 24, max_tokens=8)
    assert ei.value.status == status
    for name, v in change.items():
        setattr(good, name, v)
    block.refused(status, T=T, prefill=prefill)


@pytest.mark.parametrize("width", [8, 24, 200])
def test_width_of_an_integer_expert(width):
    """The products take K in multiples of 16, the codes in multiples of 8."""
    with pytest.raises(ops.MoeError) as ei:
        IntExpert(torch.ones((2 * width, H), device="cuda"), torch.ones((H, width), device="cuda"), 4)
    assert ei.value.status == INV
    with pytest.raises(ops.MoeError) as ei:
        IntExpert(torch.ones((64, width), device="cuda"), torch.ones((width, 32), device="cuda"), 4)
    assert ei.value.status == INV


def test_integer_expert_too_wide():
    wide = (1 << 16) + 16
    with pytest.raises(ops.MoeError) as ei:
        IntExpert(torch.ones((2 * wide, 16), device="cuda"), torch.ones((16, wide), device="cuda"), 4)
    assert ei.value.status == UNS


@pytest.mark.parametrize("T", [1, 3, 70])
def test_alignment_of_the_router(block, T):
    E = block.st.E
    odd = torch.zeros(E * H + 8, dtype=torch.bfloat16, device="cuda")[1:E * H + 1].view(E, H)
    block.spec.router = odd
    block.refused(INV, T=T)


def test_tokens_beyond_the_router(orc):
    block = Block(orc, 65536)
    block.spec.always = None
    block.refused(UNS, T=65536)


@pytest.mark.parametrize("T", [1, 3, 70])
def test_rows_of_y_behind_the_last_token(orc, T):
    """y may hold more rows: those behind the last token stay as they were."""
    st, _, _ = layers(orc, 1, 64)
    h = torch.randn((T, H), device="cuda").bfloat16()
    y = torch.full((T + 3, H), 7.0, device="cuda")
    got = st.block(0, h.clone(), None, T, y=y)
    want = st.block(0, h.clone(), None, T)
    torch.cuda.synchronize()
    assert (y[T:] == 7).all() and tuple(got.shape) == (T, H)
    assert torch.equal(y[:T], want[:T]) and got.data_ptr() == y.data_ptr()


def test_bias_on_the_host(orc):
    """The routing kernels read the bias: it has to be on the Streamer's device."""
    st, _, _ = layers(orc, 1, 24)
    spec = st.layers[0]
    with pytest.raises(AssertionError):
        Streamer([LayerSpec(**{**spec.__dict__, "route_bias": spec.route_bias.cpu()})], 24, max_tokens=8)


def test_a_bias_lives_as_long_as_the_streamer(orc):
    """The native driver keeps the bias's address: a LayerSpec that is changed afterwards does not free it."""
    st, _, _ = layers(orc, 1, 24)
    bias = weakref.ref(st.layers[0].route_bias)
    st.layers[0].route_bias = None
    gc.collect()
    assert bias() is not None and bias().data_ptr() == st._ctx[0].route_bias


@pytest.mark.parametrize("T", [1, 3, 70])
@pytest.mark.parametrize("kw,ns", [(dict(k=31, bits=4), 2), (dict(k=4, bits=16), 0)])
def test_experts_that_cannot_run(kw, ns, T):
    """33 experts a token with the shared ones; BF16 experts whose width the tensor-core path does not take."""
    d = ops.desc(64, kw["k"], H, 96, 32, kw["bits"])
    bank = torch.zeros((64, ops.moe_slot_bytes(d)), dtype=torch.uint8).pin_memory()
    block = Block.__new__(Block)
    block.st = Streamer([LayerSpec(d, bank, list(range(64)), shared=bank[:ns] if ns else None,
                                   norm=torch.ones(H, dtype=torch.bfloat16, device="cuda"),
                                   router=torch.zeros((64, H), dtype=torch.bfloat16, device="cuda"))],
                        64, max_tokens=128, n_shared=ns)
    block.refused(UNS, T=T)


@pytest.mark.parametrize("route", [None, ops.route_config("sigmoid", 8, 4, 2)])
def test_more_shared_experts_than_the_routing_takes(route):
    d = ops.desc(64, 4, H, 128, 32, 4)
    bank = torch.zeros((64, ops.moe_slot_bytes(d)), dtype=torch.uint8).pin_memory()
    with pytest.raises(ops.MoeError) as ei:
        Streamer([LayerSpec(d, bank, list(range(64)), shared=bank[:9], route=route)], 64, max_tokens=8, n_shared=9)
    assert ei.value.status == INV
