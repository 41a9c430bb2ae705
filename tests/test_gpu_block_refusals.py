"""What Streamer.block refuses leaves h (and y) as it was, so that the caller can correct
the call and make it again: arguments that only a later stage would refuse."""
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops
from streamed_quantized_expert_b200.runtime import Streamer
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
