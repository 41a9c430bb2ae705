"""Streamer.block takes tensors of its own device alone: an address of another
one would go to its kernels (stand-ins for tensors; no GPU)."""
from types import SimpleNamespace

import pytest
import torch

from streamed_quantized_expert_b200.runtime import LayerSpec, Streamer

H, E, T = 64, 8, 3
HERE, THERE = torch.device("cuda", 0), torch.device("cuda", 1)


class Tensor:
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, device=HERE):
        self.shape, self.dtype, self.device = shape, dtype, device

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        return 1 << 20


def fits(**other):
    """Streamer._block_fits with the named tensors on the other device."""
    at = lambda name: THERE if name in other else HERE  # noqa: E731
    bf = torch.bfloat16
    always = SimpleNamespace(H=H, device=at("always"))
    spec = LayerSpec(None, None, [], norm=Tensor(H, dtype=bf, device=at("norm")),
                     router=Tensor(E, H, dtype=bf, device=at("router")), always=always)
    st = SimpleNamespace(H=H, E=E, dev_err=Tensor(1, dtype=torch.int32))
    return Streamer._block_fits(st, spec, Tensor(T, H, dtype=bf, device=at("h")), Tensor(T, H, device=at("delta")), T,
                                Tensor(T, device=at("row_w")), Tensor(T, H, device=at("y")))


def test_one_device():
    assert fits()


@pytest.mark.parametrize("name", ["norm", "router", "h", "delta", "row_w", "y", "always"])
def test_another_device(name):
    assert not fits(**{name: True})
