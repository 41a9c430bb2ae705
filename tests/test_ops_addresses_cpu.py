"""Addresses and streams given to the bindings as plain numbers."""
import enum

import pytest

from streamed_quantized_expert_b200 import ops


class Address(enum.IntEnum):
    NONE = 0
    HERE = 4096


class Number(int):
    pass


@pytest.mark.parametrize("convert", [ops._ptr, ops._stream])
@pytest.mark.parametrize("value,want", [(None, None), (0, 0), (4096, 4096), (Address.HERE, 4096), (Address.NONE, 0),
                                        (Number(1 << 40), 1 << 40), (False, 0)])
def test_numbers(convert, value, want):
    assert convert(value) == want


def test_objects():
    class Tensor:
        def data_ptr(self):
            return 512

    class Stream:
        cuda_stream = 1024

    assert ops._ptr(Tensor()) == 512 and ops._stream(Stream()) == 1024
