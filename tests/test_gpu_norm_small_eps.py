"""moe_add_norm_quant with an eps so small that squares below fp32's range
count next to it.  Tolerances as in tests/test_gpu_norm_range.py."""
import numpy as np
import pytest

from streamed_quantized_expert_b200 import build, ops
from tests import _ref64 as ref
from tests.test_gpu_norm_range import compare
from tests.test_gpu_row_quant import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


@pytest.mark.parametrize("eps", [1e-6, 1e-20, 1e-32, 1e-38, 1e-42])
@pytest.mark.parametrize("hf", [False, True])
@pytest.mark.parametrize("H", [256, 520, 4096, 16392])
def test_small_rows(H, hf, eps):
    gamma = ref.round_to(1.0 + draw(2, 1, H, True)[0], False)
    size = np.array([1e-10, 1e-16, 1e-19, 1e-21, 1e-22, 0.0], np.float32)[:, None]
    h = ref.round_to(size * draw(H, 6, H, True), hf)
    compare(h, hf, None, False, gamma, eps)
    compare(ref.round_to(h * np.float32(0.5), hf), hf, ref.round_to(h * np.float32(0.5), False), False, gamma, eps,
            in_place=True)
