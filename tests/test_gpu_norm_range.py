"""moe_add_norm_quant where the squares, or their sum, leave the range of fp32:
large rows up to the 1e18 that the header allows, at every length and way a row
is held.  Tolerances as for rows of ordinary size (tests/test_gpu_row_quant.py):
(H / 512 + 16) half steps of fp32 for the scale and for x, which is rounded to
bf16 besides; a power of two that the row is taken times adds nothing."""
import numpy as np
import pytest

from streamed_quantized_expert_b200 import build, ops
from tests import _ref64 as ref
from tests.test_gpu_row_quant import close, draw, norm

import torch  # noqa: F401  (the library's tensors)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def compare(h, hf, delta, df, gamma, eps=1e-6, **kw):
    H = h.shape[1]
    ho, x, q, s = norm(h, hf, delta, df, gamma, eps, **kw)
    rh, rx, p, r = ref.add_norm(h, hf, delta, gamma, eps)
    rq, a, _ = ref.codes(p)
    if ho is not None:
        assert np.array_equal(ho, rh)
    assert np.array_equal(q, rq)
    close(x, rx, ref.UBF + (H / 512 + 16) * ref.U32)
    close(s, a * r / 127.0, (H / 512 + 16) * ref.U32)


@pytest.mark.parametrize("hf", [False, True])
@pytest.mark.parametrize("H", [256, 512, 520, 2048, 4096, 16384, 16392, 65536])
def test_large_rows(H, hf):
    r = np.random.default_rng(H)
    gamma = ref.round_to(1.0 + draw(2, 1, H, True)[0], False)
    size = np.array([0.99e18, 5e17, 7e16, 1.0], np.float32)[:, None]  # the last one of ordinary size
    h = ref.round_to(size * (0.5 + 0.5 * r.random((4, H))).astype(np.float32) * r.choice([-1, 1], (4, H)), hf)
    compare(h, hf, None, False, gamma)
    # as a sum, written over h or nowhere
    delta = ref.round_to(h * np.float32(0.25), True)
    for kw in (dict(in_place=True), dict(want_h=False), dict()):
        compare(ref.round_to(h * np.float32(0.75), hf), hf, delta, True, gamma, **kw)


@pytest.mark.parametrize("hf", [False, True])
def test_large_and_not_finite(hf):
    """An infinity or a NaN next to large values shows as before."""
    H = 4096
    h = ref.round_to(np.full((3, H), 5e17, np.float32), hf)
    h[0, 7], h[1, 9] = np.inf, np.nan
    _, x, q, s = norm(h, hf, None, False, np.ones(H, np.float32))
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all()
    assert np.isnan(x[1]).all() and np.isnan(x[0, 7]) and (np.delete(x[0], 7) == 0).all()
    assert np.all(np.abs(x[2] - 1.0) <= ref.UBF + 24 * ref.U32)
