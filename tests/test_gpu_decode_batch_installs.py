"""Decode layers of several tokens with misses, on the tensor-core grouped
GEMM (sorted x): the layer runs as two passes, the resident experts' and the
installed ones', whose lists interleave in expert id; each pass adds its own
experts' outputs only."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops, synth
from streamed_quantized_expert_b200.runtime import LayerSpec, Streamer
from tests._bank import assert_close, oracle_bank

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T", [12, 40, 64])
def test_batched_decode_with_interleaved_installs(orc, T):
    E, k, H, I, g = 64, 4, 256, 128, 32
    bank = oracle_bank(orc, E, H, I, g, 4, 4, seed=3)
    spec = LayerSpec(ops.desc(E, k, H, I, g, 4, 4), torch.from_numpy(bank).pin_memory(), list(range(E)))
    st = Streamer([spec], 40, max_tokens=64)
    assert st.uses_tc(0, T)
    st.place(0, list(range(0, E, 2)) + [1])  # every second expert resident
    slots = [bank[e] for e in range(E)]
    rng = np.random.default_rng(T)
    for step in range(5):
        x = synth.activations(0, 0, T, H, step=step)
        # all tokens choose among 36 experts, half of them resident at first
        logits = rng.standard_normal((T, E)).astype(np.float32)
        out = rng.choice(E, E - 36, replace=False)
        logits[:, out] -= 20.0
        y = st.decode_layer(0, dev(x.view(np.int16)), dev(logits), T)
        torch.cuda.synchronize()
        ids, w, _ = orc.route(logits, k)
        assert np.array_equal(st.ids[:T].cpu().numpy(), ids)
        assert_close(y.cpu().numpy(), orc.expert_ffn(x, H, I, g, 4, 4, ids, w, slots))
    assert st.check_dev_err() == 0 and st.installs > 10
