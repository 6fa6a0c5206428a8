"""The training step with 8-bit sliding activations (offload_activations 2):
the forward as before, the recompute and backward of every layer but the last
three at the values of an int8 checkpoint.

Tolerance.  A checkpointed value is off by at most a/254, a the largest of its
128; for the Gaussian residuals here a is about 2.7 deviations, so the error is
uniform with 2.7 / 127 / sqrt(12) = 0.6% of a deviation, independent from value
to value.  It reaches a layer's gradients through the normed input, q/k/v, o,
the second norm's input and its output and the FFN's hidden: six operands, each
off by about as much, in quadrature 1.5%.  With the 1% that bf16 operands add
(the bar of the exact step is 2%), 2.5% in relative L2."""
import numpy as np
import pytest

import inputs
import oracle
from inputs import TEST_CONFIGS, UNIT_EMBED, UNIT_LM_HEAD
from tests.helpers import masters, oracle_weights
from tests.test_gpu_step import compare, make_model, sf

pytestmark = pytest.mark.gpu
TOL = 2.5e-2


@pytest.mark.parametrize("layers", [3, 5, 10])
@pytest.mark.parametrize("name", ["small-gqa", "small-hd128"])
def test_step_with_8bit_checkpoints_matches_oracle(name, layers):
    cfg = TEST_CONFIGS[name].with_(n_layers=layers)
    mast = masters(cfg)
    tok, lab = inputs.tokens_and_labels(cfg)
    loss_ref, g_ref = oracle.step(oracle_weights(cfg, mast), tok, lab, cfg)
    bytes_moved = {}
    for off in (0, 2):
        with make_model(cfg, mast, offload_activations=off) as m:
            assert m.train_step(tok, lab) == sf.SF_OK, m.error()
            if off:
                compare(cfg, m, loss_ref, g_ref, tol=TOL)
            st = m.stats()
            bytes_moved[off] = (st["h2d_bytes"], st["d2h_bytes"])
    # the checkpoints up to layer L - 8 went out and came back: codes (padded to
    # 256 bytes) and a scale for each 128 values
    T = cfg.batch * cfg.seq
    one = (T * cfg.hidden + 255) // 256 * 256 + T * ((cfg.hidden + 127) // 128) * 4
    for a, b in zip(bytes_moved[2], bytes_moved[0]):
        assert a - b == max(0, layers - 7) * one


def test_8bit_checkpoints_over_steps_and_update_modes():
    """Several steps of two shapes (the second smaller than the buffers): the same
    bits whether updates overlap the next step or not, and on a second run."""
    cfg = TEST_CONFIGS["small-gqa"].with_(n_layers=10)
    mast = masters(cfg)
    batches = [inputs.tokens_and_labels(cfg, seed=70 + i) for i in range(3)]
    batches[1] = tuple(x[:1, :77].copy() for x in batches[1])
    adam = sf.Adam(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    units = (0, 2, 6, 9, UNIT_EMBED, UNIT_LM_HEAD)
    out = []
    for asyn in (0, 1, 1):
        with make_model(cfg, mast, ring_slots=2, async_update=asyn, offload_activations=2) as m:
            losses = [m.step(t, l, adam) for t, l in batches]
            m.sync()
            out.append((losses, [m.grads(u) for u in units], [m.weights(u) for u in units]))
    for other in out[1:]:
        assert other[0] == out[0][0]
        for a, b in zip(out[0][1] + out[0][2], other[1] + other[2]):
            assert np.array_equal(a, b)
