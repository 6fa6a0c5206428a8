"""8-bit sliding activations with micro-batches and with the model variants."""
import numpy as np
import pytest

import inputs
import oracle
from inputs import IGNORE_INDEX, TEST_CONFIGS
from inputs.configs import layer_tensor_shapes
from tests.helpers import masters, oracle_weights, rel_l2
from tests.test_gpu_ckpt8_step import TOL
from tests.test_gpu_step import make_model, sf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,variant", [("small-gqa", {}), ("small-qwen", dict(qkv_bias=True, tie_embeddings=True))])
def test_micro_batches_with_8bit_checkpoints(name, variant):
    """Three micro-batches whose checkpoints share the four code buffers and the
    pinned copies.  The loss and the summed gradients of the layers that keep
    fp32 inputs have the bits of the step with resident checkpoints, however far
    that is from the oracle (a key bias's gradient is a sum that nearly cancels);
    those of the layers recomputed from codes are within the step's tolerance."""
    cfg = TEST_CONFIGS[name].with_(n_layers=9, batch=3, **variant)
    mast = masters(cfg)
    tok, lab = inputs.tokens_and_labels(cfg)
    lab = lab.copy()
    lab[0, :37] = IGNORE_INDEX  # micro-batches with different valid counts
    _, g_ref = oracle.step(oracle_weights(cfg, mast), tok, lab, cfg)
    out = []
    for off in (0, 2):
        with make_model(cfg.with_(batch=1), mast, offload_activations=off) as m:
            assert m.train_step_accum(tok[:, None, :], lab[:, None, :]) == sf.SF_OK, m.error()
            out.append((m.loss(), [m.grads(l) for l in range(cfg.n_layers)]))
    (loss0, g0), (loss2, g2) = out
    assert loss0 == loss2
    for l in range(cfg.n_layers):
        if l >= cfg.n_layers - 3:
            assert np.array_equal(g0[l], g2[l]), l
            continue
        off = 0
        for tensor, shape in layer_tensor_shapes(cfg):
            n = int(np.prod(shape))
            assert rel_l2(g2[l][off:off + n].reshape(shape), g_ref["layers"][l][tensor]) <= TOL, (l, tensor)
            off += n
