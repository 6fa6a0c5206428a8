"""What 8-bit checkpoints leave as it was, bit for bit: the norm's outputs, the
step's loss, the gradients behind the first layer that is recomputed from codes."""
import numpy as np
import pytest
import torch

import inputs
import oracle
from inputs import TEST_CONFIGS, UNIT_FINAL_NORM, UNIT_LM_HEAD
from tests.gpu_util import stream, sync
from tests.helpers import masters, oracle_weights
from tests.test_gpu_attention_half import EPS, F32T, ckpt_inputs
from tests.test_gpu_ckpt8_step import TOL
from tests.test_gpu_step import compare, make_model, sf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,d", [(1, 8), (900, 384), (900, 512), (700, 520), (700, 1024), (500, 1032), (500, 2048),
                                    (300, 2056), (300, 4096), (300, 6152), (200, 8192), (200, 12288), (200, 16384)])
def test_saving_norm_is_the_norm(rows, d, fmt):
    """sf_op_rmsnorm_fwd_save8's y and rstd are sf_op_rmsnorm_fwd's."""
    x, g, _, _ = ckpt_inputs(rows, d, seed=d)
    nb, p = (d + 127) // 128, lambda t: t.data_ptr()
    y, r = [[torch.empty(*s, dtype=t, device="cuda") for _ in range(2)]
            for s, t in (((rows, d), torch.bfloat16), ((rows,), torch.float32))]
    q, s = torch.empty(rows, d, dtype=torch.uint8, device="cuda"), torch.empty(rows, nb, **F32T)
    assert sf.op_rmsnorm_fwd(p(x), p(g), p(y[0]), p(r[0]), rows, d, EPS, stream()) == 0
    assert sf.op_rmsnorm_fwd_save8(p(x), p(g), p(y[1]), p(r[1]), p(q), p(s), fmt, rows, d, EPS, stream()) == 0
    sync()
    assert torch.equal(r[0], r[1]) and torch.equal(y[0], y[1])


@pytest.mark.parametrize("fp16", [0, 1])
@pytest.mark.parametrize("name", ["small-gqa", "small-hd128"])
def test_8bit_activations_leave_the_forward_as_it_was(name, fp16):
    """The same loss and the same gradients of the last three layers, whose
    inputs stay in fp32; the others within the step's tolerance, with bf16 and
    with scaled fp16 gradients."""
    cfg = TEST_CONFIGS[name].with_(n_layers=9)
    mast = masters(cfg)
    tok, lab = inputs.tokens_and_labels(cfg)
    loss_ref, g_ref = oracle.step(oracle_weights(cfg, mast), tok, lab, cfg)
    out = []
    for off in (0, 1, 2):
        with make_model(cfg, mast, offload_activations=off, fp16_grads=fp16) as m:
            assert m.train_step(tok, lab) == sf.SF_OK, m.error()
            out.append([np.float64(m.loss())] + [m.grads(u) for u in (6, 7, 8, UNIT_FINAL_NORM, UNIT_LM_HEAD)])
            if off == 2:
                compare(cfg, m, loss_ref, g_ref, tol=TOL)
    for other in out[1:]:
        for a, b in zip(out[0], other):
            assert np.array_equal(a, b)
