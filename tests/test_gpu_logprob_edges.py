"""Log probabilities where their parts meet: large gradients beside masked logits,
through the C ABI.  Tolerances not derived here are those of the other tests of log
probabilities."""
import math

import pytest
import torch

import tests.test_gpu_logprob as base
from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

T32, I32, U, INF = base.T32, base.I32, base.U, math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sf.lib(build_if_needed=True)
    assert sf.device_error() == 0
    yield
    assert sf.device_error() == 0


# ------------------------------------------------------------------ masked logits and large gradients
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mask", [-INF, -3e38, -1e30])
@pytest.mark.parametrize("scale", [1.0, 1024.0])
def test_a_large_entropy_gradient_beside_masked_logits(scale, mask, dtype):
    """A masked logit has p = 0 and so a gradient of 0, however large dentropy is (a scaled loss)."""
    vocab, rows = 1000, 3
    z = base.logits(rows, vocab, 0, dtype, spread=0.5 / scale)
    z[:, 3:vocab:2] = mask
    tokens = torch.tensor([0, 2, -100], **I32)
    out = base.Rows(rows, 0)
    assert out.call(z, vocab, tokens, scale) == 0
    dl, de = torch.full((rows,), 1e4, **T32), torch.full((rows,), 1e6, **T32)
    dz = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    kind = sf.F32 if dtype == torch.float32 else sf.BF16
    assert sf.op_logprob_rows_bwd(z.data_ptr(), kind, z.shape[1], tokens.data_ptr(), rows, vocab, scale,
                                  out.lse.data_ptr(), out.entropy.data_ptr(), dl.data_ptr(), de.data_ptr(),
                                  dz.data_ptr(), vocab, stream=stream()) == 0
    sync()
    assert (dz[:, 3::2] == 0).all()
    ref, size, lp = base.gradient(z, vocab, tokens, scale, out.lse.double(), out.entropy.double(), dl.double(),
                                  de.double())
    base.near(dz, ref, base.BF * ref.abs() + (2.0 ** -20 + 4 * U * lp.abs()) * size + 1e-37)
