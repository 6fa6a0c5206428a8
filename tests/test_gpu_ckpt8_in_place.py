"""sf_op_rmsnorm_bwd_load8 with its result over one of its inputs."""
import pytest
import torch

from tests.gpu_util import stream, sync
from tests.test_gpu_attention_half import EPS, F32T, ckpt_inputs

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")


@pytest.mark.parametrize("over", ["dres", "dy"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,d", [(9001, 384), (2001, 4096), (1001, 12288), (1001, 16384)])
def test_norm_backward_in_place(rows, d, fmt, over):
    """dx over the residual gradient, or over dy: the bits of the call with buffers
    of their own, several rows for each thread group."""
    x, g, dy, dres = ckpt_inputs(rows, d, seed=d)
    p = lambda t: t.data_ptr()
    q, s = torch.empty(rows, d, dtype=torch.uint8, device="cuda"), torch.empty(rows, (d + 127) // 128, **F32T)
    y, r = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, **F32T)
    assert sf.op_ckpt8_save(p(x), p(q), p(s), fmt, rows, d, stream()) == 0
    assert sf.op_rmsnorm_fwd_load8(p(q), p(s), p(g), p(y), p(r), 0, fmt, rows, d, EPS, stream()) == 0
    part = torch.empty(sf.rmsnorm_bwd_scratch(rows, d), **F32T)
    out = []
    for place in (False, True):
        a, b = dy.clone(), dres.clone()
        dx = (b if over == "dres" else a) if place else torch.empty_like(dy)
        dxb, dg = torch.empty_like(y), torch.empty_like(g)
        assert sf.op_rmsnorm_bwd_load8(p(q), p(s), p(g), p(r), p(a), p(b), p(dx), p(dxb), p(dg), p(part), fmt, rows,
                                       d, stream()) == 0
        sync()
        out.append((dx, dxb, dg))
    for a, b in zip(*out):
        assert torch.equal(a, b)
