"""The join's backward where its parts meet: gradients that are not finite, through
the C ABI."""
import math

import pytest
import torch

import tests.test_gpu_join as join
from tests.gpu_util import sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

T32 = dict(dtype=torch.float32, device="cuda")
B16 = dict(dtype=torch.bfloat16, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sf.lib(build_if_needed=True)
    assert sf.device_error() == 0
    yield
    assert sf.device_error() == 0


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("nxt", [True, False])
@pytest.mark.parametrize("h32", [False, True])
@pytest.mark.parametrize("d", [136, 4096, 12288])
def test_a_gradient_that_is_not_finite_stays_with_its_dropped_element(d, h32, nxt, value):
    """dropout's gradient is 0 where the element was dropped, whatever comes back: dh is that of a zero there."""
    rows, form = 5, (True, True, nxt, h32, 0.4, 1.0, 0.5)
    x, h, gains, dy, dres = join.join_inputs(rows, d, *form[:4])
    keep = join.dropped(form, (rows, d))
    xo, _, ro, rn, _ = join.forward64(x, h, gains, form, keep)
    xo, r1, r2 = xo.float(), ro.float(), rn.float() if nxt else None
    at = [int((~keep[r]).nonzero()[r]) for r in range(rows)]
    results = []
    for there in (0.0, value):
        res = dres.clone()
        for r in range(rows):
            res[r, at[r]] = there
        dx, dh = torch.empty_like(dy), torch.empty_like(h)
        dgs = [torch.zeros(d, **B16) if g is not None else None for g in gains]
        scratch = torch.empty(sf.join_bwd_scratch(rows, d), **T32)
        assert join.call_bwd(xo, h, gains, form, r1, r2, dy if nxt else None, res, dx, dh, dgs, scratch) == 0
        sync()
        results.append((dx, dh, dgs))
    (dx0, dh0, dgs0), (dx1, dh1, dgs1) = results
    # D of the dropped element differs, and nothing else: dh and the gains' gradients see it times 0
    if nxt:
        assert torch.isfinite(dh0.float()).all()
    assert torch.equal(dh0, dh1)
    assert all(torch.equal(a, b) for a, b in zip(dgs0, dgs1) if a is not None)
    other = torch.ones(rows, d, dtype=torch.bool, device="cuda")
    for r in range(rows):
        other[r, at[r]] = False
    assert torch.equal(dx0[other], dx1[other]) and not torch.isfinite(dx1[~other]).any()
