"""The join's backward where its parts meet: gradients that are not finite, rows
shared by clusters over many turns, offsets beyond 2^31, other streams and captured
graphs, through the C ABI.  Tolerances are those of the join's other tests."""
import math

import pytest
import torch

import tests.test_gpu_join as join
from tests.dropout_reference import kept
from tests.gpu_util import stream, sync

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


@pytest.mark.parametrize("form", join.FORMS)
@pytest.mark.parametrize("rows,d", [(700, 3200), (700, 3208), (700, 3648), (700, 3656), (700, 4104), (700, 6152), (700, 8192),
                                    (700, 8200), (700, 12288), (500, 16384)])
def test_wide_rows_in_many_turns(rows, d, form):
    """Each CTA or cluster takes several rows: the ring's stages, both sets of sums and both barriers come again."""
    join.test_join_backward(rows, d, form)


def _backward_call(rows, d, form, seed):
    x, h, gains, dy, dres = join.join_inputs(rows, d, *form[:4], seed=seed)
    keep = join.dropped(form, (rows, d))
    xo, _, ro, rn, _ = join.forward64(x, h, gains, form, keep)
    fixed = (xo.float(), h, gains, form, ro.float(), rn.float(), dy, dres)
    scratch = torch.empty(sf.join_bwd_scratch(rows, d), **T32)
    out = [torch.empty_like(dy), torch.empty_like(h), *(torch.empty(d, **B16) for _ in range(3))]

    def call():
        assert join.call_bwd(*fixed, out[0], out[1], out[2:], scratch) == 0

    return call, out


@pytest.mark.parametrize("h32", [False, True])
@pytest.mark.parametrize("d", [2048, 12288, 16384])
def test_backward_on_two_streams(d, h32):
    form = (True, True, True, h32, 0.1, 1.0, 0.5)
    calls = [_backward_call(600, d, form, seed) for seed in (1, 2)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    sync()
    for _ in range(3):
        for (call, _), side in zip(calls, sides):
            with torch.cuda.stream(side):
                call()
    sync()
    for call, out in calls:
        first = [t.clone() for t in out]
        for t in out:
            t.fill_(7)
        call()
        sync()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("d", [4104, 12288, 16384])
def test_captured_backward_of_wide_rows(d):
    call, out = _backward_call(300, d, (True, True, True, False, 0.2, 1.0, 0.5), 3)
    call()
    sync()
    first = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in out:
            t.fill_(7)
        graph.replay()
        sync()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_backward_beyond_2_31_elements():
    rows, d, form = (1 << 28) + 3, 8, (True, True, True, False, 0.5, 1.0, 1.0)
    gains = [(1 + 0.25 * torch.randn(d, generator=torch.Generator().manual_seed(s))).to(**B16) for s in range(3)]
    xo, dy = torch.zeros(rows, d, **T32), torch.zeros(rows, d, **T32)
    h, dh = torch.zeros(rows, d, **B16), torch.empty(rows, d, **B16)
    n, rnd = 64, join.gen(1)
    xo[-n:], dy[-n:], h[-n:] = rnd(n, d), rnd(n, d), rnd(n, d).bfloat16()
    r1, r2 = torch.ones(rows, **T32), torch.ones(rows, **T32)
    ends = [t[-n:].double() for t in (xo, dy, h)]
    dgs, scratch = [torch.empty(d, **B16) for _ in range(3)], torch.empty(sf.join_bwd_scratch(rows, d), **T32)
    assert join.call_bwd(xo, h, gains, form, r1, r2, dy, None, dy, dh, dgs, scratch) == 0  # dx over dy
    sync()
    keep = torch.from_numpy(kept(n * d, 0.5, join.SEED, join.OFFSET, first=(rows - n) * d)).cuda().reshape(n, d)
    x, g, hh = ends
    w = g * gains[2].double()
    total = w - x * (w * x).mean(1, keepdim=True)
    size = w.abs() + x.abs() * (w * x).abs().mean(1, keepdim=True)
    join.within(dy[-n:], total, join.F32 * size)
    dv, sv = 2 * total * keep, 2 * size * keep
    wg = gains[0].double() * gains[1].double()
    q, sq = wg * dv, wg.abs() * sv
    q, sq = q - hh * (q * hh).mean(1, keepdim=True), sq + hh.abs() * (sq * hh.abs()).mean(1, keepdim=True)
    join.within(dh[-n:], q, join.BF * q.abs() + join.F32 * sq)
    assert (dy[:-n] == 0).all() and (dh[:-n] == 0).all()
    # the other rows add zeros, which change no sum: chains of at most n terms
    for got, ref, s in ((dgs[2], (g * x).sum(0), (g * x).abs().sum(0)),
                        (dgs[0], gains[1].double() * (dv * hh).sum(0), gains[1].double().abs() * (sv * hh.abs()).sum(0)),
                        (dgs[1], gains[0].double() * (dv * hh).sum(0), gains[0].double().abs() * (sv * hh.abs()).sum(0))):
        join.within(got, ref, join.BF * ref.abs() + join.F32 * s)
