"""Dropout and the join of a block's output with the residual stream, through
the C ABI, element by element against their definitions in 64 bits.

Tolerances.  A value stored in bf16 is off by at most 2^-8 of itself (half a
step).  What the kernels compute in fp32 before that is off by a few 2^-24 of
the magnitudes that are added; F32 = 2^-18 of their sum covers the longest
chains (a row of 16,384: partial sums of 32 a thread, then trees; a gain's
sum: rows of a CTA one after another, up to about 60 here, then trees)."""
import math

import numpy as np
import pytest
import torch

from tests.dropout_reference import kept, threshold
from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

BF, F32 = 2.0 ** -8, 2.0 ** -18
EPS = 1e-5
T32 = dict(dtype=torch.float32, device="cuda")
SEED, OFFSET = 0x0123456789ABCDEF, (7 << 32) + 11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sf.lib(build_if_needed=True)
    assert sf.device_error() == 0
    yield
    assert sf.device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, **T32)


def guarded(shape, dtype, tail=64):
    """A buffer of that shape followed by `tail` elements that must stay as they are."""
    n = math.prod(shape)
    flat = torch.full((n + tail,), 7, dtype=dtype, device="cuda")
    return flat[:n].view(*shape), flat[n:]


def within(got, ref, tol):
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    assert over.max().item() <= 0.0, (over.max().item(), int(over.argmax()))


def mask(shape, p, seed=SEED, offset=OFFSET):
    return torch.from_numpy(kept(math.prod(shape), p, seed, offset)).cuda().reshape(shape)


def factor(p):
    return 65536.0 / (65536.0 - threshold(p))


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,p", [(1, 0.5), (7, 0.1), (8, 0.9), (9, 0.3), (2047, 0.1), (2048, 0.0), (2049, 0.99998),
                                 (100003, 0.25), (1 << 20, 0.1)])
def test_dropout(dtype, n, p):
    x = gen(n)(n).to(dtype)
    y, tail = guarded((n,), dtype)
    kind = sf.BF16 if dtype == torch.bfloat16 else sf.F32
    assert sf.op_dropout(x.data_ptr(), y.data_ptr(), kind, n, p, SEED, OFFSET, stream=stream()) == 0
    sync()
    keep = mask((n,), p)
    ref = torch.where(keep, x.double() * factor(p), torch.zeros_like(x, dtype=torch.float64))
    # one fp32 product with a rounded factor, then one rounding
    within(y, ref, ref.abs() * (BF + 2.0 ** -22 if dtype == torch.bfloat16 else 2.0 ** -22))
    assert (y[~keep] == 0).all() and (tail == 7).all()
    assert sf.op_dropout(x.data_ptr(), x.data_ptr(), kind, n, p, SEED, OFFSET, stream=stream()) == 0
    sync()
    assert torch.equal(x, y)  # in place


def test_dropout_drops_what_is_not_finite():
    x = torch.full((4096,), math.nan, **T32)
    x[::2] = math.inf
    y = torch.empty_like(x)
    assert sf.op_dropout(x.data_ptr(), y.data_ptr(), sf.F32, 4096, 0.5, SEED, OFFSET, stream=stream()) == 0
    sync()
    keep = mask((4096,), 0.5)
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


def test_dropout_of_more_than_2_32_elements():
    n = (1 << 32) + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    assert sf.op_dropout(x.data_ptr(), x.data_ptr(), sf.BF16, n, 0.5, SEED, OFFSET, stream=stream()) == 0
    sync()
    for first in (0, (1 << 31) - 4096, (1 << 32) - 4096, (1 << 32)):
        count = min(8192, n - first)
        keep = torch.from_numpy(kept(count, 0.5, SEED, OFFSET, first=first)).cuda()
        assert torch.equal(x[first:first + count], keep.bfloat16() * 2)


def test_dropout_offset_wraps_with_the_step():
    x = torch.ones(4096, **T32)
    y = torch.empty_like(x)
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    last = 2 ** 64 - 2
    assert sf.op_dropout(x.data_ptr(), y.data_ptr(), sf.F32, 4096, 0.5, SEED, last, step=step.data_ptr(),
                         stream=stream()) == 0
    sync()
    assert torch.equal(y != 0, mask((4096,), 0.5, offset=3))


# ------------------------------------------------------------------ the join
SIZES = [(1, 8), (9, 8), (3, 24), (5, 384), (300, 512), (37, 520), (8, 1000), (9, 1032), (21, 2048), (700, 2056),
         (33, 4096), (10, 4104), (11, 8200), (6, 12288), (5, 12296), (200, 16384)]
FORMS = [  # post, gate, next, h fp32, p, alpha, beta
    (True, True, True, False, 0.1, 1.0, 0.22),
    (True, False, True, False, 0.0, 0.8, 1.0),
    (False, True, True, True, 0.3, 1.0, 1.0),
    (False, False, False, False, 0.5, 1.0, 1.0),
    (True, True, False, True, 0.05, -0.5, 2.0),
    (False, False, True, False, 0.0, 1.0, 0.0),
]


def join_inputs(rows, d, post, gate, nxt, h32, seed=3):
    rnd = gen(seed)
    x, h = 2 * rnd(rows, d), 0.5 * rnd(rows, d)
    x[:, d // 2] *= 30
    if rows > 2:
        h[1] = 0  # a block that answers nothing
    if not h32:
        h = h.bfloat16()
    gains = [(1 + 0.3 * rnd(d)).bfloat16() if there else None for there in (post, gate, nxt)]
    return x, h, gains, rnd(rows, d), rnd(rows, d)


def ptr(t):
    return t.data_ptr() if t is not None else 0


def kind(h32):
    return sf.F32 if h32 else sf.BF16


def call_fwd(x, h, gains, form, xout, y, r1, r2, p=None, **kw):
    post, gate, nxt, h32, p0, alpha, beta = form
    rows, d = x.shape
    return sf.op_join_fwd(ptr(x), ptr(h), kind(h32), *map(ptr, gains), alpha, beta, p0 if p is None else p, SEED,
                          OFFSET, ptr(xout), ptr(y), ptr(r1), ptr(r2), rows, d, EPS, stream=stream(), **kw)


def call_bwd(xout, h, gains, form, r1, r2, dy, dres, dx, dh, dgs, scratch, **kw):
    post, gate, nxt, h32, p, alpha, beta = form
    rows, d = xout.shape
    return sf.op_join_bwd(ptr(xout), ptr(h), kind(h32), *map(ptr, gains), alpha, beta, p, SEED, OFFSET, ptr(r1),
                          ptr(r2), ptr(dy), ptr(dres), ptr(dx), ptr(dh), *map(ptr, dgs), ptr(scratch), rows, d,
                          stream=stream(), **kw)


def forward64(x, h, gains, form, keep):
    """(xout, y, rstd_post, rstd_next), and the magnitudes that xout adds."""
    post, gate, nxt, h32, p, alpha, beta = form
    u, r1, r2, y = h.double(), None, None, None
    if post:
        r1 = 1 / torch.sqrt((u ** 2).mean(1) + EPS)
        u = u * r1[:, None] * gains[0].double()
    if gate:
        u = u * gains[1].double()
    v = torch.where(keep, u * factor(p), torch.zeros_like(u))
    xo = alpha * x.double() + beta * v
    size = (alpha * x.double()).abs() + (beta * v).abs()
    if nxt:
        r2 = 1 / torch.sqrt((xo ** 2).mean(1) + EPS)
        y = xo * r2[:, None] * gains[2].double()
    return xo, y, r1, r2, size


def dropped(form, shape):
    return mask(shape, form[4]) if threshold(form[4]) else torch.ones(shape, dtype=torch.bool, device="cuda")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,d", SIZES)
def test_join_forward(rows, d, form):
    post, gate, nxt, h32 = form[:4]
    x, h, gains, _, _ = join_inputs(rows, d, post, gate, nxt, h32)
    xout, t0 = guarded((rows, d), torch.float32)
    y, t1 = guarded((rows, d), torch.bfloat16)
    r1, t2 = guarded((rows,), torch.float32)
    r2, t3 = guarded((rows,), torch.float32)
    assert call_fwd(x, h, gains, form, xout, y if nxt else None, r1 if post else None, r2 if nxt else None) == 0
    sync()
    xo, yo, ro, rn, size = forward64(x, h, gains, form, dropped(form, (rows, d)))
    within(xout, xo, F32 * size)
    if post:
        within(r1, ro, F32 * ro)
    if nxt:
        within(r2, rn, F32 * rn)
        within(y, yo, BF * yo.abs() + F32 * size * (rn[:, None] * gains[2].double()).abs() + F32 * yo.abs())
    for t in (t0, t1, t2, t3):
        assert (t == 7).all()
    again = x.clone()  # in place
    assert call_fwd(again, h, gains, form, again, y if nxt else None, r1 if post else None, r2 if nxt else None) == 0
    sync()
    assert torch.equal(again, xout)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,d", SIZES + [(5003, 64), (9000, 136)])
def test_join_backward(rows, d, form):
    post, gate, nxt, h32, p, alpha, beta = form
    x, h, gains, dy, dres = join_inputs(rows, d, post, gate, nxt, h32)
    keep = dropped(form, (rows, d))
    xo, _, ro, rn, _ = forward64(x, h, gains, form, keep)
    xo, r1, r2 = xo.float(), ro.float() if post else None, rn.float() if nxt else None
    dx, t0 = guarded((rows, d), torch.float32)
    dh, t1 = guarded((rows, d), h.dtype)
    dgs = [guarded((d,), torch.bfloat16) for _ in range(3)]
    scratch, t2 = guarded((sf.join_bwd_scratch(rows, d),), torch.float32)
    given = [g if there else None for (g, _), there in zip(dgs, (post, gate, nxt))]
    for use_res in ((True, False) if nxt else (True,)):
        res = dres if use_res else None
        assert call_bwd(xo, h, gains, form, r1, r2, dy if nxt else None, res, dx, dh, given, scratch) == 0
        sync()
        # the formulas in 64 bits, from the saved row statistics
        total = dres.double() if use_res else torch.zeros_like(dy, dtype=torch.float64)
        size, bf = total.abs(), BF if not h32 else 0.0
        if nxt:
            r = r2.double()[:, None]
            u, w = xo.double() * r, dy.double() * gains[2].double()
            total = total + r * (w - u * (w * u).mean(1, keepdim=True))
            size = size + r * (w.abs() + u.abs() * (w * u).abs().mean(1, keepdim=True))
            g = (dy.double() * u).sum(0)
            within(given[2], g, BF * g.abs() + F32 * (dy.double() * u).abs().sum(0))
        within(dx, alpha * total, abs(alpha) * F32 * size)
        scale = abs(beta) * factor(p)
        dv, sv = beta * factor(p) * total * keep, scale * size * keep
        r = r1.double()[:, None] if post else 1.0
        u, w = h.double() * r, torch.ones(d, dtype=torch.float64, device="cuda")
        a, sa = (dv * u).sum(0), (sv * u.abs()).sum(0)
        if post:
            w = w * gains[0].double()
            g = a * (gains[1].double() if gate else 1.0)
            within(given[0], g, BF * g.abs() + F32 * sa * (gains[1].double().abs() if gate else 1.0))
        if gate:
            w = w * gains[1].double()
            g = a * (gains[0].double() if post else 1.0)
            within(given[1], g, BF * g.abs() + F32 * sa * (gains[0].double().abs() if post else 1.0))
        q, sq = w * dv, w.abs() * sv
        if post:
            q, sq = r * (q - u * (q * u).mean(1, keepdim=True)), \
                r * (sq + u.abs() * (sq * u.abs()).mean(1, keepdim=True))
        within(dh, q, bf * q.abs() + F32 * sq)
        for (g, t), there in zip(dgs, (post, gate, nxt)):
            assert (t == 7).all() and (there or (g == 7).all())
        for t in (t0, t1, t2):
            assert (t == 7).all()
    first = [t.clone() for t in (dx, dh, *(g for g in given if g is not None))]
    if nxt:  # over dy, the same bits again
        assert call_bwd(xo, h, gains, form, r1, r2, dy, None, dy, dh, given, scratch) == 0
    else:
        assert call_bwd(xo, h, gains, form, r1, r2, None, dres, dres, dh, given, scratch) == 0
    sync()
    for got, want in zip((dy if nxt else dres, dh, *(g for g in given if g is not None)), first):
        assert torch.equal(got, want)


def test_join_backward_over_the_residual_gradient():
    form = FORMS[0]
    x, h, gains, dy, dres = join_inputs(50, 4096, *form[:4])
    keep = dropped(form, (50, 4096))
    xo, _, ro, rn, _ = forward64(x, h, gains, form, keep)
    xo, r1, r2 = xo.float(), ro.float(), rn.float()
    dgs = [torch.empty(4096, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    scratch = torch.empty(sf.join_bwd_scratch(50, 4096), **T32)
    dx, dh, dh2 = torch.empty_like(dy), torch.empty_like(h), torch.empty_like(h)
    assert call_bwd(xo, h, gains, form, r1, r2, dy, dres, dx, dh, dgs, scratch) == 0
    assert call_bwd(xo, h, gains, form, r1, r2, dy, dres, dres, dh2, dgs, scratch) == 0
    sync()
    assert torch.equal(dx, dres) and torch.equal(dh, dh2)


@pytest.mark.parametrize("form", FORMS)
def test_join_gradient_against_autograd_and_differences(form):
    """The formulas that the kernel is held to, against autograd and central
    differences of the 64-bit forward; and the kernel's bits against them."""
    rows, d = 6, 136
    post, gate, nxt, h32, p, alpha, beta = form
    x, h, gains, dy, dres = join_inputs(rows, d, post, gate, nxt, h32)
    keep = dropped(form, (rows, d))
    leaves = [t.double().requires_grad_() for t in (x, h, *(g for g in gains if g is not None))]

    def loss(x, h, *gs):
        it = iter(gs)
        full = [next(it) if there else None for there in (post, gate, nxt)]
        xo, y, _, _, _ = forward64(x, h, full, form, keep)
        return (xo * dres.double()).sum() + ((y * dy.double()).sum() if nxt else 0.0)

    grads = torch.autograd.grad(loss(*leaves), leaves)
    g = torch.Generator().manual_seed(5)
    for i, (leaf, grad) in enumerate(zip(leaves, grads)):
        way = torch.randn(leaf.shape, generator=g, dtype=torch.float64).cuda()
        if i == 1 and post:
            way[1] = 0  # the row of zeros bends too sharply for a step
        e = 1e-5
        up, down = ([t.detach() + (s * e * way if j == i else 0) for j, t in enumerate(leaves)] for s in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * e)
        # second-order error e^2 times third derivatives (at most about 1e3 here), rounding 1e-16 / e
        assert abs((diff - (grad * way).sum()).item()) <= 1e-6 * (1 + (grad * way).abs().sum().item())
    xo, _, ro, rn, _ = forward64(x, h, gains, form, keep)
    dx, dh = torch.empty_like(dy), torch.empty_like(h)
    dgs = [torch.empty(d, dtype=torch.bfloat16, device="cuda") if there else None for there in (post, gate, nxt)]
    scratch = torch.empty(sf.join_bwd_scratch(rows, d), **T32)
    assert call_bwd(xo.float(), h, gains, form, ro.float() if post else None, rn.float() if nxt else None,
                    dy if nxt else None, dres, dx, dh, dgs, scratch) == 0
    sync()
    for got, want in zip((dx, dh, *(g for g in dgs if g is not None)), grads):
        norm = want.norm().item()
        assert (got.double() - want).norm().item() <= BF * norm + 1e-30


def test_join_of_many_rows():
    """More rows than a launch's blocks stride over at once, narrow: offsets beyond 2^31 elements."""
    rows, d = (1 << 28) + 3, 8
    form = (True, False, True, False, 0.5, 1.0, 1.0)
    h = torch.ones(rows, d, dtype=torch.bfloat16, device="cuda")
    h[-1] = 2
    x = torch.zeros(rows, d, **T32)
    gains = [torch.ones(d, dtype=torch.bfloat16, device="cuda"), None, torch.ones(d, dtype=torch.bfloat16, device="cuda")]
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    r1, r2 = torch.empty(rows, **T32), torch.empty(rows, **T32)
    assert call_fwd(x, h, gains, form, x, y, r1, r2) == 0
    sync()
    keep = torch.from_numpy(kept(64, 0.5, SEED, OFFSET, first=rows * d - 64)).cuda().reshape(8, 8)
    assert torch.equal(x[-8:] != 0, keep)
    within(r1[-1:], torch.tensor([1 / math.sqrt(4 + EPS)], dtype=torch.float64, device="cuda"), 1e-6)


def test_join_on_two_streams():
    form = FORMS[0]
    results = []
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    data = [join_inputs(400, 2048, *form[:4], seed=s) for s in (1, 2)]
    sync()
    for (x, h, gains, _, _), side in zip(data, sides):
        with torch.cuda.stream(side):
            out = [torch.empty_like(x), torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"),
                   torch.empty(400, **T32), torch.empty(400, **T32)]
            assert call_fwd(x, h, gains, form, *out) == 0
            results.append(out)
    sync()
    for (x, h, gains, _, _), out in zip(data, results):
        again = [torch.empty_like(t) for t in out]
        assert call_fwd(x, h, gains, form, *again) == 0
        sync()
        assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_join_captured_with_a_step_draws_new_masks():
    """A captured forward and backward replayed with another step: other masks, the same in both."""
    rows, d, form = 64, 1024, (True, True, True, False, 0.4, 1.0, 1.0)
    x, h, gains, dy, dres = join_inputs(rows, d, *form[:4])
    x.zero_()
    xout, y = torch.empty_like(x), torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    r1, r2 = torch.empty(rows, **T32), torch.empty(rows, **T32)
    dx, dh = torch.empty_like(x), torch.empty_like(h)
    dgs = [torch.empty(d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    scratch = torch.empty(sf.join_bwd_scratch(rows, d), **T32)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def both():
        assert call_fwd(x, h, gains, form, xout, y, r1, r2, step=step.data_ptr()) == 0
        assert call_bwd(xout, h, gains, form, r1, r2, dy, dres, dx, dh, dgs, scratch, step=step.data_ptr()) == 0

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    seen = []
    for s in (0, 1, 1 << 40):
        step.fill_(s)
        graph.replay()
        sync()
        keep = mask((rows, d), 0.4, offset=OFFSET + s)
        assert torch.equal(xout != 0, keep & (h != 0))
        seen.append([t.clone() for t in (xout, y, dx, dh, *dgs)])
        both()
        sync()
        assert all(torch.equal(a, b) for a, b in zip(seen[-1], (xout, y, dx, dh, *dgs)))
    assert not torch.equal(seen[0][0], seen[1][0])
