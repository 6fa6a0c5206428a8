"""The operators around a decoder layer's attention, through the C ABI: norms
of queries and keys with the rotation, attention with a sliding window and
sinks, and 8-bit checkpoints with the norms that write and read them.  Each is
compared element by element with its definition in 64 bits on the same inputs.

Tolerances.  A value stored in bf16 is off by at most 2^-8 of itself (half a
step).  What the kernels compute in fp32 before that rounding is off by a few
2^-24 of the magnitudes that were added; F32 = 2^-18 of their sum covers the
longest chains here (a row of 16,384: partial sums of 64 per thread, then
trees).  The attention rounds P and dS to bf16 for the tensor core, which adds
2^-8 of the sum of the magnitudes that they multiply; SC = 2^-11 covers what
the fp32 scores (128 products) and the exponentials add to P."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

BF = 2.0 ** -8
F32 = 2.0 ** -18
SC = 2.0 ** -11
EPS = 1e-5
D64 = dict(dtype=torch.float64, device="cuda")
F32T = dict(dtype=torch.float32, device="cuda")  # another test module changes the default type


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sf.lib(build_if_needed=True)
    assert sf.device_error() == 0
    yield
    assert sf.device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, **F32T)


def within(got, ref, tol):
    """Every element within its tolerance (and finite)."""
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    assert over.max().item() <= 0.0, (over.max().item(), int(over.argmax()))


def guarded(shape, dtype, tail=256):
    """A buffer of that shape followed by `tail` elements that must stay as they are."""
    n = math.prod(shape)
    flat = torch.full((n + tail,), 7, dtype=dtype, device="cuda")
    return flat[:n].view(*shape), flat[n:]


def untouched(*tails):
    for t in tails:
        assert (t == 7).all()


def table(seq, hd, base=10000.0):
    return torch.from_numpy(sf.rope_table(seq, hd, base)).cuda()


def rotate(z, cos, sin):
    h = z.shape[-1] // 2
    return torch.cat([z[..., :h] * cos - z[..., h:] * sin, z[..., h:] * cos + z[..., :h] * sin], -1)


# ------------------------------------------------------------------ query/key norms
def qk_inputs(T, Hq, Hkv, hd, pad=0, seed=1):
    rnd = gen(seed)
    W = (Hq + 2 * Hkv) * hd
    x = torch.full((T, W + pad), 3.0, device="cuda", dtype=torch.bfloat16)
    x[:, :W] = rnd(T, W) * torch.exp(rnd(Hq + 2 * Hkv)).repeat_interleave(hd)
    gq, gk = (1 + 0.3 * rnd(hd)).bfloat16(), (1 + 0.3 * rnd(hd)).bfloat16()
    dy = torch.full((T, W + pad), 5.0, device="cuda", dtype=torch.bfloat16)
    dy[:, :W] = rnd(T, W)
    return x, gq, gk, dy, W


def qk_ref(x, gq, gk, dy, Hq, Hkv, hd, pos, tab, eps=EPS):
    """y, dx, dgq, dgk of the query and key heads in float64, and their tolerances."""
    n = (Hq + Hkv) * hd
    xs = x[:, :n].double().reshape(-1, Hq + Hkv, hd)
    g = torch.cat([gq.double().expand(Hq, -1), gk.double().expand(Hkv, -1)])
    cos, sin = (tab[pos][:, None, :, i].double() for i in (0, 1))
    r = 1.0 / torch.sqrt((xs ** 2).mean(-1, keepdim=True) + eps)
    xh = xs * r
    z = xh * g
    y = rotate(z, cos, sin)
    za = z.abs()
    h = hd // 2
    pair = za + torch.cat([za[..., h:], za[..., :h]], -1)
    ytol = BF * y.abs() + F32 * pair
    d = dy[:, :n].double().reshape(-1, Hq + Hkv, hd)
    dz = rotate(d, cos, -sin)
    da = d.abs() + torch.cat([d[..., h:], d[..., :h]], -1).abs()
    w = dz * g
    dx = r * (w - xh * (w * xh).mean(-1, keepdim=True))
    wa = da * g.abs()
    size = r * (wa + xh.abs() * (wa * xh.abs()).mean(-1, keepdim=True))
    dg, dga = (dz * xh), (da * xh.abs())
    out = []
    for s in (slice(0, Hq), slice(Hq, Hq + Hkv)):
        v = dg[:, s].sum((0, 1))
        out += [v, BF * v.abs() + F32 * dga[:, s].sum((0, 1))]
    return y.reshape(-1, n), ytol.reshape(-1, n), dx.reshape(-1, n), \
        (BF * dx.abs() + F32 * size).reshape(-1, n), out


QK_CASES = [  # T, seq, Hq, Hkv, hd, pad, positions given
    (1, 1, 1, 1, 16, 0, False),
    (1, 5, 4, 4, 64, 0, True),
    (70, 35, 6, 2, 64, 8, False),
    (333, 700, 16, 2, 128, 64, True),
    (257, 257, 5, 5, 96, 0, False),
    (65, 33, 12, 3, 80, 16, True),
    (129, 129, 32, 8, 128, 0, False),
    (40, 40, 3, 1, 256, 0, False),
    (31, 31, 2, 1, 240, 0, True),
    (3001, 1500, 16, 16, 32, 0, False),
    (900, 900, 40, 8, 128, 0, True),
]


@pytest.mark.parametrize("T,seq,Hq,Hkv,hd,pad,given", QK_CASES)
def test_qknorm_rope_forward_and_backward(T, seq, Hq, Hkv, hd, pad, given):
    x, gq, gk, dy, W = qk_inputs(T, Hq, Hkv, hd, pad)
    tab, ld, n = table(seq, hd), W + pad, (Hq + Hkv) * hd
    pos = torch.arange(T, device="cuda") % seq
    if given:
        pos = (pos * 7 + 3) % seq
    pos32 = pos.to(torch.int32)
    pp = pos32.data_ptr() if given else 0
    y_ref, y_tol, dx_ref, dx_tol, (dq, dqt, dk, dkt) = qk_ref(x, gq, gk, dy, Hq, Hkv, hd, pos, tab)
    (y, yt), (dx, dxt) = guarded((T, ld), torch.bfloat16), guarded((T, ld), torch.bfloat16)
    assert sf.op_qknorm_rope_fwd(x.data_ptr(), ld, y.data_ptr(), ld, T, seq, Hq, Hkv, hd, gq.data_ptr(),
                                 gk.data_ptr(), EPS, tab.data_ptr(), pp, stream()) == 0
    sc, sct = guarded((sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd),), torch.float32)
    (dgq, t1), (dgk, t2) = guarded((hd,), torch.bfloat16), guarded((hd,), torch.bfloat16)
    args = (T, seq, Hq, Hkv, hd, gq.data_ptr(), gk.data_ptr(), EPS, tab.data_ptr(), pp, sc.data_ptr(),
            dgq.data_ptr(), dgk.data_ptr(), stream())
    assert sf.op_qknorm_rope_bwd(x.data_ptr(), ld, dy.data_ptr(), ld, dx.data_ptr(), ld, *args) == 0
    sync()
    within(y[:, :n], y_ref, y_tol)
    within(dx[:, :n], dx_ref, dx_tol)
    within(dgq, dq, dqt)
    within(dgk, dk, dkt)
    assert torch.equal(y[:, n:W], x[:, n:W]) and torch.equal(dx[:, n:W], dy[:, n:W])
    assert (y[:, W:] == 7).all() and (dx[:, W:] == 7).all()  # padding columns are not written
    untouched(yt, dxt, sct, t1, t2)
    # in place: the same bits, the value heads and padding as they were
    x2, dy2, g2 = x.clone(), dy.clone(), (dgq.clone(), dgk.clone())
    assert sf.op_qknorm_rope_fwd(x2.data_ptr(), ld, x2.data_ptr(), ld, T, seq, Hq, Hkv, hd, gq.data_ptr(),
                                 gk.data_ptr(), EPS, tab.data_ptr(), pp, stream()) == 0
    assert sf.op_qknorm_rope_bwd(x.data_ptr(), ld, dy2.data_ptr(), ld, dy2.data_ptr(), ld, *args) == 0
    sync()
    assert torch.equal(x2[:, :W], y[:, :W]) and torch.equal(x2[:, W:], x[:, W:])
    assert torch.equal(dy2[:, :W], dx[:, :W]) and torch.equal(dy2[:, W:], dy[:, W:])
    assert torch.equal(dgq, g2[0]) and torch.equal(dgk, g2[1])  # fixed order of the sums


def test_qknorm_zero_rows_and_tiny_eps():
    """Rows of zeros norm to zeros; their gradient is r g dz with r = 1/sqrt(eps)."""
    T, Hq, Hkv, hd = 9, 2, 1, 64
    x, gq, gk, dy, W = qk_inputs(T, Hq, Hkv, hd)
    x[::2] = 0
    tab, pos = table(T, hd), torch.arange(T, device="cuda")
    for eps in (1e-5, 1e-30):
        y_ref, y_tol, dx_ref, dx_tol, _ = qk_ref(x, gq, gk, dy, Hq, Hkv, hd, pos, tab, eps)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        sc = torch.empty(sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd), **F32T)
        dg = torch.empty(2, hd, dtype=torch.bfloat16, device="cuda")
        a = (T, T, Hq, Hkv, hd, gq.data_ptr(), gk.data_ptr(), eps, tab.data_ptr(), 0)
        assert sf.op_qknorm_rope_fwd(x.data_ptr(), W, y.data_ptr(), W, *a, stream()) == 0
        assert sf.op_qknorm_rope_bwd(x.data_ptr(), W, dy.data_ptr(), W, dx.data_ptr(), W, *a, sc.data_ptr(),
                                     dg[0].data_ptr(), dg[1].data_ptr(), stream()) == 0
        sync()
        n = (Hq + Hkv) * hd
        within(y[:, :n], y_ref, y_tol)
        within(dx[:, :n], dx_ref, dx_tol)


def test_qknorm_gradient_against_differences():
    """Directional derivatives of sum(y * dy) by central differences in float64."""
    T, Hq, Hkv, hd = 20, 3, 1, 32
    x, gq, gk, dy, W = qk_inputs(T, Hq, Hkv, hd, seed=5)
    tab, pos, n = table(T, hd), torch.arange(T, device="cuda"), (Hq + Hkv) * hd
    _, _, _, tol, (_, dqt, _, dkt) = qk_ref(x, gq, gk, dy, Hq, Hkv, hd, pos, tab)
    dx = torch.empty_like(x)
    sc = torch.empty(sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd), **F32T)
    dg = torch.empty(2, hd, dtype=torch.bfloat16, device="cuda")
    assert sf.op_qknorm_rope_bwd(x.data_ptr(), W, dy.data_ptr(), W, dx.data_ptr(), W, T, T, Hq, Hkv, hd,
                                 gq.data_ptr(), gk.data_ptr(), EPS, tab.data_ptr(), 0, sc.data_ptr(),
                                 dg[0].data_ptr(), dg[1].data_ptr(), stream()) == 0
    sync()

    def loss(xx, a, b):
        return (qk_ref(xx, a, b, dy, Hq, Hkv, hd, pos, tab)[0] * dy[:, :n].double()).sum()

    rnd = gen(9)
    vx, vq, vk = rnd(T, W).double(), rnd(hd).double(), rnd(hd).double()
    vx[:, n:] = 0
    x64, q64, k64 = x.double(), gq.double(), gk.double()
    h = 1e-6
    num = ((loss(x64 + h * vx, q64 + h * vq, k64 + h * vk) - loss(x64 - h * vx, q64 - h * vq, k64 - h * vk))
           / (2 * h)).item()
    got = ((dx.double() * vx)[:, :n].sum() + (dg[0].double() * vq).sum() + (dg[1].double() * vk).sum()).item()
    bound = ((tol * vx[:, :n].abs()).sum() + (dqt * vq.abs()).sum() + (dkt * vk.abs()).sum()).item()
    assert abs(got - num) <= bound + 1e-6 * abs(num)


def test_qknorm_position_outside_the_table():
    """Its token is normed but not rotated, and the error word says so; the others are right."""
    T, Hq, Hkv, hd, seq = 6, 2, 1, 64, 4
    x, gq, gk, dy, W = qk_inputs(T, Hq, Hkv, hd)
    tab = table(seq, hd)
    pos = torch.tensor([0, 3, 4, 1, -1, 2], dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    assert sf.op_qknorm_rope_fwd(x.data_ptr(), W, y.data_ptr(), W, T, seq, Hq, Hkv, hd, gq.data_ptr(),
                                 gk.data_ptr(), EPS, tab.data_ptr(), pos.data_ptr(), stream()) == 0
    sync()
    assert sf.device_error() == 5 and sf.device_error() == 0
    ok = torch.where((pos >= 0) & (pos < seq), pos, torch.zeros_like(pos)).long()  # position 0 turns nothing
    y_ref, y_tol, *_ = qk_ref(x, gq, gk, dy, Hq, Hkv, hd, ok, tab)
    within(y[:, :(Hq + Hkv) * hd], y_ref, y_tol)


# ------------------------------------------------------------------ windowed attention
def visible(S, window, sinks):
    q, k = torch.arange(S, device="cuda")[:, None], torch.arange(S, device="cuda")[None, :]
    return (k <= q) & ((q - k < window) | (k < sinks))


def split_heads(qkv, B, S, Hq, Hkv, hd):
    x = qkv.double().reshape(B, S, Hq + 2 * Hkv, hd).transpose(1, 2)
    rep = Hq // Hkv
    return x[:, :Hq], x[:, Hq:Hq + Hkv].repeat_interleave(rep, 1), x[:, Hq + Hkv:].repeat_interleave(rep, 1)


def attn_ref(qkv, B, S, Hq, Hkv, hd, window, sinks):
    """o [B*S, Hq*hd], its tolerance, and lse [B, Hq, S] in float64."""
    q, k, v = split_heads(qkv, B, S, Hq, Hkv, hd)
    s = (q @ k.transpose(-1, -2)) * hd ** -0.5
    s = s.masked_fill(~visible(S, window, sinks), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    o, a = p @ v, p @ v.abs()
    flat = lambda t: t.transpose(1, 2).reshape(B * S, -1)
    return flat(o), flat(BF * o.abs() * (1 + BF) + (BF + SC) * a), lse


def attn_bwd_ref(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab=None):
    """dqkv in float64 from the forward's stored o and lse, and its tolerance."""
    q, k, v = split_heads(qkv, B, S, Hq, Hkv, hd)
    heads = lambda t: t.double().reshape(B, S, Hq, hd).transpose(1, 2)
    do, oo, sc = heads(dout), heads(o), hd ** -0.5
    p = torch.exp((q @ k.transpose(-1, -2)) * sc - lse.double()[..., None])
    p = p * visible(S, window, sinks)
    D = (do * oo).sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - D)
    # what dS is off by: its rounding, P's error, and the fp32 sums of dP and D
    e = (BF + SC) * ds.abs() + 2.0 ** -15 * p * (do.abs() @ v.abs().transpose(-1, -2) +
                                                 (do * oo).abs().sum(-1, keepdim=True))
    dq, dqe = sc * (ds @ k), sc * (e @ k.abs())
    grp = lambda t: t.reshape(B, Hkv, Hq // Hkv, S, hd).sum(2)
    T = lambda t: t.transpose(-1, -2)
    dk, dke = grp(sc * (T(ds) @ q)), grp(sc * (T(e) @ q.abs()))
    dv, dve = grp(T(p) @ do), grp((BF + SC) * (T(p) @ do.abs()))
    x, xe = torch.cat([dq, dk], 1), torch.cat([dqe, dke], 1)
    if tab is not None:
        cos, sin = tab[:S, :, 0].double(), tab[:S, :, 1].double()
        h = hd // 2
        size = x.abs() + torch.cat([x[..., h:], x[..., :h]], -1).abs()
        x, xe = rotate(x, cos, -sin), xe + torch.cat([xe[..., h:], xe[..., :h]], -1) + F32 * size
    g, ge = torch.cat([x, dv], 1), torch.cat([xe, dve], 1)
    flat = lambda t: t.transpose(1, 2).reshape(B * S, -1)
    return flat(g), flat(BF * g.abs() * (1 + BF) + ge * (1 + BF))


WIN_CASES = [  # B, S, Hq, Hkv, hd, window, sinks
    (1, 1, 2, 1, 64, 1, 0),
    (2, 1, 1, 1, 128, 5, 3),
    (1, 64, 2, 2, 128, 1, 0),        # every query sees itself only
    (1, 130, 4, 2, 64, 1, 1),
    (2, 127, 3, 1, 64, 64, 0),       # odd group: query blocks are paired instead of heads
    (1, 128, 2, 1, 128, 65, 2),
    (1, 129, 3, 3, 128, 128, 0),
    (2, 300, 6, 2, 64, 63, 4),
    (1, 300, 4, 2, 128, 129, 130),   # sinks over two blocks
    (1, 700, 2, 1, 128, 100, 4),     # a gap between the sinks' block and the window's
    (1, 700, 3, 1, 64, 100, 4),
    (2, 641, 4, 4, 128, 127, 0),     # windows that start inside a tile, no sinks
    (1, 777, 5, 5, 64, 200, 1),
    (1, 1025, 8, 2, 128, 256, 64),
    (1, 900, 2, 2, 128, 320, 300),
    (1, 385, 2, 1, 128, 4000, 0),    # wider than the sequence: plain causal attention
    (1, 260, 2, 1, 64, 40, 900),     # every token is a sink
    # long enough that the backward splits the queries behind the sinks' window
    (1, 2100, 2, 1, 128, 100, 4),
    (1, 2500, 4, 2, 64, 64, 130),
    (2, 3000, 3, 1, 128, 64, 130),
    (1, 4000, 2, 1, 64, 1, 1),
    (2, 2600, 2, 2, 128, 300, 17),
]


def win_inputs(B, S, Hq, Hkv, hd, seed=1):
    rnd = gen(seed)
    return rnd(B * S, (Hq + 2 * Hkv) * hd).bfloat16(), rnd(B * S, Hq * hd).bfloat16()


def win_fwd(qkv, B, S, Hq, Hkv, hd, window, sinks):
    (o, ot), (lse, lt) = guarded((B * S, Hq * hd), torch.bfloat16), guarded((B, Hq, S), torch.float32)
    assert sf.op_attn_window_fwd(qkv.data_ptr(), o.data_ptr(), lse.data_ptr(), B, S, Hq, Hkv, hd, window,
                                 sinks, stream()) == 0
    sync()
    untouched(ot, lt)
    return o, lse


def win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab=None, det=0):
    dqkv, gt = guarded(tuple(qkv.shape), torch.bfloat16)
    delta, dt = guarded((B, Hq, S), torch.float32)
    n = sf.attn_window_dq_scratch_floats(B, S, Hq, hd, window, sinks, det)
    acc, at = guarded((n,), torch.float32)
    acc.fill_(float("nan"))  # no slot is read that was not written
    assert sf.op_attn_window_bwd(qkv.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                                 delta.data_ptr(), acc.data_ptr(), dqkv.data_ptr(), B, S, Hq, Hkv, hd, window,
                                 sinks, tab.data_ptr() if tab is not None else 0, stream(), det) == 0
    sync()
    untouched(gt, dt, at)
    return dqkv


@pytest.mark.parametrize("B,S,Hq,Hkv,hd,window,sinks", WIN_CASES)
def test_window_forward(B, S, Hq, Hkv, hd, window, sinks):
    qkv, _ = win_inputs(B, S, Hq, Hkv, hd)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, window, sinks)
    ref, tol, lref = attn_ref(qkv, B, S, Hq, Hkv, hd, window, sinks)
    within(o, ref, tol)
    # fp32 scores of 128 products, the exponentials' 2^-22 and the logarithm
    within(lse, lref, 2.0 ** -15 + 2.0 ** -21 * lref.abs())


@pytest.mark.parametrize("det", [0, 1])
@pytest.mark.parametrize("B,S,Hq,Hkv,hd,window,sinks", WIN_CASES)
def test_window_backward(B, S, Hq, Hkv, hd, window, sinks, det):
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=2)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, window, sinks)
    for tab in (None, table(S, hd)):
        got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab, det)
        ref, tol = attn_bwd_ref(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab)
        within(got, ref, tol)
    if det:
        again = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab, det)
        assert torch.equal(again, got)


@pytest.mark.parametrize("det", [0, 1])
@pytest.mark.parametrize("B,S,Hq,Hkv,hd", [
    (8, 390, 16, 16, 128),   # 128 heads and batches of four key blocks: one chunk and the rest
    (3, 1000, 80, 40, 128),  # 120 of eight: several chunks
    (3, 1000, 80, 40, 64),
])
def test_backward_of_many_heads(B, S, Hq, Hkv, hd, det):
    """Without a window the backward takes heads in chunks where there are many."""
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=4)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, S, 0)
    got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, S, 0, None, det)
    for b in range(B):  # one sequence at a time: the float64 scores of all are too large
        rows = slice(b * S, (b + 1) * S)
        ref, tol = attn_bwd_ref(qkv[rows], o[rows], dout[rows], lse[b:b + 1], 1, S, Hq, Hkv, hd, S, 0)
        within(got[rows], ref, tol)


@pytest.mark.parametrize("hd,Hq", [(64, 4), (128, 4), (128, 3)])
def test_window_wider_than_the_sequence_is_causal_attention(hd, Hq):
    B, S, Hkv = 2, 390, 1
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=3)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, S, 0)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    assert sf.op_attn_fwd(qkv.data_ptr(), o2.data_ptr(), lse2.data_ptr(), B, S, Hq, Hkv, hd, stream()) == 0
    sync()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, 2 ** 31 - 1, 2 ** 31 - 1, None, 1)
    dqkv = torch.empty_like(qkv)
    delta = torch.empty_like(lse)
    acc = torch.empty(sf.attn_dq_scratch_floats(B, S, Hq, hd, 1), **F32T)
    assert sf.op_attn_bwd(qkv.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(), delta.data_ptr(),
                          acc.data_ptr(), dqkv.data_ptr(), B, S, Hq, Hkv, hd, 0, stream(), 1) == 0
    sync()
    ref, tol = attn_bwd_ref(qkv, o, dout, lse, B, S, Hq, Hkv, hd, S, 0)
    within(got, ref, tol)
    within(dqkv, ref, tol)


def test_window_ignores_what_is_masked():
    """Keys and queries of other positions may be anything; infinite keys and
    values outside every window's blocks are never read."""
    B, S, Hq, Hkv, hd, W = 1, 700, 4, 2, 128, 96
    qkv, _ = win_inputs(B, S, Hq, Hkv, hd, seed=4)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, W, 0)
    bad = qkv.clone()
    kv = bad[:, Hq * hd:]
    kv[:128] = float("nan")          # blocks before the windows of queries from 384 on
    bad[600:, Hq * hd:(Hq + Hkv) * hd] = float("inf")  # later keys (masked in the diagonal blocks)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    assert sf.op_attn_window_fwd(bad.data_ptr(), o2.data_ptr(), lse2.data_ptr(), B, S, Hq, Hkv, hd, W, 0,
                                 stream()) == 0
    sync()
    assert torch.equal(o2[384:600], o[384:600]) and torch.equal(lse2[:, :, 384:600], lse[:, :, 384:600])


def test_window_gradient_against_differences():
    B, S, Hq, Hkv, hd, W, n = 1, 150, 2, 1, 64, 40, 3
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=6)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, W, n)
    got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, W, n)
    _, tol = attn_bwd_ref(qkv, o, dout, lse, B, S, Hq, Hkv, hd, W, n)
    # the stored o is rounded: D moves by up to 2^-8 sum |do o|, dS by p of that
    q, k, v = split_heads(qkv, B, S, Hq, Hkv, hd)
    oh, dh = (t.double().reshape(B, S, Hq, hd).transpose(1, 2) for t in (o, dout))
    e = torch.exp(q @ k.transpose(-1, -2) * hd ** -0.5 - lse.double()[..., None]) * visible(S, W, n)
    e = e * (BF + BF * BF + 2 * SC) * (dh * oh).abs().sum(-1, keepdim=True)
    tol = tol.reshape(S, Hq + 2 * Hkv, hd).clone()
    tol[:, :Hq] += (hd ** -0.5 * (e @ k.abs()))[0].transpose(0, 1)
    tol[:, Hq:Hq + Hkv] += (hd ** -0.5 * (e.transpose(-1, -2) @ q.abs())).sum(1)[0][:, None]
    v64 = gen(7)(*qkv.shape).double()
    loss = lambda x: (attn_ref(x, B, S, Hq, Hkv, hd, W, n)[0] * dout.double()).sum()
    h = 1e-6
    num = ((loss(qkv.double() + h * v64) - loss(qkv.double() - h * v64)) / (2 * h)).item()
    dot = (got.double() * v64).sum().item()
    assert abs(dot - num) <= (tol.reshape(S, -1) * v64.abs()).sum().item() + 1e-6 * abs(num)


# ------------------------------------------------------------------ 8-bit checkpoints
FMTS = [("int8", 0, 127.0), ("e4m3", 1, 448.0)]


def ckpt_ref(x, top):
    """Codes (as their values), scales and loaded values by the stated fp32 rule."""
    rows, d = x.shape
    nb = (d + 127) // 128
    xb = torch.zeros(rows, nb * 128, **F32T)
    xb[:, :d] = x
    xb = xb.reshape(rows, nb, 128).cpu().numpy()
    a = np.abs(xb).max(-1)
    with np.errstate(all="ignore"):
        live = np.isfinite(a) & (a >= np.float32(2.0 ** -100))
        inv = np.where(live, np.float32(top) / a, np.float32(0)).astype(np.float32)
        s = np.where(live, a / np.float32(top), np.where(np.isfinite(a), np.float32(0), np.float32("nan")))
        v = np.where(live[..., None], xb * inv[..., None], np.float32(0)).astype(np.float32)
    if top == 127.0:
        c = np.rint(v)
    else:
        c = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    s = s.astype(np.float32)
    val = (c.astype(np.float32) * s[..., None]).astype(np.float32)
    cut = lambda t: torch.from_numpy(t.reshape(rows, -1)[:, :d].copy()).cuda()
    return cut(c), torch.from_numpy(s).cuda(), cut(val)


def codes_of(q, fmt):
    return (q.view(torch.int8) if fmt == 0 else q.view(torch.float8_e4m3fn)).float()


def same(a, b):
    assert torch.equal(a.nan_to_num(nan=1e30), b.nan_to_num(nan=1e30))


def ckpt_inputs(rows, d, seed=1):
    rnd = gen(seed)
    x = rnd(rows, d)
    x[:, ::37] *= 50.0        # outlier channels
    x[rows // 2] *= 1e-3
    return x, (1 + 0.2 * rnd(d)).bfloat16(), rnd(rows, d), rnd(rows, d)


CK_CASES = [(1, 8), (3, 128), (5, 136), (37, 384), (200, 1000), (300, 4096), (7, 6152), (5, 12288), (3, 16384),
            (1201, 520)]


@pytest.mark.parametrize("name,fmt,top", FMTS)
@pytest.mark.parametrize("rows,d", CK_CASES)
def test_ckpt8_norm_round_trip(rows, d, name, fmt, top):
    """Save (alone and with the norm), load, the norm of the loaded values and
    its backward."""
    x, g, dy, dres = ckpt_inputs(rows, d)
    nb = (d + 127) // 128
    assert sf.ckpt8_scales(rows, d) == rows * nb
    c_ref, s_ref, v_ref = ckpt_ref(x, top)
    (q, qt), (s, st), (v, vt) = (guarded((rows, d), torch.uint8), guarded((rows, nb), torch.float32),
                                 guarded((rows, d), torch.float32))
    assert sf.op_ckpt8_save(x.data_ptr(), q.data_ptr(), s.data_ptr(), fmt, rows, d, stream()) == 0
    assert sf.op_ckpt8_load(q.data_ptr(), s.data_ptr(), v.data_ptr(), fmt, rows, d, stream()) == 0
    sync()
    same(codes_of(q, fmt), c_ref)
    same(s, s_ref)
    same(v, v_ref)
    untouched(qt, st, vt)
    # half a step of the code: 1/254 of the block's largest (int8), 2^-4 of the value (e4m3)
    step = s_ref.repeat_interleave(128, 1)[:, :d].double()
    err = (v.double() - x.double()).abs()
    tol = step * 0.5 if fmt == 0 else torch.maximum(x.double().abs() * 2.0 ** -4, step * 2.0 ** -10)
    assert (err <= tol * (1 + 2.0 ** -20) + step * 2.0 ** -16).all()

    (q2, q2t), (s2, s2t), (y, yt), (r, rt) = (guarded((rows, d), torch.uint8), guarded((rows, nb), torch.float32),
                                              guarded((rows, d), torch.bfloat16), guarded((rows,), torch.float32))
    assert sf.op_rmsnorm_fwd_save8(x.data_ptr(), g.data_ptr(), y.data_ptr(), r.data_ptr(), q2.data_ptr(),
                                   s2.data_ptr(), fmt, rows, d, EPS, stream()) == 0
    sync()
    assert torch.equal(q2, q)
    same(s2, s)
    untouched(q2t, s2t, yt, rt)

    def norm(xx):
        rr = 1.0 / torch.sqrt((xx.double() ** 2).mean(1) + EPS)
        return xx.double() * rr[:, None] * g.double(), rr

    y_ref, r_ref = norm(x)
    within(r, r_ref, F32 * r_ref)
    within(y, y_ref, (BF + F32) * y_ref.abs())
    (y2, y2t), (r2, r2t), (v2, v2t) = (guarded((rows, d), torch.bfloat16), guarded((rows,), torch.float32),
                                       guarded((rows, d), torch.float32))
    assert sf.op_rmsnorm_fwd_load8(q.data_ptr(), s.data_ptr(), g.data_ptr(), y2.data_ptr(), r2.data_ptr(),
                                   v2.data_ptr(), fmt, rows, d, EPS, stream()) == 0
    y3, r3 = torch.empty_like(y2), torch.empty_like(r2)
    assert sf.op_rmsnorm_fwd_load8(q.data_ptr(), s.data_ptr(), g.data_ptr(), y3.data_ptr(), r3.data_ptr(), 0,
                                   fmt, rows, d, EPS, stream()) == 0
    sync()
    same(v2, v_ref)
    y_ref, r_ref = norm(v_ref)
    within(r2, r_ref, F32 * r_ref)
    within(y2, y_ref, (BF + F32) * y_ref.abs())
    assert torch.equal(y3, y2) and torch.equal(r3, r2)
    untouched(y2t, r2t, v2t)

    for res in (dres, None):
        (dx, dt), (dxb, bt), (dg, gt) = (guarded((rows, d), torch.float32), guarded((rows, d), torch.bfloat16),
                                         guarded((d,), torch.bfloat16))
        sc, sct = guarded((sf.rmsnorm_bwd_scratch(rows, d),), torch.float32)
        assert sf.op_rmsnorm_bwd_load8(q.data_ptr(), s.data_ptr(), g.data_ptr(), r2.data_ptr(), dy.data_ptr(),
                                       res.data_ptr() if res is not None else 0, dx.data_ptr(), dxb.data_ptr(),
                                       dg.data_ptr(), sc.data_ptr(), fmt, rows, d, stream()) == 0
        sync()
        rr = r2.double()[:, None]
        xh, w = v_ref.double() * rr, dy.double() * g.double()
        base = res.double() if res is not None else torch.zeros(rows, d, **D64)
        dx_ref = base + rr * (w - xh * (w * xh).mean(1, keepdim=True))
        size = base.abs() + rr * (w.abs() + xh.abs() * (w * xh).abs().mean(1, keepdim=True))
        within(dx, dx_ref, F32 * size)
        within(dxb, dx_ref, BF * dx_ref.abs() + F32 * size)
        ref = (dy.double() * xh).sum(0)
        within(dg, ref, BF * ref.abs() + F32 * (dy.double() * xh).abs().sum(0))
        untouched(dt, bt, gt, sct)


@pytest.mark.parametrize("name,fmt,top", FMTS)
def test_ckpt8_special_blocks(name, fmt, top):
    """Zeros, tiny and huge magnitudes, infinities and NaN, each in its own block."""
    d = 128 * 7 + 8
    x = torch.zeros(2, d, **F32T)
    x[0, 128:256] = 1e-38
    x[0, 256:384] = torch.linspace(-3e38, 3e38, 128, **F32T)
    x[0, 384:512] = 1.0
    x[0, 400] = float("inf")
    x[0, 512:640] = 2.0
    x[0, 600] = float("nan")
    x[0, 640:768] = 2.0 ** -100
    x[0, 768:896] = -2.0 ** -99
    x[0, 896:] = torch.tensor([1.0, -1.0, 0.5, 1e-9, 0.0, -0.25, 0.9999, 2.0], **F32T)
    x[1] = torch.linspace(-1, 1, d, **F32T)
    c_ref, s_ref, v_ref = ckpt_ref(x, top)
    q = torch.empty(2, d, dtype=torch.uint8, device="cuda")
    s, v = torch.empty(2, 8, **F32T), torch.empty(2, d, **F32T)
    assert sf.op_ckpt8_save(x.data_ptr(), q.data_ptr(), s.data_ptr(), fmt, 2, d, stream()) == 0
    assert sf.op_ckpt8_load(q.data_ptr(), s.data_ptr(), v.data_ptr(), fmt, 2, d, stream()) == 0
    sync()
    same(codes_of(q, fmt), c_ref)
    same(s, s_ref)
    same(v, v_ref)
    # a block loads as NaN exactly when it held something that is not finite (the
    # linspace does: its step, 6e38, overflows)
    pad = lambda t: torch.nn.functional.pad(t, (0, 8 * 128 - d)).reshape(2, 8, 128)
    bad = (~torch.isfinite(pad(x))).any(-1, keepdim=True).expand(-1, -1, 128)
    assert bool((torch.isnan(pad(v))[:, :7] == bad[:, :7]).all())
    assert not v[0, 128:256].any()


@pytest.mark.parametrize("name,fmt,top", FMTS)
def test_ckpt8_huge_magnitudes(name, fmt, top):
    x = torch.empty(1, 256, **F32T)
    x[0, :128] = torch.linspace(-1.5e38, 1.5e38, 128, **F32T) * 2
    x[0, 128:] = 3.4028234663852886e38
    x[0, 130] = -3.4028234663852886e38
    c_ref, s_ref, v_ref = ckpt_ref(x, top)
    q = torch.empty(1, 256, dtype=torch.uint8, device="cuda")
    s, v = torch.empty(1, 2, **F32T), torch.empty(1, 256, **F32T)
    assert sf.op_ckpt8_save(x.data_ptr(), q.data_ptr(), s.data_ptr(), fmt, 1, 256, stream()) == 0
    assert sf.op_ckpt8_load(q.data_ptr(), s.data_ptr(), v.data_ptr(), fmt, 1, 256, stream()) == 0
    sync()
    same(codes_of(q, fmt), c_ref)
    same(s, s_ref)
    same(v, v_ref)
    assert torch.isfinite(s).all()


def test_ckpt8_backward_against_differences():
    """sum(dy * y) of the norm of the loaded values, by central differences."""
    rows, d = 6, 264
    x, g, dy, _ = ckpt_inputs(rows, d, seed=3)
    _, s, v = ckpt_ref(x, 127.0)
    q = torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    sc = torch.empty_like(s)
    assert sf.op_ckpt8_save(x.data_ptr(), q.data_ptr(), sc.data_ptr(), 0, rows, d, stream()) == 0
    y, r = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, **F32T)
    assert sf.op_rmsnorm_fwd_load8(q.data_ptr(), sc.data_ptr(), g.data_ptr(), y.data_ptr(), r.data_ptr(), 0, 0,
                                   rows, d, EPS, stream()) == 0
    dx, dxb = torch.empty(rows, d, **F32T), torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    dg = torch.empty(d, dtype=torch.bfloat16, device="cuda")
    part = torch.empty(sf.rmsnorm_bwd_scratch(rows, d), **F32T)
    assert sf.op_rmsnorm_bwd_load8(q.data_ptr(), sc.data_ptr(), g.data_ptr(), r.data_ptr(), dy.data_ptr(), 0,
                                   dx.data_ptr(), dxb.data_ptr(), dg.data_ptr(), part.data_ptr(), 0, rows, d,
                                   stream()) == 0
    sync()
    u, ug = gen(8)(rows, d).double(), gen(9)(d).double()

    def loss(t):
        xx, gg = v.double() + t * u, g.double() + t * ug
        return (xx / torch.sqrt((xx ** 2).mean(1, keepdim=True) + EPS) * gg * dy.double()).sum().item()

    h = 1e-6
    num = (loss(h) - loss(-h)) / (2 * h)
    got = (dx.double() * u).sum().item() + (dg.double() * ug).sum().item()
    rr = r.double()[:, None]
    xh, w = (v.double() * rr).abs(), (dy.double() * g.double()).abs()
    tol = (F32 * rr * (w + xh * (w * xh).mean(1, keepdim=True)) * u.abs()).sum().item()
    tol += (((dy.double() * xh).sum(0).abs() * BF + F32 * (dy.double().abs() * xh).sum(0)) * ug.abs()).sum().item()
    assert abs(got - num) <= tol + 1e-6 * abs(num)


# ------------------------------------------------------------------ as they are used together
def test_attention_half_of_a_layer_with_a_checkpoint():
    """A layer's attention half: the norm that saves the checkpoint, the Q/K/V
    projection, the query/key norm in place, windowed attention; then the
    recompute from the checkpoint and the whole backward, captured in a CUDA
    graph on another stream and replayed, against float64 from the loaded
    values.  The projections are the framework's own GEMM."""
    B, S, d, Hq, Hkv, hd, W, n = 2, 200, 384, 6, 2, 64, 72, 4
    T, Wd = B * S, (Hq + 2 * Hkv) * hd
    rnd = gen(21)
    x, g1 = rnd(T, d), (1 + 0.1 * rnd(d)).bfloat16()
    wqkv = (0.05 * rnd(Wd, d)).bfloat16()
    gq, gk = (1 + 0.2 * rnd(hd)).bfloat16(), (1 + 0.2 * rnd(hd)).bfloat16()
    dout = rnd(T, Hq * hd).bfloat16()
    tab = table(S, hd)
    nb = d // 128
    E = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")
    u, r1, q8, s8 = E(torch.bfloat16, T, d), E(torch.float32, T), E(torch.uint8, T, d), E(torch.float32, T, nb)
    qkv, o, lse = E(torch.bfloat16, T, Wd), E(torch.bfloat16, T, Hq * hd), E(torch.float32, B, Hq, S)
    raw, xv = E(torch.bfloat16, T, Wd), E(torch.float32, T, d)
    dqkv, delta = E(torch.bfloat16, T, Wd), E(torch.float32, B, Hq, S)
    acc = E(torch.float32, sf.attn_window_dq_scratch_floats(B, S, Hq, hd, W, n, 1))
    sq = E(torch.float32, sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd))
    dgq, dgk, du = E(torch.bfloat16, hd), E(torch.bfloat16, hd), E(torch.float32, T, d)
    dx, dxb, dg1 = E(torch.float32, T, d), E(torch.bfloat16, T, d), E(torch.bfloat16, d)
    sn = E(torch.float32, sf.rmsnorm_bwd_scratch(T, d))
    p = lambda t: t.data_ptr()

    def half(st):
        qk = (T, S, Hq, Hkv, hd, p(gq), p(gk), EPS, p(tab), 0)
        shape = (B, S, Hq, Hkv, hd, W, n)
        rc = [sf.op_rmsnorm_fwd_save8(p(x), p(g1), p(u), p(r1), p(q8), p(s8), 0, T, d, EPS, st),
              sf.op_gemm(sf.NT, sf.EPI_BF16, T, Wd, d, p(u), d, p(wqkv), d, p(qkv), Wd, stream=st),
              sf.op_qknorm_rope_fwd(p(qkv), Wd, p(qkv), Wd, *qk, st),
              sf.op_attn_window_fwd(p(qkv), p(o), p(lse), *shape, st),
              # the layer's backward: from the checkpoint on
              sf.op_rmsnorm_fwd_load8(p(q8), p(s8), p(g1), p(u), p(r1), p(xv), 0, T, d, EPS, st),
              sf.op_gemm(sf.NT, sf.EPI_BF16, T, Wd, d, p(u), d, p(wqkv), d, p(raw), Wd, stream=st),
              sf.op_qknorm_rope_fwd(p(raw), Wd, p(qkv), Wd, *qk, st),
              sf.op_attn_window_fwd(p(qkv), p(o), p(lse), *shape, st),
              sf.op_attn_window_bwd(p(qkv), p(o), p(dout), p(lse), p(delta), p(acc), p(dqkv), *shape, 0, st, 1),
              sf.op_qknorm_rope_bwd(p(raw), Wd, p(dqkv), Wd, p(dqkv), Wd, *qk, p(sq), p(dgq), p(dgk), st),
              sf.op_gemm(sf.NN, sf.EPI_F32, T, d, Wd, p(dqkv), Wd, p(wqkv), d, p(du), d, stream=st),
              sf.op_rmsnorm_bwd_load8(p(q8), p(s8), p(g1), p(r1), p(du), 0, p(dx), p(dxb), p(dg1), p(sn), 0, T,
                                      d, st)]
        assert rc == [0] * len(rc), rc

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        half(stream())
    side.synchronize()
    first = [t.clone() for t in (o, lse, dqkv, dgq, dgk, dx, dxb, dg1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        half(stream())
    for t in (u, qkv, o, lse, raw, dqkv, dx, dxb, dg1, dgq, dgk):
        t.zero_()
    graph.replay()
    sync()
    for a, b in zip(first, (o, lse, dqkv, dgq, dgk, dx, dxb, dg1)):
        assert torch.equal(a, b)
    # float64 from the loaded values (no rounding between the operators)
    xx = xv.double().requires_grad_(True)
    a = [t.double().requires_grad_(True) for t in (g1, gq, gk)]
    uu = xx / torch.sqrt((xx ** 2).mean(1, keepdim=True) + EPS) * a[0]
    z = (uu @ wqkv.double().T).reshape(B, S, Hq + 2 * Hkv, hd)
    cos, sin = tab[:, None, :, 0].double(), tab[:, None, :, 1].double()
    rms = lambda t: t / torch.sqrt((t ** 2).mean(-1, keepdim=True) + EPS)
    qk = torch.cat([rotate(rms(z[:, :, :Hq]) * a[1], cos, sin),
                    rotate(rms(z[:, :, Hq:Hq + Hkv]) * a[2], cos, sin), z[:, :, Hq + Hkv:]], 2)
    ref = attn_ref(qk.reshape(T, Wd), B, S, Hq, Hkv, hd, W, n)[0]
    grads = torch.autograd.grad((ref * dout.double()).sum(), [xx] + a)
    # every bf16 tensor on the way (u, the projection, the normed heads, P, dS,
    # dqkv, du's operands) adds at most 2^-8 of itself: ten of them forward and
    # backward, in the 2-norm
    rel = lambda got, want: ((got.double() - want).norm() / want.norm()).item()
    assert rel(o, ref) <= 5 * BF
    for got, want in zip((dx, dgq, dgk, dg1), (grads[0], grads[2], grads[3], grads[1])):
        assert rel(got, want) <= 10 * BF


def test_calls_on_two_streams_at_once():
    """Two training-like chains with their own buffers on two streams, launched
    without waiting: the same bits as one after the other."""
    def chain(seed):
        B, S, Hq, Hkv, hd, W, n, T, d = 1, 1100, 8, 2, 128, 200, 4, 1100, 1024
        rnd = gen(seed)
        qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=seed)
        x, gq, gk, dy, Wd = qk_inputs(T, Hq, Hkv, hd, seed=seed)
        h, g, dyn = rnd(T, d), (1 + 0.1 * rnd(d)).bfloat16(), rnd(T, d)
        tab = table(S, hd)
        E = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")
        o, lse, dqkv = E(torch.bfloat16, T, Hq * hd), E(torch.float32, B, Hq, S), torch.empty_like(qkv)
        delta = torch.empty_like(lse)
        acc = E(torch.float32, sf.attn_window_dq_scratch_floats(B, S, Hq, hd, W, n, 1))
        y, dx, sq = torch.empty_like(x), torch.empty_like(x), E(torch.float32, sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd))
        dgq, dgk = E(torch.bfloat16, hd), E(torch.bfloat16, hd)
        q8, s8, yn, r = E(torch.uint8, T, d), E(torch.float32, T, d // 128), E(torch.bfloat16, T, d), E(torch.float32, T)
        dh, dhb, dg, part = E(torch.float32, T, d), E(torch.bfloat16, T, d), E(torch.bfloat16, d), \
            E(torch.float32, sf.rmsnorm_bwd_scratch(T, d))
        p = lambda t: t.data_ptr()
        keep = (qkv, dout, x, gq, gk, dy, h, g, dyn, tab, delta, acc, sq, part)

        def run(st):
            shape, qk = (B, S, Hq, Hkv, hd, W, n), (T, S, Hq, Hkv, hd, p(gq), p(gk), EPS, p(tab), 0)
            for _ in range(3):
                rc = [sf.op_attn_window_fwd(p(qkv), p(o), p(lse), *shape, st),
                      sf.op_attn_window_bwd(p(qkv), p(o), p(dout), p(lse), p(delta), p(acc), p(dqkv), *shape, 0, st, 1),
                      sf.op_qknorm_rope_fwd(p(x), Wd, p(y), Wd, *qk, st),
                      sf.op_qknorm_rope_bwd(p(x), Wd, p(dy), Wd, p(dx), Wd, *qk, p(sq), p(dgq), p(dgk), st),
                      sf.op_rmsnorm_fwd_save8(p(h), p(g), p(yn), p(r), p(q8), p(s8), 1, T, d, EPS, st),
                      sf.op_rmsnorm_bwd_load8(p(q8), p(s8), p(g), p(r), p(dyn), 0, p(dh), p(dhb), p(dg), p(part), 1,
                                              T, d, st)]
                assert rc == [0] * 6, rc
        return run, (o, lse, dqkv, y, dx, dgq, dgk, q8, s8, yn, dh, dg), keep

    a, b = chain(31), chain(32)
    for c in (a, b):
        c[0](stream())
        sync()
    want = [[t.clone() for t in c[1]] for c in (a, b)]
    for c in (a, b):
        for t in c[1]:
            t.zero_()
    sync()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a[0](s1.cuda_stream)
    b[0](s2.cuda_stream)
    sync()
    for c, w in zip((a, b), want):
        for got, ref in zip(c[1], w):
            assert torch.equal(got, ref)


# ------------------------------------------------------------------ offsets beyond 2^31 elements
def test_qknorm_beyond_32_bit_offsets():
    T, Hq, Hkv, hd = 360001, 32, 8, 128
    W, tail = (Hq + 2 * Hkv) * hd, 5
    assert T * W > 2 ** 31
    small, gq, gk, dy_s, _ = qk_inputs(tail, Hq, Hkv, hd, seed=41)
    tab = table(64, hd)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-tail:] = torch.arange(7, 7 + tail, dtype=torch.int32, device="cuda")
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[-tail:], dy[-tail:] = small, dy_s
    p = lambda t: t.data_ptr()
    outs = []
    for xx, dd, pp, n in ((x, dy, pos, T), (small, dy_s, pos[-tail:].contiguous(), tail)):
        sc = torch.empty(sf.qknorm_rope_bwd_scratch(n, Hq, Hkv, hd), **F32T)
        dg = torch.empty(2, hd, dtype=torch.bfloat16, device="cuda")
        y, dx = torch.empty_like(xx), torch.empty_like(xx)
        qk = (n, 64, Hq, Hkv, hd, p(gq), p(gk), EPS, p(tab), p(pp))
        assert sf.op_qknorm_rope_fwd(p(xx), W, p(y), W, *qk, stream()) == 0
        assert sf.op_qknorm_rope_bwd(p(xx), W, p(dd), W, p(dx), W, *qk, p(sc), p(dg[0]), p(dg[1]), stream()) == 0
        sync()
        outs.append((y[-tail:].clone(), dx[-tail:].clone()))
        assert n == tail or not (y[:-tail].any() or dx[:-tail].any())
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_window_beyond_32_bit_offsets():
    B, S, Hq, Hkv, hd, W, n = 11, 2 ** 20 + 40, 1, 1, 64, 70, 2
    assert B * S * 3 * hd > 2 ** 31
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=42)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, W, n)
    got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, W, n, None, 1)
    last = slice((B - 1) * S, B * S)
    o1, lse1 = win_fwd(qkv[last], 1, S, Hq, Hkv, hd, W, n)
    assert torch.equal(o[last], o1) and torch.equal(lse[-1:], lse1)
    one = win_bwd(qkv[last], o1, dout[last].contiguous(), lse1, 1, S, Hq, Hkv, hd, W, n, None, 1)
    assert torch.equal(got[last], one)
    # and its first 600 tokens against the definition
    c = 600
    ref, tol, _ = attn_ref(qkv[last][:c], 1, c, Hq, Hkv, hd, W, n)
    within(o1[:c], ref, tol)


def test_ckpt8_beyond_32_bit_offsets():
    rows, d = 140000, 16384
    assert rows * d > 2 ** 31
    x = torch.zeros(rows, d, **F32T)
    small, g, dy_s, _ = ckpt_inputs(3, d, seed=43)
    x[-3:] = small
    p = lambda t: t.data_ptr()
    E = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")
    outs = []
    for xx, n in ((x, rows), (small, 3)):
        q, s, v, y, r = E(torch.uint8, n, d), E(torch.float32, n, d // 128), E(torch.float32, n, d), \
            E(torch.bfloat16, n, d), E(torch.float32, n)
        assert sf.op_ckpt8_save(p(xx), p(q), p(s), 0, n, d, stream()) == 0
        assert sf.op_ckpt8_load(p(q), p(s), p(v), 0, n, d, stream()) == 0
        assert sf.op_rmsnorm_fwd_load8(p(q), p(s), p(g), p(y), p(r), 0, 0, n, d, EPS, stream()) == 0
        dy = torch.zeros(n, d, **F32T)
        dy[-3:] = dy_s
        part, dg, dxb = E(torch.float32, sf.rmsnorm_bwd_scratch(n, d)), E(torch.bfloat16, d), E(torch.bfloat16, n, d)
        dx = E(torch.float32, n, d)
        assert sf.op_rmsnorm_bwd_load8(p(q), p(s), p(g), p(r), p(dy), 0, p(dx), p(dxb), p(dg), p(part), 0, n, d,
                                       stream()) == 0
        sync()
        outs.append([t[-3:].clone() for t in (q, s, v, y, r, dx, dxb)])
        del q, s, v, y, dy, dx, dxb
    for a, b in zip(*outs):
        assert torch.equal(a, b)
