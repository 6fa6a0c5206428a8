"""The same operators where their loops run many times: rings in shared memory
that wrap, thread groups that take several rows, and persistent CTAs that go from
item to item, on a device of any size.  Definitions, inputs and tolerances are
those of the tests of single passes."""
import pytest
import torch

from tests.gpu_util import stream, sync
from tests.test_gpu_attention_half import (BF, D64, EPS, F32, F32T, _lib, attn_bwd_ref, attn_ref, ckpt_inputs,
                                           ckpt_ref, guarded, qk_inputs, qk_ref, table, untouched, win_bwd, win_fwd,
                                           win_inputs, within)

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ norm backward from the codes
@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("fmt,top", [(0, 127.0), (1, 448.0)])
@pytest.mark.parametrize("d,groups", [(128, 16), (1000, 8), (4096, 2), (8192, 1), (12288, 1), (16384, 1)])
def test_norm_backward_of_many_rows(d, groups, fmt, top, with_res):
    """At most `groups` rows at a time in each of the device's CTAs: six rows or
    more for each thread group, so the ring (two or three rows) wraps, and an
    uneven end.  dx and dxb of every row, dg over all of them."""
    rows = 6 * sms() * groups + groups + 1
    x, g, dy, dres = ckpt_inputs(rows, d, seed=d + fmt)
    p = lambda t: t.data_ptr()
    nb = (d + 127) // 128
    q, s = torch.empty(rows, d, dtype=torch.uint8, device="cuda"), torch.empty(rows, nb, **F32T)
    v, y = torch.empty(rows, d, **F32T), torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    r = torch.empty(rows, **F32T)
    assert sf.op_ckpt8_save(p(x), p(q), p(s), fmt, rows, d, stream()) == 0
    assert sf.op_rmsnorm_fwd_load8(p(q), p(s), p(g), p(y), p(r), p(v), fmt, rows, d, EPS, stream()) == 0
    (dx, dt), (dxb, bt), (dg, gt) = (guarded((rows, d), torch.float32), guarded((rows, d), torch.bfloat16),
                                     guarded((d,), torch.bfloat16))
    sc, sct = guarded((sf.rmsnorm_bwd_scratch(rows, d),), torch.float32)
    assert sf.op_rmsnorm_bwd_load8(p(q), p(s), p(g), p(r), p(dy), p(dres) if with_res else 0, p(dx), p(dxb), p(dg),
                                   p(sc), fmt, rows, d, stream()) == 0
    sync()
    untouched(dt, bt, gt, sct)
    if rows * d < 2 ** 22:  # the rule itself, on the host
        assert torch.equal(v, ckpt_ref(x, top)[2])
    ref, size_g = torch.zeros(d, **D64), torch.zeros(d, **D64)
    for a in range(0, rows, 512):  # float64 in slices
        c = slice(a, a + 512)
        rr = r[c].double()[:, None]
        assert ((rr[:, 0] * torch.sqrt((v[c].double() ** 2).mean(1) + EPS) - 1).abs() <= F32).all()
        xh, w = v[c].double() * rr, dy[c].double() * g.double()
        base = dres[c].double() if with_res else torch.zeros_like(xh)
        dx_ref = base + rr * (w - xh * (w * xh).mean(1, keepdim=True))
        size = base.abs() + rr * (w.abs() + xh.abs() * (w * xh).abs().mean(1, keepdim=True))
        within(dx[c], dx_ref, F32 * size)
        within(dxb[c], dx_ref, BF * dx_ref.abs() + F32 * size)
        ref += (dy[c].double() * xh).sum(0)
        size_g += (dy[c].double() * xh).abs().sum(0)
    within(dg, ref, BF * ref.abs() + F32 * size_g)


# ------------------------------------------------------------------ query/key norms
@pytest.mark.parametrize("Hq,Hkv,hd,pads", [
    (16, 4, 128, (0, 8, 24, 16)),
    (12, 3, 80, (8, 0, 16, 40)),
    (4, 4, 256, (16, 64, 0, 8)),
    (6, 2, 16, (0, 0, 8, 0)),
])
def test_qknorm_of_many_steps_and_four_strides(Hq, Hkv, hd, pads):
    """Twelve or more steps for each warp of a full grid, so its ring of five wraps;
    x, y, dy and dx each with a row stride of its own."""
    per = 32 // max(1, 2 ** ((hd // 16 - 1).bit_length()))  # heads of a step
    steps = min(-(-Hq // per), -(-Hkv // per))              # of a token, in the shorter phase
    T = 12 * 4 * 5 * sms() // steps + 3
    seq = 700
    x, gq, gk, _, W = qk_inputs(T, Hq, Hkv, hd, pads[0], seed=hd)
    _, _, _, dy, _ = qk_inputs(T, Hq, Hkv, hd, pads[2], seed=hd)
    ldx, ldy, lddy, lddx = (W + pad for pad in pads)
    tab, n = table(seq, hd), (Hq + Hkv) * hd
    pos = (torch.arange(T, device="cuda") * 7 + 3) % seq
    pos32 = pos.to(torch.int32)
    p = lambda t: t.data_ptr()
    (y, yt), (dx, dxt) = guarded((T, ldy), torch.bfloat16), guarded((T, lddx), torch.bfloat16)
    sc, sct = guarded((sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd),), torch.float32)
    (dgq, t1), (dgk, t2) = guarded((hd,), torch.bfloat16), guarded((hd,), torch.bfloat16)
    qk = (T, seq, Hq, Hkv, hd, p(gq), p(gk), EPS, p(tab), p(pos32))
    assert sf.op_qknorm_rope_fwd(p(x), ldx, p(y), ldy, *qk, stream()) == 0
    assert sf.op_qknorm_rope_bwd(p(x), ldx, p(dy), lddy, p(dx), lddx, *qk, p(sc), p(dgq), p(dgk), stream()) == 0
    sync()
    untouched(yt, dxt, sct, t1, t2)
    assert torch.equal(y[:, n:W], x[:, n:W]) and torch.equal(dx[:, n:W], dy[:, n:W])
    assert (y[:, W:] == 7).all() and (dx[:, W:] == 7).all()
    sums = [0.0] * 4
    for a in range(0, T, 4096):  # float64 in slices
        c = slice(a, a + 4096)
        y_ref, y_tol, dx_ref, dx_tol, out = qk_ref(x[c], gq, gk, dy[c], Hq, Hkv, hd, pos[c], tab)
        within(y[c, :n], y_ref, y_tol)
        within(dx[c, :n], dx_ref, dx_tol)
        # a slice's tolerance holds 2^-8 of its own sum; of the whole's is wanted
        for i in (0, 2):
            sums[i] = sums[i] + out[i]
            sums[i + 1] = sums[i + 1] + (out[i + 1] - BF * out[i].abs())
    within(dgq, sums[0], BF * sums[0].abs() + sums[1])
    within(dgk, sums[2], BF * sums[2].abs() + sums[3])


@pytest.mark.parametrize("T,Hq,Hkv,hd", [(5948, 3, 1, 64), (3, 8, 8, 144), (5, 9, 3, 176), (55, 8, 8, 256),
                                         (47, 16, 8, 80), (2748, 35, 5, 256), (5003, 16, 2, 128), (1, 1, 1, 16)])
def test_qknorm_gain_sums_in_place_and_beside(T, Hq, Hkv, hd):
    """The same order of the gains' sums whether the value heads are copied or stay."""
    x, gq, gk, dy, W = qk_inputs(T, Hq, Hkv, hd)
    tab, p = table(T, hd), lambda t: t.data_ptr()
    out = []
    for place in (False, True, False):
        d = dy.clone()
        dx = d if place else torch.empty_like(d)
        sc = torch.empty(sf.qknorm_rope_bwd_scratch(T, Hq, Hkv, hd), **F32T)
        dg = torch.empty(2, hd, dtype=torch.bfloat16, device="cuda")
        assert sf.op_qknorm_rope_bwd(p(x), W, p(d), W, p(dx), W, T, T, Hq, Hkv, hd, p(gq), p(gk), EPS, p(tab), 0,
                                     p(sc), p(dg[0]), p(dg[1]), stream()) == 0
        sync()
        out.append((dx, dg, sc))
    for other in out[1:]:
        for a, b in zip(out[0], other):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ windowed attention
MANY_ITEMS = [  # B, S, Hq, Hkv, hd, window, sinks: several items for each SM, forward and (head dim 64) backward
    (8, 1001, 16, 16, 64, 250, 0),
    (6, 2500, 16, 16, 64, 64, 130),   # with the sinks' far queries as items of their own
    (24, 1300, 12, 4, 64, 300, 17),   # odd groups: query blocks are paired in the forward
    (30, 600, 12, 12, 64, 1, 1),
    (8, 1001, 16, 16, 128, 250, 0),
    (24, 1300, 12, 4, 128, 300, 17),
    (6, 2500, 32, 8, 128, 64, 130),
]


@pytest.mark.parametrize("B,S,Hq,Hkv,hd,window,sinks", MANY_ITEMS)
def test_window_of_many_items(B, S, Hq, Hkv, hd, window, sinks):
    assert (S + 127) // 128 * Hkv * B > 2 * sms()
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=51)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, window, sinks)
    tab = table(S, hd)
    got = [win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, window, sinks, tab, det) for det in (0, 1)]
    for b in range(B):  # one sequence at a time: the float64 scores of all are too large
        rows = slice(b * S, (b + 1) * S)
        ref, tol, lref = attn_ref(qkv[rows], 1, S, Hq, Hkv, hd, window, sinks)
        within(o[rows], ref, tol)
        within(lse[b:b + 1], lref, 2.0 ** -15 + 2.0 ** -21 * lref.abs())
        ref, tol = attn_bwd_ref(qkv[rows], o[rows], dout[rows], lse[b:b + 1], 1, S, Hq, Hkv, hd, window, sinks, tab)
        for g in got:
            within(g[rows], ref, tol)


@pytest.mark.parametrize("det", [0, 1])
def test_window_gradients_beyond_32_bit_offsets(det):
    """The last of eleven long sequences (hundreds of items for each SM): the
    gradients of its first tokens against the definition."""
    B, S, Hq, Hkv, hd, W = 11, 2 ** 20 + 40, 1, 1, 64, 70
    c = 600
    qkv, dout = win_inputs(B, S, Hq, Hkv, hd, seed=42)
    o, lse = win_fwd(qkv, B, S, Hq, Hkv, hd, W, 0)
    got = win_bwd(qkv, o, dout, lse, B, S, Hq, Hkv, hd, W, 0, None, det)
    for b in (0, 5, B - 1):
        rows = slice(b * S, b * S + c)
        ref, tol = attn_bwd_ref(qkv[rows], o[rows], dout[rows], lse[b:b + 1, :, :c], 1, c, Hq, Hkv, hd, W, 0)
        within(got[rows, :hd], ref[:, :hd], tol[:, :hd])
        keys = slice(0, c - W)  # every query that sees them is among the first c
        within(got[rows][keys, hd:], ref[keys, hd:], tol[keys, hd:])
