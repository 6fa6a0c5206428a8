"""Log probabilities of given tokens, entropies and alternatives, and their
gradients, through the C ABI, against their definitions in 64 bits.

Tolerances.  An exponential is off by 2^-21 of itself and by 2^-23 of its
argument's size, which where it matters is below 32: 2^-18 in all.  A sum's
chain (a thread's logits, at most vocab / 128 of them, then trees of about 64
in all) adds 2^-24 a step.  REL(vocab) is the sum of both; the logarithm turns
it into an absolute error."""
import math

import pytest
import torch

from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

BF, U = 2.0 ** -8, 2.0 ** -24
T32 = dict(dtype=torch.float32, device="cuda")
I32 = dict(dtype=torch.int32, device="cuda")
INF = math.inf


def REL(vocab):
    return 2.0 ** -18 + (vocab / 128 + 64) * U


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


def logits(rows, vocab, pad, dtype, seed=1, spread=2.0):
    z = torch.full((rows, (vocab + 7) // 8 * 8 + pad), 1e30, **T32).to(dtype)  # never to be looked at
    z[:, :vocab] = spread * gen(seed)(rows, vocab)
    return z


class Rows:
    """One call's outputs, each followed by elements that must stay as they are."""

    def __init__(self, rows, top):
        f = lambda n, dt: torch.full((n + 16,), 7, dtype=dt, device="cuda")
        self.rows, self.top = rows, top
        self.flat = [f(rows, torch.float32) for _ in range(3)] + [f(rows * top, torch.int32), f(rows * top, torch.float32)]
        self.logp, self.lse, self.entropy = (t[:rows] for t in self.flat[:3])
        self.ids, self.top_logp = (t[:rows * top].view(rows, top) for t in self.flat[3:])

    def call(self, z, vocab, tokens, scale=1.0, entropy=True):
        kind = sf.F32 if z.dtype == torch.float32 else sf.BF16
        return sf.op_logprob_rows(z.data_ptr(), kind, z.shape[1], tokens.data_ptr(), self.rows, vocab, scale,
                                  self.logp.data_ptr(), self.lse.data_ptr(), self.entropy.data_ptr() if entropy else 0,
                                  self.top, self.ids.data_ptr(), self.top_logp.data_ptr(), stream=stream())

    def untouched(self):
        for t, n in zip(self.flat, [self.rows] * 3 + [self.rows * self.top] * 2):
            assert (t[n:] == 7).all()


def near(got, ref, tol):
    """Equal where the reference is not finite, within tol elsewhere."""
    got, fine = got.double(), torch.isfinite(ref)
    assert torch.equal(got[~fine], ref[~fine]), (got[~fine][:4], ref[~fine][:4])
    over = (got[fine] - ref[fine]).abs() - (tol[fine] if torch.is_tensor(tol) else tol)
    assert over.numel() == 0 or over.max().item() <= 0.0, over.max().item()


def reference(z, vocab, tokens, scale):
    t = z[:, :vocab].double() * scale
    # differences to the largest first: the lowest value of a type leaves nothing of a logarithm beside it
    m = t.amax(1, keepdim=True)
    x = torch.where(torch.isinf(t), t, t - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    ls = torch.log(torch.exp(x).sum(1))
    lse = torch.where(torch.isinf(ls), ls, m[:, 0] + ls)
    lp = torch.where(torch.isinf(x), x, x - torch.where(torch.isinf(ls), torch.zeros_like(ls), ls)[:, None])
    p = torch.exp(lp)
    h = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    at = torch.gather(lp, 1, tokens.clamp(0, vocab - 1).long()[:, None])[:, 0]
    logp = torch.where(tokens < 0, torch.zeros_like(at), at)
    values, ids = torch.sort(t, dim=1, descending=True, stable=True)
    return lse, lp, p, h, logp, ids, torch.gather(lp, 1, ids)


def check(z, vocab, tokens, top, scale=1.0):
    out = Rows(z.shape[0], top)
    assert out.call(z, vocab, tokens, scale) == 0
    sync()
    lse, lp, p, h, logp, ids, tl = reference(z, vocab, tokens, scale)
    rel = REL(vocab)
    big = (z[:, :vocab].double() * scale)
    big = torch.where(torch.isfinite(big), big.abs(), torch.zeros_like(big)).amax(1)
    near(out.lse, lse, rel + 4 * U * (big + 1))
    near(out.logp, logp, rel + 4 * U * torch.where(torch.isfinite(logp), logp.abs(), torch.zeros_like(logp)) + 4 * U)
    # log S and T / S, each to its relative error; T / S is at most the entropy
    near(out.entropy, h, rel * (1 + 3 * h) + 4 * U * (1 + h))
    assert torch.equal(out.ids, ids[:, :top].int())
    tl = tl[:, :top]
    near(out.top_logp, tl, rel + 4 * U * (1 + torch.where(torch.isfinite(tl), tl.abs(), torch.zeros_like(tl))))
    out.untouched()
    return out


SIZES = [(1, 1, 0, 1), (3, 7, 8, 7), (5, 50, 0, 20), (4, 255, 8, 32), (2, 2048, 0, 5), (3, 2049, 64, 32),
         (700, 3000, 0, 3), (2, 8197, 0, 20), (5, 32000, 0, 32), (3, 128256, 8, 20), (1, 152064, 0, 32),
         (2, 300001, 0, 20), (160, 128256, 0, 20), (1, 1 << 20, 0, 32), (1300, 2051, 0, 32), (2500, 2051, 0, 32), (2501, 4096, 8, 20), (12, 1000, 0, 17)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,pad,top", SIZES)
def test_rows(rows, vocab, pad, top, dtype):
    z = logits(rows, vocab, pad, dtype)
    tokens = torch.randint(0, vocab, (rows,), **I32)
    tokens[::3] = z[::3, :vocab].float().argmax(1).int()
    tokens[1::4] = -100
    for scale in (1.0, 0.37):
        check(z, vocab, tokens, top, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 2050, 20011, 128256])
def test_rows_with_ties_and_masks(vocab, dtype):
    """Equal logits anywhere, masked ones of -inf and of the type's lowest value,
    rows with fewer unmasked logits than alternatives, peaked and large rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    low = torch.finfo(dtype).min
    rows = []
    base = 2 * torch.randn(vocab, generator=g, **T32)
    rows.append(torch.zeros(vocab, **T32))                      # all equal
    rows.append(torch.round(base))                              # few values
    rows.append(torch.randint(-1, 2, (vocab,), generator=g, **T32) * 0.0)  # zeros of both signs
    rows.append(torch.full((vocab,), -INF, **T32))              # nothing left
    for value in (-INF, low):
        one = torch.full((vocab,), value, **T32)
        one[vocab - 1] = 3.0                                    # one left, the last
        rows.append(one)
        few = torch.full((vocab,), value, **T32)
        few[torch.randperm(vocab, generator=g, device="cuda")[:17]] = base[:17]
        rows.append(few)
        half = base.clone()
        half[vocab // 3:] = value
        rows.append(half)
        rows.append(torch.where(torch.rand(vocab, generator=g, **T32) < 0.5, base, torch.full_like(base, value)))
    rows.append(torch.full((vocab,), low, **T32))               # the lowest value everywhere
    peak = base.clone()
    peak[vocab // 2] = 90.0
    rows.append(peak)
    rows.append(base * 500)                                     # far apart
    rows.append(base + 30000)                                   # large
    block = base.clone()
    block[vocab // 4:vocab // 4 + min(vocab // 2, 5000)] = 7.5  # a long run of the largest value
    rows.append(block)
    rows.append(torch.sort(base).values)                        # rising
    rows.append(torch.sort(base, descending=True).values)       # falling
    z = torch.zeros(len(rows), (vocab + 7) // 8 * 8, **T32).to(dtype)
    z[:, :vocab] = torch.stack(rows)
    z[2, ::3] = -0.0
    tokens = torch.full((len(rows),), vocab - 1, **I32)
    check(z, vocab, tokens, 32)
    check(z, vocab, tokens, 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [9, 5000, 128256])
def test_rows_that_are_not_finite(vocab, dtype):
    z = logits(6, vocab, 0, dtype)
    for r, (at, value) in enumerate([(0, math.nan), (vocab - 1, math.nan), (vocab // 2, INF), (vocab // 3, INF)]):
        z[r, at] = value
    z[3, vocab // 2] = -INF
    tokens = torch.tensor([1, 0, vocab // 2, -100, 2, -1], **I32)
    out = Rows(6, 5)
    assert out.call(z, vocab, tokens) == 0
    sync()
    assert torch.isnan(out.lse[:4]).all() and torch.isnan(out.entropy[:4]).all()
    assert torch.isnan(out.logp[:3]).all() and out.logp[3] == 0 and out.logp[5] == 0
    assert (out.ids[:4] == -1).all() and torch.isnan(out.top_logp[:4]).all()
    lse, _, _, _, _, ids, _ = reference(z[4:], vocab, tokens[4:], 1.0)
    near(out.lse[4:], lse, REL(vocab) + 1e-6)
    assert torch.equal(out.ids[4:], ids[:, :5].int())
    out.untouched()


def test_rows_without_entropy_or_alternatives():
    z = logits(10, 4099, 0, torch.float32)
    tokens = torch.arange(10, **I32)
    full, part = Rows(10, 4), Rows(10, 0)
    assert full.call(z, 4099, tokens) == 0 and part.call(z, 4099, tokens, entropy=False) == 0
    sync()
    # without the entropy a row's sums may be taken in another order
    near(part.lse, full.lse.double(), 2 * REL(4099))
    near(part.logp, full.logp.double(), 2 * REL(4099))
    assert (part.entropy == 7).all()
    part.untouched()


def test_a_token_beyond_the_vocabulary_is_reported():
    z = logits(4, 100, 0, torch.float32)
    tokens = torch.tensor([3, 100, 2 ** 31 - 1, 99], **I32)
    out = Rows(4, 2)
    assert out.call(z, 100, tokens) == 0
    assert sf.device_error() == 4
    assert (out.logp[1:3] == 0).all() and (out.logp[[0, 3]] < 0).all()
    dz = torch.full((4, 104), 5.0, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(4, **T32)
    assert sf.op_logprob_rows_bwd(z.data_ptr(), sf.F32, 104, tokens.data_ptr(), 4, 100, 1.0, out.lse.data_ptr(), 0,
                                  ones.data_ptr(), 0, dz.data_ptr(), 104, stream=stream()) == 0
    assert sf.device_error() == 4
    assert (dz[1:3, :100] == 0).all() and (dz[[0, 3], :100] != 0).any() and (dz[:, 100:] == 5).all()


def test_rows_beyond_2_31_logits():
    rows, vocab = 17000, 128256
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    z[-1] = logits(1, vocab, 0, torch.bfloat16, seed=7)[0]
    tokens = torch.full((rows,), vocab - 1, **I32)
    out = Rows(rows, 3)
    assert out.call(z, vocab, tokens) == 0
    dl, de = torch.full((rows,), 0.5, **T32), torch.full((rows,), 0.25, **T32)
    assert sf.op_logprob_rows_bwd(z.data_ptr(), sf.BF16, vocab, tokens.data_ptr(), rows, vocab, 1.0,
                                  out.lse.data_ptr(), out.entropy.data_ptr(), dl.data_ptr(), de.data_ptr(),
                                  z.data_ptr(), vocab, stream=stream()) == 0  # in place
    sync()
    near(out.lse[:-1], torch.full((rows - 1,), math.log(vocab), dtype=torch.float64, device="cuda"), REL(vocab) + 1e-6)
    assert (out.ids[:-1] == torch.arange(3, **I32)).all()
    last = logits(1, vocab, 0, torch.bfloat16, seed=7)
    lse, _, _, h, _, ids, _ = reference(last, vocab, tokens[-1:], 1.0)
    near(out.lse[-1:], lse, REL(vocab) + 8 * U * lse.abs())
    assert torch.equal(out.ids[-1:], ids[:, :3].int())
    ref, size, lp = gradient(last, vocab, tokens[-1:], 1.0, out.lse[-1:].double(), out.entropy[-1:].double(),
                             dl[-1:].double(), de[-1:].double())
    near(z[-1:], ref, BF * ref.abs() + (2.0 ** -20 + 4 * U * lp.abs()) * size + 1e-37)


def test_rows_on_two_streams():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    data = [(logits(400, 5003, 0, torch.float32, seed=s), torch.arange(400, **I32)) for s in (1, 2)]
    outs = [Rows(400, 7), Rows(400, 7)]
    sync()
    for (z, tokens), out, side in zip(data, outs, sides):
        with torch.cuda.stream(side):
            assert out.call(z, 5003, tokens) == 0
    sync()
    for (z, tokens), out in zip(data, outs):
        again = Rows(400, 7)
        assert again.call(z, 5003, tokens) == 0
        sync()
        assert all(torch.equal(a, b) for a, b in zip(again.flat, out.flat))


def test_rows_of_few_sets_of_large_logits():
    """Many logits above the bound that the threads' maxima give, rising: the list overflows again and again."""
    vocab = 128256
    z = logits(400, vocab, 0, torch.float32)
    own = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    own[(torch.arange(vocab, device="cuda") // 8) % 256 < 60] = True  # 15 sets of 4 threads of a row's 256
    z[:, own] = torch.linspace(10, 20, int(own.sum()), **T32)
    check(z[::50].contiguous(), vocab, torch.zeros(8, **I32), 32)
    check(z, vocab, torch.zeros(400, **I32), 32)


# ------------------------------------------------------------------ gradients of rows
def gradient(z, vocab, tokens, scale, lse, h, dl, de):
    t = z[:, :vocab].double() * scale
    lp = t - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]
    p = torch.exp(lp)
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    hot = torch.zeros_like(p)
    live = (tokens >= 0) & (tokens < vocab)
    hot[torch.arange(len(tokens), device="cuda")[live], tokens[live].long()] = 1.0
    dl = torch.where(live, dl, torch.zeros_like(dl))[:, None]
    g = dl * (hot - p) - de[:, None] * p * (lp + h[:, None])
    size = dl.abs() * (hot + p) + de.abs()[:, None] * p * (lp.abs() + h.abs()[:, None])
    return scale * g, scale * size, lp


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,pad,top", SIZES)
def test_rows_backward(rows, vocab, pad, top, dtype):
    z = logits(rows, vocab, pad, dtype, seed=2)
    tokens = torch.randint(0, vocab, (rows,), **I32)
    tokens[1::4] = -1
    scale = 0.8
    rnd = gen(5)
    dl, de = rnd(rows), 0.1 * rnd(rows)
    de[1::8] = 0.0  # with no token either: zeros, whatever the logits
    z[1::8] = math.nan
    lse, _, _, h, _, _, _ = reference(torch.nan_to_num(z), vocab, tokens, scale)
    lse32, h32 = lse.float(), h.float()
    lse32[1::8] = math.nan
    ld = z.shape[1] + 8
    flat = torch.full((rows * ld + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    dz = flat[:rows * ld].view(rows, ld)
    kind = sf.F32 if dtype == torch.float32 else sf.BF16
    args = (lse32.data_ptr(), h32.data_ptr(), dl.data_ptr(), de.data_ptr())
    assert sf.op_logprob_rows_bwd(z.data_ptr(), kind, z.shape[1], tokens.data_ptr(), rows, vocab, scale, *args,
                                  dz.data_ptr(), ld, stream=stream()) == 0
    sync()
    ref, size, lp = gradient(torch.nan_to_num(z), vocab, tokens, scale, lse32.nan_to_num().double(), h32.double(),
                             dl.double(), de.double())
    ref[1::8], size[1::8] = 0.0, 0.0
    # an exponential's error, and the rounding of lp (2^-24 of its size) in it and beside it
    rel = 2.0 ** -20 + 4 * U * lp.abs()
    near(dz[:, :vocab], ref, BF * ref.abs() + (rel * size) + 1e-37)
    assert (dz[:, vocab:] == 7).all() and (flat[rows * ld:] == 7).all()
    if dtype == torch.bfloat16:  # in place
        pad_before = z[:, vocab:].clone()
        assert sf.op_logprob_rows_bwd(z.data_ptr(), kind, z.shape[1], tokens.data_ptr(), rows, vocab, scale, *args,
                                      z.data_ptr(), z.shape[1], stream=stream()) == 0
        sync()
        assert torch.equal(z[:, :vocab], dz[:, :vocab]) and torch.equal(z[:, vocab:].nan_to_num(), pad_before.nan_to_num())


def test_rows_backward_with_masks():
    vocab = 5000
    z = logits(4, vocab, 0, torch.float32)
    z[0, ::2] = -INF
    z[1] = -INF                        # nothing left
    z[2] = torch.finfo(torch.float32).min
    z[2, 7] = 1.0                      # one left
    z[3, 5] = math.nan
    tokens = torch.tensor([1, 3, 7, 2], **I32)
    out = Rows(4, 0)
    assert out.call(z, vocab, tokens) == 0
    dl, de = torch.ones(4, **T32), torch.full((4,), 0.5, **T32)
    dz = torch.empty(4, vocab, dtype=torch.bfloat16, device="cuda")
    assert sf.op_logprob_rows_bwd(z.data_ptr(), sf.F32, vocab, tokens.data_ptr(), 4, vocab, 1.0, out.lse.data_ptr(),
                                  out.entropy.data_ptr(), dl.data_ptr(), de.data_ptr(), dz.data_ptr(), vocab,
                                  stream=stream()) == 0
    sync()
    ref, size, lp = gradient(z[:1], vocab, tokens[:1], 1.0, out.lse[:1].double(), out.entropy[:1].double(),
                             dl[:1].double(), de[:1].double())
    near(dz[:1], ref, BF * ref.abs() + 2.0 ** -18 * size)
    assert (dz[0, ::2] == 0).all() and (dz[1] == 0).all()
    # p is 1: the gradient is that of a sure thing, up to lse's rounding
    assert (dz[2].float().abs() <= 1e-6).all() and torch.isnan(dz[3]).all()


def test_rows_gradient_against_differences():
    """Central differences of the kernel's own forward along a direction."""
    vocab, rows = 1000, 16
    z = logits(rows, vocab, 0, torch.float32, spread=1.0)
    tokens = torch.randint(0, vocab, (rows,), **I32)
    rnd = gen(9)
    dl, de, way = rnd(rows), rnd(rows), rnd(rows, vocab)
    out = Rows(rows, 0)
    assert out.call(z, vocab, tokens, 0.9) == 0
    dz = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    assert sf.op_logprob_rows_bwd(z.data_ptr(), sf.F32, vocab, tokens.data_ptr(), rows, vocab, 0.9, out.lse.data_ptr(),
                                  out.entropy.data_ptr(), dl.data_ptr(), de.data_ptr(), dz.data_ptr(), vocab,
                                  stream=stream()) == 0
    e, values = 2.0 ** -6, []
    for s in (1, -1):
        shifted = z + s * e * way
        o = Rows(rows, 0)
        assert o.call(shifted, vocab, tokens, 0.9) == 0
        sync()
        values.append(dl.double() * o.logp.double() + de.double() * o.entropy.double())
    diff = (values[0] - values[1]) / (2 * e)
    slope = (dz.double() * way.double()).sum(1)
    # the forward's error over 2e, the third derivative (logits move by at most 4 e: cumulants of a
    # direction of unit size, at most about 30 with the entropy's factors) and dz's rounding
    size = dl.abs().double() + 8 * de.abs().double()
    tol = 2 * REL(vocab) * 8 * size / (2 * e) + 30 * e * e * size + BF * (dz.double() * way.double()).abs().sum(1)
    assert ((diff - slope).abs() <= tol).all()


# ------------------------------------------------------------------ the head
LM = [(1, 8, 8, 1), (5, 64, 104, 2), (130, 136, 520, 64), (300, 384, 3000, 128), (129, 512, 4096, 1000),
      (257, 256, 32000, 100), (70, 64, 104, 1), (700, 128, 520, 100), (128, 1024, 512, 7), (128, 64, 20000, 500)]


def lm_inputs(n, d, v, seed=4):
    rnd = gen(seed)
    h, w = rnd(n, d).bfloat16(), (1.5 / math.sqrt(d) * rnd(v, d)).bfloat16()
    tokens = torch.randint(0, v, (n,), **I32)
    tokens[2::5] = -100
    return h, w, tokens


def lm_errors(h, w, scale):
    """What fp32 sums of d products leave on a logit."""
    d = h.shape[1]
    return scale * (2.0 ** -20 * math.sqrt(d) + d * U) * (h.double().norm(dim=1) * w.double().norm(dim=1).max())


@pytest.mark.parametrize("n,d,v,chunk", LM)
def test_lm_logprob(n, d, v, chunk):
    h, w, tokens = lm_inputs(n, d, v)
    top, scale = min(v, 9), 0.7
    out = Rows(n, top)
    size = sf.lm_logprob_workspace_bytes(n, v, chunk)
    ws = torch.full((size + 256,), 7, dtype=torch.uint8, device="cuda")
    assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, scale, chunk, ws.data_ptr(),
                            out.logp.data_ptr(), out.lse.data_ptr(), out.entropy.data_ptr(), top, out.ids.data_ptr(),
                            out.top_logp.data_ptr(), stream=stream()) == 0
    sync()
    z = h.double() @ w.double().t()
    lse, lp, p, ent, logp, ids, tl = reference(z, v, tokens, scale)
    te, rel = lm_errors(h, w, scale), REL(v)
    near(out.lse, lse, te + rel + 4 * U * lse.abs() + 8 * U)
    near(out.logp, logp, 2 * te + rel + 4 * U * logp.abs() + 8 * U)
    near(out.entropy, ent, te * 2 * (1 + ent) + rel * (1 + 3 * ent) + 8 * U * (1 + ent))
    # logits nearer than their errors may change places
    near(out.top_logp, tl[:, :top], (2 * te + rel)[:, None] + 8 * U * (1 + tl[:, :top].abs()))
    got = torch.gather(lp, 1, out.ids.long())
    assert ((got - tl[:, :top]).abs() <= 4 * te[:, None]).all()
    assert all(len(set(r)) == top for r in out.ids.tolist())
    out.untouched()
    assert (ws[size:] == 7).all()


@pytest.mark.parametrize("entropy", [True, False])
@pytest.mark.parametrize("n,d,v,chunk", LM)
def test_lm_logprob_backward(n, d, v, chunk, entropy):
    h, w, tokens = lm_inputs(n, d, v)
    scale, rnd = 0.7, gen(8)
    dl, de = rnd(n), 0.1 * rnd(n) * entropy
    z = h.double() @ w.double().t()
    lse, _, _, ent, _, _, _ = reference(z, v, tokens, scale)
    lse, ent = lse.float(), ent.float()
    size = sf.lm_logprob_bwd_workspace_bytes(n, d, v, chunk)
    ws = torch.full((size + 256,), 7, dtype=torch.uint8, device="cuda")
    dh = torch.full((n + 1, d), 7, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((v + 1, d), 7, dtype=torch.bfloat16, device="cuda")
    assert sf.op_lm_logprob_bwd(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, scale, chunk, lse.data_ptr(),
                                ent.data_ptr() if entropy else 0, dl.data_ptr(), de.data_ptr() if entropy else 0,
                                ws.data_ptr(), dh.data_ptr(), dw.data_ptr(), stream=stream()) == 0
    sync()
    dz, size_z, lp = gradient(z, v, tokens, scale, lse.double(), ent.double(), dl.double(), de.double())
    # dz's bf16 rounding (up to 128 rows what it leaves is kept), the exponential, the logit's error in p and in log p
    te = lm_errors(h, w, scale)[:, None]
    ez = (BF * BF if n <= 128 else BF) * dz.abs() + (2.0 ** -20 + 4 * U * lp.abs() + 2 * te) * size_z + te * (scale * de.abs().double()[:, None] * torch.exp(lp))
    f32 = 2.0 ** -18
    ref = dz @ w.double()
    near(dh[:n], ref, BF * ref.abs() + ez @ w.double().abs() + f32 * (dz.abs() @ w.double().abs()))
    ref = dz.t() @ h.double()
    near(dw[:v], ref, BF * ref.abs() + ez.t() @ h.double().abs() + f32 * (dz.abs().t() @ h.double().abs()))
    assert (dh[n:] == 7).all() and (dw[v:] == 7).all() and (ws[size:] == 7).all()


def test_lm_logprob_agrees_with_the_loss():
    """The head's mean loss and its gradient are those of sf_op_lce with dlogp = -1 / n_valid."""
    n, d, v, chunk = 300, 256, 3000, 128
    h, w, tokens = lm_inputs(n, d, v)
    valid = int((tokens >= 0).sum())
    loss, dh, dw = torch.empty(1, **T32), torch.empty(n, d, **T32), torch.empty(v, d, **T32)
    ws = torch.empty(sf.lce_workspace_bytes(n, v, chunk), dtype=torch.uint8, device="cuda")
    assert sf.op_lce(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, valid, chunk, ws.data_ptr(),
                     loss.data_ptr(), dh.data_ptr(), dw.data_ptr(), stream=stream()) == 0
    out = Rows(n, 0)
    wf = torch.empty(sf.lm_logprob_workspace_bytes(n, v, chunk), dtype=torch.uint8, device="cuda")
    assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 1.0, chunk, wf.data_ptr(),
                            out.logp.data_ptr(), out.lse.data_ptr(), stream=stream()) == 0
    wb = torch.empty(sf.lm_logprob_bwd_workspace_bytes(n, d, v, chunk), dtype=torch.uint8, device="cuda")
    dl = torch.full((n,), -1.0 / valid, **T32)
    dh2, dw2 = torch.empty(n, d, dtype=torch.bfloat16, device="cuda"), torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    assert sf.op_lm_logprob_bwd(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 1.0, chunk, out.lse.data_ptr(),
                                0, dl.data_ptr(), 0, wb.data_ptr(), dh2.data_ptr(), dw2.data_ptr(), stream=stream()) == 0
    sync()
    assert abs(loss.item() + out.logp.double().sum().item() / valid) <= 1e-5 * loss.item()
    for a, b in ((dh, dh2), (dw, dw2)):
        # both round dz to bf16 (the exponentials' last bits may round apart), the second its result too
        assert (a.double() - b.double()).norm() <= 1.5 * BF * a.double().norm()
