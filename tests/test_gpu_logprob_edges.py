"""Log probabilities where their parts meet: rows that are nearly certain, large
gradients beside masked logits, the head's product that leaves only sums, tokens
beyond the vocabulary, captured graphs and repeated calls, through the C ABI.
Tolerances not derived here are those of the other tests of log probabilities."""
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


# ------------------------------------------------------------------ rows that are nearly certain
@pytest.mark.parametrize("rows,vocab", [(4, 64), (4, 1000), (3000, 2048), (5, 2051), (4, 8192), (4, 32000), (200, 32000),
                                        (400, 32000)])
@pytest.mark.parametrize("rest", ["one beside it", "all"])
def test_rows_that_are_nearly_certain(rows, vocab, rest):
    """log p of the likely token is -log(1 + q), q the others' weights, and keeps q's digits.

    With x = z - m, an exponential is off by 2^-21 of itself and by what the roundings of x, of the
    constant and of their product (2^-24 of |x| each, x below 32) leave: 4 * 32 * 2^-24 = 2^-17.  The
    others' sum takes vocab / 128 + 64 steps of 2^-24 at most; the maximum, 1, has to enter beside it
    without rounding it away."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.full((rows, (vocab + 7) // 8 * 8), -INF, **T32)
    at = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    near = (at // 8 * 8 + (at + 3) % 8).clamp(max=vocab - 1)  # in the same eight logits, or the last
    near = torch.where(near == at, (at + 1) % vocab, near)
    if rest == "all":
        z[:, :vocab] = -14.0 + torch.randn(rows, vocab, generator=g, **T32)
    r = torch.arange(rows, device="cuda")
    z[r, near] = -15.0 - 3 * torch.rand(rows, generator=g, **T32)
    z[r, at] = 7.0 if rest == "all" else 0.0
    out = base.Rows(rows, 1)
    assert out.call(z, vocab, at.int()) == 0
    sync()
    x = z[:, :vocab].double() - z[r, at].double()[:, None]
    x[r, at] = -INF
    q = torch.exp(x).sum(1)
    ref = -torch.log1p(q)
    rel = 2.0 ** -21 + 2.0 ** -17 + (vocab / 128 + 64) * U + 2 * U
    over = (out.logp.double() - ref).abs() / ref.abs()
    assert over.max().item() <= rel, over.max().item()
    over = (out.top_logp[:, 0].double() - ref).abs() / ref.abs()
    assert over.max().item() <= rel
    # entropy: log(1 + q) + sum of e |x| / (1 + q), each term to its relative error
    t = torch.where(torch.isinf(x), torch.zeros_like(x), -torch.exp(x) * x).sum(1)
    ent = torch.log1p(q) + t / (1 + q)
    assert ((out.entropy.double() - ent).abs() <= (rel + (vocab / 128 + 64) * U) * ent).all()


@pytest.mark.parametrize("n,d,v", [(3, 64, 520), (300, 64, 104), (130, 128, 3000)])
def test_the_head_of_nearly_certain_rows(n, d, v):
    """The same through the head's product: hidden states and weights whose logits are exact."""
    g = torch.Generator(device="cuda").manual_seed(v)
    tokens = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    # h of a row: 1 in one column; w of a token: the logits of that column's rows, small whole numbers
    w = torch.randint(-20, -14, (v, d), generator=g, device="cuda").to(torch.bfloat16)
    h = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    cols = torch.arange(n, device="cuda") % d
    h[torch.arange(n, device="cuda"), cols] = 1.0
    tokens = tokens[torch.arange(n, device="cuda") % d]  # one likely token for each column
    w[tokens.long(), cols] = 4.0
    out = base.Rows(n, 0)
    ws = torch.empty(sf.lm_logprob_workspace_bytes(n, v, 64), dtype=torch.uint8, device="cuda")
    assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 1.0, 64, ws.data_ptr(),
                            out.logp.data_ptr(), out.lse.data_ptr(), out.entropy.data_ptr(), stream=stream()) == 0
    sync()
    z = h.double() @ w.double().t()
    r = torch.arange(n, device="cuda")
    x = z - z[r, tokens.long()][:, None]
    x[r, tokens.long()] = -INF
    ref = -torch.log1p(torch.exp(x).sum(1))
    rel = 2.0 ** -21 + 2.0 ** -17 + (v / 128 + 64) * U + 2 * U
    over = (out.logp.double() - ref).abs() / ref.abs()
    assert over.max().item() <= rel, over.max().item()


# ------------------------------------------------------------------ the head's sums
def fused(h, w, tokens, scale, chunk, entropy=True):
    n, d, v = *h.shape, w.shape[0]
    out = base.Rows(n, 0)
    size = sf.lm_logprob_workspace_bytes(n, v, chunk)
    ws = torch.full((size + 256,), 7, dtype=torch.uint8, device="cuda")
    assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, scale, chunk, ws.data_ptr(),
                            out.logp.data_ptr(), out.lse.data_ptr(), out.entropy.data_ptr() if entropy else 0,
                            stream=stream()) == 0
    sync()
    assert (ws[size:] == 7).all()
    out.untouched()
    return out


def check_head(h, w, tokens, scale, out):
    v = w.shape[0]
    lse, _, _, ent, logp, _, _ = base.reference(h.double() @ w.double().t(), v, tokens, scale)
    te, rel = base.lm_errors(h, w, scale), base.REL(v)
    base.near(out.lse, lse, te + rel + 4 * U * lse.abs() + 8 * U)
    base.near(out.logp, logp, 2 * te + rel + 4 * U * logp.abs() + 8 * U)
    base.near(out.entropy, ent, te * 2 * (1 + ent) + rel * (1 + 3 * ent) + 8 * U * (1 + ent))


@pytest.mark.parametrize("scale", [1.0, 0.7, 1.6])
@pytest.mark.parametrize("n,d,v,chunk", base.LM + [(3000, 64, 104, 100), (40, 64, 8, 3), (33, 64, 128, 1), (64, 64, 136, 2)])
def test_lm_logprob_without_alternatives(n, d, v, chunk, scale):
    """The logits leave the product as sums, in one pass or in several, on tiles of 128 and of 256 columns."""
    h, w, tokens = base.lm_inputs(n, d, v)
    out = fused(h, w, tokens, scale, chunk)
    check_head(h, w, tokens, scale, out)
    part = fused(h, w, tokens, scale, chunk, entropy=False)
    assert torch.equal(part.logp, out.logp) and torch.equal(part.lse, out.lse) and (part.entropy == 7).all()


def test_head_tokens_beyond_the_vocabulary_are_reported():
    n, d, v = 200, 64, 520
    for few in (n, 20):
        h, w, tokens = base.lm_inputs(n, d, v)
        h, tokens = h[:few], tokens[:few]
        ref = fused(h, w, torch.where(torch.arange(few, device="cuda") % 3 == 0, -100, tokens).int(), 1.0, 64)
        tokens[::3] = v + torch.arange(len(tokens[::3]), **I32) * 1000
        out = fused(h, w, tokens, 1.0, 64)
        assert sf.device_error() == 4
        assert torch.equal(out.logp, ref.logp) and torch.equal(out.lse, ref.lse) and (out.logp[::3] == 0).all()
        dl, grads = torch.ones(few, **T32), []
        for t in (tokens, torch.where(tokens >= v, -1, tokens).int()):
            ws = torch.empty(sf.lm_logprob_bwd_workspace_bytes(few, d, v, 64), dtype=torch.uint8, device="cuda")
            dh, dw = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((few, d), (v, d)))
            assert sf.op_lm_logprob_bwd(h.data_ptr(), w.data_ptr(), t.data_ptr(), few, d, v, 1.0, 64,
                                        out.lse.data_ptr(), 0, dl.data_ptr(), 0, ws.data_ptr(), dh.data_ptr(),
                                        dw.data_ptr(), stream=stream()) == 0
            assert sf.device_error() == (4 if t is tokens else 0)
            grads.append((dh, dw))
        assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
        assert (grads[0][0][::3] == 0).all()


@pytest.mark.parametrize("n,d,v,chunk", [(5, 256, 3000, 2), (300, 256, 3000, 256), (1200, 128, 1032, 256)])
def test_head_repeated_and_captured(n, d, v, chunk):
    """The same bits from every call: again, after other work in the same workspace, and replayed."""
    h, w, tokens = base.lm_inputs(n, d, v)
    rnd = base.gen(3)
    dl, de = rnd(n), 0.1 * rnd(n)
    f, b = sf.lm_logprob_workspace_bytes(n, v, chunk), sf.lm_logprob_bwd_workspace_bytes(n, d, v, chunk)
    ws = torch.empty(max(f, b), dtype=torch.uint8, device="cuda")  # of both directions
    out = [torch.empty(n, **T32) for _ in range(3)] + [torch.empty_like(h), torch.empty_like(w)]
    p = [t.data_ptr() for t in out]

    def both():
        assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 0.9, chunk, ws.data_ptr(),
                                *p[:3], stream=stream()) == 0
        assert sf.op_lm_logprob_bwd(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 0.9, chunk, p[1], p[2],
                                    dl.data_ptr(), de.data_ptr(), ws.data_ptr(), p[3], p[4], stream=stream()) == 0

    both()
    sync()
    first = [t.clone() for t in out]

    def again(call):
        for t in out:
            t.fill_(7)
        ws.fill_(255)  # NaN wherever it is read before it is written
        call()
        sync()
        assert all(torch.equal(x, y) for x, y in zip(first, out))

    for _ in range(3):
        again(both)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        again(graph.replay)


def test_head_on_two_streams():
    n, d, v, chunk = 300, 256, 3000, 128
    data = [base.lm_inputs(n, d, v, seed=s) for s in (1, 2)]
    sides, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [base.Rows(n, 0), base.Rows(n, 0)]
    spaces = [torch.empty(sf.lm_logprob_workspace_bytes(n, v, chunk), dtype=torch.uint8, device="cuda") for _ in data]

    def call(x, out, ws):
        h, w, tokens = x
        assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), n, d, v, 1.0, chunk, ws.data_ptr(),
                                out.logp.data_ptr(), out.lse.data_ptr(), out.entropy.data_ptr(), stream=stream()) == 0

    sync()
    for _ in range(4):
        for x, out, ws, side in zip(data, outs, spaces, sides):
            with torch.cuda.stream(side):
                call(x, out, ws)
    sync()
    for x, out, ws in zip(data, outs, spaces):
        alone = base.Rows(n, 0)
        call(x, alone, ws)
        sync()
        assert all(torch.equal(a, b) for a, b in zip(alone.flat, out.flat))


# ------------------------------------------------------------------ rows, captured
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (20, 128256), (70, 32000), (160, 32000), (400, 32000), (9, 8192),
                                        (3000, 2048)])
def test_captured_rows_follow_their_inputs(rows, vocab, dtype):
    """Each shape of a row's threads and clusters in a graph, replayed over other logits and tokens."""
    z, tokens = base.logits(rows, vocab, 0, dtype), torch.zeros(rows, **I32)
    out = base.Rows(rows, 20)
    dl, de = torch.full((rows,), 0.5, **T32), torch.full((rows,), 0.25, **T32)
    dz = torch.empty(z.shape, dtype=torch.bfloat16, device="cuda")
    kind = sf.F32 if dtype == torch.float32 else sf.BF16

    def both():
        assert out.call(z, vocab, tokens, 0.9) == 0
        assert sf.op_logprob_rows_bwd(z.data_ptr(), kind, z.shape[1], tokens.data_ptr(), rows, vocab, 0.9,
                                      out.lse.data_ptr(), out.entropy.data_ptr(), dl.data_ptr(), de.data_ptr(),
                                      dz.data_ptr(), z.shape[1], stream=stream()) == 0

    both()
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (5, 6):
        z.copy_(base.logits(rows, vocab, 0, dtype, seed=seed))
        tokens.copy_(torch.randint(0, vocab, (rows,), **I32))
        graph.replay()
        sync()
        replayed = [t.clone() for t in (*out.flat, dz)]
        both()
        sync()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (*out.flat, dz)))
        assert torch.equal(out.ids, base.reference(z, vocab, tokens, 0.9)[5][:, :20].int())
