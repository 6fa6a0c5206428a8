"""Log probabilities where their parts meet: large gradients beside masked logits and
rows that are nearly certain, through the C ABI.  Tolerances not derived here are those of the other tests of log
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
