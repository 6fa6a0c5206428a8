"""Dropout, residual joins and the head's log probabilities run together as a
policy-gradient step uses them, against autograd of the same model in 64 bits:
embedding dropout, a join, a projection, a second join with the final norm, the
head, and everything's gradients."""
import math

import pytest
import torch

from tests.dropout_reference import kept, threshold
from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")

T32 = dict(dtype=torch.float32, device="cuda")
B16 = dict(dtype=torch.bfloat16, device="cuda")
EPS, SEED, P = 1e-5, 99, 0.15
# two bf16 operands' roundings (2^-8 each at worst) enter each product, and three products follow one
# another; the step's own bar for bf16 compute with fp32 sums is 2e-2 of a tensor
BAR = 2e-2


def drop_mask(shape, offset):
    return torch.from_numpy(kept(math.prod(shape), P, SEED, offset)).cuda().reshape(shape).double() * \
        (65536.0 / (65536 - threshold(P)))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n,d,v,chunk", [(50, 128, 520, 64), (300, 384, 3000, 128)])
def test_policy_step(n, d, v, chunk, captured):
    sf.lib(build_if_needed=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, **T32)
    emb, h1 = rnd(n, d), rnd(n, d).bfloat16()
    gains = [(1 + 0.2 * rnd(d)).bfloat16() for _ in range(6)]  # post, gate, next of both joins
    w2, wl = (rnd(d, d) / math.sqrt(d)).bfloat16(), (1.5 / math.sqrt(d) * rnd(v, d)).bfloat16()
    tokens = torch.randint(0, v, (n,), generator=g, dtype=torch.int32, device="cuda")
    tokens[3::7] = -100
    live = (tokens >= 0).float()
    adv, bonus = rnd(n) * live / n, 0.02 * live / n  # the loss: -sum adv logp - sum bonus entropy
    dl, de = -adv, -bonus

    new = torch.empty
    x0, x1, x2 = (new(n, d, **T32) for _ in range(3))
    y1, h2, y2 = (new(n, d, **B16) for _ in range(3))
    r = [new(n, **T32) for _ in range(4)]
    logp, lse, ent, top = new(n, **T32), new(n, **T32), new(n, **T32), new(n, 5, **T32)
    ids = new(n, 5, dtype=torch.int32, device="cuda")
    ws = new(sf.lm_logprob_workspace_bytes(n, v, chunk), dtype=torch.uint8, device="cuda")
    wb = new(sf.lm_logprob_bwd_workspace_bytes(n, d, v, chunk), dtype=torch.uint8, device="cuda")
    scratch = new(sf.join_bwd_scratch(n, d), **T32)
    dy2b, dw, dw2 = new(n, d, **B16), new(v, d, **B16), new(d, d, **B16)
    dy2, dx2, dy1, dx1, dx0 = (new(n, d, **T32) for _ in range(5))
    dh2, dh1 = new(n, d, **B16), new(n, d, **B16)
    dg = [new(d, **B16) for _ in range(6)]
    q = lambda *ts: [t.data_ptr() for t in ts]

    def step():
        s = stream()
        ok = [sf.op_dropout(*q(emb, x0), sf.F32, n * d, P, SEED, 0, stream=s)]
        ok.append(sf.op_join_fwd(*q(x0, h1), sf.BF16, *q(*gains[:3]), 1.0, 0.5, P, SEED, 1, *q(x1, y1, r[0], r[1]),
                                 n, d, EPS, stream=s))
        ok.append(sf.op_gemm(sf.NT, sf.EPI_BF16, n, d, d, y1.data_ptr(), d, w2.data_ptr(), d, h2.data_ptr(), d,
                             stream=s))
        ok.append(sf.op_join_fwd(*q(x1, h2), sf.BF16, *q(*gains[3:]), 1.0, 0.5, P, SEED, 2, *q(x2, y2, r[2], r[3]),
                                 n, d, EPS, stream=s))
        ok.append(sf.op_lm_logprob(*q(y2, wl, tokens), n, d, v, 0.9, chunk, *q(ws, logp, lse, ent), 5, *q(ids, top),
                                   stream=s))
        ok.append(sf.op_lm_logprob_bwd(*q(y2, wl, tokens), n, d, v, 0.9, chunk, *q(lse, ent, dl, de, wb, dy2b, dw),
                                       stream=s))
        dy2.copy_(dy2b)
        ok.append(sf.op_join_bwd(*q(x2, h2), sf.BF16, *q(*gains[3:]), 1.0, 0.5, P, SEED, 2, *q(r[2], r[3], dy2), 0,
                                 *q(dx2, dh2, *dg[3:], scratch), n, d, stream=s))
        ok.append(sf.op_gemm(sf.NN, sf.EPI_F32, n, d, d, dh2.data_ptr(), d, w2.data_ptr(), d, dy1.data_ptr(), d,
                             stream=s))
        ok.append(sf.op_gemm(sf.TN, sf.EPI_BF16, d, d, n, dh2.data_ptr(), d, y1.data_ptr(), d, dw2.data_ptr(), d,
                             stream=s))
        ok.append(sf.op_join_bwd(*q(x1, h1), sf.BF16, *q(*gains[:3]), 1.0, 0.5, P, SEED, 1, *q(r[0], r[1], dy1, dx2),
                                 *q(dx1, dh1, *dg[:3], scratch), n, d, stream=s))
        ok.append(sf.op_dropout(*q(dx1, dx0), sf.F32, n * d, P, SEED, 0, stream=s))
        assert ok == [0] * len(ok), ok

    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (x1, y1, logp, dw, dx0, dh1):
            t.zero_()
        graph.replay()
    else:
        step()
    sync()
    assert sf.device_error() == 0

    leaves = [t.double().requires_grad_() for t in (emb, h1, *gains, w2, wl)]
    e, b1, p1, t1, n1, p2, t2, n2, m2, ml = leaves
    norm = lambda x: x / torch.sqrt((x ** 2).mean(1, keepdim=True) + EPS)
    a = e * drop_mask((n, d), 0)
    a = a + 0.5 * drop_mask((n, d), 1) * (norm(b1) * p1 * t1)
    b2 = (norm(a) * n1) @ m2.t()
    a = a + 0.5 * drop_mask((n, d), 2) * (norm(b2) * p2 * t2)
    lp = torch.log_softmax(0.9 * (norm(a) * n2) @ ml.t(), 1)
    chosen = torch.gather(lp, 1, tokens.clamp(min=0).long()[:, None])[:, 0]
    entropy = -(lp.exp() * lp).sum(1)
    loss = -(adv.double() * chosen).sum() - (bonus.double() * entropy).sum()
    grads = torch.autograd.grad(loss, leaves)
    far = lambda got, ref: ((got.double() - ref).norm() / ref.norm()).item()
    assert far(logp, torch.where(tokens >= 0, chosen, torch.zeros_like(chosen)).detach()) <= BAR
    assert far(ent, entropy.detach()) <= BAR
    assert far(top, torch.sort(lp, 1, descending=True).values[:, :5].detach()) <= BAR
    for name, got, ref in zip(("emb", "h1", "post1", "gate1", "next1", "post2", "gate2", "next2", "w2", "head"),
                              (dx0, dh1, *dg, dw2, dw), grads):
        assert far(got, ref) <= BAR, (name, far(got, ref))
