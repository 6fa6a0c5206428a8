"""Captured graphs of the attention half's backward passes that use the same
scratch buffers, replayed in turn with new inputs in between."""
import pytest
import torch

from tests.gpu_util import sync
from tests.test_gpu_attention_half import EPS, F32T, _lib, qk_inputs, table, win_fwd, win_inputs

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")


@pytest.mark.parametrize("hd,sinks", [(64, 0), (64, 4), (128, 4)])
def test_two_graphs_share_their_scratch(hd, sinks):
    """Graph A and graph B: the windowed and the causal backward and the query/key
    norm's, on tensors of their own, with one dq_acc, delta and gain scratch for
    all.  Replayed A, B, A with A's inputs exchanged before the last replay; each
    result is the eager call's."""
    B, S, Hq, Hkv, W = 1, 2500, 4, 2, 100
    E = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")
    p = lambda t: t.data_ptr()
    delta = E(torch.float32, B, Hq, S)
    acc = E(torch.float32, max(sf.attn_window_dq_scratch_floats(B, S, Hq, hd, W, sinks, 1),
                               sf.attn_dq_scratch_floats(B, S, Hq, hd, 1)))
    part = torch.empty(sf.qknorm_rope_bwd_scratch(S, Hq, Hkv, hd), **F32T)
    tab = table(S, hd)

    class Work:
        def __init__(self, seed):
            self.qkv, self.dout = win_inputs(B, S, Hq, Hkv, hd, seed=seed)
            self.x, self.gq, self.gk, _, self.W = qk_inputs(S, Hq, Hkv, hd, seed=seed)
            self.o, self.lse = win_fwd(self.qkv, B, S, Hq, Hkv, hd, W, sinks)
            self.oc, self.lc = win_fwd(self.qkv, B, S, Hq, Hkv, hd, S, 0)
            self.dw, self.dc, self.dx = (torch.empty_like(self.qkv) for _ in range(3))
            self.dg = E(torch.bfloat16, 2, hd)

        def inputs(self):
            return self.qkv, self.dout, self.x, self.o, self.lse, self.oc, self.lc

        def run(self, st):
            shape = (B, S, Hq, Hkv, hd)
            rc = [sf.op_attn_window_bwd(p(self.qkv), p(self.o), p(self.dout), p(self.lse), p(delta), p(acc), p(self.dw),
                                        *shape, W, sinks, 0, st, 1),
                  sf.op_attn_bwd(p(self.qkv), p(self.oc), p(self.dout), p(self.lc), p(delta), p(acc), p(self.dc),
                                 *shape, p(tab), st, 1),
                  sf.op_qknorm_rope_bwd(p(self.x), self.W, p(self.dw), self.W, p(self.dx), self.W, S, S, Hq, Hkv, hd,
                                        p(self.gq), p(self.gk), EPS, p(tab), 0, p(part), p(self.dg[0]), p(self.dg[1]), st)]
            assert rc == [0] * 3, rc

        def results(self):
            sync()
            return [t.clone() for t in (self.dw, self.dc, self.dx, self.dg)]

    a, b, c = (Work(s) for s in (61, 62, 63))
    st = torch.cuda.Stream()
    want = {}
    for name, w in (("a", a), ("b", b), ("c", c)):
        w.gq, w.gk = a.gq, a.gk
        sync()
        w.run(st.cuda_stream)
        want[name] = w.results()
    graphs = []
    for w in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            w.run(torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    acc.fill_(float("nan"))
    sync()

    def replay(g, w, expected):
        for t in (w.dw, w.dc, w.dx, w.dg):
            t.zero_()
        g.replay()
        for got, ref in zip(w.results(), expected):
            assert torch.equal(got, ref)

    replay(graphs[0], a, want["a"])
    replay(graphs[1], b, want["b"])
    for mine, new in zip(a.inputs(), c.inputs()):
        mine.copy_(new)
    replay(graphs[0], a, want["c"])
