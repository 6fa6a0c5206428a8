"""Argument checks and sizes of dropout, the residual join and the log
probabilities: all answered on the host, before any launch."""
import pytest


@pytest.fixture(scope="module")
def sf():
    import offloaded_fine_tuning_gb300 as sfp
    sfp.lib(build_if_needed=True)
    return sfp


A = 4096  # an aligned address that is never read: every call below is refused
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(y=0), dict(x=A + 8), dict(y=A + 4), dict(type=2), dict(type=-1), dict(n=-1), dict(n=2 ** 40 + 1),
    dict(p=-0.1), dict(p=1.0), dict(p=1.5), dict(p=NAN), dict(p=1 - 2.0 ** -18), dict(step=A + 4)])
def test_dropout_refuses(sf, bad):
    a = dict(x=A, y=A, type=sf.BF16, n=16, p=0.1, seed=1, offset=2, step=0)
    a.update(bad)
    assert sf.op_dropout(**a) == sf.SF_EINVAL


def test_dropout_of_nothing_is_a_no_op(sf):
    assert sf.op_dropout(0, 0, sf.F32, 0, 0.5, 1, 2) == sf.SF_OK


def fwd_args(sf, **kw):
    a = dict(x=A, h=A, h_type=sf.BF16, g_post=A, gate=A, g_next=A, alpha=1.0, beta=1.0, p=0.1, seed=1, offset=2,
             xout=A, y=A, rstd_post=A, rstd_next=A, rows=4, d=64, eps=1e-5, step=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(h=0), dict(xout=0), dict(y=0), dict(rstd_post=0), dict(rstd_next=0), dict(x=A + 8), dict(h=A + 8),
    dict(xout=A + 4), dict(y=A + 2), dict(rstd_post=A + 2), dict(rstd_next=A + 1), dict(g_post=A + 8),
    dict(gate=A + 2), dict(g_next=A + 8), dict(h_type=2), dict(alpha=NAN), dict(alpha=INF), dict(beta=-INF),
    dict(p=1.0), dict(p=-1.0), dict(step=A + 1), dict(rows=-1), dict(rows=2 ** 31), dict(d=0), dict(d=12),
    dict(d=16392), dict(eps=0.0), dict(eps=NAN)])
def test_join_forward_refuses(sf, bad):
    assert sf.op_join_fwd(**fwd_args(sf, **bad)) == sf.SF_EINVAL


def test_join_forward_of_no_rows_is_a_no_op(sf):
    assert sf.op_join_fwd(**fwd_args(sf, rows=0)) == sf.SF_OK


@pytest.mark.parametrize("bad", [
    dict(xout=0), dict(h=0), dict(dx=0), dict(dh=0), dict(dy=0), dict(rstd_post=0), dict(rstd_next=0),
    dict(dg_post=0), dict(dgate=0), dict(dg_next=0), dict(scratch=0), dict(scratch=A + 4), dict(dx=A), dict(dh=2 * A),
    dict(dy=A + 8), dict(dres=A + 8), dict(dx=7 * A + 8), dict(dh=7 * A + 8), dict(dg_post=A + 1), dict(dgate=A + 1),
    dict(dg_next=A + 1), dict(rows=0), dict(rows=2 ** 31), dict(d=20), dict(h_type=5), dict(p=2.0), dict(beta=NAN),
    dict(g_next=0, dres=0), dict(rstd_post=A + 2), dict(rstd_next=A + 2)])
def test_join_backward_refuses(sf, bad):
    a = dict(xout=A, h=2 * A, h_type=sf.F32, g_post=A, gate=A, g_next=A, alpha=1.0, beta=1.0, p=0.1, seed=1, offset=2,
             rstd_post=A, rstd_next=A, dy=3 * A, dres=4 * A, dx=5 * A, dh=6 * A, dg_post=A, dgate=A, dg_next=A,
             scratch=A, rows=4, d=64, step=0)
    a.update(bad)
    assert sf.op_join_bwd(**a) == sf.SF_EINVAL


def test_join_scratch_sizes(sf):
    assert sf.join_bwd_scratch(1, 8) == 16
    for rows, d in ((1, 8), (5, 4096), (100000, 16384), (2 ** 31 - 1, 8)):
        n = sf.join_bwd_scratch(rows, d)
        assert n >= 2 * d and n % (2 * d) == 0
    for rows, d in ((-1, 64), (4, 0), (4, 12), (4, 16392), (2 ** 31, 64)):
        assert sf.join_bwd_scratch(rows, d) == -1


def rows_args(sf, **kw):
    a = dict(z=A, z_type=sf.F32, ldz=104, tokens=A, rows=4, vocab=100, scale=1.0, logp=A, lse=A, entropy=A, top=5,
             ids=A, top_logp=A)
    a.update(kw)
    return a


SIZES = [dict(z=0), dict(z=A + 8), dict(z_type=2), dict(ldz=96), dict(ldz=108), dict(tokens=0), dict(tokens=A + 2),
         dict(rows=-1), dict(rows=2 ** 31), dict(vocab=0), dict(vocab=2 ** 24 + 1, ldz=2 ** 25), dict(scale=0.0),
         dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(scale=2.0 ** -21), dict(scale=2.0 ** 21), dict(lse=0),
         dict(lse=A + 2)]


@pytest.mark.parametrize("bad", SIZES + [
    dict(logp=0), dict(logp=A + 1), dict(entropy=A + 2), dict(top=-1), dict(top=33), dict(top=9, vocab=8), dict(ids=0),
    dict(top_logp=0), dict(ids=A + 2), dict(top_logp=A + 2)])
def test_logprob_rows_refuses(sf, bad):
    assert sf.op_logprob_rows(**rows_args(sf, **bad)) == sf.SF_EINVAL


@pytest.mark.parametrize("bad", SIZES + [
    dict(dlogp=0), dict(dlogp=A + 2), dict(dentropy=A + 2), dict(entropy=0), dict(entropy=A + 1), dict(dz=0),
    dict(dz=A + 8), dict(lddz=96), dict(lddz=101), dict(dz=A), dict(dz=A, z_type=0, lddz=112)])
def test_logprob_rows_backward_refuses(sf, bad):
    a = dict(z=A, z_type=sf.F32, ldz=104, tokens=A, rows=4, vocab=100, scale=1.0, lse=A, entropy=A, dlogp=A,
             dentropy=A, dz=2 * A, lddz=104)
    a.update(bad)
    assert sf.op_logprob_rows_bwd(**a) == sf.SF_EINVAL


def test_logprob_of_no_rows_is_a_no_op(sf):
    assert sf.op_logprob_rows(**rows_args(sf, rows=0)) == sf.SF_OK
    assert sf.op_logprob_rows_bwd(A, sf.F32, 104, A, 0, 100, 1.0, A, A, A, A, 2 * A, 104) == sf.SF_OK


LM = [dict(h=0), dict(w=0), dict(tokens=0), dict(workspace=0), dict(h=A + 8), dict(w=A + 2), dict(workspace=A + 16),
      dict(tokens=A + 1), dict(n=0), dict(n=2 ** 31), dict(d=4), dict(d=20), dict(v=4), dict(v=100), dict(v=2 ** 24 + 8),
      dict(scale=0.0), dict(scale=NAN), dict(chunk_rows=0), dict(lse=0)]


@pytest.mark.parametrize("bad", LM + [dict(logp=0), dict(top=33), dict(top=3), dict(top=3, ids=A, top_logp=A + 2)])
def test_lm_logprob_refuses(sf, bad):
    a = dict(h=A, w=A, tokens=A, n=4, d=64, v=104, scale=1.0, chunk_rows=2, workspace=A, logp=A, lse=A, entropy=A)
    a.update(bad)
    assert sf.op_lm_logprob(**a) == sf.SF_EINVAL


@pytest.mark.parametrize("bad", LM + [dict(dh=0), dict(dw=0), dict(dh=A + 8), dict(dw=A + 8), dict(dlogp=0),
                                      dict(entropy=0), dict(dentropy=A + 2)])
def test_lm_logprob_backward_refuses(sf, bad):
    a = dict(h=A, w=A, tokens=A, n=4, d=64, v=104, scale=1.0, chunk_rows=2, lse=A, entropy=A, dlogp=A, dentropy=A,
             workspace=A, dh=A, dw=A)
    a.update(bad)
    assert sf.op_lm_logprob_bwd(**a) == sf.SF_EINVAL


def test_lm_logprob_workspaces(sf):
    assert sf.lm_logprob_workspace_bytes(1000, 104, 300) == 300 * 104 * 4 // 256 * 256 + 256
    assert sf.lm_logprob_workspace_bytes(64, 128, 1 << 40) == 64 * 128 * 4
    assert sf.lm_logprob_bwd_workspace_bytes(64, 32, 128, 1) == 64 * 128 * 6 + 64 * 32 * 12  # few rows: one chunk
    whole = sf.lm_logprob_bwd_workspace_bytes(256, 32, 128, 256)
    assert whole == 256 * 128 * 6  # one chunk: no sum of dw
    assert sf.lm_logprob_bwd_workspace_bytes(257, 32, 128, 256) == whole + 128 * 32 * 4
    for bad in ((0, 104, 2), (4, 100, 2), (4, 104, 0), (4, 2 ** 24 + 8, 2), (2 ** 31, 104, 2)):
        assert sf.lm_logprob_workspace_bytes(*bad) == -1
        assert sf.lm_logprob_bwd_workspace_bytes(bad[0], 64, *bad[1:]) == -1
    assert sf.lm_logprob_bwd_workspace_bytes(4, 20, 104, 2) == -1
