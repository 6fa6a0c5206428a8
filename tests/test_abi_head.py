"""Refusals of the head's log probabilities with an address of its own for each
argument, so that nothing but the named one can be the reason, and the limit of the
vocabulary: all answered on the host, before any launch."""
import pytest


@pytest.fixture(scope="module")
def sf():
    import offloaded_fine_tuning_gb300 as sfp
    sfp.lib(build_if_needed=True)
    return sfp


A = 4096  # aligned addresses that are never read: every call below is refused


def backward(sf, **bad):
    names = ("h", "w", "tokens", "lse", "entropy", "dlogp", "dentropy", "workspace", "dh", "dw")
    a = {name: A * (i + 1) for i, name in enumerate(names)}
    a.update(n=4, d=64, v=104, scale=1.0, chunk_rows=2)
    a.update(bad)
    return sf.op_lm_logprob_bwd(**a)


@pytest.mark.parametrize("n", [1, 128, 129, 100000])
def test_dh_over_h_is_refused(sf, n):
    """dw's product reads h after dh has been written, so their gradient would be that of dh's values."""
    assert backward(sf, n=n, dh=A) == sf.SF_EINVAL


@pytest.mark.parametrize("bad", [
    dict(h=0), dict(w=0), dict(tokens=0), dict(workspace=0), dict(h=A + 8), dict(w=A + 2), dict(workspace=A + 16),
    dict(tokens=A + 1), dict(n=0), dict(n=2 ** 31), dict(d=4), dict(d=20), dict(v=4), dict(v=100), dict(v=2 ** 20 + 8),
    dict(scale=0.0), dict(scale=float("nan")), dict(chunk_rows=0), dict(lse=0), dict(dh=0), dict(dw=0), dict(dh=A + 8),
    dict(dw=A + 8), dict(dlogp=0), dict(entropy=0), dict(dentropy=A + 2), dict(dlogp=A + 1), dict(lse=A + 2)])
def test_the_backward_refuses_each_by_itself(sf, bad):
    assert backward(sf, **bad) == sf.SF_EINVAL


def test_the_vocabulary_has_a_limit(sf):
    top = 2 ** 20
    rows = dict(z=A, z_type=sf.F32, ldz=top + 8, tokens=2 * A, rows=4, scale=1.0, lse=4 * A, entropy=5 * A)
    assert sf.op_logprob_rows(**rows, vocab=top + 1, logp=3 * A) == sf.SF_EINVAL
    assert sf.op_logprob_rows_bwd(**rows, vocab=top + 1, dlogp=6 * A, dentropy=7 * A, dz=8 * A, lddz=top + 8) == \
        sf.SF_EINVAL
    assert sf.op_lm_logprob(A, 2 * A, 3 * A, 4, 64, top + 8, 1.0, 2, 4 * A, 5 * A, 6 * A) == sf.SF_EINVAL
    assert sf.lm_logprob_workspace_bytes(4, top, 2) == 2 * top * 4
    assert sf.lm_logprob_workspace_bytes(4, top + 8, 2) == -1
    assert sf.lm_logprob_bwd_workspace_bytes(4, 64, top + 8, 2) == -1
