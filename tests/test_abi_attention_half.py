"""Argument checks and sizes of the query/key norm, windowed attention and
8-bit checkpoint entry points: all answered on the host, before any launch."""
import pytest


@pytest.fixture(scope="module")
def sf():
    import offloaded_fine_tuning_gb300 as sfp
    sfp.lib(build_if_needed=True)
    return sfp


A = 4096  # an aligned address that is never read: every call below is refused


def qk_args(**kw):
    a = dict(x=A, ldx=384, y=A, ldy=384, tokens=4, seq=8, Hq=4, Hkv=1, head_dim=64, gq=A, gk=A, eps=1e-5,
             table=A, pos=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(y=0), dict(gq=0), dict(gk=0), dict(table=0), dict(x=A + 8), dict(y=A + 8), dict(gq=A + 2),
    dict(table=A + 8), dict(pos=A + 2), dict(ldx=376), dict(ldy=376), dict(ldx=388), dict(ldy=392), dict(tokens=-1),
    dict(seq=0), dict(Hq=0), dict(Hkv=0), dict(head_dim=8), dict(head_dim=72), dict(head_dim=272), dict(eps=0.0),
    dict(eps=float("nan")), dict(Hq=2 ** 31 - 1), dict(tokens=2 ** 40), dict(Hq=70000, ldx=2 ** 30, ldy=2 ** 30)])
def test_qknorm_forward_refuses(sf, bad):
    assert sf.op_qknorm_rope_fwd(**qk_args(**bad)) == sf.SF_EINVAL


def test_qknorm_forward_of_no_tokens_is_a_no_op(sf):
    assert sf.op_qknorm_rope_fwd(**qk_args(tokens=0)) == sf.SF_OK


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(dy=0), dict(dx=0), dict(scratch=0), dict(dgq=0), dict(dgk=0), dict(tokens=0), dict(dx=A),
    dict(dx=3 * A, lddx=392), dict(scratch=A + 4), dict(dgq=A + 1), dict(lddy=376), dict(lddx=380), dict(head_dim=0)])
def test_qknorm_backward_refuses(sf, bad):
    a = dict(x=A, ldx=384, dy=3 * A, lddy=384, dx=2 * A, lddx=384, tokens=4, seq=8, Hq=4, Hkv=1, head_dim=64, gq=A,
             gk=A, eps=1e-5, table=A, pos=0, scratch=A, dgq=A, dgk=A)
    a.update(bad)
    assert sf.op_qknorm_rope_bwd(**a) == sf.SF_EINVAL


def test_qknorm_scratch_sizes(sf):
    assert sf.qknorm_rope_bwd_scratch(1, 4, 1, 64) >= 128
    assert sf.qknorm_rope_bwd_scratch(100000, 4, 1, 64) % 128 == 0
    for bad in ((-1, 4, 1, 64), (4, 0, 1, 64), (4, 4, 0, 64), (4, 4, 1, 60)):
        assert sf.qknorm_rope_bwd_scratch(*bad) == -1


@pytest.mark.parametrize("bad", [
    dict(qkv=0), dict(o=0), dict(lse=0), dict(qkv=A + 8), dict(B=-1), dict(S=-1), dict(Hq=0), dict(Hkv=0),
    dict(Hkv=3), dict(hd=96), dict(window=0), dict(window=-5), dict(sinks=-1), dict(B=65536), dict(S=2 ** 30 + 1),
    dict(Hq=65536, Hkv=65536), dict(Hq=2 ** 22, Hkv=1)])
def test_window_forward_refuses(sf, bad):
    a = dict(qkv=A, o=A, lse=A, B=1, S=16, Hq=4, Hkv=2, hd=64, window=8, sinks=1)
    a.update(bad)
    assert sf.op_attn_window_fwd(**a) == sf.SF_EINVAL


@pytest.mark.parametrize("bad", [
    dict(qkv=0), dict(o=0), dict(dout=0), dict(lse=0), dict(delta=0), dict(dq_acc=0), dict(dqkv=0),
    dict(dq_acc=A + 4), dict(dqkv=A + 8), dict(dout=A + 8), dict(table=A + 4), dict(Hkv=3), dict(hd=32),
    dict(window=0), dict(sinks=-1), dict(B=65536), dict(S=2 ** 31 - 1)])
def test_window_backward_refuses(sf, bad):
    a = dict(qkv=A, o=A, dout=A, lse=A, delta=A, dq_acc=A, dqkv=A, B=1, S=16, Hq=4, Hkv=2, hd=64, window=8, sinks=1)
    a.update(bad)
    assert sf.op_attn_window_bwd(**a) == sf.SF_EINVAL


def test_window_of_an_empty_batch_is_a_no_op(sf):
    assert sf.op_attn_window_fwd(A, A, A, 0, 16, 4, 2, 64, 8, 1) == sf.SF_OK
    assert sf.op_attn_window_fwd(A, A, A, 1, 0, 4, 2, 64, 8, 1) == sf.SF_OK
    assert sf.op_attn_window_bwd(A, A, A, A, A, A, A, 1, 0, 4, 2, 64, 8, 1) == sf.SF_OK


def blocks_seen(S, window, sinks, qb):
    """Most 128-key blocks that the queries of an aligned block of qb see, sinks' blocks
    and the others apart."""
    ns = (min(sinks, S) + 127) // 128
    most = 0
    for q0 in range(0, S, qb):
        lo = max(0, q0 - window + 1) // 128
        most = max(most, q0 // 128 - max(lo, ns) + 1)
    return ns, most


@pytest.mark.parametrize("S", [1, 127, 128, 129, 640, 1000, 2049, 5000])
@pytest.mark.parametrize("window", [1, 2, 64, 65, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 128, 129, 4000])
def test_window_scratch_holds_every_visited_block(sf, S, window, sinks):
    B, Hq = 2, 3
    for hd, qb in ((64, 128), (128, 128)):
        per = B * S * Hq * hd
        # behind dQ: whole 128-key tiles of partial dK and dV, for sinks only
        extra = sf.attn_window_dq_scratch_floats(B, S, Hq, hd, window, sinks, 0) - per
        assert extra >= 0 and extra % (256 * hd * B * Hq) == 0 and (sinks > 0 or extra == 0)
        n = sf.attn_window_dq_scratch_floats(B, S, Hq, hd, window, sinks, 1) - extra
        ns, most = blocks_seen(S, window, sinks, qb)
        assert n % per == 0 and ns + max(0, most) <= n // per <= (S + 127) // 128
    for bad in ((-1, S, Hq, 64, 1, 0, 1), (B, -1, Hq, 64, 1, 0, 1), (B, S, 0, 64, 1, 0, 1), (B, S, Hq, 96, 1, 0, 1),
                (B, S, Hq, 64, 0, 0, 1), (B, S, Hq, 64, 1, -1, 1), (65536, S, Hq, 64, 1, 0, 1),
                (B, 2 ** 31 - 1, Hq, 64, 1, 0, 1)):
        assert sf.attn_window_dq_scratch_floats(*bad) == -1


def test_window_of_more_elements_than_a_device_holds_is_refused(sf):
    """Each size alone is allowed; their product would pass 64 bits in the scratch size."""
    for B, S, Hq, Hkv, hd in ((65535, 1 << 30, 1 << 21, 1, 128), (1, 1 << 30, 1 << 20, 16, 64),
                              (65535, 1 << 20, 512, 512, 128)):
        assert sf.attn_window_dq_scratch_floats(B, S, Hq, hd, 64, 4, 1) == -1
        assert sf.op_attn_window_fwd(A, A, A, B, S, Hq, Hkv, hd, 64, 4) == sf.SF_EINVAL
        assert sf.op_attn_window_bwd(A, A, A, A, A, A, A, B, S, Hq, Hkv, hd, 64, 4) == sf.SF_EINVAL
    # the largest one allowed: 2^38 elements of Q, K and V, a slot for each of its blocks
    n = sf.attn_window_dq_scratch_floats(1, 1 << 30, 2, 64, 1 << 30, 0, 1)
    assert n == (1 << 23) * (1 << 30) * 128


def test_ckpt8_refuses(sf):
    assert sf.ckpt8_scales(10, 136) == 20 and sf.ckpt8_scales(0, 8) == 0
    for rows, d in ((-1, 128), (4, 0), (4, 12), (4, 16392), (2 ** 31, 128)):
        assert sf.ckpt8_scales(rows, d) == -1
    for fmt, rows, d in ((2, 4, 128), (-1, 4, 128), (0, -1, 128), (0, 4, 4), (0, 4, 132), (1, 4, 16392),
                         (0, 2 ** 31, 128)):
        assert sf.op_ckpt8_save(A, A, A, fmt, rows, d) == sf.SF_EINVAL
        assert sf.op_ckpt8_load(A, A, A, fmt, rows, d) == sf.SF_EINVAL
        assert sf.op_rmsnorm_fwd_save8(A, A, A, A, A, A, fmt, rows, d, 1e-5) == sf.SF_EINVAL
        assert sf.op_rmsnorm_fwd_load8(A, A, A, A, A, A, fmt, rows, d, 1e-5) == sf.SF_EINVAL
        assert sf.op_rmsnorm_bwd_load8(A, A, A, A, A, A, A, A, A, A, fmt, rows, d) == sf.SF_EINVAL
    assert sf.op_rmsnorm_bwd_load8(A, A, A, A, A, A, A, A, A, A, 0, 0, 128) == sf.SF_EINVAL  # no rows, no gain sum
    assert sf.op_rmsnorm_fwd_save8(A, A, A, A, A, A, 0, 4, 128, 0.0) == sf.SF_EINVAL
    for i in range(3):
        p = [A, A, A]
        for v in (0, A + 8):
            p[i] = v
            assert sf.op_ckpt8_save(*p, 0, 4, 128) == sf.SF_EINVAL
            assert sf.op_ckpt8_load(*p, 0, 4, 128) == sf.SF_EINVAL
    for i in range(6):
        p = [A] * 6
        p[i] = 0
        assert sf.op_rmsnorm_fwd_save8(*p, 0, 4, 128, 1e-5) == sf.SF_EINVAL
        if i != 5:  # the loaded values are optional
            assert sf.op_rmsnorm_fwd_load8(*p, 0, 4, 128, 1e-5) == sf.SF_EINVAL
    for i in range(10):
        if i == 5:  # the residual gradient is optional
            continue
        p = [A] * 10
        p[i] = 0
        assert sf.op_rmsnorm_bwd_load8(*p, 0, 4, 128) == sf.SF_EINVAL
    for call in (lambda: sf.op_ckpt8_save(A, A, A, 0, 0, 128), lambda: sf.op_ckpt8_load(A, A, A, 1, 0, 128),
                 lambda: sf.op_rmsnorm_fwd_save8(A, A, A, A, A, A, 0, 0, 128, 1e-5)):
        assert call() == sf.SF_OK
