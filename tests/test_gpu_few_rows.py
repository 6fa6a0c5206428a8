"""Products with few rows, whose left operand is less than 128 KB (its tensor map
has planes behind the matrix, which nothing may load), and dropout that drops
nothing, through the C ABI.

A row's products do not depend on the number of rows, so those of few rows are the
same bits as in a call with enough rows for a plain map; those are held against
64 bits: a sum of K fp32 products of bf16 values is off by K 2^-24 of the sum of
their sizes (any order)."""
import math

import pytest
import torch

from tests.gpu_util import stream, sync

pytestmark = pytest.mark.gpu
sf = pytest.importorskip("offloaded_fine_tuning_gb300")
F32 = dict(dtype=torch.float32, device="cuda")  # another test module changes the default type


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sf.lib(build_if_needed=True)
    assert sf.device_error() == 0
    yield
    assert sf.device_error() == 0


def product(layout, a, b, rows, N, K):
    """The fp32 product of a's first rows, and 64 elements behind it."""
    c = torch.full((rows * N + 64,), 7.0, **F32)
    assert sf.op_gemm(layout, 1, rows, N, K, a.data_ptr(), a.shape[1], b.data_ptr(), b.shape[1], c.data_ptr(), N,
                      stream=stream()) == 0
    sync()
    assert (c[rows * N:] == 7).all()
    return c[:rows * N].view(rows, N)


@pytest.mark.parametrize("layout", ["NT", "NN"])
@pytest.mark.parametrize("rows,N,K", [(1, 4096, 4096), (15, 1000, 4096), (16, 1000, 4096), (7, 520, 8192), (1, 8, 8),
                                      (130, 64, 72), (300, 304, 200), (3, 128, 1000)])
def test_products_of_few_rows(layout, rows, N, K):
    g = torch.Generator(device="cuda").manual_seed(rows + N + K)
    many = max(rows + 8, 65536 // K + 1)
    full = torch.randn(many, K + 8, generator=g, **F32).bfloat16()
    full[:, K:] = math.nan  # between the rows
    few = full.clone()
    few[rows:] = math.nan   # behind them
    shape = (N, K) if layout == "NT" else (K, N)
    b = torch.randn(*shape, generator=g, **F32).bfloat16()
    got = product(getattr(sf, layout), few, b, rows, N, K)
    assert torch.equal(got, product(getattr(sf, layout), full, b, many, N, K)[:rows])
    a, b = few[:rows, :K].double(), (b.t() if layout == "NT" else b).double()
    over = (got.double() - a @ b).abs() - (a.abs() @ b.abs()) * (K * 2.0 ** -24)
    assert over.max().item() <= 0.0


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("n", [1, 3, 15])
def test_head_of_few_rows(n, top):
    d, v, many = 4096, 2056, 64
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randn(v, d, generator=g, **F32).bfloat16()
    full = (torch.randn(many, d, generator=g, **F32) * 0.02).bfloat16()
    few = full.clone()
    few[n:] = math.nan
    tokens = torch.randint(0, v, (many,), generator=g, device="cuda", dtype=torch.int32)

    def call(h, rows):
        ws = torch.empty(sf.lm_logprob_workspace_bytes(rows, v, rows), dtype=torch.uint8, device="cuda")
        logp, lse, ent = (torch.empty(rows, **F32) for _ in range(3))
        ids = torch.empty(rows, max(top, 1), dtype=torch.int32, device="cuda")
        top_logp = torch.empty(rows, max(top, 1), **F32)
        assert sf.op_lm_logprob(h.data_ptr(), w.data_ptr(), tokens.data_ptr(), rows, d, v, 1.0, rows, ws.data_ptr(),
                                logp.data_ptr(), lse.data_ptr(), ent.data_ptr(), top, ids.data_ptr() if top else 0,
                                top_logp.data_ptr() if top else 0, stream=stream()) == 0
        sync()
        return logp, lse, ent, ids

    got, ref = call(few, n), call(full, many)
    z = few[:n].double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    # logits: K products (|h| about 0.016, |w| 0.8 on average, 4096 of them: 52), then
    # the sums' relative 2^-18 + (v / 128 + 64) 2^-24 as an error of the logarithm
    tol = 2 * 52 * d * 2.0 ** -24 + 2.0 ** -18 + (v / 128 + 64) * 2.0 ** -24
    assert (got[1].double() - lse).abs().max().item() <= tol
    at = z.gather(1, tokens[:n, None].long())[:, 0]
    assert (got[0].double() - (at - lse)).abs().max().item() <= 2 * tol
    if top:
        assert torch.equal(got[3], ref[3][:n])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 4096, 4097, 100003])
def test_dropout_that_drops_nothing(n, kind):
    dtype, code = (torch.bfloat16, sf.BF16) if kind == "bf16" else (torch.float32, sf.F32)
    x = torch.randn(n, **F32).to(dtype)
    x[n // 2] = math.inf
    y = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    assert sf.op_dropout(x.data_ptr(), y.data_ptr(), code, n, 0.0, 5, 9, step.data_ptr(), stream=stream()) == 0
    sync()
    assert torch.equal(y[:n], x) and (y[n:] == 7).all()
