"""NaN in the norm's E4M3 output: an element of y that is NaN, by the input or by
an x + residual past bf16's range, has the code of NaN, as its bf16 copy has NaN,
and products of the codes show it."""

import pytest
import torch

from fp8_block_scaled_05_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def is_nan(q):
    return (q & 0x7F) == 0x7F


def inputs(M, K, case):
    x = synth.act(M, K, case=case, tensor=0, device="cuda")
    r = synth.act(M, K, case=case, tensor=1, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(case)
    return x, r, 1 + 0.2 * torch.randn(K, generator=g, device="cuda")


# rows of one wave, of several, of sixteen with two and four loads per thread
@pytest.mark.parametrize("M,K", [(9, 512), (5, 7168), (3, 16384), (3, 16512)])
def test_codes_keep_nan(fp8bs, M, K):
    """A NaN element makes its row's codes NaN, no other row's."""
    x, r, g = inputs(M, K, 1300)
    q0, s0 = fp8bs.fp8_quant_rmsnorm(x, g, residual=r)
    bad = x.clone()
    bad[1, 100] = float("nan")
    y = torch.empty_like(x)
    q, s = fp8bs.fp8_quant_rmsnorm(bad, g, residual=r, y=y)
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[:, keep], s0[:, keep])
    assert torch.all(y[1].isnan())
    assert torch.all(is_nan(q[1])) and not torch.any(is_nan(q[keep]))


@pytest.mark.parametrize("M,K", [(9, 512), (5, 7168), (3, 16384), (3, 16512)])
def test_codes_keep_an_overflowed_sum(fp8bs, M, K):
    """Finite x and residual whose sum leaves bf16: h is infinite there, rstd 0, y
    NaN at that element and 0 beside it."""
    x, r, g = inputs(M, K, 1301)
    x[2, 70], r[2, 70] = 3e38, 3e38
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(M, device="cuda")
    q, _ = fp8bs.fp8_quant_rmsnorm(x, g, residual=r, h=h, y=y, rstd=rstd)
    assert h[2, 70] == float("inf") and rstd[2] == 0
    where = torch.zeros(M, K, dtype=torch.bool, device="cuda")
    where[2, 70] = True
    assert torch.equal(y.isnan(), where)
    assert torch.equal(is_nan(q), where)
    rest = torch.arange(K, device="cuda") != 70
    assert torch.all(y[2, rest] == 0) and torch.all(q[2, rest] & 0x7F == 0)


def test_a_weight_of_nan_takes_its_column(fp8bs):
    x, r, g = inputs(40, 384, 1302)
    g[130] = float("nan")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, residual=r)
    assert torch.all(is_nan(q[:, 130])) and is_nan(q).sum() == 40 and torch.all(s.isfinite())


@pytest.mark.parametrize("M", [3, 40, 100, 600])
def test_products_of_the_codes_show_it(fp8bs, M):
    """Few-row and tiled products: a NaN row stays one, the others are as before."""
    K, N = 384, 256
    x, r, g = inputs(M, K, 1303)
    qw, sw = fp8bs.fp8_quant_w_128x128(synth.weight(N, K, case=1303, tensor=2, device="cuda"))
    clean = fp8bs.fp8_block_gemm(*fp8bs.fp8_quant_rmsnorm(x, g, residual=r), qw, sw)
    x[2, 5], r[2, 5] = 3e38, 3e38
    c = fp8bs.fp8_block_gemm(*fp8bs.fp8_quant_rmsnorm(x, g, residual=r), qw, sw)
    keep = [m for m in range(M) if m != 2]
    assert torch.all(c[2].isnan()) and torch.equal(c[keep], clean[keep])
