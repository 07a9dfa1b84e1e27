"""The norm, the gated product and their backward passes where offsets pass 31 and
32 bits, over long contractions, and with strided experts.

Large results are held to the same call on a part of the rows (or on compact
operands), bit for bit: the parts are checked against float64 elsewhere, and no
result depends on its row's place.
"""

import numpy as np
import pytest
import torch

from fp8_block_scaled_05_amd import synth
from tests.test_gpu_gated import check_codes, check_y, check_z, exact_sums, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def codes(*shape):
    """Finite E4M3 codes (of positive values)."""
    return torch.randint(0, 255, shape, dtype=torch.uint8, device="cuda").remainder_(127)


def values(M, N):
    """bf16 in [-1, 1), quick to make."""
    x = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    return x.uniform_(-1, 1)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("M", [1, 20, 40, 130, 333])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_long_contraction(fp8bs, M, act):
    """56 groups."""
    N, K = 640, 7168
    _, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1200)
    z = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, act=act)
    check_y(y, fp8bs.fp8_block_gemm(qx, sx, qw, sw, out_dtype=torch.float32), act)
    qc, sc = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw, act=act, z=z)
    sums = exact_sums(qx, sx, qw, sw)
    check_z(z, sums)
    check_codes(qc, sc, sums, act)


@pytest.mark.parametrize("M", [1, 20, 50, 100, 300])
def test_weight_up_to_the_last_32_bit_offset(fp8bs, M):
    """2N ldb just below 2^32: the up rows begin near 2^31."""
    N, K, ld = 130944, 256, 16384
    assert 2 ** 32 - 2 ** 23 < 2 * N * ld < 2 ** 32
    qw = codes(2 * N, K)
    wide = torch.empty(2 * N, ld, dtype=torch.uint8, device="cuda")
    wide[:, :K] = qw
    sw = torch.rand(2 * N // 128, K // 128, device="cuda") * 1e-3
    qx, sx = codes(M, K), torch.rand(K // 128, M, device="cuda") * 1e-3
    z = [torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, z=z[0])
    b = fp8bs.fp8_block_gemm_gated(qx, sx, wide[:, :K], sw, z=z[1])
    assert same(a, b) and same(*z) and same(z[0], fp8bs.fp8_block_gemm(qx, sx, qw, sw))
    a = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw)
    b = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, wide[:, :K], sw)
    assert same(a[0], b[0]) and same(a[1], b[1])


@pytest.mark.parametrize("rows", [[3, 0, 70], [300, 1, 500], [2000, 3000, 0]])
def test_strided_experts(fp8bs, rows):
    """Experts' weights apart from each other, rows of W too."""
    N, K, G, M = 384, 256, len(rows), sum(rows)
    qw, sw = codes(G, 2 * N, K), torch.rand(G, N // 64, K // 128, device="cuda") * 1e-3
    apart = torch.full((G, 2 * N + 5, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    apart[:, :2 * N, :K] = qw
    qx, sx = codes(M, K), torch.rand(K // 128, M, device="cuda") * 1e-3
    wide = torch.full((M, K + 16), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :K] = qx
    off = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    a = fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off)
    b = fp8bs.fp8_block_grouped_gemm_gated(wide[:, :K], sx, apart[:, :2 * N, :K], sw, off)
    assert same(a, b)
    a = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off)
    b = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(wide[:, :K], sx, apart[:, :2 * N, :K], sw, off)
    assert same(a[0], b[0]) and same(a[1], b[1])


def test_gated_outputs_past_32_bits(fp8bs):
    """z of 2.3e9 elements, y of 1.2e9; the last rows."""
    M, N, K, last = 70001, 16384, 128, 400
    qw, sw = codes(2 * N, K), torch.rand(2 * N // 128, 1, device="cuda") * 1e-3
    qx, sx = codes(M, K), torch.rand(1, M, device="cuda") * 1e-3
    z = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    zl = torch.empty(last, 2 * N, dtype=torch.bfloat16, device="cuda")
    ql, sl = qx[-last:], sx[:, -last:].contiguous()
    y = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, z=z)
    assert same(y[-last:], fp8bs.fp8_block_gemm_gated(ql, sl, qw, sw, z=zl)) and same(z[-last:], zl)
    del y
    off = torch.tensor([0, M - last, M], dtype=torch.int32, device="cuda")
    two, stwo = torch.stack([qw, qw]), torch.stack([sw, sw])
    qc, sc = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw, z=z)
    part = fp8bs.fp8_block_gemm_gated_e4m3_out(ql, sl, qw, sw, z=zl)
    assert same(qc[-last:], part[0]) and same(sc[:, -last:], part[1]) and same(z[-last:], zl)
    z.zero_()
    qc, sc = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, two, stwo, off, z=z)
    assert same(qc[-last:], part[0]) and same(sc[:, -last:], part[1]) and same(z[-last:], zl)


def test_norm_past_32_bits(fp8bs):
    """4.3e9 elements and more than 2^31 bytes a tensor; the last rows."""
    M, K, last = 131080, 32768, 77
    assert M * K > 2 ** 32
    x, g = values(M, K), 1 + 0.2 * torch.randn(K, device="cuda")
    h, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, residual=x, h=h, rstd=rstd)
    hl, rl = torch.empty_like(x[-last:]), torch.empty(last, device="cuda")
    ql, sl = fp8bs.fp8_quant_rmsnorm(x[-last:], g, residual=x[-last:], h=hl, rstd=rl)
    assert same(q[-last:], ql) and same(s[:, -last:], sl)
    assert same(h[-last:], hl) and same(rstd[-last:], rl)
    del q, s
    dx, dw = fp8bs.bf16_rmsnorm_backward(x, h, rstd, g)
    dl, _ = fp8bs.bf16_rmsnorm_backward(x[-last:], hl, rl, g)
    assert same(dx[-last:], dl)
    # dweight of some columns in float64, M FP32 terms and sums in parts of at most
    # M / 256 + 1 rows and 256 of them
    c = slice(K - 128, K)
    n = h[:, c].double() * rstd.double()[:, None]
    t = x[:, c].double() * n
    tol = (M / 256 + 260) * 2.0 ** -24 * t.abs().sum(0)
    assert torch.all((dw[c].double() - t.sum(0)).abs() <= tol)


def test_gated_backward_past_32_bits(fp8bs):
    """z of 2.3e9 elements and its codes, both ways round; the last rows."""
    M, N, first = 70001, 16384, 70001 // 128 * 128 - 256
    dy, z = values(M, N), values(M, 2 * N)
    q, s, qt, st, yt, syt = fp8bs.fp8_quant_gated_backward(dy, z)
    want = fp8bs.fp8_quant_gated_backward(dy[first:], z[first:])
    b = first // 128
    got = (q[first:], s[:, first:], qt[:, first:], st[b:], yt[:, first:], syt[b:])
    for a, w in zip(got, want):
        assert same(a, w)
