"""NaN in the gated product's E4M3 output: an element of y that is NaN has the code
of NaN, whatever else its tile holds, on the tiled paths and on that of few rows."""

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


def operands(fp8bs, M, N, K, case):
    x = synth.act(M, K, case=case, tensor=0, device="cuda")
    w = synth.weight(2 * N, K, case=case, tensor=1, device="cuda").float() * (50 / K ** 0.5)
    return x, *fp8bs.fp8_quant_act_1x128(x), *fp8bs.fp8_quant_w_128x128(w.to(torch.bfloat16))


# few rows by one, two and four row tiles; tiles of 32, 64 and 128 rows
SHAPES = [(1, 256), (16, 384), (20, 256), (50, 256), (70, 256), (200, 4096), (1000, 4096)]


@pytest.mark.parametrize("bf16_in", [False, True])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("M,N", SHAPES)
def test_a_column(fp8bs, M, N, up, bf16_in):
    """A NaN in one row of W makes its column of y NaN; the tile's other codes are
    what they are beside a column of zeros."""
    K, n = 384, 200
    x, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1310)
    a, sa = (x, None) if bf16_in else (qx, sx)
    row = n + N * up
    qw[row] = 0
    q0, s0 = fp8bs.fp8_block_gemm_gated_e4m3_out(a, sa, qw, sw)
    qw[row, 77] = 0x7F
    z = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    q, s = fp8bs.fp8_block_gemm_gated_e4m3_out(a, sa, qw, sw, z=z)
    assert torch.all(z[:, row].isnan()) and z.isnan().sum() == M
    assert torch.all(is_nan(q[:, n]))
    rest = torch.arange(N, device="cuda") != n
    assert torch.equal(q[:, rest], q0[:, rest]) and torch.equal(s, s0)


@pytest.mark.parametrize("M,N", [s for s in SHAPES if s[0] > 1])
def test_a_row(fp8bs, M, N):
    """A NaN code of A makes its row NaN and no other, in both output types."""
    K, m = 384, M // 2
    _, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1311)
    q0, s0 = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw)
    y0 = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw)
    qx[m, 300] = 0x7F
    q, s = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw)
    y = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw)
    keep = torch.arange(M, device="cuda") != m
    assert torch.all(is_nan(q[m])) and torch.all(y[m].isnan())
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[:, keep], s0[:, keep])
    assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("rows,N", [([40, 0, 130], 256), ([300, 200, 140], 1536),
                                    ([900, 500, 600], 4096)])
def test_experts(fp8bs, rows, N):
    """One expert's NaN stays with its rows (tiles of 32, 64 and 128 rows)."""
    K, M, n = 256, sum(rows), 131
    _, qx, sx, _, _ = operands(fp8bs, M, 128, K, 1312)
    w = [fp8bs.fp8_quant_w_128x128(synth.weight(2 * N, K, case=1312, tensor=1 + e, device="cuda"))
         for e in range(3)]
    qw, sw = torch.stack([c for c, _ in w]), torch.stack([s for _, s in w])
    off = torch.tensor([0] + rows, device="cuda").cumsum(0).to(torch.int32)
    qw[2, n] = 0
    q0, s0 = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off)
    qw[2, n, 9] = 0x7F
    q, s = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off)
    where = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    where[rows[0] + rows[1]:, n] = True
    assert torch.equal(is_nan(q), where)
    assert torch.equal(q[~where], q0[~where]) and torch.equal(s, s0)


def test_a_training_step_shows_it():
    """A NaN that the E4M3 operands alone carry (a norm's weight, the gate's codes)
    reaches the loss and the gradients."""
    from fp8_block_scaled_05_amd import train_step as ts
    for rows in (50, 700):
        cfg = ts.Config(block="gated", act="silu", layers=1)
        p = ts.init(cfg)
        p["norm0"][5] = float("nan")
        loss, grads = ts.loss_and_grads(cfg, p, *ts.batch(cfg, rows, 3))
        assert loss.isnan() and torch.all(grads["head"].isnan().any(dim=1))
