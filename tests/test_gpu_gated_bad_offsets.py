"""Expert offsets that break the contract (decreasing, negative, overlong): results
are unspecified, but nothing outside z, the codes, their scales and the bf16 output
is written, by any tile shape, and the next call is right."""

import pytest
import torch

from fp8_block_scaled_05_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def framed(rows, cols, frame, dtype, fill):
    """(buffer full of ``fill``, the view of rows x cols inside a frame of it)"""
    buf = torch.full((rows + 2, cols + 2 * frame), fill, dtype=dtype, device="cuda")
    return buf, buf[1:rows + 1, frame:frame + cols]


def untouched(buf, view, fill):
    """The frame as it was; clears the view."""
    view.fill_(fill)
    return bool(torch.all(buf == fill))


# E4M3 tiles of 32, 64, 64 and 128 rows; bf16 of 32x64, 64x64, 128x256 and 256x256
@pytest.mark.parametrize("M,N", [(300, 256), (640, 1536), (700, 2048), (2000, 4096)])
def test_nothing_outside_is_written(fp8bs, M, N):
    G, K = 3, 256
    qx, sx = fp8bs.fp8_quant_act_1x128(synth.act(M, K, case=1320, device="cuda"))
    w = [fp8bs.fp8_quant_w_128x128(synth.weight(2 * N, K, case=1320, tensor=1 + e, device="cuda"))
         for e in range(G)]
    qw, sw = torch.stack([c for c, _ in w]), torch.stack([s for _, s in w])
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    zb, z = framed(M, 2 * N, 3, bf, 9)
    yb, y = framed(M, N, 5, bf, 9)
    qb, q = framed(M, N, 16, u8, 7)
    sb, s = framed(N // 128, M, 3, f32, 7)
    third = M // 3
    good = torch.tensor([0, third, 2 * third, M], dtype=torch.int32, device="cuda")
    want = (fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, good),
            *fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, good))
    big = 2 ** 31 - 1
    for off in ([0, 2 * third, third, M], [-50, third, 2 * third, M], [0, third, 9 * M, big],
                [M, 0, 0, M], [big, -big, big, -big], [M, M, M, M], [0, M, 0, M]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, o, z=z, out=y)
        torch.cuda.synchronize()
        assert untouched(zb, z, 9) and untouched(yb, y, 9), off
        fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, o, z=z, qc=q, sc=s)
        torch.cuda.synchronize()
        assert untouched(zb, z, 9) and untouched(qb, q, 7) and untouched(sb, s, 7), off
    fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, good, z=z, out=y)
    fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, good, qc=q, sc=s)
    assert all(torch.equal(a, b) for a, b in zip((y, q, s), want))
