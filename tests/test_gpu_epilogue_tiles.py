"""The epilogue at the ends of its tile choice: sizes around the counts where the
next tile shape takes over, with odd strides and the residual in place.
Tolerances as derived in test_gpu_epilogue.py."""

import pytest
import torch

from oracle import epilogue
from tests import _gpu_util as gu
from tests.test_gpu_epilogue import check, extras, fp8bs, operands  # noqa: F401

pytestmark = pytest.mark.gpu

# 32x64 tiles up to 128 tiles of 64x64 (128 and 129 of them), those up to 768
# (768 and 784), half and large tiles beyond
SHAPES = [(100, 4096, 128), (65, 4160, 256), (129, 2752, 384), (1536, 2048, 128),
          (1560, 2000, 256), (1300, 2600, 384), (1100, 8200, 128), (2000, 5001, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_part(fp8bs, M, N, K):  # noqa: F811
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 910)
    bias, res = extras(M, N, M)
    z = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act="gelu", residual=res, z=z)
    want, wz = epilogue.forward(C, gu.host_f64(bias), "gelu", gu.host_f64(res))
    check(y, want, wz, B)
    check(z, wz, wz, B)
    plain = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw)
    assert torch.equal(plain, fp8bs.fp8_block_gemm(qx, sx, qw, sw))


@pytest.mark.parametrize("ld,shift", [(3, 0), (1, 1), (6, 2)])
@pytest.mark.parametrize("M,N", [(520, 1990), (1300, 2600), (1100, 8198)])
def test_strides_in_place(fp8bs, M, N, ld, shift):  # noqa: F811
    """Row strides of N + ld elements from an offset; the residual is the output.
    Nothing outside the output's rows and columns is written."""
    K, ld = 256, N + ld
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 911)
    bias, _ = extras(M, N, 4)
    bufs = [torch.full((M * ld + 8,), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z, out = [torch.as_strided(b, (M, N), (ld, 1), shift) for b in bufs]
    out.copy_(torch.randn(M, N, device="cuda"))
    want, wz = epilogue.forward(C, gu.host_f64(bias), "silu", gu.host_f64(out))
    fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act="silu", residual=out, z=z, out=out)
    check(out, want, wz, B)
    check(z, wz, wz, B)
    for b, v in zip(bufs, (z, out)):
        v.fill_(9.0)
        assert torch.all(b == 9.0)
