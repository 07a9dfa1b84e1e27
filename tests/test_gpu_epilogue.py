"""The GEMM's epilogue and its backward on the GPU against the float64 oracle.

Tolerances: the FP32 sums C are held to the library's bar 2e-3 * sum|a b|
(tests/_gpu_util.py).  act has a slope of at most 1.13 (gelu at 1.41; silu
1.10), so y is off by at most 1.13 of that, by its activation's own error
(sigma by hardware exp and reciprocal: below 2^-18 of |z| for |z| <= 20, the
argument's rounding being |z| 2^-23), and by 2^-8 of its value for bf16.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import epilogue
from fp8_block_scaled_05_amd import synth
from tests import _gpu_util as gu

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu"]
SLOPE = 1.13


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def operands(fp8bs, M, N, K, case):
    x = synth.act(M, K, case=case, tensor=0, device="cuda")
    w = (synth.weight(N, K, case=case, tensor=1, device="cuda").float() * (50 / K ** 0.5)).to(
        torch.bfloat16)
    qw, sw = fp8bs.fp8_quant_w_128x128(w)
    qx, sx = fp8bs.fp8_quant_act_1x128(x)
    C, B = oracle.block_gemm(gu.host(qx), gu.host(sx), gu.host(qw), gu.host(sw))
    return x, qx, sx, qw, sw, C, B


def extras(M, N, seed, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bias = torch.randn(N, generator=g, device="cuda")
    res = torch.randn(M, ld or N, generator=g, device="cuda").to(torch.bfloat16)[:, :N]
    return bias, res


def check(got, want, z, B):
    got = gu.host_f64(got)
    assert np.all(np.isfinite(got))
    tol = SLOPE * 2e-3 * B + 2.0 ** -18 * np.abs(z) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol)


# few-row kernels (fused quantizer, codes, shared), every tile shape, ragged
SHAPES = [(1, 100, 128), (3, 261, 1280), (16, 2050, 512), (20, 300, 384), (64, 777, 256),
          (65, 128, 128), (100, 130, 512), (333, 2050, 640), (300, 8200, 256), (1100, 4100, 256)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_codes_in_bf16_out(fp8bs, M, N, K, act):
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 900)
    bias, res = extras(M, N, M + N)
    z = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act=act, residual=res, z=z)
    want, wz = epilogue.forward(C, gu.host_f64(bias), act, gu.host_f64(res))
    check(y, want, wz, B)
    check(z, wz, wz, B)


@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 64, 70])
def test_bf16_in(fp8bs, M):
    N, K = 515, 640
    x, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 901)
    bias, res = extras(M, N, M)
    s = torch.zeros(K // 128, M, device="cuda")
    y = fp8bs.fp8_block_gemm_epilogue(x, s, qw, sw, bias=bias, act="silu", residual=res)
    assert torch.equal(s, sx)
    want, wz = epilogue.forward(C, gu.host_f64(bias), "silu", gu.host_f64(res))
    check(y, want, wz, B)
    # the same as from the quantizer's codes
    y2 = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act="silu", residual=res)
    check(y2, want, wz, B)


@pytest.mark.parametrize("bias,residual,z", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)])
@pytest.mark.parametrize("M", [8, 50, 200])
def test_parts_left_out(fp8bs, M, bias, residual, z):
    N, K = 390, 256
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 902)
    b, r = extras(M, N, 3)
    zk = torch.empty(M, N, dtype=torch.bfloat16, device="cuda") if z else None
    y = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=b if bias else None, act="gelu",
                                      residual=r if residual else None, z=zk)
    want, wz = epilogue.forward(C, gu.host_f64(b) if bias else None, "gelu",
                                gu.host_f64(r) if residual else None)
    check(y, want, wz, B)
    if z:
        check(zk, wz, wz, B)


def test_nothing_in_the_epilogue_is_the_plain_product(fp8bs):
    for M, N in ((4, 300), (40, 300), (90, 300), (700, 5000)):
        _, qx, sx, qw, sw, _, _ = operands(fp8bs, M, N, 256, 903)
        y = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw)
        assert torch.equal(y, fp8bs.fp8_block_gemm(qx, sx, qw, sw))


@pytest.mark.parametrize("M", [7, 33, 129])
@pytest.mark.parametrize("ld,shift", [(400, 0), (401, 1), (406, 2)])
def test_strides_and_alignment(fp8bs, M, ld, shift):
    """Odd row strides and offsets of residual, z and output; nothing outside
    the output's rows and columns is written."""
    N, K = 390, 256
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 904)
    bias, _ = extras(M, N, 4)
    bufs = [torch.full((M * ld + 8,), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    view = [torch.as_strided(b, (M, N), (ld, 1), shift) for b in bufs]
    res, z, out = view
    res.copy_(torch.randn(M, N, device="cuda"))
    fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act="silu", residual=res, z=z, out=out)
    want, wz = epilogue.forward(C, gu.host_f64(bias), "silu", gu.host_f64(res))
    check(out, want, wz, B)
    check(z, wz, wz, B)
    for b, v in zip(bufs[1:], view[1:]):
        v.fill_(9.0)
        assert torch.all(b == 9.0)


@pytest.mark.parametrize("M", [9, 50, 150])
def test_residual_in_place(fp8bs, M):
    N, K = 256, 256
    _, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 905)
    _, res = extras(M, N, 5)
    want, wz = epilogue.forward(C, None, "none", gu.host_f64(res))
    y = fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, residual=res, out=res)
    assert y is res
    check(y, want, wz, B)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,a_bf16", [(1, 128, False), (12, 256, True), (64, 384, False),
                                        (333, 2048, False), (600, 4096, True)])
def test_e4m3_out(fp8bs, M, N, a_bf16, act):
    """The codes' values against y: an E4M3 value is off by at most 2^-4 of it
    or, below the normal range, half a step of 2^-9, both times the scale,
    which is (largest |y| of the tile) / 448 within the tile's tolerance."""
    K = 256
    x, qx, sx, qw, sw, C, B = operands(fp8bs, M, N, K, 906)
    bias, res = extras(M, N, 6)
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qc, sc = fp8bs.fp8_block_gemm_epilogue_e4m3_out(
        x if a_bf16 else qx, None if a_bf16 else sx, qw, sw, bias=bias, act=act, residual=res, z=z)
    y, wz = epilogue.forward(C, gu.host_f64(bias), act, gu.host_f64(res))
    check(z, wz, wz, B)
    tol = SLOPE * 2e-3 * B + 2.0 ** -18 * np.abs(wz)
    s = gu.host_f64(sc).T  # [M][N/128]
    t = lambda a: a.reshape(M, N // 128, 128)
    top = np.abs(t(y)).max(axis=2)
    assert np.all(np.abs(s * 448 - top) <= t(tol).max(axis=2) + 2.0 ** -20 * top)
    got = t(oracle.decode(gu.host(qc)).astype(np.float64)) * s[:, :, None]
    lim = (np.abs(t(y)) + t(tol)) * 2.0 ** -4 + 2.0 ** -10 * s[:, :, None] + t(tol)
    assert np.all(np.abs(got - t(y)) <= lim * (1 + 2.0 ** -16))


# ----------------------------------------------------------------------------
# backward


def grads(M, N, seed, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(M, ld or N, generator=g, device="cuda").to(torch.bfloat16)[:, :N]
    z = (2 * torch.randn(M, ld or N, generator=g, device="cuda")).to(torch.bfloat16)[:, :N]
    return dy, z


def padded(dz):
    M, N = dz.shape
    out = torch.zeros((M + 127) // 128 * 128, N, dtype=dz.dtype, device=dz.device)
    out[:M] = dz
    return out


@pytest.mark.parametrize("M,N", [(1, 128), (127, 256), (128, 128), (333, 2048), (700, 640)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_equals_the_quantizers(fp8bs, M, N, act):
    """Where dz is a bf16 value (no activation, relu) both quantized forms are
    the library's quantizers' on it, bit for bit."""
    dy, z = grads(M, N, M)
    q, s, qt, st, db = fp8bs.fp8_quant_epilogue_backward(dy, z if act == "relu" else None, act)
    dz = dy if act == "none" else torch.where(z > 0, dy, torch.zeros_like(dy))
    q2, s2 = fp8bs.fp8_quant_act_1x128(dz)
    qt2, st2 = fp8bs.fp8_quant_act_128x1_t(padded(dz))
    # a masked negative value may keep its sign (code 0x80)
    plain = lambda c: torch.where(c == 0x80, torch.zeros_like(c), c)
    assert torch.equal(plain(q), plain(q2)) and torch.equal(s, s2)
    assert torch.equal(plain(qt), plain(qt2)) and torch.equal(st, st2)
    d = gu.host_f64(dz)
    assert np.all(np.abs(gu.host_f64(db) - d.sum(0)) <= (M + 8) * 2.0 ** -24 * np.abs(d).sum(0))


@pytest.mark.parametrize("M,N", [(1, 128), (130, 384), (333, 2048)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_values(fp8bs, M, N, act):
    """dz in FP32 is off by less than 2^-20 (|dy| (1 + |z|)): sigma and its
    products carry a few 2^-24 each, times |z| where z multiplies them.  The
    codes' values add an E4M3 rounding (2^-4 of the value, or half a step of
    2^-9, times the scale)."""
    dy, z = grads(M, N, M + 1)
    q, s, qt, st, db = fp8bs.fp8_quant_epilogue_backward(dy, z, act)
    hy, hz = gu.host_f64(dy), gu.host_f64(z)
    dz, want_db = epilogue.backward(hy, hz, act)
    tol = 2.0 ** -20 * np.abs(hy) * (1 + np.abs(hz))
    assert np.all(np.abs(gu.host_f64(db) - want_db) <=
                  tol.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(dz).sum(0))
    Mp = (M + 127) // 128 * 128
    pad = lambda a: np.concatenate([a, np.zeros((Mp - M, N))]).T
    for codes, scale, d, e in ((q, s, dz, tol), (qt, st, pad(dz), pad(tol))):
        R, W = d.shape
        t = lambda a: a.reshape(R, W // 128, 128)
        sc = gu.host_f64(scale).T
        top = np.maximum(np.abs(t(d)).max(axis=2), 2.0 ** -64)
        assert np.all(np.abs(sc * 448 - top) <= t(e).max(axis=2) + 2.0 ** -22 * top)
        got = t(oracle.decode(gu.host(codes)).astype(np.float64)) * sc[:, :, None]
        lim = (np.abs(t(d)) + t(e)) * 2.0 ** -4 + 2.0 ** -10 * sc[:, :, None] + t(e)
        assert np.all(np.abs(got - t(d)) <= lim * (1 + 2.0 ** -16))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_far_arguments(fp8bs, act):
    """z out to bf16's largest values: slopes 0 and 1, nothing that is not
    finite."""
    M, N = 128, 128
    z = torch.tensor([30.0, -30.0, 200.0, -200.0, 1e5, -1e5, 3e38, -3e38], device="cuda")
    z = z.to(torch.bfloat16).repeat(M, N // 8)
    dy = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    q, s, qt, st, db = fp8bs.fp8_quant_epilogue_backward(dy, z, act)
    got = torch.from_numpy(oracle.decode(gu.host(q)).astype(np.float64))
    want = torch.tensor([448.0, 0.0] * 4, dtype=torch.float64).repeat(M, N // 8)
    assert torch.all((got - want).abs() < 1e-2)
    assert torch.allclose(db.cpu().double(), want[0] * M / 448, atol=1e-2)


def test_backward_strides(fp8bs):
    M, N = 200, 256
    dy, z = grads(M, N, 8, ld=N + 48)
    ref = fp8bs.fp8_quant_epilogue_backward(dy.contiguous(), z.contiguous(), "gelu")
    q = torch.full((M, N + 32), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((N // 128, M + 5), 7.0, device="cuda")
    qt = torch.full((N, 256 + 16), 7, dtype=torch.uint8, device="cuda")
    st = torch.full((2, N + 3), 7.0, device="cuda")
    fp8bs.fp8_quant_epilogue_backward(dy, z, "gelu", q=q, s=s, qt=qt, st=st)
    assert torch.equal(q[:, :N], ref[0]) and torch.all(q[:, N:] == 7)
    assert torch.equal(s[:, :M], ref[1]) and torch.all(s[:, M:] == 7)
    assert torch.equal(qt[:, :256], ref[2]) and torch.all(qt[:, 256:] == 7)
    assert torch.equal(st[:, :N], ref[3]) and torch.all(st[:, N:] == 7)


def test_backward_of_the_layer(fp8bs):
    """The whole layer's gradients through the library's backward GEMMs against
    float64 products of the same quantized operands' values, and a directional
    difference of the oracle's layer."""
    M, N, K = 200, 256, 384
    x = synth.act(M, K, case=910, device="cuda", row_lognormal=False, outlier_frac=0)
    w = (synth.weight(N, K, case=910, device="cuda").float() * 3).to(torch.bfloat16)
    qx, sx = fp8bs.fp8_quant_act_1x128(x)
    qw, sw, qwt, swt = fp8bs.fp8_quant_w_128x128_t(w)
    bias, _ = extras(M, N, 9)
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8_block_gemm_epilogue(qx, sx, qw, sw, bias=bias, act="gelu", z=z)
    dy, _ = grads(M, N, 10)
    q, s, qt, st, db = fp8bs.fp8_quant_epilogue_backward(dy, z, "gelu")
    dx = fp8bs.fp8_block_gemm(q, s, qwt, swt)
    xt, sxt = fp8bs.fp8_quant_act_128x1_t(padded(x))
    dw = fp8bs.fp8_block_gemm_rowscaled(qt, st, xt, sxt)
    X, W, dY = gu.host_f64(x), gu.host_f64(w), gu.host_f64(dy)
    b = gu.host_f64(bias)
    layer = lambda X, W, b: (epilogue.act(X @ W.T + b, "gelu") * dY).sum()
    rng = np.random.default_rng(0)
    h = 1e-4
    # E4M3 keeps 3 mantissa bits: every operand is off by up to 2^-4 of its
    # value, so a derivative along a random direction is off by about 3 such
    # relative errors (two operands and z) of the root sum of squares; 0.25
    # of that norm is more than four standard deviations
    for which, g in ((0, gu.host_f64(dx)), (1, gu.host_f64(dw)), (2, gu.host_f64(db))):
        u = rng.normal(size=g.shape)
        args = [[X, W, b], [X, W, b]]
        args[0][which] = args[0][which] + h * u
        args[1][which] = args[1][which] - h * u
        diff = (layer(*args[0]) - layer(*args[1])) / (2 * h)
        assert abs(diff - (g * u).sum()) <= 0.25 * np.sqrt((g ** 2).sum())
