"""Refusals of the gated product's and the norm's calls, at the C ABI (fake
device addresses: validation comes before any HIP call) and in the binding (no
GPU needed)."""

import pytest
import torch

from fp8_block_scaled_05_amd import fp8bs

P = 1 << 20
lib = fp8bs.lib


def gemm(a_kind=0, a=P, lda=256, sa=P, ldsa=64, b=P, ldb=256, sb=P, act=2, z=0, ldz=0, c=P,
         ldc=128, M=64, N=128, K=256, ws=0, n=0):
    return lib.fp8_block_gemm_gated(a_kind, a, lda, sa, ldsa, b, ldb, sb, act, z, ldz, c, ldc, M, N,
                                    K, ws, n, None)


def test_gated_gemm():
    assert gemm(act=4) == fp8bs.ERR_DTYPE and gemm(act=-1) == fp8bs.ERR_DTYPE
    assert gemm(a_kind=2) == fp8bs.ERR_DTYPE
    assert gemm(K=100) == fp8bs.ERR_SHAPE and gemm(K=0) == fp8bs.ERR_SHAPE
    assert gemm(N=200) == fp8bs.ERR_SHAPE and gemm(N=64) == fp8bs.ERR_SHAPE
    assert gemm(M=-1) == fp8bs.ERR_SHAPE and gemm(N=-128) == fp8bs.ERR_SHAPE
    assert gemm(M=0, a=0, c=0) == fp8bs.OK and gemm(N=0, b=0) == fp8bs.OK
    for k in ("a", "sa", "b", "sb", "c"):
        assert gemm(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("lda", 128), ("lda", 264), ("ldb", 255), ("ldb", (1 << 24) + 16), ("ldsa", 63),
                 ("ldc", 127), ("a", P + 8), ("b", P + 8), ("sb", P + 2), ("sa", P + 1),
                 ("c", P + 1)):
        assert gemm(**{k: v}) == fp8bs.ERR_LAYOUT, (k, v)
    # W within 32-bit offsets
    assert gemm(N=1 << 20, ldb=2048, ldc=1 << 20) == fp8bs.ERR_LAYOUT
    assert gemm(N=1 << 62, ldc=1 << 62) == fp8bs.ERR_LAYOUT
    assert gemm(z=P, ldz=255) == fp8bs.ERR_LAYOUT and gemm(z=P + 1, ldz=256) == fp8bs.ERR_LAYOUT
    need = fp8bs.workspace_bytes(fp8bs.OP_GEMM_BF16, 64, 128, 256)
    assert gemm(a_kind=1, sa=0) == fp8bs.ERR_WORKSPACE
    assert gemm(a_kind=1, sa=0, ws=P, n=need - 1) == fp8bs.ERR_WORKSPACE
    assert gemm(a_kind=1, sa=0, ws=P + 128, n=need) == fp8bs.ERR_LAYOUT


def test_gated_gemm_e4m3_out():
    def g(a_kind=0, act=2, z=0, ldz=0, qc=P, ldqc=256, sc=P, ldsc=200, M=200, N=256, ws=0, n=0):
        return lib.fp8_block_gemm_gated_e4m3_out(a_kind, P, 256, P, 200, P, 256, P, act, z, ldz, qc,
                                                 ldqc, sc, ldsc, M, N, 256, ws, n, None)

    assert g(N=200) == fp8bs.ERR_SHAPE and g(act=9) == fp8bs.ERR_DTYPE
    assert g(sc=0) == fp8bs.ERR_NULL and g(qc=0) == fp8bs.ERR_NULL
    assert g(ldsc=199) == fp8bs.ERR_LAYOUT and g(ldqc=248) == fp8bs.ERR_LAYOUT
    assert g(qc=P + 8) == fp8bs.ERR_LAYOUT and g(z=P, ldz=256) == fp8bs.ERR_LAYOUT
    # few rows and a bf16 A need room
    need = fp8bs.workspace_bytes(fp8bs.OP_GEMM_GATED_E4M3, 64, 256, 256)
    assert need >= 64 * 256 * 4 + 64 * 256
    assert g(M=64) == fp8bs.ERR_WORKSPACE and g(M=64, ws=P, n=need - 1) == fp8bs.ERR_WORKSPACE
    assert g(M=64, ws=P + 16, n=need) == fp8bs.ERR_LAYOUT
    assert g(a_kind=1) == fp8bs.ERR_WORKSPACE
    assert (fp8bs.workspace_bytes(fp8bs.OP_GEMM_GATED_E4M3, 65, 256, 256) ==
            fp8bs.workspace_bytes(fp8bs.OP_GEMM_BF16, 65, 256, 256))
    assert fp8bs.workspace_bytes(fp8bs.OP_GEMM_GATED_E4M3, 0, 256, 256) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_grouped(e4m3):
    def g(a=P, lda=256, sa=P, ldsa=64, b=P, ldb=256, stride=512 * 256, sb=P, act=2, z=0, ldz=0, c=P,
          ldc=256, sc=P, ldsc=64, off=P, G=3, M=64, N=256, K=256):
        head = (a, lda, sa, ldsa, b, ldb, stride, sb, act, z, ldz, c, ldc)
        tail = (off, G, M, N, K, None)
        if e4m3:
            return lib.fp8_block_grouped_gemm_gated_e4m3_out(*head, sc, ldsc, *tail)
        return lib.fp8_block_grouped_gemm_gated(*head, *tail)

    assert g(act=5) == fp8bs.ERR_DTYPE
    for k, v in (("G", 0), ("G", 4097), ("M", -1), ("N", 200), ("K", 100)):
        assert g(**{k: v}) == fp8bs.ERR_SHAPE, (k, v)
    assert g(M=0) == fp8bs.OK and g(N=0) == fp8bs.OK
    for k in ("a", "sa", "b", "sb", "c", "off") + (("sc",) if e4m3 else ()):
        assert g(**{k: 0}) == fp8bs.ERR_NULL, k
    # the stride covers gate and up rows
    for k, v in (("stride", 512 * 256 - 16), ("stride", 512 * 256 + 8), ("ldsa", 63), ("ldc", 255),
                 ("lda", 255), ("ldb", 264), ("off", P + 2), ("sa", P + 2)):
        assert g(**{k: v}) == fp8bs.ERR_LAYOUT, (k, v)
    assert g(z=P, ldz=511) == fp8bs.ERR_LAYOUT
    if e4m3:
        assert g(ldsc=63) == fp8bs.ERR_LAYOUT


def test_gated_backward():
    def b(dy=P, lddy=256, z=P, ldz=512, act=2, M=200, N=256, q=P, ldq=512, s=P, lds=200, qt=P,
          ldqt=256, st=P, ldst=512, yt=P, ldyt=256, syt=P, ldsyt=256):
        return lib.fp8_quant_gated_backward(dy, lddy, z, ldz, act, M, N, q, ldq, s, lds, qt, ldqt,
                                            st, ldst, yt, ldyt, syt, ldsyt, None)

    assert b(act=7) == fp8bs.ERR_DTYPE
    assert b(N=200) == fp8bs.ERR_SHAPE and b(M=-1) == fp8bs.ERR_SHAPE
    assert b(M=0) == fp8bs.OK and b(N=0) == fp8bs.OK
    for k in ("dy", "z", "q", "s", "qt", "st", "yt", "syt"):
        assert b(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("lddy", 255), ("ldz", 256), ("ldq", 256), ("lds", 199), ("ldqt", 208),
                 ("ldst", 511), ("ldyt", 208), ("ldsyt", 255), ("dy", P + 8), ("qt", P + 8),
                 ("yt", P + 8), ("syt", P + 2), ("s", P + 2)):
        assert b(**{k: v}) == fp8bs.ERR_LAYOUT, (k, v)


@pytest.mark.parametrize("codes", [False, True])
def test_rmsnorm(codes):
    def f(x=P, ldx=256, r=0, ldr=0, w=P, eps=1e-6, h=0, ldh=0, y=P, ldy=256, rstd=0, q=P, ldq=256,
          s=P, lds=100, M=100, K=256):
        if codes:
            return lib.fp8_quant_rmsnorm(x, ldx, r, ldr, w, eps, h, ldh, y, ldy, rstd, q, ldq, s,
                                         lds, M, K, None)
        return lib.bf16_rmsnorm(x, ldx, r, ldr, w, eps, h, ldh, rstd, y, ldy, M, K, None)

    for k, v in (("K", 0), ("K", 200), ("K", 32768 + 128), ("M", -1), ("eps", 0.0), ("eps", -1.0),
                 ("eps", 2.0 ** -101), ("eps", float("inf")), ("eps", float("nan"))):
        assert f(**{k: v}) == fp8bs.ERR_SHAPE, (k, v)
    assert f(M=0, x=0, y=0, q=0) == fp8bs.OK
    for k in ("x", "w") + (("q", "s") if codes else ("y",)):
        assert f(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("ldx", 128), ("ldx", 264), ("x", P + 8), ("w", P + 4), ("ldy", 240), ("y", P + 2),
                 ("rstd", P + 2)) + ((("ldq", 255), ("q", P + 8), ("lds", 99), ("s", P + 1))
                                     if codes else ()):
        assert f(**{k: v}) == fp8bs.ERR_LAYOUT, (k, v)
    assert f(r=P, ldr=240) == fp8bs.ERR_LAYOUT and f(r=P + 8, ldr=256) == fp8bs.ERR_LAYOUT
    assert f(h=P, ldh=240) == fp8bs.ERR_LAYOUT and f(h=P + 8, ldh=256) == fp8bs.ERR_LAYOUT


def test_rmsnorm_backward():
    need = fp8bs.workspace_bytes(fp8bs.OP_RMSNORM_BACKWARD, 1000, 0, 512)
    assert 0 < need <= 1024 * 512
    assert fp8bs.workspace_bytes(fp8bs.OP_RMSNORM_BACKWARD, 10 ** 9, 0, 512) <= 1024 * 512

    def f(dy=P, lddy=512, h=P, ldh=512, rstd=P, w=P, dh=0, lddh=0, dx=P, lddx=512, dw=P, M=1000,
          K=512, ws=P, n=need):
        return lib.bf16_rmsnorm_backward(dy, lddy, h, ldh, rstd, w, dh, lddh, dx, lddx, dw, M, K,
                                         ws, n, None)

    for k, v in (("K", 0), ("K", 200), ("K", 32768 + 128), ("M", -1)):
        assert f(**{k: v}) == fp8bs.ERR_SHAPE, (k, v)
    for k in ("dy", "h", "rstd", "w", "dx", "dw"):
        assert f(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("lddy", 496), ("ldh", 520), ("lddx", 128), ("dy", P + 8), ("dx", P + 8),
                 ("w", P + 8), ("dw", P + 4), ("rstd", P + 2), ("ws", P + 64)):
        assert f(**{k: v}) == fp8bs.ERR_LAYOUT, (k, v)
    assert f(dh=P, lddh=496) == fp8bs.ERR_LAYOUT and f(dh=P + 4, lddh=512) == fp8bs.ERR_LAYOUT
    assert f(n=need - 1) == fp8bs.ERR_WORKSPACE and f(ws=0) == fp8bs.ERR_WORKSPACE


def test_binding():
    bf, u8 = torch.bfloat16, torch.uint8
    a, sa = torch.zeros(70, 256, dtype=u8), torch.zeros(2, 70)
    b, sb = torch.zeros(512, 256, dtype=u8), torch.zeros(4, 2)
    f = fp8bs.fp8_block_gemm_gated
    with pytest.raises(ValueError, match="act must be one of"):
        f(a, sa, b, sb, act="swish")
    with pytest.raises(ValueError, match="multiple of 128 each"):
        f(a, sa, b[:384], sb[:3])
    with pytest.raises(ValueError, match="z must be a 2-D tensor"):
        f(a, sa, b, sb, z=torch.zeros(70, 256, dtype=bf))
    with pytest.raises(ValueError, match="z must be torch.bfloat16"):
        f(a, sa, b, sb, z=torch.zeros(70, 512))
    with pytest.raises(ValueError, match="out must be torch.bfloat16"):
        f(a, sa, b, sb, out=torch.zeros(70, 256))
    with pytest.raises(ValueError, match="sb must be a 2-D tensor"):
        f(a, sa, b, sb[:2])
    with pytest.raises(ValueError, match="need their scales"):
        f(a, None, b, sb)
    with pytest.raises(ValueError, match="GPU tensors only"):
        f(a, sa, b, sb)
    g = fp8bs.fp8_block_gemm_gated_e4m3_out
    with pytest.raises(ValueError, match="qc must be a 2-D tensor"):
        g(a, sa, b, sb, qc=torch.zeros(70, 128, dtype=u8))
    with pytest.raises(ValueError, match="sc must be a 2-D tensor"):
        g(a, sa, b, sb, sc=torch.zeros(1, 70))
    with pytest.raises(ValueError, match="GPU tensors only"):
        g(a, sa, b, sb)
    b3, sb3, off = torch.zeros(2, 512, 256, dtype=u8), torch.zeros(2, 4, 2), torch.zeros(3).int()
    for call in (fp8bs.fp8_block_grouped_gemm_gated, fp8bs.fp8_block_grouped_gemm_gated_e4m3_out):
        with pytest.raises(ValueError, match="group_offsets must be int32"):
            call(a, sa, b3, sb3, off.long())
        with pytest.raises(ValueError, match="vector of G"):
            call(a, sa, b3, sb3, off[:2])
        with pytest.raises(ValueError, match="multiple of 128 each"):
            call(a, sa, b3[:, :384], sb3[:, :3].contiguous(), off)
        with pytest.raises(ValueError, match="z must be a 2-D tensor"):
            call(a, sa, b3, sb3, off, z=torch.zeros(69, 512, dtype=bf))
        with pytest.raises(ValueError, match="GPU tensors only"):
            call(a, sa, b3, sb3, off)
    h = fp8bs.fp8_quant_gated_backward
    dy, z = torch.zeros(10, 256, dtype=bf), torch.zeros(10, 512, dtype=bf)
    with pytest.raises(ValueError, match="multiple of 128"):
        h(torch.zeros(10, 200, dtype=bf), z)
    with pytest.raises(ValueError, match="z must be a 2-D tensor"):
        h(dy, dy)
    with pytest.raises(ValueError, match="qt must be a 2-D tensor"):
        h(dy, z, qt=torch.zeros(256, 128, dtype=u8))
    with pytest.raises(ValueError, match="outputs of product=True"):
        h(dy, z, yt=torch.zeros(256, 128, dtype=u8), product=False)
    with pytest.raises(ValueError, match="GPU tensors only"):
        h(dy, z)
    w = torch.ones(256)
    for call in (fp8bs.fp8_quant_rmsnorm, fp8bs.bf16_rmsnorm):
        with pytest.raises(ValueError, match="x must be torch.bfloat16"):
            call(dy.float(), w)
        with pytest.raises(ValueError, match="weight must be torch.float32"):
            call(dy, w.to(bf))
        with pytest.raises(ValueError, match="weight must be a contiguous vector"):
            call(dy, w[:128])
        with pytest.raises(ValueError, match="K = 200"):
            call(dy[:, :200], w)
        with pytest.raises(ValueError, match="residual must be a 2-D tensor"):
            call(dy, w, residual=dy[:9])
        with pytest.raises(ValueError, match="rstd must be a contiguous vector"):
            call(dy, w, rstd=torch.zeros(9))
        with pytest.raises(ValueError, match="GPU tensors only"):
            call(dy, w)
    n = fp8bs.bf16_rmsnorm_backward
    with pytest.raises(ValueError, match="rstd must be torch.float32"):
        n(dy, dy, torch.zeros(10, dtype=bf), w)
    with pytest.raises(ValueError, match="h must be a 2-D tensor"):
        n(dy, dy[:5], torch.zeros(10), w)
    with pytest.raises(ValueError, match="dh must be torch.bfloat16"):
        n(dy, dy, torch.zeros(10), w, dh=dy.float())
    with pytest.raises(ValueError, match="dweight must be a contiguous vector"):
        n(dy, dy, torch.zeros(10), w, dweight=torch.zeros(128))
    with pytest.raises(ValueError, match="GPU tensors only"):
        n(dy, dy, torch.zeros(10), w)
