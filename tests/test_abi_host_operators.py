"""Refusals of the epilogue, epilogue-backward and cross-entropy calls, at the C
ABI (fake device addresses: validation comes before any HIP call) and in the
binding (no GPU needed)."""

import ctypes

import pytest

from fp8_block_scaled_05_amd import fp8bs

P = 1 << 20
lib = fp8bs.lib


def ep(bias=0, residual=0, ldr=0, z=0, ldz=0, act=0):
    return fp8bs._Epilogue(bias, residual, ldr, z, ldz, act)


def gemm(e=None, a_kind=0, a=P, lda=256, sa=P, ldsa=64, b=P, ldb=256, sb=P, c=P, ldc=128, M=64,
         N=128, K=256, ws=0, ws_bytes=0, null=False):
    e = None if null else ctypes.byref(e or ep())
    return lib.fp8_block_gemm_epilogue(a_kind, a, lda, sa, ldsa, b, ldb, sb, e, c, ldc, M, N, K, ws,
                                       ws_bytes, None)


def test_epilogue_gemm():
    assert gemm(null=True) == fp8bs.ERR_NULL
    assert gemm(ep(act=4)) == fp8bs.ERR_DTYPE
    assert gemm(ep(act=-1)) == fp8bs.ERR_DTYPE
    assert gemm(ep(residual=P, ldr=127)) == fp8bs.ERR_LAYOUT
    assert gemm(ep(z=P, ldz=127)) == fp8bs.ERR_LAYOUT
    assert gemm(ep(z=P + 1, ldz=128)) == fp8bs.ERR_LAYOUT
    assert gemm(ep(residual=P + 1, ldr=128)) == fp8bs.ERR_LAYOUT
    assert gemm(ep(bias=P + 2)) == fp8bs.ERR_LAYOUT
    assert gemm(K=100) == fp8bs.ERR_SHAPE
    assert gemm(M=0, a=0, c=0) == fp8bs.OK
    assert gemm(N=0) == fp8bs.OK
    assert gemm(a_kind=5) == fp8bs.ERR_DTYPE
    assert gemm(sa=0) == fp8bs.ERR_NULL
    assert gemm(ldc=127) == fp8bs.ERR_LAYOUT
    assert gemm(a_kind=1, sa=0) == fp8bs.ERR_WORKSPACE


def test_epilogue_gemm_e4m3_out():
    def g(e=None, qc=P, ldqc=256, sc=P, ldsc=64, N=256):
        return lib.fp8_block_gemm_epilogue_e4m3_out(0, P, 256, P, 64, P, 256, P,
                                                    ctypes.byref(e or ep()), qc, ldqc, sc, ldsc,
                                                    64, N, 256, 0, 0, None)

    assert g(N=200) == fp8bs.ERR_SHAPE
    assert g(ep(act=9)) == fp8bs.ERR_DTYPE
    assert g(sc=0) == fp8bs.ERR_NULL
    assert g(ldsc=63) == fp8bs.ERR_LAYOUT
    assert g(qc=P + 8) == fp8bs.ERR_LAYOUT


def test_epilogue_backward():
    need = fp8bs.workspace_bytes(fp8bs.OP_EPILOGUE_BACKWARD, 200, 256, 0)
    assert need == 2 * 256 * 4

    def b(dy=P, lddy=256, z=P, ldz=256, act=2, M=200, N=256, q=P, ldq=256, s=P, lds=200, qt=P,
          ldqt=256, st=P, ldst=256, db=P, ws=P, ws_bytes=need):
        return lib.fp8_quant_epilogue_backward(dy, lddy, z, ldz, act, M, N, q, ldq, s, lds, qt,
                                               ldqt, st, ldst, db, ws, ws_bytes, None)

    assert b(act=7) == fp8bs.ERR_DTYPE
    assert b(N=200) == fp8bs.ERR_SHAPE
    assert b(M=-1) == fp8bs.ERR_SHAPE
    assert b(M=0) == fp8bs.OK and b(N=0) == fp8bs.OK
    for k in ("dy", "z", "q", "s", "qt", "st", "db"):
        assert b(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("lddy", 255), ("ldz", 128), ("ldq", 255), ("lds", 199), ("ldqt", 208),
                 ("ldst", 255), ("dy", P + 8), ("qt", P + 8), ("db", P + 2), ("ws", P + 16)):
        assert b(**{k: v}) == fp8bs.ERR_LAYOUT, k
    assert b(ws_bytes=need - 1) == fp8bs.ERR_WORKSPACE
    assert b(ws=0) == fp8bs.ERR_WORKSPACE


def test_xent():
    need = fp8bs.workspace_bytes(fp8bs.OP_XENT, 100, 1000, 256)
    assert need > 0 and need % 256 == 0

    def f(x=P, ldx=256, w=P, ldw=256, t=P, loss=P, lse=P, M=100, V=1000, K=256, ws=P, n=need):
        return lib.bf16_linear_xent(x, ldx, w, ldw, t, -100, loss, lse, M, V, K, ws, n, None)

    assert f(M=-1) == fp8bs.ERR_SHAPE and f(V=0) == fp8bs.ERR_SHAPE
    assert f(K=100) == fp8bs.ERR_SHAPE and f(K=0) == fp8bs.ERR_SHAPE
    assert f(V=1 << 31) == fp8bs.ERR_SHAPE and f(M=1 << 31) == fp8bs.ERR_SHAPE
    assert f(M=0, x=0, loss=0) == fp8bs.OK
    for k in ("x", "w", "t", "loss", "lse"):
        assert f(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("ldx", 255), ("ldw", 264), ("ldw", (1 << 22) + 16), ("x", P + 8), ("t", P + 4),
                 ("ws", P + 64)):
        assert f(**{k: v}) == fp8bs.ERR_LAYOUT, k
    assert f(n=need - 1) == fp8bs.ERR_WORKSPACE and f(ws=0) == fp8bs.ERR_WORKSPACE


def test_xent_backward():
    need = fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, 100, 1000, 256)

    def f(x=P, ldx=256, w=P, ldw=256, t=P, lse=P, dl=P, dx=P, lddx=256, dw=P, lddw=256, M=100,
          V=1000, K=256, ws=P, n=need):
        return lib.bf16_linear_xent_backward(x, ldx, w, ldw, t, -100, lse, dl, dx, lddx, dw, lddw,
                                             M, V, K, ws, n, None)

    assert f(V=0) == fp8bs.ERR_SHAPE and f(K=64) == fp8bs.ERR_SHAPE
    for k in ("x", "w", "t", "lse", "dl", "dx", "dw"):
        assert f(**{k: 0}) == fp8bs.ERR_NULL, k
    for k, v in (("lddx", 128), ("lddw", 255), ("dx", P + 8), ("dw", P + 8), ("dl", P + 2),
                 ("ldx", (1 << 22) + 16)):
        assert f(**{k: v}) == fp8bs.ERR_LAYOUT, k
    assert f(n=need - 1) == fp8bs.ERR_WORKSPACE
    # the workspace does not grow with the vocabulary times the rows
    big = fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, 65536, 129280, 7168)
    assert big < 65536 * 129280 * 2 / 2


def test_binding():
    import torch
    bf, u8 = torch.bfloat16, torch.uint8
    a, sa = torch.zeros(64, 256, dtype=u8), torch.zeros(2, 64)
    b, sb = torch.zeros(300, 256, dtype=u8), torch.zeros(3, 2)
    f = fp8bs.fp8_block_gemm_epilogue
    with pytest.raises(ValueError, match="act must be one of"):
        f(a, sa, b, sb, act="tanh")
    with pytest.raises(ValueError, match="bias must be torch.float32"):
        f(a, sa, b, sb, bias=torch.zeros(300, dtype=bf))
    with pytest.raises(ValueError, match="bias must be a contiguous vector"):
        f(a, sa, b, sb, bias=torch.zeros(299))
    with pytest.raises(ValueError, match="residual must be a 2-D tensor"):
        f(a, sa, b, sb, residual=torch.zeros(64, 299, dtype=bf))
    with pytest.raises(ValueError, match="z must be torch.bfloat16"):
        f(a, sa, b, sb, z=torch.zeros(64, 300))
    with pytest.raises(ValueError, match="out must be torch.bfloat16"):
        f(a, sa, b, sb, out=torch.zeros(64, 300))
    with pytest.raises(ValueError, match="GPU tensors only"):
        f(a, sa, b, sb, bias=torch.zeros(300), act="silu")
    with pytest.raises(ValueError, match="multiple of 128"):
        fp8bs.fp8_block_gemm_epilogue_e4m3_out(a, sa, b, sb)
    g = fp8bs.fp8_quant_epilogue_backward
    dy = torch.zeros(10, 256, dtype=bf)
    with pytest.raises(ValueError, match="needs z"):
        g(dy, None, "gelu")
    with pytest.raises(ValueError, match="multiple of 128"):
        g(torch.zeros(10, 200, dtype=bf), None)
    with pytest.raises(ValueError, match="qt must be a 2-D tensor"):
        g(dy, None, qt=torch.zeros(256, 10, dtype=u8))
    with pytest.raises(ValueError, match="GPU tensors only"):
        g(dy, dy, "relu")
    x, w, t = torch.zeros(5, 256, dtype=bf), torch.zeros(9, 256, dtype=bf), torch.zeros(5).long()
    with pytest.raises(ValueError, match="target must be torch.int64"):
        fp8bs.bf16_linear_xent(x, w, t.int())
    with pytest.raises(ValueError, match="target must be a contiguous vector"):
        fp8bs.bf16_linear_xent(x, w, t[:4])
    with pytest.raises(ValueError, match="w must be a 2-D tensor"):
        fp8bs.bf16_linear_xent(x, w[:, :128], t)
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        fp8bs.bf16_linear_xent(x.float(), w, t)
    with pytest.raises(ValueError, match="K = 200"):
        fp8bs.bf16_linear_xent(x[:, :200], w[:, :200], t)
    with pytest.raises(ValueError, match="at least one row"):
        fp8bs.bf16_linear_xent(x, w[:0], t)
    with pytest.raises(ValueError, match="dloss must be a contiguous vector"):
        fp8bs.bf16_linear_xent_backward(x, w, t, torch.zeros(5), torch.zeros(4))
    with pytest.raises(ValueError, match="dw must be a 2-D tensor"):
        fp8bs.bf16_linear_xent_backward(x, w, t, torch.zeros(5), torch.zeros(5), dw=w[:8])
    with pytest.raises(ValueError, match="GPU tensors only"):
        fp8bs.bf16_linear_xent(x, w, t)
