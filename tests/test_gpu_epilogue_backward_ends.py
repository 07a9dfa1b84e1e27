"""The epilogue's backward at its ends."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N", [(1, 128), (130, 384)])
def test_nan_pre_activation(fp8bs, M, N, act):
    """A NaN z is a NaN of dz: in its code of both forms and in dbias of its
    column, and nowhere else; infinities keep the slopes' limits."""
    g = torch.Generator(device="cuda").manual_seed(M)
    dy = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    dy[0, 9] = 1.0
    z[0, 9] = float("inf")
    z[0, 10] = float("-inf")
    ref = fp8bs.fp8_quant_epilogue_backward(dy, z, act)
    z[M - 1, 5], z[M // 2, N - 1] = float("nan"), float("nan")
    q, s, qt, st, db = fp8bs.fp8_quant_epilogue_backward(dy, z, act)
    hit = torch.isnan(z)
    nan = lambda c: (c & 0x7F) == 0x7F
    assert torch.equal(nan(q), hit)
    assert torch.equal(nan(qt)[:, :M], hit.t()) and not nan(qt)[:, M:].any()
    assert torch.equal(torch.isnan(db), hit.any(dim=0))
    assert torch.isfinite(ref[4]).all() and torch.isfinite(s).all() and torch.isfinite(st).all()
    rest = ~hit.any(dim=0)
    assert torch.equal(db[rest], ref[4][rest])


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("N", [128, 640])
def test_no_rows(fp8bs, N, act):
    """The bias gradient of an empty batch is zero, as the head's weight gradient."""
    dy = torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    z = dy if act != "none" else None
    db = torch.full((N + 3,), 7.0, device="cuda")
    q, s, qt, st, got = fp8bs.fp8_quant_epilogue_backward(dy, z, act, dbias=db)
    assert got is db and torch.all(db[:N] == 0) and torch.all(db[N:] == 7)
    assert q.shape == (0, N) and s.shape == (N // 128, 0) and qt.shape == (N, 0)
    assert st.shape == (0, N)
    # freed memory holds what was there: a fresh dbias is cleared too
    junk = torch.full((N,), 3.0, device="cuda")
    del junk
    assert torch.all(fp8bs.fp8_quant_epilogue_backward(dy, z, act)[4] == 0)
