"""Gradients of the cross entropy over three and more pieces of the vocabulary, the
last of them as short as one column, against float64 on the GPU.  The plan is
recomputed here and held to the library's workspace, so that a change of its
constants shows.  Tolerances as derived in test_gpu_xent.py."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
PIECE, PARTS, MOST_PARTS, TILE, PAD = 1 << 30, 256 << 20, 32, 256, 128


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def cdiv(a, b):
    return -(-a // b)


def plan(M, V, K):
    """(pieces, columns of a piece, columns of the last, workspace bytes)"""
    Mt = cdiv(M, TILE) * TILE
    most = max(TILE, PIECE // (2 * Mt) // TILE * TILE)
    ld = cdiv(cdiv(V, cdiv(V, most)), TILE) * TILE
    pieces = cdiv(V, ld)
    dx_rows = max(M, min(MOST_PARTS * M, PARTS // (4 * K)))
    r = lambda n: cdiv(n, 256) * 256
    size = 256 + 5 * r(4 * M) + 2 * r(2 * cdiv(M, PAD) * PAD * K) + r(2 * Mt * ld) + r(4 * dx_rows * K)
    return pieces, ld, V - (pieces - 1) * ld, size


@pytest.mark.parametrize("M,valid,V,K,weights,pieces,last", [
    # every row counts and is used in place
    (12032, 12032, 100001, 128, "mean", 3, 32929),
    # packed rows, dloss by row
    (65536, 3200, 20001, 128, "signed", 3, 6177),
    # a last piece of one column, shorter than dx's parts are many: small tiles
    (1 << 20, 300, 1537, 128, "signed", 4, 1),
    # the same, large tiles
    (400000, 300, 5121, 5120, "mean", 5, 1),
])
def test_pieces(fp8bs, M, valid, V, K, weights, pieces, last):
    n, ld, rest, size = plan(M, V, K)
    assert (n, rest) == (pieces, last)
    assert fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, M, V, K) == size
    g = torch.Generator(device="cuda").manual_seed(M + V)
    rows = torch.randperm(M, generator=g, device="cuda")[:valid].sort().values
    x = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[rows] = torch.randn(valid, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, K, generator=g, device="cuda") * (1.5 / K ** 0.5)).to(torch.bfloat16)
    t = torch.full((M,), -100, device="cuda")
    t[rows] = torch.randint(V, (valid,), generator=g, device="cuda")
    t[rows[::5]] = V - 1  # the last piece's
    d = torch.full((M,), 1.0 / valid, device="cuda") if weights == "mean" else \
        torch.randn(M, generator=g, device="cuda")
    ws = w.double()
    lse = torch.zeros(M, device="cuda")
    for r in rows.split(2048):
        lse[r] = torch.logsumexp(x[r].double() @ ws.t(), dim=1).float()
    # the workspace holds NaN: nothing is read that was not written
    space = torch.full((size // 4,), float("nan"), device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d, workspace=space)
    del space
    want_dw = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    tol_dw = torch.zeros_like(want_dw)
    for r in rows.split(2048):
        xs = x[r].double()
        err = 2 * K * U * (xs.abs() @ ws.abs().t()).amax(dim=1)
        G = torch.exp(xs @ ws.t() - lse[r].double()[:, None])
        E = 4 * G * (err + 6e-5)[:, None]
        G[torch.arange(len(r), device="cuda"), t[r]] -= 1.0
        E += G.abs() * (2.0 ** -8 + 2 * max(valid, V) * U)
        dr = d[r].double()[:, None]
        want = (dr * G) @ ws
        tol = (dr.abs() * E) @ ws.abs()
        assert torch.all((dx[r].double() - want).abs() <= tol + 2.0 ** -8 * want.abs())
        want_dw += (dr * G).t() @ xs
        tol_dw += (dr.abs() * (E + 2.0 ** -8 * G.abs())).t() @ xs.abs()
    assert torch.all((dw.double() - want_dw).abs() <= tol_dw + 2.0 ** -8 * want_dw.abs())
    dx[rows] = 0
    assert torch.all(dx == 0)
