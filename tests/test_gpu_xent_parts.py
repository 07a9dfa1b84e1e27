"""Gradients of the cross entropy where the vocabulary is taken in more than one
piece and dx in many parts, against float64 on the GPU: every row's dx, and dw
as a whole.  Tolerances as derived in test_gpu_xent.py."""

import pytest
import torch

from tests.test_gpu_xent_shapes import U, fp8bs, logits, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,V,K,ignored", [
    # two pieces (9216 padded rows of half of 60001 columns, at most 2^30 bytes)
    (9000, 60001, 128, 0.05),
    # one tile of dx in 32 parts, of large and of small tiles
    (250, 70001, 256, 0.0), (1000, 70001, 256, 0.3), (60, 70001, 128, 0.0),
    # parts that do not divide the contraction; dw tiles fewer than workgroups
    (1030, 6100, 1024, 0.0), (1000, 4100, 1152, 0.5), (2050, 20003, 512, 0.1),
    # two rounds of large tiles for the logits but for the last rows
    (613, 32003, 128, 0.0), (1531, 32003, 256, 0.6),
])
def test_parts(fp8bs, M, V, K, ignored):  # noqa: F811
    x, w, t = make(M, V, K, M + V + K, ignored)
    rows, xs, ws, l, err = logits(x, w, t)
    lse = torch.zeros(M, device="cuda")
    lse[rows] = torch.logsumexp(l, dim=1).float()
    d = torch.randn(M, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    G = torch.exp(l - lse[rows].double()[:, None])
    E = 4 * G * (err + 6e-5)[:, None]
    G[torch.arange(len(rows), device="cuda"), t[rows]] -= 1.0
    E += G.abs() * (2.0 ** -8 + 2 * max(M, V) * U)
    dr = d[rows].double()[:, None]
    want = (dr * G) @ ws
    tol = (dr.abs() * E) @ ws.abs()
    assert torch.all((dx[rows].double() - want).abs() <= tol + 2.0 ** -8 * want.abs())
    assert torch.all(dx[t == -100] == 0)
    E = dr.abs() * (E + 2.0 ** -8 * G.abs())
    want = (dr * G).t() @ xs
    tol = E.t() @ xs.abs()
    assert torch.all((dw.double() - want).abs() <= tol + 2.0 ** -8 * want.abs())
    # the same call again gives the same bits
    again = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


# the last rows' tiles cut in four (two rows of large tiles, 1, 101 and 128 rows
# more), an uncut last tile (129), and a vocabulary that ends inside each
@pytest.mark.parametrize("M", [513, 613, 640, 641])
@pytest.mark.parametrize("V", [32003, 32640, 30721])
def test_forward_last_rows(fp8bs, M, V):  # noqa: F811
    x, w, t = make(M, V, 128, M + V, 0.0)
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    rows, _, _, l, err = logits(x, w, t)
    want_lse = torch.logsumexp(l, dim=1)
    want = want_lse - l[torch.arange(M, device="cuda"), t]
    tol = err + 6e-5 + 2 * U * want_lse.abs()
    assert torch.all((lse.double() - want_lse).abs() <= tol)
    assert torch.all((loss.double() - want).abs() <= 2 * tol)


# heads whose tiles are the narrow ones, ending inside the first and the second
# half of a 128-column step of dx; one row to several tiles of them
@pytest.mark.parametrize("M,K", [(1, 256), (16, 128), (17, 640), (55, 384), (130, 512)])
@pytest.mark.parametrize("V", [1, 63, 65, 700, 1090, 1615, 3969])
def test_narrow_tiles(fp8bs, M, V, K):  # noqa: F811
    x, w, t = make(M, V, K, M + V + K, 0.0)
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    rows, xs, ws, l, err = logits(x, w, t)
    want_lse = torch.logsumexp(l, dim=1)
    want = want_lse - l[torch.arange(M, device="cuda"), t]
    tol = err + 6e-5 + 2 * U * want_lse.abs()
    assert torch.all((lse.double() - want_lse).abs() <= tol)
    assert torch.all((loss.double() - want).abs() <= 2 * tol)
    d = torch.randn(M, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    # the workspace holds NaN: nothing is read that was not written
    ws_bytes = fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, M, V, K)
    space = torch.full(((ws_bytes + 3) // 4,), float("nan"), device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d, workspace=space)
    G = torch.exp(l - lse.double()[:, None])
    E = 4 * G * (err + 6e-5)[:, None]
    G[torch.arange(M, device="cuda"), t] -= 1.0
    E += G.abs() * (2.0 ** -8 + 2 * max(M, V) * U)
    dr = d.double()[:, None]
    want = (dr * G) @ ws
    assert torch.all((dx.double() - want).abs() <=
                     (dr.abs() * E) @ ws.abs() + 2.0 ** -8 * want.abs())
    E = dr.abs() * (E + 2.0 ** -8 * G.abs())
    want = (dr * G).t() @ xs
    assert torch.all((dw.double() - want).abs() <= E.t() @ xs.abs() + 2.0 ** -8 * want.abs())
