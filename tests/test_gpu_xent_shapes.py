"""The cross entropy at sizes that take the large tiles, their half tiles, several
pieces and parts, against float64 on the GPU.  Tolerances as derived in
test_gpu_xent.py."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def make(M, V, K, seed, ignored):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, K, generator=g, device="cuda") * (1.5 / K ** 0.5)).to(torch.bfloat16)
    t = torch.randint(V, (M,), generator=g, device="cuda")
    t[torch.randperm(M, generator=g, device="cuda")[:int(M * ignored)]] = -100
    x[t == -100] = float("nan")
    return x, w, t


def logits(x, w, t):
    rows = torch.nonzero(t != -100)[:, 0]
    xs, ws = x[rows].double(), w.double()
    l = xs @ ws.t()
    err = 2 * x.shape[1] * U * (xs.abs() @ ws.abs().t()).amax(dim=1)
    return rows, xs, ws, l, err


# large tiles; with 300 and 100 rows over 200 tiles of w, half tiles; exact ends
@pytest.mark.parametrize("M,V,K,ignored", [
    (300, 51000, 128, 0.0), (100, 51000, 128, 0.0), (700, 51000, 256, 0.45), (513, 30001, 256, 0.0),
    (1100, 8193, 384, 0.1), (256, 65536, 128, 0.0), (2000, 5000, 2048, 0.3), (9000, 700, 128, 0.2),
])
def test_forward(fp8bs, M, V, K, ignored):
    x, w, t = make(M, V, K, M + V, ignored)
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    rows, _, _, l, err = logits(x, w, t)
    want_lse = torch.logsumexp(l, dim=1)
    want = want_lse - l[torch.arange(len(rows), device="cuda"), t[rows]]
    tol = err + 6e-5 + 2 * U * want_lse.abs()
    assert torch.all((lse[rows].double() - want_lse).abs() <= tol)
    assert torch.all((loss[rows].double() - want).abs() <= 2 * tol)
    rest = t == -100
    assert torch.all(loss[rest] == 0) and torch.all(lse[rest] == 0)


@pytest.mark.parametrize("M,V,K,ignored,weights", [
    (300, 12545, 1024, 0.0, "mean"), (700, 12500, 1152, 0.4, "signed"), (64, 25100, 640, 0.0, "mean"),
    (1000, 51000, 256, 0.0, "mean"), (2500, 60001, 256, 0.1, "signed"), (129, 40000, 384, 0.0, "mean"),
    (9000, 700, 256, 0.2, "signed"), (8192, 513, 1536, 0.0, "mean"),
])
def test_backward(fp8bs, M, V, K, ignored, weights):
    x, w, t = make(M, V, K, M + V, ignored)
    rows, xs, ws, l, err = logits(x, w, t)
    lse = torch.zeros(M, device="cuda")
    lse[rows] = torch.logsumexp(l, dim=1).float()
    d = torch.full((M,), 1.0 / M, device="cuda") if weights == "mean" else \
        torch.randn(M, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
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
