"""The head's cross entropy and its gradients on the GPU against the float64
oracle on the same bf16 inputs.

Tolerances, derived from the arithmetic (u = 2^-24, products of bf16 values
are exact in FP32):
- a logit is an FP32 sum of K products, each step off by at most 2 u of the
  running sum (truncation allowed): |dl| <= 2 K u B, B = sum_k |x w|;
- lse moves by at most the largest logit error; its own sum of at most V
  terms, the exponentials (argument rounded to 2^-23 of |l| log2 e, and the
  exp itself) and the logarithm add less than 2^-19 (1 + |l - max|) over the
  terms that count (below 2^-19 * 30 = 6e-5);
- G is off by P (e^(2 d) - 1) <= 4 P d, d the logit error plus 6e-5 (and the
  given lse's own), and by 2^-9 |G| from bf16; the sums over v and m are FP32
  (2 n u of the sum of magnitudes); dw's operand x dloss / c is off by 2^-9
  more where dloss is not one value; bf16 outputs are off by 2^-9 of their
  value.  2^-8 stands for each 2^-9, which covers the products of errors.
"""

import numpy as np
import pytest
import torch

from oracle import xent as oracle
from tests import _gpu_util as gu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def make(M, V, K, seed=0, ignored=0.0, std=1.5, pad=0):
    """bf16 x [M][K], w [V][K] (row strides K + pad), targets, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K + pad, generator=g).to(torch.bfloat16).cuda()[:, :K]
    w = (torch.randn(V, K + pad, generator=g) * (std / K ** 0.5)).to(torch.bfloat16).cuda()[:, :K]
    t = torch.randint(V, (M,), generator=g)
    t[torch.randperm(M, generator=g)[:int(M * ignored)]] = -100
    return x, w, t.cuda()


def logit_error(x, w):
    """Largest error of each row's logits."""
    return 2 * x.shape[1] * U * (np.abs(x) @ np.abs(w).T).max(axis=1)


def check_forward(fp8bs, x, w, t, **kw):
    loss, lse = fp8bs.bf16_linear_xent(x, w, t, **kw)
    xs, ws, ts = gu.host_f64(x), gu.host_f64(w), gu.host(t)
    want, want_lse = oracle.linear_xent(xs, ws, ts, kw.get("ignore_index", -100))
    ok = oracle.valid_rows(ts, ws.shape[0], kw.get("ignore_index", -100))
    tol = np.where(ok, logit_error(np.where(ok[:, None], xs, 0.0), ws) + 6e-5, 0.0)
    loss, lse = gu.host_f64(loss)[:len(ok)], gu.host_f64(lse)[:len(ok)]
    assert np.all(np.abs(lse - want_lse) <= tol + 2 * U * np.abs(want_lse))
    assert np.all(np.abs(loss - want) <= 2 * tol + 2 * U * np.abs(want_lse))
    return want_lse


def check_backward(fp8bs, x, w, t, lse, dloss, **kw):
    """lse, dloss: float64 host arrays; the GPU gets them rounded to FP32."""
    l32, d32 = gu.f32(lse), gu.f32(dloss)
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, l32, d32, **kw)
    xs, ws, ts = gu.host_f64(x), gu.host_f64(w), gu.host(t)
    d = gu.host_f64(d32)
    rows = np.nonzero(oracle.valid_rows(ts, ws.shape[0]))[0]
    G, _ = oracle.softmax_minus_onehot(xs, ws, ts, gu.host_f64(l32))
    want_dx, want_dw = oracle.linear_xent_backward(xs, ws, ts, gu.host_f64(l32), d)
    P = np.abs(G)
    P[np.arange(rows.size), ts[rows]] = 1.0
    err = 2.0 ** -8 * np.abs(G) + 4 * P * (logit_error(xs[rows], ws) + 6e-5)[:, None]
    n = max(xs.shape[0], ws.shape[0])
    err += 2 * n * U * np.abs(G)
    tx = np.zeros(want_dx.shape)
    tx[rows] = np.abs(d[rows])[:, None] * (err @ np.abs(ws))
    tw = (np.abs(d[rows])[:, None] * (err + 2.0 ** -8 * np.abs(G))).T @ np.abs(xs[rows])
    got_dx, got_dw = gu.host_f64(dx), gu.host_f64(dw)
    assert np.all(np.isfinite(got_dx)) and np.all(np.isfinite(got_dw))
    assert np.all(np.abs(got_dx - want_dx) <= tx + 2.0 ** -8 * np.abs(want_dx))
    assert np.all(np.abs(got_dw - want_dw) <= tw + 2.0 ** -8 * np.abs(want_dw))
    return dx, dw


@pytest.mark.parametrize("M,V,K", [
    (1, 1, 128), (1, 1003, 256), (2, 129, 128), (17, 4099, 512), (33, 65, 128), (64, 2050, 384),
    (65, 1, 128), (65, 257, 128), (130, 1003, 512), (255, 769, 256), (257, 256, 640),
    (600, 3001, 256),
])
def test_forward(fp8bs, M, V, K):
    check_forward(fp8bs, *make(M, V, K, seed=M + V))


@pytest.mark.parametrize("M", [5, 64, 65, 300])
@pytest.mark.parametrize("ignored", [0.3, 1.0])
def test_forward_with_ignored_rows(fp8bs, M, ignored):
    x, w, t = make(M, 517, 256, seed=M, ignored=ignored)
    # what a row without a loss holds reaches nothing
    x[t == -100] = float("nan")
    check_forward(fp8bs, x, w, t)


def test_forward_targets_outside_the_vocabulary(fp8bs):
    for M in (6, 100):
        x, w, t = make(M, 300, 128, seed=2)
        t[0], t[3], t[5] = -1, 300, 1 << 40
        check_forward(fp8bs, x, w, t)
        # another ignore_index: -100 is then only a target out of range
        t[1] = 7
        check_forward(fp8bs, x, w, t, ignore_index=7)


@pytest.mark.parametrize("M", [3, 200])
def test_forward_strides_and_outputs(fp8bs, M):
    x, w, t = make(M, 421, 256, seed=4, pad=48)
    loss = torch.full((M + 3,), -5.0, device="cuda")
    lse = torch.full((M + 1,), -5.0, device="cuda")
    check_forward(fp8bs, x, w, t, loss=loss, lse=lse)
    assert torch.all(loss[M:] == -5.0) and torch.all(lse[M:] == -5.0)


@pytest.mark.parametrize("M", [4, 70])
def test_forward_large_and_infinite_logits(fp8bs, M):
    """Logits of thousands; a vocabulary row that makes one logit -inf (and
    whole blocks of them); and a row whose logits are all -inf or hold NaN,
    which gives what the formula gives."""
    x, w, t = make(M, 600, 128, seed=6, std=500.0)
    check_forward(fp8bs, x, w, t)
    x, w, t = make(M, 600, 128, seed=7)
    x[:, 0] = 1.0
    w[130:599, 0] = float("-inf")
    t[:] = 3
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    keep = torch.cat([w[:130], w[599:]])
    ref, ref_lse = fp8bs.bf16_linear_xent(x, keep, t)
    assert torch.equal(loss, ref) or torch.allclose(loss, ref, rtol=0, atol=6e-5)
    assert torch.allclose(lse, ref_lse, rtol=0, atol=6e-5)
    x[1] = float("nan")
    loss, lse = fp8bs.bf16_linear_xent(x, keep, t)
    assert torch.isnan(loss[1]) and torch.isnan(lse[1])
    assert torch.isfinite(torch.cat([loss[:1], loss[2:]])).all()


@pytest.mark.parametrize("M,V,K", [
    (1, 1, 128), (1, 1003, 256), (3, 300, 128), (64, 517, 256), (65, 257, 128), (130, 1003, 512),
    (256, 512, 256), (300, 2049, 384),
])
def test_backward(fp8bs, M, V, K):
    x, w, t = make(M, V, K, seed=M + V + 1)
    lse = oracle.linear_xent(gu.host_f64(x), gu.host_f64(w), gu.host(t))[1]
    check_backward(fp8bs, x, w, t, lse, np.full(M, 1.0 / M))


@pytest.mark.parametrize("M,ignored,weights", [
    (200, 0.4, "mean"), (200, 0.4, "signed"), (128, 0.0, "signed"), (64, 0.0, "negative"),
    (70, 1.0, "mean"), (90, 0.0, "zero"), (129, 0.9, "signed"),
])
def test_backward_rows_and_weights(fp8bs, M, ignored, weights):
    x, w, t = make(M, 700, 256, seed=M, ignored=ignored)
    xs, ws, ts = gu.host_f64(x), gu.host_f64(w), gu.host(t)
    lse = oracle.linear_xent(xs, ws, ts)[1]
    d = {"mean": np.full(M, 1 / 77.0), "negative": np.full(M, -0.3), "zero": np.zeros(M),
         "signed": np.random.default_rng(M).normal(size=M)}[weights]
    x[t == -100] = float("nan")  # reaches nothing
    # the oracle's rows without a loss hold NaN too, and are left out there
    dx, dw = check_backward(fp8bs, x, w, t, lse, d)
    assert torch.all(dx[t == -100] == 0)


def test_backward_pieces_and_splits(fp8bs):
    """Shapes whose plan has several pieces of the vocabulary, and one that
    splits dx's contraction, at a hidden size small enough for the oracle."""
    M, V, K = 2300, 70000, 128  # 2304 rows of G: 58112 columns per piece at most
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, K, generator=g, device="cuda") * 0.13).to(torch.bfloat16)
    t = torch.randint(V, (M,), generator=g, device="cuda")
    l = x.double() @ w.double().t()
    lse = torch.logsumexp(l, dim=1)
    d = torch.full((M,), 1.0 / M, device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse.float(), d)
    G = torch.exp(l - lse.float().double()[:, None])
    G[torch.arange(M, device="cuda"), t] -= 1.0
    E = G.abs() * (2.0 ** -8 + 2 * V * U) + 4 * torch.exp(l - lse[:, None]) * 1e-4
    for got, want, tol in ((dx, G @ w.double(), E @ w.double().abs()),
                           (dw, G.t() @ x.double(), E.t() @ x.double().abs())):
        want, tol = want / M, tol / M
        assert torch.all((got.double() - want).abs() <= tol + 2.0 ** -8 * want.abs())


def test_backward_no_rows(fp8bs):
    x, w, t = make(0, 300, 128)
    e = torch.empty(0, device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, e, e, dw=torch.ones_like(w))
    assert dx.shape == (0, 128) and torch.all(dw == 0)
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    assert loss.shape == lse.shape == (0,)


def test_backward_strides_and_outputs(fp8bs):
    M, V, K = 140, 333, 256
    x, w, t = make(M, V, K, seed=9, pad=16)
    lse = oracle.linear_xent(gu.host_f64(x), gu.host_f64(w), gu.host(t))[1]
    dx = torch.full((M, K + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((V + 2, K + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    check_backward(fp8bs, x, w, t, lse, np.full(M, 0.01), dx=dx[:, :K], dw=dw[:V, :K])
    assert torch.all(dx[:, K:] == 7) and torch.all(dw[:, K:] == 7) and torch.all(dw[V:] == 7)


def test_gradient_against_differences(fp8bs):
    """Directional derivatives of the GPU's own loss.  Steps of 2^-4 in x and
    w (exact in bf16 on these grids): the loss is off by 6e-5 + its logits'
    error per row, so a difference quotient is off by at most 2 * 1e-4 / 2^-3
    per unit of weight; the third derivative along the direction (every |logit
    step| <= 0.6) adds less than 0.6^3 / 6 per unit step cubed."""
    M, V, K = 96, 200, 128
    g = torch.Generator().manual_seed(11)
    grid = lambda *s: (torch.randint(-16, 17, s, generator=g) / 16).to(torch.bfloat16).cuda()
    x, w = grid(M, K), grid(V, K) / 8
    t = torch.randint(V, (M,), generator=g).cuda()
    d = torch.full((M,), 1.0 / M, device="cuda")
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    h = 2.0 ** -4
    ux = torch.where(torch.rand(M, K, generator=g).cuda() < 0.5, 1.0, -1.0)
    mean = lambda a, b: (fp8bs.bf16_linear_xent(a, b, t)[0].double() * d.double()).sum().item()
    up = mean((x.float() + h * ux).to(torch.bfloat16), w)
    down = mean((x.float() - h * ux).to(torch.bfloat16), w)
    assert abs((up - down) / (2 * h) - (dx.double() * ux.double()).sum().item()) < 0.02
    hw = 2.0 ** -7  # w's grid is 2^-7
    uw = torch.where(torch.rand(V, K, generator=g).cuda() < 0.5, 1.0, -1.0)
    up = mean(x, (w.float() + hw * uw).to(torch.bfloat16))
    down = mean(x, (w.float() - hw * uw).to(torch.bfloat16))
    assert abs((up - down) / (2 * hw) - (dw.double() * uw.double()).sum().item()) < 0.1


def test_repeated_calls_and_streams(fp8bs):
    """The same bits again, also on a stream of the caller's own and with a
    workspace that holds anything."""
    x, w, t = make(300, 1500, 256, seed=12, ignored=0.2)
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    d = torch.rand(300, device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n = fp8bs.workspace_bytes(fp8bs.OP_XENT, 300, 1500, 256)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        loss2, lse2 = fp8bs.bf16_linear_xent(x, w, t, workspace=ws)
        n = fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, 300, 1500, 256)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        dx2, dw2 = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d, workspace=ws)
    s.synchronize()
    for a, b in ((loss, loss2), (lse, lse2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)


def test_graph_capture(fp8bs):
    """Forward and backward in a captured graph, replayed on new inputs with
    eager work in between."""
    M, V, K = 100, 900, 128
    x, w, t = make(M, V, K, seed=13)
    d = torch.full((M,), 0.01, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    w1 = torch.empty(fp8bs.workspace_bytes(fp8bs.OP_XENT, M, V, K), dtype=torch.uint8,
                     device="cuda")
    w2 = torch.empty(fp8bs.workspace_bytes(fp8bs.OP_XENT_BACKWARD, M, V, K), dtype=torch.uint8,
                     device="cuda")

    def step():
        fp8bs.bf16_linear_xent(x, w, t, loss=loss, lse=lse, workspace=w1)
        fp8bs.bf16_linear_xent_backward(x, w, t, lse, d, dx=dx, dw=dw, workspace=w2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        xn, wn, tn = make(M, V, K, seed=20 + k, ignored=0.1 * k)
        x.copy_(xn), w.copy_(wn), t.copy_(tn)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in (loss, lse, dx, dw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (loss, lse, dx, dw)):
            assert torch.equal(a, b)
