"""The norm and its backward on the GPU against the float64 oracle.

Tolerances.  A row's sum of squares is taken in at most 32 multiply-adds per
thread, 6 steps over a wave and 16 over waves, each off by 2^-24 of the sum;
with the mean's division and eps that is below 58 * 2^-24, half of it after the
root, and 2 roundings of root and division: rstd is within 31 * 2^-24 < 2^-19
of its value.  y has two more roundings: below 2^-18 (REL).  bf16 outputs add
2^-8 of their value; an E4M3 value 2^-4 of it or, below the normal range, half a
step of 2^-9, times the scale.

Backward: c = mean(u n) is off by at most (58 + 3) * 2^-24 < 2^-18 of
mean|u n|; u, n and their products carry a few 2^-24 each.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import rmsnorm
from fp8_block_scaled_05_amd import synth
from tests import _gpu_util as gu

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18
EPS = 1e-6


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def inputs(M, K, case):
    x = synth.act(M, K, case=case, tensor=0, device="cuda", outlier_mult=20.0)
    r = synth.act(M, K, case=case, tensor=1, device="cuda", outlier_mult=20.0)
    g = torch.Generator(device="cuda").manual_seed(case)
    return x, r, 1 + 0.2 * torch.randn(K, generator=g, device="cuda")


def added(x, r):
    return x if r is None else (x.float() + r.float()).to(torch.bfloat16)


def check_codes(q, s, y):
    """Codes [R][C] with scales [C/128][R] against values y off by REL."""
    R, C = y.shape
    t = np.abs(y).reshape(R, C // 128, 128)
    s = gu.host_f64(s).T[:R]
    top = np.maximum(t.max(axis=2), 2.0 ** -64)
    assert np.all(np.abs(s * 448 - top) <= 2 * REL * top)
    got = oracle.decode(gu.host(q)).astype(np.float64).reshape(t.shape) * s[:, :, None]
    lim = t * (2.0 ** -4 + 2 * REL) + 2.0 ** -10 * s[:, :, None]
    assert np.all(np.abs(got - y.reshape(t.shape)) <= lim * (1 + 2.0 ** -16))


def check_forward(q, s, h, y, rstd, want_h, g, eps=EPS):
    if h is not None:
        assert torch.equal(h.view(torch.int16), want_h.view(torch.int16))
    wy, wr = rmsnorm.forward(gu.host_f64(want_h), gu.host_f64(g), eps)
    if rstd is not None:
        assert np.all(np.abs(gu.host_f64(rstd) - wr) <= 2.0 ** -19 * wr)
    if y is not None:
        assert np.all(np.abs(gu.host_f64(y) - wy) <= (2.0 ** -8 + 2 * REL) * np.abs(wy))
    if q is not None:
        check_codes(q, s, wy)


# one wave to a row, several, sixteen; a last workgroup with rows to spare; the
# ends of the choice of threads and loads per thread
SHAPES = [(1, 128), (1, 7168), (3, 256), (5, 512), (333, 2048), (64, 640), (9, 4096), (7, 4224),
          (50, 7168), (2, 8192), (3, 8320), (2, 16384), (3, 16512), (2, 32768), (1025, 384)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(fp8bs, M, K, residual):
    x, r, g = inputs(M, K, 1000)
    r = r if residual else None
    h = torch.full((M, K), 9.0, dtype=torch.bfloat16, device="cuda")
    y, rstd = torch.empty_like(h), torch.empty(M, device="cuda")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, EPS, residual=r, h=h, y=y, rstd=rstd)
    check_forward(q, s, h, y, rstd, added(x, r), g)
    # the outputs that are left out change nothing
    q2, s2 = fp8bs.fp8_quant_rmsnorm(x, g, EPS, residual=r)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    y2 = fp8bs.bf16_rmsnorm(x, g, EPS, residual=r)
    assert torch.equal(y, y2)
    h3, rstd3 = torch.empty_like(h), torch.empty_like(rstd)
    y3 = fp8bs.bf16_rmsnorm(x, g, EPS, residual=r, h=h3, rstd=rstd3)
    assert torch.equal(y, y3) and torch.equal(h, h3) and torch.equal(rstd, rstd3)


@pytest.mark.parametrize("M,K", [(40, 128), (17, 2048), (5, 7168)])
def test_exact_where_rstd_is_a_power_of_two(fp8bs, M, K):
    """Rows of 2^j (three of +-1.5, five of +-0.5 in eight): mean h^2 = 4^j, so y
    is a bf16 value and the codes are the quantizer's, bit for bit."""
    rng = np.random.default_rng(3)
    v = np.tile(np.array([1.5] * 3 + [0.5] * 5), K // 8)
    v = np.stack([rng.permutation(v) for _ in range(M)]) * rng.choice([-1, 1], size=(M, K))
    scale = 2.0 ** rng.integers(-20, 20, size=(M, 1))
    x = torch.tensor(v * scale, device="cuda").to(torch.bfloat16)
    g = torch.tensor(rng.choice([-2.0, 1.0, 0.5], size=K), dtype=torch.float32, device="cuda")
    y = torch.empty_like(x)
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, 2.0 ** -100, y=y)
    want = (torch.tensor(v, device="cuda") * g.double()).to(torch.bfloat16)
    assert torch.equal(y, want)
    q2, s2 = fp8bs.fp8_quant_act_1x128(want)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("K", [256, 2048, 7168])
def test_zero_tiny_and_huge_rows(fp8bs, K):
    """A zero row; rows whose squares would leave FP32 on either side."""
    x, _, g = inputs(6, K, 1001)
    x = x.float()
    x[0] = 0
    x[1] *= 1e-30
    x[2] = x[2].sign() * 2e38 * torch.rand_like(x[2])
    x[3] = 0
    x[3, 5] = 3e38
    x[4] *= 1e25
    x = x.to(torch.bfloat16)
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, EPS, y=y, rstd=rstd)
    wy, wr = rmsnorm.forward(gu.host_f64(x), gu.host_f64(g), EPS)
    # rstd below the normal range has steps of 2^-149
    err = np.abs(gu.host_f64(rstd) - wr)
    assert np.all(err <= 2.0 ** -19 * wr + 2.0 ** -149)
    rel = 2 * REL + 2.0 ** -149 / wr[:, None]
    # y below the normal range of FP32 and bf16: a step of bf16 there
    assert np.all(np.abs(gu.host_f64(y) - wy) <= (2.0 ** -8 + rel) * np.abs(wy) + 2.0 ** -133)
    assert np.all(gu.host(q[0]) & 0x7F == 0)
    for m in (2, 4, 5):
        check_codes(q[m:m + 1], s[:, m:m + 1], wy[m:m + 1])


@pytest.mark.parametrize("eps", [1e20, 1e36, 3.4e38])
def test_large_eps(fp8bs, eps):
    """An eps that counts beside a mean of squares past FP32's range, and one that
    leaves it together with the mean."""
    eps = float(np.float32(eps))
    x, _, g = inputs(5, 512, 1005)
    x = (x.float() * torch.tensor([1.0, 1e10, 1e18, 1e19, 1e20], device="cuda")[:, None])
    x = x.to(torch.bfloat16)
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, eps, y=y, rstd=rstd)
    wy, wr = rmsnorm.forward(gu.host_f64(x), gu.host_f64(g), eps)
    assert np.all(np.abs(gu.host_f64(rstd) - wr) <= 2.0 ** -19 * wr)
    assert np.all(np.abs(gu.host_f64(y) - wy) <= (2.0 ** -8 + 2 * REL) * np.abs(wy))


@pytest.mark.parametrize("M,K", [(1, 7168), (70, 512), (33, 2048)])
def test_strides_and_untouched_memory(fp8bs, M, K):
    x, r, g = inputs(M, K + 48, 1002)
    x, r, g = x[:, :K], r[:, 16:K + 16], g[:K].clone()
    bufs = [torch.full((M + 2, K + 32), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "hy"]
    h, y = (b[1:M + 1, 16:K + 16] for b in bufs)
    q = torch.full((M + 1, K + 16), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((K // 128 + 1, M + 3), 7.0, device="cuda")
    rstd = torch.full((M + 1,), 7.0, device="cuda")
    fp8bs.fp8_quant_rmsnorm(x, g, EPS, residual=r, h=h, y=y, rstd=rstd, q=q, s=s)
    check_forward(q[:M, :K], s[:K // 128, :M], h, y, rstd[:M], added(x, r), g)
    for b, v in zip(bufs, (h, y)):
        v.fill_(9.0)
        assert torch.all(b == 9.0)
    assert torch.all(q[M:] == 7) and torch.all(q[:, K:] == 7)
    assert torch.all(s[K // 128:] == 7) and torch.all(s[:, M:] == 7) and rstd[M] == 7


@pytest.mark.parametrize("M,K", [(3, 256), (200, 7168)])
def test_in_place(fp8bs, M, K):
    x, r, g = inputs(M, K, 1003)
    want = fp8bs.fp8_quant_rmsnorm(x, g, EPS, residual=r)
    h = added(x, r)
    for into in (0, 1):
        a = [x.clone(), r.clone()]
        got = fp8bs.fp8_quant_rmsnorm(a[0], g, EPS, residual=a[1], h=a[into])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(a[into], h) and torch.equal(a[1 - into], (x, r)[1 - into])


def test_one_token_views(fp8bs):
    """A single row of any torch stride (a broadcast row, a column's view)."""
    x, r, g = inputs(4, 256, 1004)
    want = fp8bs.fp8_quant_rmsnorm(x[2:3].clone(), g, residual=r[2:3].clone())
    got = fp8bs.fp8_quant_rmsnorm(x[2:3], g, residual=r[2].expand(1, 256))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    seq = x.view(1, 4, 256)[:, 2]
    got = fp8bs.fp8_quant_rmsnorm(seq, g, residual=r[2:3])
    assert torch.equal(got[0], want[0])


def test_no_rows(fp8bs):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, device="cuda")
    q, s = fp8bs.fp8_quant_rmsnorm(x, g, residual=x)
    assert q.shape == (0, 256) and s.shape == (2, 0)
    assert fp8bs.bf16_rmsnorm(x, g).shape == (0, 256)
    dw = torch.full((256,), 7.0, device="cuda")
    dx, dw = fp8bs.bf16_rmsnorm_backward(x, x, torch.empty(0, device="cuda"), g, dweight=dw)
    assert dx.shape == (0, 256) and torch.all(dw == 0)


def check_backward(dx, dw, dy, h, rstd, g, dh):
    M = dy.shape[0]
    hy, hh, hr, hg = (gu.host_f64(t) for t in (dy, h, rstd, g))
    want, want_dg = rmsnorm.backward(hy, hh, hr, hg)
    n, u = hh * hr[:, None], hy * hg
    tol = hr[:, None] * (2.0 ** -22 * np.abs(u) +
                         np.abs(n) * REL * np.abs(u * n).mean(axis=1, keepdims=True))
    if dh is not None:
        want = want + gu.host_f64(dh)
    got = gu.host_f64(dx)
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 1.01 * tol)
    # a column's sum: M terms with 2 roundings each, added in at most M steps,
    # then over at most 64 + 8 sums
    lim = (M + 80) * 2.0 ** -24 * np.abs(hy * n).sum(axis=0)
    assert np.all(np.abs(gu.host_f64(dw) - want_dg) <= lim)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("M,K", SHAPES + [(1531, 512), (2000, 128), (700, 4096), (1, 16512)])
def test_backward(fp8bs, M, K, with_dh):
    x, dh, g = inputs(M, K, 1005)
    dy = (1e-2 * synth.act(M, K, case=1005, tensor=2, device="cuda").float()).to(torch.bfloat16)
    dh = dh if with_dh else None
    rstd = torch.empty(M, device="cuda")
    fp8bs.bf16_rmsnorm(x, g, EPS, rstd=rstd)
    dx, dw = fp8bs.bf16_rmsnorm_backward(dy, x, rstd, g, dh=dh)
    check_backward(dx, dw, dy, x, rstd, g, dh)
    # the same again, from a workspace of NaN and without timing's influence
    ws = torch.full((fp8bs.workspace_bytes(fp8bs.OP_RMSNORM_BACKWARD, M, 0, K) // 4,), float("nan"),
                    device="cuda")
    dx2, dw2 = fp8bs.bf16_rmsnorm_backward(dy, x, rstd, g, dh=dh, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("M,K", [(5, 256), (300, 2048)])
def test_backward_in_place_and_strides(fp8bs, M, K):
    x, dh, g = inputs(M, K, 1006)
    dy = synth.act(M, K, case=1006, tensor=2, device="cuda")
    rstd = torch.empty(M, device="cuda")
    fp8bs.bf16_rmsnorm(x, g, EPS, rstd=rstd)
    want, wdw = fp8bs.bf16_rmsnorm_backward(dy, x, rstd, g, dh=dh)
    for k in ("dy", "dh"):
        t = {"dy": dy.clone(), "dh": dh.clone()}
        dx, dw = fp8bs.bf16_rmsnorm_backward(t["dy"], x, rstd, g, dh=t["dh"], dx=t[k])
        assert dx is t[k] and torch.equal(dx, want) and torch.equal(dw, wdw)
    wide = [torch.full((M + 1, K + 32), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    v = [w[:M, 16:K + 16] for w in wide]
    for a, b in zip(v, (dy, x, dh)):
        a.copy_(b)
    dwide = torch.full((K + 4,), 7.0, device="cuda")
    fp8bs.bf16_rmsnorm_backward(v[0], v[1], rstd, g, dh=v[2], dx=v[3], dweight=dwide[:K])
    assert torch.equal(v[3], want) and torch.equal(dwide[:K], wdw) and torch.all(dwide[K:] == 7)
    v[3].fill_(9.0)
    assert torch.all(wide[3] == 9.0)


def test_gradient_against_differences(fp8bs):
    """dx and dg along random directions against central differences of the
    float64 norm: both are sums of bf16-rounded or FP32 products, so the bound is
    the rounding of dx, 2^-8 of its values along the direction."""
    M, K = 37, 384
    x, _, g = inputs(M, K, 1007)
    dy = synth.act(M, K, case=1007, tensor=2, device="cuda")
    rstd = torch.empty(M, device="cuda")
    fp8bs.bf16_rmsnorm(x, g, EPS, rstd=rstd)
    dx, dg = fp8bs.bf16_rmsnorm_backward(dy, x, rstd, g)
    X, G, Y = gu.host_f64(x), gu.host_f64(g), gu.host_f64(dy)
    f = lambda X, G: (rmsnorm.forward(X, G, EPS)[0] * Y).sum()
    rng = np.random.default_rng(7)
    u, v, e = rng.normal(size=X.shape), rng.normal(size=G.shape), 1e-5
    # the difference's own error: third derivatives times e^2, and f's rounding / e
    slack = 1e-6 * np.abs(Y).sum()
    ax, ag = gu.host_f64(dx), gu.host_f64(dg)
    d = (f(X + e * u, G) - f(X - e * u, G)) / (2 * e)
    assert abs(d - (ax * u).sum()) <= 2.0 ** -8 * np.abs(ax * u).sum() + slack
    d = (f(X, G + e * v) - f(X, G - e * v)) / (2 * e)
    assert abs(d - (ag * v).sum()) <= 2.0 ** -16 * np.abs(ag * v).sum() + slack


def test_nan_rows_stay_alone(fp8bs):
    """A NaN element makes its row's bf16 outputs and gradients NaN, no other
    row's."""
    x, _, g = inputs(9, 512, 1008)
    clean = fp8bs.bf16_rmsnorm(x, g)
    bad = x.clone()
    bad[4, 100] = float("nan")
    rstd = torch.empty(9, device="cuda")
    y = fp8bs.bf16_rmsnorm(bad, g, rstd=rstd)
    keep = [m for m in range(9) if m != 4]
    assert torch.equal(y[keep], clean[keep]) and torch.all(y[4].isnan())
    dx, dw = fp8bs.bf16_rmsnorm_backward(x, bad, rstd, g)
    assert torch.all(dx[4].isnan()) and torch.all(dx[keep].isfinite())
    assert torch.all(dw.isnan())


def test_graph_and_streams(fp8bs):
    """Captured and replayed between eager calls, on its own stream; two calls at
    once with workspaces of their own."""
    M, K = 300, 1024
    x, r, g = inputs(M, K, 1009)
    dy = synth.act(M, K, case=1009, tensor=2, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, y, dx = torch.empty(M, K, **bf), torch.empty(M, K, **bf), torch.empty(M, K, **bf)
    rstd, dw = torch.empty(M, device="cuda"), torch.empty(K, device="cuda")
    q, s = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(8, M, device="cuda")
    ws = torch.empty(fp8bs.workspace_bytes(fp8bs.OP_RMSNORM_BACKWARD, M, 0, K), dtype=torch.uint8,
                     device="cuda")

    def step():
        fp8bs.fp8_quant_rmsnorm(x, g, EPS, residual=r, h=h, y=y, rstd=rstd, q=q, s=s)
        fp8bs.bf16_rmsnorm_backward(dy, h, rstd, g, dx=dx, dweight=dw, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        x.copy_(synth.act(M, K, case=1010 + turn, device="cuda"))
        for t in (h, y, dx, rstd, dw, s):
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, s, h, y, rstd, dx, dw)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, s, h, y, rstd, dx, dw)))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for st in (a, b, a, b):
        with torch.cuda.stream(st):
            outs.append(fp8bs.bf16_rmsnorm_backward(dy, h, rstd, g))
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], dx) and torch.equal(o[1], dw) for o in outs)
