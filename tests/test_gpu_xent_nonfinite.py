"""The head's cross entropy where logits are NaN or infinite: what the formulas
give, also where such a logit stands alone in the last columns of the vocabulary
or among -inf, for every tile shape.  Finite results are held to the tolerance
derived in test_gpu_xent.py."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

# one row to 16 (narrow and wide tiles), 64, more (narrow, small), large tiles, and
# large tiles with their half and quarter ones; V = 1 more than whole blocks of
# columns, so that the last column is the only one of its block
SHAPES = [(4, 1), (4, 33), (4, 2049), (4, 40001), (40, 129), (40, 2049), (40, 20097), (70, 65),
          (70, 2049), (70, 20097), (300, 51073), (600, 30081), (613, 32001)]


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def make(M, V, K=128, seed=0):
    """x with ones in its first column, so that w's first column adds to every
    row's logits; every seventh row carries no loss."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, K, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    x[:, 0] = 1.0
    t = torch.randint(V, (M,), generator=g, device="cuda")
    t[::7] = -100
    return x, w, t


def check(fp8bs, x, w, t):
    """lse and loss against the formulas in float64, with NaN and infinities in
    the same places."""
    loss, lse = fp8bs.bf16_linear_xent(x, w, t)
    l = x.double() @ w.double().t()
    finite = torch.where(torch.isfinite(w), w, torch.zeros_like(w)).double()
    tol = 2 * x.shape[1] * U * (x.double().abs() @ finite.abs().t()).amax(dim=1) + 6e-5
    keep = t >= 0
    zero = torch.zeros(len(t), dtype=torch.float64, device="cuda")
    want = torch.where(keep, torch.logsumexp(l, dim=1), zero)
    at = torch.where(keep, l.gather(1, t.clamp_min(0)[:, None])[:, 0], zero)
    for got, ref, k in ((lse, want, 1), (loss, want - at, 2)):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        # a loss past FP32's range is infinite there
        ref = torch.where(torch.isinf(ref.float()), ref.float().double(), ref)
        ok = torch.isfinite(ref)
        assert torch.equal(got[~ok & ~torch.isnan(ref)], ref[~ok & ~torch.isnan(ref)])
        assert torch.all((got - ref).abs()[ok] <= (k * tol + 2 * U * want.abs())[ok])
    return lse, keep


@pytest.mark.parametrize("M,V", SHAPES)
def test_nan_in_the_last_column(fp8bs, M, V):
    x, w, t = make(M, V)
    w[V - 1, 0] = float("nan")
    lse, keep = check(fp8bs, x, w, t)
    assert torch.isnan(lse[keep]).all()


@pytest.mark.parametrize("M,V", SHAPES)
def test_nan_among_minus_infinities(fp8bs, M, V):
    x, w, t = make(M, V, seed=1)
    w[V // 2:, 0] = float("-inf")
    w[V // 2 + (V - V // 2) // 3, 0] = float("nan")
    lse, keep = check(fp8bs, x, w, t)
    assert torch.isnan(lse[keep]).all()


@pytest.mark.parametrize("M,V", SHAPES)
def test_all_minus_infinity(fp8bs, M, V):
    x, w, t = make(M, V, seed=2)
    w[:, 0] = float("-inf")
    lse, keep = check(fp8bs, x, w, t)
    assert torch.all(lse[keep] == float("-inf"))


@pytest.mark.parametrize("M,V", SHAPES)
def test_one_finite_column(fp8bs, M, V):
    x, w, t = make(M, V, seed=3)
    w[:V - 1, 0] = float("-inf")
    t[t >= 0] = V - 1
    lse, keep = check(fp8bs, x, w, t)
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("where", ["first", "last", "both"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_plus_infinity(fp8bs, M, V, where):
    """lse is +inf and so is the loss, but for a target whose own logit is."""
    x, w, t = make(M, V, seed=4)
    if where != "last":
        w[0, 0] = float("inf")
    if where != "first":
        w[V - 1, 0] = float("inf")
    lse, keep = check(fp8bs, x, w, t)
    assert torch.all(lse[keep] == float("inf"))


@pytest.mark.parametrize("top", [2.6e38, -2.6e38])
@pytest.mark.parametrize("M,V", SHAPES)
def test_logits_at_the_end_of_the_range(fp8bs, M, V, top):
    """Logits whose product with log2 e is past FP32's range.  w's first column
    alone is not zero, so logits are exact and the gradients are 0 or as many
    shares of -x and w as the formula gives."""
    x, w, t = make(M, V, seed=5)
    w.zero_()
    w[:, 0] = top
    w[:V // 2, 0] = -3e38
    lse, keep = check(fp8bs, x, w, t)
    d = torch.full((M,), 2.0 ** -20, device="cuda")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    # lse is the largest logit: log of at most V is less than its last bit
    P = (w[:, 0].double()[None, :] == lse.double()[:, None]).double() * keep[:, None]
    G = P.clone()
    rows = torch.nonzero(keep)[:, 0]
    G[rows, t[rows]] -= 1.0
    want = (G.t() @ (2.0 ** -20 * x.double()))
    # G is 0, 1 or -1: FP32 sums of exact products, one bf16 rounding
    tol = 2 * M * U * (G.abs().t() @ (2.0 ** -20 * x.double().abs()))
    assert torch.all((dw.double() - want).abs() <= tol + 2.0 ** -8 * want.abs())


@pytest.mark.parametrize("M,V,K", [(64, 200, 128), (200, 333, 256), (256, 512, 128),
                                   (5000, 300, 128)])
@pytest.mark.parametrize("which", ["all", "half", "one"])
def test_infinite_dloss(fp8bs, M, V, K, which):
    """An overflowed scale of the loss reaches dx of its rows and all of dw."""
    x, w, t = make(M, V, K, seed=6)
    _, lse = fp8bs.bf16_linear_xent(x, w, t)
    d = torch.full((M,), 0.5, device="cuda")
    hit = {"all": slice(None), "half": slice(M // 2, None), "one": slice(1, 2)}[which]
    d[hit] = float("inf")
    dx, dw = fp8bs.bf16_linear_xent_backward(x, w, t, lse, d)
    assert not torch.isfinite(dw).any()
    rows = torch.isinf(d) & (t >= 0)
    assert not torch.isfinite(dx[rows]).any()
    assert torch.isfinite(dx[~rows]).all()
