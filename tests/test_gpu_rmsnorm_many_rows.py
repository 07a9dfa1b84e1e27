"""More rows than one grid holds: workgroups of a row each reach the 2^32 threads
that a launch may have (rows of 640 first, at 2^25 of them)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def test_rows_past_one_grid(fp8bs):
    """2^25 + 3 rows (64 GB of operands): every row is formed, the ends of the
    grids' shares as in a call of their own; h and rstd go along."""
    M, K = 2 ** 25 + 3, 640
    try:
        x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        x.view(torch.int16).random_(0x3F00, 0x4000)  # values of 0.5 to 2
        g = 1 + 0.2 * torch.randn(K, device="cuda")
        q = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
        s = torch.zeros(K // 128, M, device="cuda")
        rstd = torch.zeros(M, device="cuda")
        ends = [slice(0, 3)] + [slice(m - 3, m + 3) for m in (2 ** 23, 2 ** 24, 2 ** 25)]
        ends = [slice(e.start, min(e.stop, M)) for e in ends]
        want = []
        for e in ends:
            h, r = torch.empty_like(x[e]), torch.empty(e.stop - e.start, device="cuda")
            want.append((*fp8bs.fp8_quant_rmsnorm(x[e].clone(), g, residual=x[e].clone(), h=h,
                                                  rstd=r), h, r))
        # h onto x itself
        fp8bs.fp8_quant_rmsnorm(x, g, residual=x, h=x, rstd=rstd, q=q, s=s)
        assert bool((s > 0).all()) and bool((rstd > 0).all())
        for e, (wq, ws, wh, wr) in zip(ends, want):
            assert torch.equal(q[e], wq) and torch.equal(s[:, e], ws)
            assert torch.equal(x[e], wh) and torch.equal(rstd[e], wr)
    finally:
        x = q = s = rstd = None
        torch.cuda.empty_cache()
