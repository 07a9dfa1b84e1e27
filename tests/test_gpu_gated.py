"""The gated product, dense and by experts, on the GPU.

bf16 output: its gate and up sums are the plain products' (fp8_block_gemm and
fp8_block_grouped_gemm on the stacked weight) in the same order, so the kept z is
held to theirs bit for bit, and those are held to the oracle elsewhere.  y is
checked against float64 from the plain product's FP32 sums: sigma by hardware
exp and reciprocal is within 2^-18 of |gate| (|gate| <= 20, the argument's
rounding being |gate| 2^-23), the product adds 2^-24, bf16 2^-8 of the value.

E4M3 output: its sums are of exact products, checked against float64 sums of the
decoded operands.  A group's 128 products are added in FP32, one rounding (of at
most 2^-23: the adder may cut) per product at worst, then scaled and added to the
groups before: within (128 + K/128 + 4) 2^-23 of B = sum|ab|.  That holds for any
order; the roundings are independent, so the scales, taken over all tiles, come
far closer: within 2^-18 in the 2-norm, a quarter of what the FP8 instruction's
sums leave (1.5e-5).
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import gated
from fp8_block_scaled_05_amd import synth
from tests import _gpu_util as gu

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def fp8bs():
    from fp8_block_scaled_05_amd import fp8bs as mod
    return mod


def operands(fp8bs, M, N, K, case):
    """Pre-activations of order one."""
    x = synth.act(M, K, case=case, tensor=0, device="cuda")
    w = (synth.weight(2 * N, K, case=case, tensor=1, device="cuda").float() * (50 / K ** 0.5)).to(
        torch.bfloat16)
    qw, sw = fp8bs.fp8_quant_w_128x128(w)
    qx, sx = fp8bs.fp8_quant_act_1x128(x)
    return x, qx, sx, qw, sw


def value_tol(z, err=0.0):
    """of y, where the pre-activations are off by err (act has slopes up to 1.13)"""
    gate, up = gated.split(z)
    tol = 2.0 ** -18 * np.abs(gate) * np.abs(up) + 2.0 ** -140
    if np.ndim(err):
        eg, eu = gated.split(err)
        tol = tol + 1.13 * eg * (np.abs(up) + eu) + np.abs(gate) * eu
    return tol


def decoded(qx, sx, qw, sw):
    """The operands' values in float64 on the GPU."""
    M, K = qx.shape
    a = qx.view(torch.float8_e4m3fn).double().view(M, K // 128, 128)
    a = a * sx[:, :M].t().double()[:, :, None]
    w = qw.view(torch.float8_e4m3fn).double().view(-1, K // 128, 128)
    w = w * sw.double().repeat_interleave(128, dim=0)[:, :, None]
    return a.view(M, K), w.view(-1, K)


def exact_sums(qx, sx, qw, sw):
    """(z, bound of its error) in float64."""
    a, w = decoded(qx, sx, qw, sw)
    K = a.shape[1]
    z, B = torch.mm(a, w.t()), torch.mm(a.abs(), w.abs().t())
    return z.cpu().numpy(), ((128 + K // 128 + 4) * 2.0 ** -23 * B).cpu().numpy()


def check_y(y, z32, act):
    z = gu.host_f64(z32)
    want = gated.forward(z, act)
    got = gu.host_f64(y)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= value_tol(z) + 2.0 ** -8 * np.abs(want))


def check_codes(qc, sc, sums, act):
    z, err = sums
    y, tol = gated.forward(z, act), value_tol(z, err)
    M, N = y.shape
    t = lambda a: a.reshape(M, N // 128, 128)
    s = gu.host_f64(sc).T[:M]
    top = np.maximum(np.abs(t(y)).max(axis=2), 2.0 ** -64)
    assert np.all(np.abs(s * 448 - top) <= t(tol).max(axis=2) + 2.0 ** -20 * top)
    assert np.sqrt(((s * 448 - top) ** 2).sum()) <= 2.0 ** -18 * np.sqrt((top ** 2).sum())
    got = t(oracle.decode(gu.host(qc)).astype(np.float64)) * s[:, :, None]
    lim = (np.abs(t(y)) + t(tol)) * 2.0 ** -4 + 2.0 ** -10 * s[:, :, None] + t(tol)
    assert np.all(np.abs(got - t(y)) <= lim * (1 + 2.0 ** -16))


def check_z(z, sums):
    want, err = sums
    assert np.all(np.abs(gu.host_f64(z) - want) <= err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want))


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


# few-row kernels (one, two, four and shared row tiles; 8 to 72 weight rows per
# workgroup, in one round of workgroups and two), ragged rows, odd numbers of 128-column blocks; K of one to seven
# groups (fewer than the stages, every end of their turn)
SHAPES = [(1, 128, 128), (1, 3456, 256), (3, 384, 1280), (2, 2048, 256), (16, 1152, 512),
          (16, 2816, 384), (16, 4096, 640), (17, 128, 384), (20, 1920, 256), (32, 3456, 128),
          (32, 3968, 256), (33, 896, 256), (50, 2048, 256), (64, 4224, 384), (65, 128, 128),
          (100, 256, 512), (129, 384, 256), (333, 2048, 640), (300, 8192, 256), (1100, 4096, 256),
          (2100, 3968, 128)] + [(m, n, 256) for m in (1, 16, 20, 33, 64)
                                for n in (4608, 5248, 6784, 7552, 9088)] + [
          (2, 12416, 128), (40, 10752, 128), (1, 19456, 128)]
# tiles: E4M3 of 32, 64 and 128 rows, a last round in halves of 64; bf16 of 32x64,
# 64x64, 128x256 and 256x256, a last round in halves of 128
TILES = [(70, 1024, 768), (200, 4096, 896), (700, 2048, 384), (1000, 4096, 256), (1200, 8192, 128),
         (520, 5120, 128), (2600, 4096, 256), (700, 16384, 128)]


@pytest.mark.parametrize("act,M,N,K", [(a, *s) for s in SHAPES for a in ACTS] +
                         [("silu", *s) for s in TILES])
def test_codes_in(fp8bs, M, N, K, act):
    _, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1100)
    z32 = fp8bs.fp8_block_gemm(qx, sx, qw, sw, out_dtype=torch.float32)
    zb = fp8bs.fp8_block_gemm(qx, sx, qw, sw)
    z = torch.full((M, 2 * N), 9.0, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, act=act, z=z)
    assert same(z, zb)
    check_y(y, z32, act)
    z.fill_(9.0)
    qc, sc = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw, act=act, z=z)
    sums = exact_sums(qx, sx, qw, sw)
    check_z(z, sums)
    check_codes(qc, sc, sums, act)
    # without z
    assert same(fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, act=act), y)
    q2, s2 = fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw, act=act)
    assert torch.equal(q2, qc) and torch.equal(s2, sc)


@pytest.mark.parametrize("M", [1, 2, 16, 17, 40, 64, 65, 200])
def test_bf16_in(fp8bs, M):
    N, K = 384, 640
    x, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1101)
    z32 = fp8bs.fp8_block_gemm(qx, sx, qw, sw, out_dtype=torch.float32)
    s = torch.zeros(K // 128, M, device="cuda")
    z = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_gemm_gated(x, s, qw, sw, z=z)
    assert torch.equal(s, sx) and same(z, fp8bs.fp8_block_gemm(qx, sx, qw, sw))
    check_y(y, z32, "silu")
    s.zero_()
    qc, sc = fp8bs.fp8_block_gemm_gated_e4m3_out(x, s, qw, sw)
    assert torch.equal(s, sx)
    check_codes(qc, sc, exact_sums(qx, sx, qw, sw), "silu")
    # the codes' own call, and no scales asked for
    q2, s2 = fp8bs.fp8_block_gemm_gated_e4m3_out(x, None, qw, sw)
    assert torch.equal(q2, qc) and torch.equal(s2, sc)


@pytest.mark.parametrize("M", [7, 40, 129, 700])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_strides_and_alignment(fp8bs, M, shift):
    """Odd row strides and offsets of z and the bf16 output, strided codes;
    nothing outside the outputs' rows and columns is written."""
    N, K = 256, 256
    _, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1102)
    z32 = fp8bs.fp8_block_gemm(qx, sx, qw, sw, out_dtype=torch.float32)
    want_z = fp8bs.fp8_block_gemm(qx, sx, qw, sw)
    bufs = [torch.full((M * (n + 3 + shift) + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
            for n in (2 * N, N)]
    z, out = (torch.as_strided(b, (M, n), (n + 3 + shift, 1), shift)
              for b, n in zip(bufs, (2 * N, N)))
    fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw, act="gelu", z=z, out=out)
    assert torch.equal(z, want_z)
    check_y(out, z32, "gelu")
    qc = torch.full((M + 1, N + 16), 7, dtype=torch.uint8, device="cuda")
    sc = torch.full((N // 128 + 1, M + 5), 7.0, device="cuda")
    z.fill_(9.0)
    fp8bs.fp8_block_gemm_gated_e4m3_out(qx, sx, qw, sw, act="gelu", z=z, qc=qc, sc=sc)
    sums = exact_sums(qx, sx, qw, sw)
    check_z(z, sums)
    check_codes(qc[:M, :N], sc[:N // 128, :M], sums, "gelu")
    assert torch.all(qc[M:] == 7) and torch.all(qc[:, N:] == 7)
    assert torch.all(sc[N // 128:] == 7) and torch.all(sc[:, M:] == 7)
    z.fill_(9.0)
    out.fill_(9.0)
    assert all(torch.all(b == 9.0) for b in bufs)


@pytest.mark.parametrize("M", [5, 40, 200])
def test_strided_operands(fp8bs, M):
    N, K = 256, 384
    _, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1103)
    want = fp8bs.fp8_block_gemm_gated(qx, sx, qw, sw)
    a = torch.full((M, K + 32), 0x7F, dtype=torch.uint8, device="cuda")
    b = torch.full((2 * N, K + 16), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((K // 128, M + 9), float("nan"), device="cuda")
    a[:, :K], b[:, :K], s[:, :M] = qx, qw, sx
    assert same(fp8bs.fp8_block_gemm_gated(a[:, :K], s[:, :M], b[:, :K], sw), want)


def test_no_rows(fp8bs):
    _, _, _, qw, sw = operands(fp8bs, 1, 128, 256, 1104)
    a, s = torch.empty(0, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 0, device="cuda")
    assert fp8bs.fp8_block_gemm_gated(a, s, qw, sw).shape == (0, 128)
    qc, sc = fp8bs.fp8_block_gemm_gated_e4m3_out(a, s, qw, sw)
    assert qc.shape == (0, 128) and sc.shape == (1, 0)


# ----------------------------------------------------------------------------
# experts


def experts(fp8bs, rows, N, K, case, gap=0):
    G, M = len(rows), sum(rows) + gap
    x = synth.act(M, K, case=case, tensor=0, device="cuda")
    qx, sx = fp8bs.fp8_quant_act_1x128(x)
    w = synth.expert_weights(G, 2 * N, K, case=case, device="cuda", std=1.0 / K ** 0.5)
    qw = torch.empty(G, 2 * N, K, dtype=torch.uint8, device="cuda")
    sw = torch.empty(G, N // 64, K // 128, device="cuda")
    for g in range(G):
        qw[g], sw[g] = fp8bs.fp8_quant_w_128x128(w[g])
    off = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    return qx, sx, qw, sw, off


# N = 384 in tiles of every number of rows: few rows in all, few to each group,
# whole and ragged tile-rows
ROWS = [[1], [0, 5, 0, 300, 1, 0], [128, 256, 129, 255], [1] * 70, [0, 0, 700], [513, 0, 40],
        [3] * 90, [700, 0, 64, 65, 1900, 129], [130] * 12, [7000, 0, 9000, 2000]]


@pytest.mark.parametrize("act", ["silu", "gelu", "none", "relu"])
@pytest.mark.parametrize("rows", ROWS)
def test_grouped(fp8bs, rows, act):
    N, K = 384, 256
    qx, sx, qw, sw, off = experts(fp8bs, rows, N, K, 1105)
    z32 = fp8bs.fp8_block_grouped_gemm(qx, sx, qw, sw, off, out_dtype=torch.float32)
    zb = fp8bs.fp8_block_grouped_gemm(qx, sx, qw, sw, off)
    z = torch.full((sum(rows), 2 * N), 9.0, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off, act=act, z=z)
    assert same(z, zb)
    check_y(y, z32, act)
    z.fill_(9.0)
    qc, sc = fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off, act=act, z=z)
    at, parts = 0, []
    for g, n in enumerate(rows):
        if n:
            parts.append(exact_sums(qx[at:at + n], sx[:, at:at + n], qw[g], sw[g]))
        at += n
    sums = tuple(np.concatenate(p) for p in zip(*parts))
    check_z(z, sums)
    check_codes(qc, sc, sums, act)
    assert same(fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off, act=act), y)


def test_grouped_is_the_dense_product_of_each_expert(fp8bs):
    rows, N, K = [70, 0, 200, 333], 256, 384
    qx, sx, qw, sw, off = experts(fp8bs, rows, N, K, 1106)
    y = fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off)
    at = 0
    for g, n in enumerate(rows):
        if n:
            c = slice(at, at + n)
            assert same(y[c], fp8bs.fp8_block_gemm_gated(qx[c], sx[:, c], qw[g], sw[g]))
        at += n


def test_grouped_rows_of_no_expert_stay(fp8bs):
    rows, N, K, gap = [40, 0, 130], 128, 256, 50
    qx, sx, qw, sw, off = experts(fp8bs, rows, N, K, 1107, gap)
    M, used = sum(rows) + gap, sum(rows)
    z = torch.full((M, 2 * N), 9.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((M, N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off, z=z, out=out[:, :N])
    assert torch.all(z[used:] == 9) and torch.all(out[used:] == 9) and torch.all(out[:, N:] == 9)
    assert same(z[:used], fp8bs.fp8_block_grouped_gemm(qx[:used], sx[:, :used], qw, sw, off))
    qc = torch.full((M, N), 7, dtype=torch.uint8, device="cuda")
    sc = torch.full((1, M), 7.0, device="cuda")
    fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off, qc=qc, sc=sc)
    assert torch.all(qc[used:] == 7) and torch.all(sc[:, used:] == 7)
    assert not torch.any(sc[:, :used] == 7)


def test_grouped_bad_offsets_stay_inside(fp8bs):
    """Decreasing, negative and overlong offsets: unspecified results, nothing
    outside the outputs is written."""
    rows, N, K = [100, 100, 100], 128, 256
    qx, sx, qw, sw, _ = experts(fp8bs, rows, N, K, 1108)
    buf = torch.full((302, N), 9.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 200, 100, 300], [-50, 100, 200, 300], [0, 100, 900, 5000], [300, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, o, out=buf[1:301])
        torch.cuda.synchronize()
        assert torch.all(buf[0] == 9) and torch.all(buf[301] == 9)


@pytest.mark.parametrize("M", [60, 400, 5000])
def test_grouped_graph_follows_the_offsets(fp8bs, M):
    """A captured call takes the offsets that the device holds at its replay."""
    N, K, G = 256, 384, 5
    cuts = np.random.default_rng(6)
    qx, sx, qw, sw, off = experts(fp8bs, [M] + [0] * (G - 1), N, K, 1111)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qc, sc = torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.empty(2, M, device="cuda")

    def step():
        fp8bs.fp8_block_grouped_gemm_gated(qx, sx, qw, sw, off, out=y)
        fp8bs.fp8_block_grouped_gemm_gated_e4m3_out(qx, sx, qw, sw, off, qc=qc, sc=sc)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        inner = np.sort(cuts.integers(0, M + 1, G - 1))
        off.copy_(torch.tensor([0, *inner, M], dtype=torch.int32))
        y.fill_(5.0)
        sc.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, qc, sc)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, qc, sc)))
    # an expert's rows by themselves (few rows of a dense call are summed in another order)
    g = int(np.argmax(np.diff([0, *inner, M])))
    lo, hi = (int(c) for c in [0, *inner, M][g:g + 2])
    one = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
    assert same(y[lo:hi], fp8bs.fp8_block_grouped_gemm_gated(
        qx[lo:hi], sx[:, lo:hi], qw[g:g + 1], sw[g:g + 1], one))


def test_graph_and_streams(fp8bs):
    """Captured and replayed between eager calls; calls on two streams at once."""
    M, N, K = 40, 512, 640
    x, qx, sx, qw, sw = operands(fp8bs, M, N, K, 1109)
    qc, sc = torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.empty(4, M, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = [torch.empty(fp8bs.workspace_bytes(op, M, N, K), dtype=torch.uint8, device="cuda")
          for op in (fp8bs.OP_GEMM_GATED_E4M3, fp8bs.OP_GEMM_BF16)]

    def step():
        fp8bs.fp8_block_gemm_gated_e4m3_out(x, None, qw, sw, qc=qc, sc=sc, workspace=ws[0])
        fp8bs.fp8_block_gemm_gated(x, None, qw, sw, out=y, workspace=ws[1])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        x.copy_(synth.act(M, K, case=1110 + turn, device="cuda"))
        y.fill_(5.0)
        sc.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qc, sc, y)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (qc, sc, y)))
    torch.cuda.synchronize()
    outs = []
    for st in [torch.cuda.Stream(), torch.cuda.Stream()] * 2:
        with torch.cuda.stream(st):
            outs.append((*fp8bs.fp8_block_gemm_gated_e4m3_out(x, None, qw, sw),
                         fp8bs.fp8_block_gemm_gated(x, None, qw, sw)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, (qc, sc, y)))
