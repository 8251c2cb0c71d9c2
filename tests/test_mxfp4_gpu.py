"""The 4-bit floating point operators on the GPU against the 64-bit reference (mxfp4_ref): the codec bit
for bit, the product on lattices whose sums are exact (bit for bit) and on random data (derived
bounds), values that are not finite, the longest sides; captured, on another stream, in caller-owned
buffers between canaries."""
import math

import pytest
import torch

import int8_quantized_matmul_rowwise_amd as lm
from tests import mxfp4_ref as ref
from tests.test_fp8_gpu import frame_untouched, framed, gen, lattice, outliers, randn, trits, u8

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16]
E8 = torch.float8_e8m0fnu


# ---- codec

@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R,C", [(1, 16), (3, 32), (31, 48), (32, 256), (33, 272), (70, 1040), (5, 4112), (129, 528)])
def test_quantize_rows(R, C, dt):
    print(f"\n[case] quantize rows {dt} {R}x{C}", flush=True)
    g = gen(R + C)
    X = outliers(g, randn(g, R, C) * torch.exp2(torch.randint(-6, 3, (R, 1), generator=g).float())).to(dt)
    q, s = lm.mxfp4_quantize(X.cuda())
    v, rq, rs = ref.coded(X)
    assert torch.equal(u8(q), rq) and torch.equal(u8(s), rs)
    assert torch.equal(lm.mxfp4_dequantize(q, s, C, dt).cpu().double(), v)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("K,N", [(16, 8), (32, 136), (144, 128), (256, 520), (272, 264), (2064, 136), (528, 8), (16, 1288)])
def test_quantize_columns(K, N, dt):
    print(f"\n[case] quantize columns {dt} {K}x{N}", flush=True)
    g = gen(K + N)
    W = (randn(g, K, N) * 0.02 * torch.exp2(torch.randint(-6, 3, (K, 1), generator=g).float()))
    W[: min(K, 32), : min(N, 40)] = 0
    W = W.to(dt)
    q, s = lm.mxfp4_quantize(W.cuda(), columns=True)
    v, rq, rs = ref.coded(W.t())
    assert torch.equal(u8(q), rq) and torch.equal(u8(s), rs)
    assert torch.equal(lm.mxfp4_dequantize(q, s, K, dt).cpu().double(), v)
    if N % 16 == 0 and K % 16 == 0:  # the same codes from the transposed matrix
        q2, s2 = lm.mxfp4_quantize(W.t().contiguous().cuda())
        assert torch.equal(u8(q2), rq) and torch.equal(u8(s2), rs)


def border_groups(dt):
    """Groups whose largest magnitude is 7 times a power of two, a step to either side of it, the type's
    largest and smallest numbers, and every tie between two codes with a step to either side."""
    fi = torch.finfo(dt)
    step = fi.eps
    rows = []
    for a in (7.0, 7.0 * (1 + step), 7.0 * (1 - step / 2), 1.75, 3.5 * 2.0 ** -9, 6.0, 6.0 * (1 + step), fi.max, fi.tiny, fi.smallest_normal * step, 1.0, 0.0):
        v = torch.linspace(-1, 1, 32, dtype=torch.float64) * a
        v[0], v[1] = a, -a
        rows.append(v)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    for e in (-9, -3, 0, 2, 8):
        v = torch.cat([ties, ties * (1 + step), ties * (1 - step / 2), torch.tensor([6.0])]) * 2.0 ** e
        rows.append(torch.cat([v, -v[:10]])[:32])
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("dt", DTS)
def test_quantize_border_values(dt):
    X = border_groups(dt)
    v, rq, rs = ref.coded(X)
    q, s = lm.mxfp4_quantize(X.cuda())
    assert torch.equal(u8(q), rq) and torch.equal(u8(s), rs)
    W = torch.zeros(32, 24, dtype=dt)
    W[:, : X.shape[0]] = X.t()
    q, s = lm.mxfp4_quantize(W.cuda(), columns=True)
    v, rq, rs = ref.coded(W.t())
    assert torch.equal(u8(q), rq) and torch.equal(u8(s), rs)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("v", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("columns", [False, True])
def test_quantize_not_finite(v, dt, columns):
    """The group becomes NaN as a whole; every other one keeps its bits."""
    g = gen(21)
    X = randn(g, 80, 272).to(dt)
    bad = [(0, 0), (33, 31), (34, 32), (79, 271), (50, 256)]
    Y = X.clone()
    for r, c in bad:
        Y[r, c] = v
    if columns:
        X, Y = X.t().contiguous(), Y.t().contiguous()
    q0, s0 = lm.mxfp4_quantize(X.cuda(), columns=columns)
    q1, s1 = lm.mxfp4_quantize(Y.cuda(), columns=columns)
    n = X.shape[0] if columns else X.shape[1]
    v0, v1 = (lm.mxfp4_dequantize(q, s, n, dt).cpu() for q, s in ((q0, s0), (q1, s1)))
    hit = torch.zeros(80, 288, dtype=torch.bool)
    for r, c in bad:
        hit[r, c // 32 * 32: c // 32 * 32 + 32] = True
    hit = hit[:, :272]
    assert torch.isnan(v1[hit]).all() and torch.equal(v1[~hit], v0[~hit])
    assert int((u8(s1) == 255).sum()) == len(bad) and int((u8(s0) == 255).sum()) == 0


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("v", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("n", [16, 48, 272, 528])
def test_padding_of_groups_that_are_not_finite(n, columns, v, dt):
    """Codes past n are zeros, in a last group of 16 values that is not finite too; scales past the last group and
    row are zeros, and the other groups keep their codes."""
    X = randn(gen(n), 40, n).to(dt)
    Y = X.clone()
    Y[3, n - 1] = Y[39, n - 16] = v
    if columns:
        X, Y = X.t().contiguous(), Y.t().contiguous()
    q0, s0 = lm.mxfp4_quantize(X.cuda(), columns=columns)
    q1, s1 = lm.mxfp4_quantize(Y.cuda(), columns=columns)
    assert not q0[:, n // 2:].any() and not q1[:, n // 2:].any()
    _, _, rs = ref.coded(Y.t() if columns else Y)
    assert torch.equal(u8(s1), rs) and int((rs == 255).sum()) == 2
    a, b = q0.cpu(), q1.cpu()
    for r in (3, 39):
        b[r, (n - 16) // 32 * 16:] = a[r, (n - 16) // 32 * 16:]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt", DTS)
def test_dequantize_every_code_and_scale(dt):
    n = 256
    q = torch.arange(256, dtype=torch.uint8)[:128].repeat(256, 1)
    q[:, 1::2] = torch.arange(128, 256, dtype=torch.uint8)[::2]
    b = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 8).clone()
    s = ref.tiles(b)
    want = ref.values(q, s, n)
    got = lm.mxfp4_dequantize(q.cuda(), s.cuda(), n, dt).cpu()
    # a value that the type cannot hold becomes infinite, as its conversion makes it
    w = want.float().to(dt)
    assert torch.equal(torch.isnan(got), torch.isnan(w)) and torch.equal(got.nan_to_num(0, 7, -7), w.nan_to_num(0, 7, -7))


def test_codec_empty():
    for shape, columns in (((0, 32), False), ((5, 0), False), ((0, 8), True), ((32, 0), True)):
        x = torch.zeros(shape, dtype=torch.float16, device="cuda")
        q, s = lm.mxfp4_quantize(x, columns=columns)
        rows, n = (shape[1], shape[0]) if columns else shape
        assert q.shape == (rows, lm.fp4_code_pitch(n)) and lm.mxfp4_dequantize(q, s, n).shape == (rows, n)


@pytest.mark.parametrize("R,C,columns", [(1 << 22, 16, False), (1 << 22, 272, False), (2, 1 << 22, False), (1 << 22, 8, True), (16, 1 << 22, True), (272, 1 << 20, True)])
def test_codec_longest_sides(R, C, columns):
    """Whole numbers up to 3, which the format holds exactly."""
    print(f"\n[case] codec longest side {R}x{C} columns={columns}", flush=True)
    X = trits(5, R, C) * 3
    q, s = lm.mxfp4_quantize(X, columns=columns)
    n = R if columns else C
    assert torch.equal(lm.mxfp4_dequantize(q, s, n, X.dtype), X.t() if columns else X)
    del X, q, s
    torch.cuda.empty_cache()


def test_codec_past_32_bits():
    """A matrix of more than 2^32 values."""
    R, C = (1 << 20) + 40, 4112
    print(f"\n[case] codec past 32 bits {R}x{C}", flush=True)
    X = torch.zeros(R, C, dtype=torch.float16, device="cuda")
    rows = [0, 1, (1 << 19) + 7, 1 << 20, R - 33, R - 1]
    X[rows] = trits(6, len(rows), C) * 2
    q, s = lm.mxfp4_quantize(X)
    out = lm.mxfp4_dequantize(q, s, C, X.dtype)
    assert torch.equal(out[rows], X[rows])
    assert int(out.count_nonzero()) == int(X.count_nonzero())
    del X, q, s, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R,C,columns", [(33, 272, False), (272, 136, True)])
def test_codec_writes_its_outputs_alone(R, C, columns):
    X = randn(gen(8), R, C).half().cuda()
    q0, s0 = lm.mxfp4_quantize(X, columns=columns)
    rows, n = (C, R) if columns else (R, C)
    q, qw = framed(tuple(q0.shape), torch.uint8, 90)
    s, sw = framed(tuple(s0.shape), torch.uint8, 90)
    assert lm.lib().mxfp4_quantize(X.data_ptr(), R, C, lm.F16, int(columns), q.data_ptr(), s.data_ptr(), torch.cuda.current_stream().cuda_stream) == lm.OK
    out, ow = framed((rows, n), torch.float16)
    lm.mxfp4_dequantize(q, s, n, torch.float16, out=out)
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(s, u8(s0).cuda())
    assert frame_untouched(qw, q.numel(), 90) and frame_untouched(sw, s.numel(), 90) and frame_untouched(ow, rows * n)


# ---- product

SHAPES = [(1, 16, 8), (1, 4096, 264), (3, 144, 1032), (4, 528, 72), (5, 272, 136), (16, 272, 520), (17, 1040, 264), (33, 528, 136), (64, 1664, 72),
          (65, 256, 136), (100, 640, 2056), (128, 2064, 264), (129, 128, 264), (300, 1040, 520), (257, 400, 1288),
          (520, 144, 776),
          # split sums: few columns and many steps, with parts of unequal length
          (2, 16384, 520), (16, 4240, 264), (30, 8208, 72), (64, 4112, 264), (40, 4096, 8200), (64, 1040, 12296),
          (100, 4240, 264), (300, 8208, 520), (260, 8208, 2056), (6, 1040, 16392), (4, 16400, 8200)]
# several pieces of columns with A coded in the kernel; tiles of 128, of 256 (one and several a workgroup, odd and even
# counts of steps), and tiles whose sums are split
LARGE = [(1, 4112, 8200), (4, 1040, 12296), (3, 272, 16392), (2048, 528, 2056), (2400, 272, 4360), (4100, 144, 4360), (4100, 400, 4360),
         (4100, 800, 4360), (1200, 12304, 4104), (2056, 16400, 4104), (1000, 8208, 1032), (8200, 528, 2056)]


def product(X, W):
    """Exact: whole numbers."""
    return (X.double() @ W.double()).float().to(X.dtype)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", SHAPES + LARGE)
def test_matmul_exact_lattice(M, K, N, dt):
    print(f"\n[case] mxfp4 lattice {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X = lattice(g, M, K, dt=dt, spread=3).cuda()
    W = lattice(g, N, K, dt=dt, spread=3).t().contiguous().cuda()
    # another scale for some of the groups
    X[:, 32:64] *= 2
    W[64:96] *= 4
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    want = product(X, W)
    assert torch.equal(lm.mxfp4_matmul(X, Wq, s), want)
    Xq, sx = lm.mxfp4_quantize(X)
    assert torch.equal(lm.mxfp4_matmul_coded(Xq, sx, Wq, s, dt), want)
    assert torch.equal(lm.mxfp4_matmul_coded(Xq.view(torch.float4_e2m1fn_x2), sx.view(torch.uint8), Wq, s, dt), want)


# few rows of wide weights: one or two pieces of 16 rows against one, two and four of 16 columns, several steps a wave,
# and shares of them that are not equal
WIDE = [(12, 4240, 4104), (17, 1040, 8200), (30, 4240, 8200), (32, 8208, 8456), (5, 4240, 24584), (16, 8208, 28680), (16, 272, 24576)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", WIDE)
def test_matmul_few_rows_of_wide_weights(M, K, N, dt):
    print(f"\n[case] mxfp4 wide {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X = lattice(g, M, K, dt=dt, spread=3).cuda()
    W = lattice(g, N, K, dt=dt, spread=3).t().contiguous().cuda()
    X[:, 32:64] *= 2
    W[64:96] *= 4
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    want = product(X, W)
    assert torch.equal(lm.mxfp4_matmul(X, Wq, s), want)
    assert torch.equal(lm.mxfp4_matmul_coded(*lm.mxfp4_quantize(X), Wq, s, dt), want)


@pytest.mark.parametrize("seed", range(24))
def test_matmul_sweep(seed):
    g = gen(3000 + seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    M, K, N, dt = rnd(1, (20, 130, 700)[seed % 3]), 16 * rnd(1, 300), 8 * rnd(1, 400), DTS[seed // 3 % 2]
    print(f"\n[case] mxfp4 sweep {dt} {M}x{K}x{N}", flush=True)
    X, W = lattice(g, M, K, dt=dt).cuda(), lattice(g, K, N, dt=dt).cuda()
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    want = product(X, W)
    assert torch.equal(lm.mxfp4_matmul(X, Wq, s), want)
    assert torch.equal(lm.mxfp4_matmul_coded(*lm.mxfp4_quantize(X), Wq, s, dt), want)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", [(4100, 16, 4104), (4100, 256, 4104), (4100, 512, 4104), (4100, 768, 4104), (4200, 1040, 8200), (12000, 272, 4360)])
def test_matmul_many_tiles(M, K, N, dt):
    """Several tiles a workgroup: one step a tile, two, three, and more."""
    print(f"\n[case] mxfp4 many tiles {dt} {M}x{K}x{N}", flush=True)
    X, W = trits(M + K, M, K, dt=dt), trits(N + K, K, N, dt=dt)
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    assert torch.equal(lm.mxfp4_matmul(X, Wq, s), product(X, W))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", [x for x in SHAPES if x[1] * x[2] < 3 << 20])
def test_matmul_random(M, K, N, dt):
    print(f"\n[case] mxfp4 random {dt} {M}x{K}x{N}", flush=True)
    g = gen(M * 3 + K + N)
    X, W = outliers(g, randn(g, M, K)).to(dt), (randn(g, N, K) * 0.02).to(dt)
    Wq, s = lm.mxfp4_quantize(W.cuda())
    Y = lm.mxfp4_matmul(X.cuda(), Wq, s)
    want, err = ref.product(ref.coded(X)[0], ref.coded(W)[0])
    ref.assert_close(Y, want, err, "Y")
    Yc = lm.mxfp4_matmul_coded(*lm.mxfp4_quantize(X.cuda()), Wq, s, dt)
    ref.assert_close(Yc, want, err, "Y of codes")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M", [3, 37, 70, 300])
def test_matmul_rows_do_not_meet(M, dt):
    """A row that is not finite is NaN and leaves the others as they were, bit for bit, whatever its place."""
    K, N = 400, 264
    g = gen(5)
    X, W = randn(g, M, K).to(dt), (randn(g, N, K) * 0.02).to(dt)
    Wq, s = lm.mxfp4_quantize(W.cuda())
    Y = lm.mxfp4_matmul(X.cuda(), Wq, s).cpu()
    for row, v in ((0, math.nan), (M - 1, math.inf), (M // 2, -math.inf)):
        X2 = X.clone()
        X2[row, 7] = v
        Y2 = lm.mxfp4_matmul(X2.cuda(), Wq, s).cpu()
        keep = torch.arange(M) != row
        assert torch.equal(Y2[keep], Y[keep])
        assert torch.isnan(Y2[row].float()).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M", [2, 20, 100, 12000])
def test_matmul_weights_not_finite(M, dt):
    K, N = 272, 264
    g = gen(M)
    X, W = lattice(g, M, K, dt=dt).cuda(), lattice(g, K, N, dt=dt).cuda()
    want = product(X, W)
    W[5, 17], W[271, 263] = math.inf, math.nan
    Y = lm.mxfp4_matmul(X, *lm.mxfp4_quantize(W, columns=True))
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[17] = keep[263] = False
    assert torch.equal(Y[:, keep], want[:, keep]) and torch.isnan(Y[:, ~keep]).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M", [4, 20, 140])
def test_matmul_far_scales(M, dt):
    """Rows and groups at the ends of the type's range: the scales are applied without a detour
    through values that overflow or vanish."""
    K, N = 256, 136
    g = gen(6)
    lo, hi = (-12, 8) if dt == torch.float16 else (-90, 90)
    X = lattice(g, M, K, dt=torch.float64)
    X = (X * torch.exp2(torch.linspace(lo, hi, M).round().double())[:, None]).to(dt).cuda()
    W = (lattice(g, K, N, dt=torch.float64) * 2.0 ** (-4 if dt == torch.float16 else -20)).to(dt).cuda()
    assert torch.equal(lm.mxfp4_matmul(X, *lm.mxfp4_quantize(W, columns=True)), product(X, W))


def test_matmul_smallest_scales():
    """bf16 values below 2^-124 have the least scale, 2^-127, and codes below the usual range."""
    dt = torch.bfloat16
    X = torch.tensor([[2.0 ** -126, 2.0 ** -127, 2.0 ** -128, 3 * 2.0 ** -126] + [0.0] * 12], dtype=torch.float64).to(dt).cuda()
    W = torch.zeros(16, 8, dtype=torch.float64)
    W[0], W[1], W[2], W[3] = 2.0 ** 100, 2.0 ** 101, 2.0 ** 101, 2.0 ** 101
    W = W.to(dt).cuda()
    for rep in (1, 40, 200):
        Y = lm.mxfp4_matmul(X.expand(rep, 16).contiguous(), *lm.mxfp4_quantize(W, columns=True))
        assert torch.equal(Y.double().cpu(), torch.full((rep, 8), 2.0 ** -26 + 2.0 ** -26 + 2.0 ** -27 + 6 * 2.0 ** -26, dtype=torch.float64).float().to(dt).double())


def test_matmul_empty():
    q = lm.mxfp4_quantize(torch.zeros(0, 64, dtype=torch.float16, device="cuda"), columns=True)
    Y = lm.mxfp4_matmul(torch.zeros(5, 0, dtype=torch.float16, device="cuda"), *q)
    assert Y.shape == (5, 64) and not Y.any()
    q = lm.mxfp4_quantize(torch.zeros(64, 8, dtype=torch.float16, device="cuda"), columns=True)
    assert lm.mxfp4_matmul(torch.zeros(0, 64, dtype=torch.float16, device="cuda"), *q).shape == (0, 8)
    x = lm.mxfp4_quantize(torch.zeros(0, 64, dtype=torch.float16, device="cuda"))
    assert lm.mxfp4_matmul_coded(*x, *q).shape == (0, 8)


@pytest.mark.parametrize("M,N", [(1, 8), (3, 2056), (20, 136), (64, 72), (130, 136), (300, 264), (2056, 2056)])
def test_matmul_longest_sum(M, N):
    K, dt = 1 << 22, torch.bfloat16
    print(f"\n[case] mxfp4 longest sum {M}x{K}x{N}", flush=True)
    X, W = trits(M, M, K, dt=dt), trits(M + N, K, N, dt=dt)
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    Y = lm.mxfp4_matmul(X, Wq, s)
    if M > 2000:
        want = torch.cat([lm.mxfp4_matmul(X[a: a + 128], Wq, s) for a in range(0, M, 128)])
    else:
        want = sum(X[:, a: a + (1 << 18)].double() @ W[a: a + (1 << 18)].double() for a in range(0, K, 1 << 18)).float().to(dt)
    assert Y.any() and torch.equal(Y, want)
    assert torch.equal(lm.mxfp4_matmul_coded(*lm.mxfp4_quantize(X), Wq, s, dt), want)
    del X, W, Wq, s, Y, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,N", [(1 << 22, 144, 136), (1 << 22, 16, 8), (40, 144, 1 << 22), (3, 272, 1 << 22), (300, 16, 1 << 22)])
def test_matmul_longest_sides(M, K, N):
    print(f"\n[case] mxfp4 longest side {M}x{K}x{N}", flush=True)
    X, W = trits(1, M, K), trits(2, K, N)
    Wq, s = lm.mxfp4_quantize(W, columns=True)
    assert torch.equal(lm.mxfp4_matmul(X, Wq, s), product(X, W))
    del X, W, Wq, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,N", [(1, 144, 72), (19, 272, 136), (70, 400, 264), (300, 1040, 520), (30, 8208, 72)])
def test_matmul_writes_its_output_alone(M, K, N):
    g = gen(7)
    X, W = randn(g, M, K).half().cuda(), randn(g, N, K).half().cuda()
    Wq, s = lm.mxfp4_quantize(W)
    Xq, sx = lm.mxfp4_quantize(X)
    for coded in (False, True):
        call = (lambda **kw: lm.mxfp4_matmul_coded(Xq, sx, Wq, s, torch.float16, **kw)) if coded else (lambda **kw: lm.mxfp4_matmul(X, Wq, s, **kw))
        nb = (lm.mxfp4_matmul_coded_workspace_bytes if coded else lm.mxfp4_matmul_workspace_bytes)(M, K, N)
        Y, yw = framed((M, N), torch.float16)
        ws, wsw = framed((nb,), torch.uint8, 90)
        call(Y=Y, workspace=ws)
        torch.cuda.synchronize()
        assert frame_untouched(yw, M * N) and frame_untouched(wsw, nb, 90)
        # the workspace's old contents do not matter, and equal calls give equal bits
        ws.fill_(255)
        assert torch.equal(call(workspace=ws), Y)


@pytest.mark.parametrize("M", [20, 100, 300])
def test_scales_of_rows_past_the_last_have_no_effect(M):
    g = gen(9)
    K, N = 272, 136
    X, W = randn(g, M, K).half().cuda(), randn(g, N, K).half().cuda()
    (Xq, sx), (Wq, s) = lm.mxfp4_quantize(X), lm.mxfp4_quantize(W)
    want = lm.mxfp4_matmul_coded(Xq, sx, Wq, s, X.dtype)
    for rows, t in ((M, sx), (N, s)):  # every byte of the rows past the last: NaN
        b = t.view(torch.uint8)
        for r in range(rows, -(-rows // 32) * 32):
            at = [(r % 16) * 4 + r % 32 // 16 + (x // 8) * 256 + (x % 4) * 64 + (x % 8 // 4) * 2 for x in range(16)]
            b[r // 32, at] = 255
    assert torch.equal(lm.mxfp4_matmul_coded(Xq, sx, Wq, s, X.dtype), want)


# (sums split over workgroups among them)
@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("M,K,N", [(2, 272, 136), (16, 4240, 264), (100, 4240, 264), (300, 8208, 520), (1200, 12304, 4104), (2048, 528, 2056)])
def test_workspaces_graphs_and_streams(M, K, N, coded):
    print(f"\n[case] mxfp4 graphs {M}x{K}x{N} coded={coded}", flush=True)
    g = gen(M + K + N)
    dt = torch.bfloat16
    X, W = randn(g, M, K).to(dt).cuda(), randn(g, N, K).to(dt).cuda()
    Wq, s = lm.mxfp4_quantize(W)
    if coded:
        Xq, sx = lm.mxfp4_quantize(X)
        nb, f = lm.mxfp4_matmul_coded_workspace_bytes(M, K, N), lambda ws: lm.mxfp4_matmul_coded(Xq, sx, Wq, s, dt, workspace=ws)
    else:
        nb, f = lm.mxfp4_matmul_workspace_bytes(M, K, N), lambda ws: lm.mxfp4_matmul(X, Wq, s, workspace=ws)
    want = f(None)
    ws, whole = framed((nb,), torch.uint8, 90)
    for fill in (255, 0, 129):
        ws.fill_(fill)
        assert torch.equal(f(ws), want), fill
    assert frame_untouched(whole, nb, 90)
    graphs = []
    for _ in range(2):  # with one workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f(ws)
        graphs.append((graph, out))
    for r in range(3):
        ws.fill_(255)
        for graph, out in graphs:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want), r
    sides = [(torch.cuda.Stream(), torch.full((nb,), 255, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for side, own in sides:
            with torch.cuda.stream(side):
                outs.append(f(own))
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_on_another_stream():
    g = gen(14)
    X, W = randn(g, 40, 272).half().cuda(), randn(g, 264, 272).half().cuda()
    q = lm.mxfp4_quantize(W)
    want = lm.mxfp4_matmul(X, *q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for i in range(8):
        st = side if i % 2 else side.cuda_stream
        Xq, sx = lm.mxfp4_quantize(X, stream=st)
        outs += [lm.mxfp4_matmul(X, *q, stream=st), lm.mxfp4_matmul_coded(Xq, sx, *q, X.dtype, stream=st)]
        outs.append(lm.mxfp4_dequantize(Xq, sx, 272, stream=st))
    side.synchronize()
    values = lm.mxfp4_dequantize(*lm.mxfp4_quantize(X), 272)
    for i, o in enumerate(outs):
        assert torch.equal(o, values if i % 3 == 2 else want)
    assert torch.cuda.current_stream() != side


def test_refusals_of_gpu_tensors():
    X, W = torch.zeros(5, 272, dtype=torch.float16, device="cuda"), torch.zeros(264, 272, dtype=torch.float16, device="cuda")
    Wq, s = lm.mxfp4_quantize(W)
    Xq, sx = lm.mxfp4_quantize(X)
    for bad in (lambda: lm.mxfp4_quantize(X.float()), lambda: lm.mxfp4_matmul(X.float(), Wq, s), lambda: lm.mxfp4_matmul(X, Wq.view(torch.int8), s),
                lambda: lm.mxfp4_matmul(X, Wq, s.cpu()), lambda: lm.mxfp4_matmul(X, Wq, s, Y=torch.zeros(5, 264, device="cuda")),
                lambda: lm.mxfp4_matmul_coded(Xq, sx, Wq, s, torch.float32), lambda: lm.mxfp4_dequantize(Xq, sx, 272, torch.float32),
                lambda: lm.mxfp4_matmul(X, Wq, s, workspace=torch.zeros(1 << 20, device="cuda")),
                lambda: lm.fp8_matmul_block_coded(X, sx, Wq, s)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lm.mxfp4_quantize(W.t()), lambda: lm.mxfp4_quantize(X[0]), lambda: lm.mxfp4_matmul(X[:, ::2], Wq, s),
                lambda: lm.mxfp4_matmul(X, Wq[:, :128].contiguous(), s), lambda: lm.mxfp4_matmul(X, Wq, s[:1]),
                lambda: lm.mxfp4_matmul(X, Wq, s, Y=X), lambda: lm.mxfp4_matmul_coded(Xq, s, Wq, s), lambda: lm.mxfp4_matmul_coded(Xq[:, :100].contiguous(), sx, Wq, s),
                lambda: lm.mxfp4_dequantize(Xq, sx, 600), lambda: lm.mxfp4_dequantize(Xq, s, 272), lambda: lm.mxfp4_dequantize(Xq, sx, 272, X.dtype, out=W)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lm.mxfp4_quantize(torch.zeros(5, 264, dtype=torch.float16, device="cuda")),  # no multiple of 16
                lambda: lm.mxfp4_quantize(torch.zeros(5, 16, dtype=torch.float16, device="cuda"), columns=True),
                lambda: lm.mxfp4_dequantize(Xq, sx, 264),
                lambda: lm.mxfp4_matmul(torch.zeros(100, 272, dtype=torch.float16, device="cuda"), Wq, s, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                lambda: lm.mxfp4_matmul(torch.zeros(100, 272, dtype=torch.float16, device="cuda"), Wq, s, workspace=Wq.view(-1))):
        with pytest.raises(lm.LLMInt8Error):
            bad()
    torch.cuda.synchronize()
