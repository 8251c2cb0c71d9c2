"""The e4m3 block-scaled operators on the GPU against the 64-bit reference (fp8_ref): weight
conversion and its transposed form bit for bit, the product and its gradient on lattices whose
sums are exact (bit for bit) and on random data (derived bounds), and the mixture-of-experts
layer; captured, on another stream, in caller-owned buffers between canaries."""
import math

import pytest
import torch

import int8_quantized_matmul_rowwise_amd as lm
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16]
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def outliers(g, x):
    """A few columns far larger, one row of zeros, one group of zeros."""
    x = x.clone()
    x[:, torch.randint(0, x.shape[1], (3,), generator=g)] *= 30
    if x.shape[0] > 2:
        x[1] = 0
    x[0, :128] = 0
    return x


def u8(t):
    return t.view(torch.uint8).cpu()


def codes_equal(got, want_values, what):
    assert torch.equal(got.cpu().view(F8).float().double(), want_values), f"{what}: codes differ"


# ---- weight conversion

@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 136), (2064, 520), (400, 1032), (528, 8), (16, 1288)])
def test_quantize_weight(K, N, dt):
    print(f"\n[case] quantize {dt} {K}x{N}", flush=True)
    g = gen(K + N)
    W = (randn(g, K, N) * 0.02 * torch.exp2(torch.randint(-6, 3, (K, 1), generator=g).float()))
    W[: min(K, 128), : min(N, 128)] *= 0  # a block of zeros
    W = W.to(dt)
    Wd = W.cuda()
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(Wd, transposed=True)
    q1, s1 = lm.fp8_quantize_weight_block(Wd)
    _, rq, rs, rqt, rst = ref.coded_weight(W)
    codes_equal(Wq, rq, "Wq")
    codes_equal(WqT, rqt, "WqT")
    assert torch.equal(u8(s), rs) and torch.equal(u8(sT), rst)
    assert torch.equal(u8(q1), u8(Wq)) and torch.equal(u8(s1), u8(s))


@pytest.mark.parametrize("dt", DTS)
def test_quantize_border_values(dt):
    """Blocks whose largest magnitude is 448 times a power of two, one step to either side of it,
    the type's largest and smallest numbers, and every tie between two codes."""
    fi = torch.finfo(dt)
    step = torch.finfo(dt).eps
    tops = [448.0, 448.0 * (1 + step), 448.0 * (1 - step / 2), 1.75, 3.5 * 2.0 ** -9, fi.max, fi.tiny,
            fi.smallest_normal * step, 1.0, 0.0]
    cols = []
    for a in tops:
        v = torch.linspace(-1, 1, 128, dtype=torch.float64) * a
        v[0], v[1] = a, -a
        cols.append(v)
    grid = torch.tensor([m * 2.0 ** e for e in range(-9, 9) for m in (1.0, 1.0625, 1.1875, 1.3125, 1.4375, 1.5625, 1.6875)]
                        + [448.0, 0.0], dtype=torch.float64)  # ties at the odd sixteenths
    cols.append(grid[-128:])
    # one block per value: 128 equal columns each
    W = torch.cat([c[:, None].expand(128, 128) for c in cols], dim=1).to(dt).contiguous()
    Wq, s = lm.fp8_quantize_weight_block(W.cuda())
    _, rq, rs, _, _ = ref.coded_weight(W)
    codes_equal(Wq, rq, "Wq")
    assert torch.equal(u8(s), rs)


# ---- product

def lattice(g, *shape, dt, spread=0):
    """Whole numbers -3 .. 3 times a power of two per row: their codes are exact, and so is every
    sum of their products here."""
    x = torch.randint(-3, 4, shape, generator=g).double()
    if spread:
        x = x * torch.exp2(torch.randint(0, spread + 1, (shape[0], 1), generator=g).double())
    return x.to(dt)


SHAPES = [(1, 16, 8), (1, 4096, 264), (3, 144, 1032), (16, 272, 520), (17, 1040, 264), (33, 528, 136), (64, 1664, 72),
          (65, 256, 136), (100, 640, 2056), (128, 2064, 264), (129, 128, 264), (300, 1040, 520), (257, 400, 1288),
          (520, 144, 776),
          # split sums: few columns and many groups, with parts of unequal length
          (2, 16384, 520), (16, 4240, 264), (30, 8208, 72), (64, 2192, 264), (40, 4096, 8200), (64, 1040, 12296),
          (100, 4240, 264), (300, 8208, 520), (260, 4240, 2056), (6, 1040, 16392), (4, 16400, 8200)]


# two pieces of columns with A coded in the kernel; the persistent tiled kernels: tiles of 128, of 256 (one and several a workgroup, odd and even counts
# of groups), and tiles of 256 whose sums are split
LARGE = [(1, 4112, 8200), (4, 1040, 12296), (3, 272, 16392), (2048, 272, 2056), (2400, 272, 4360), (4100, 144, 4360), (4100, 400, 4360), (1200, 12304, 4104)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", SHAPES + LARGE)
def test_matmul_exact_lattice(M, K, N, dt):
    print(f"\n[case] matmul lattice {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X = lattice(g, M, K, dt=dt, spread=3)
    W = lattice(g, N, K, dt=dt, spread=3).t().contiguous()
    Wq, s = lm.fp8_quantize_weight_block(W.cuda())
    Y = lm.fp8_matmul_block(X.cuda(), Wq, s)
    want = (X.double() @ W.double()).float().to(dt)
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("seed", range(16))
def test_matmul_and_backward_sweep(seed):
    g = gen(2000 + seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    M, K, N, dt = rnd(1, 20 if seed % 2 else 700), 16 * rnd(1, 300), 8 * rnd(1, 400), DTS[seed // 2 % 2]
    print(f"\n[case] matmul, backward sweep {dt} {M}x{K}x{N}", flush=True)
    X, W, dY = lattice(g, M, K, dt=dt).cuda(), lattice(g, K, N, dt=dt).cuda(), lattice(g, M, N, dt=dt).cuda()
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    assert torch.equal(lm.fp8_matmul_block(X, Wq, s), (X.double() @ W.double()).float().to(dt))
    dX, dW = lm.fp8_matmul_block_backward(dY, X, WqT, sT)
    assert torch.equal(dX, (dY.double() @ W.double().t()).float().to(dt))
    assert torch.equal(dW, (X.double().t() @ dY.double()).float().to(dt))


# many tiles, several per workgroup, with few and many groups along K (the sums of the lattice are
# exact in 64 bits on the GPU too)
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", [(4100, 16, 4104), (4100, 128, 4104), (4100, 256, 4104), (4100, 272, 4360), (4100, 512, 4104),
                                   (4100, 640, 4104), (5000, 1040, 4104), (3800, 16, 4000), (3800, 144, 4000),
                                   (3800, 400, 4000), (3800, 1664, 4000), (2049, 912, 8200)])
def test_matmul_many_tiles(M, K, N, dt):
    print(f"\n[case] matmul many tiles {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X = lattice(g, M, K, dt=dt, spread=3).cuda()
    W = lattice(g, N, K, dt=dt, spread=3).t().contiguous().cuda()
    Y = lm.fp8_matmul_block(X, *lm.fp8_quantize_weight_block(W))
    assert torch.equal(Y, (X.double() @ W.double()).float().to(dt))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", [(130, 4112, 4104), (700, 4112, 4104), (4100, 4112, 520), (520, 1040, 8200)])
def test_backward_many_tiles(M, K, N, dt):
    print(f"\n[case] backward many tiles {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X, W, dY = (lattice(g, *sh, dt=dt).cuda() for sh in ((M, K), (K, N), (M, N)))
    _, _, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    dX, dW = lm.fp8_matmul_block_backward(dY, X, WqT, sT)
    assert torch.equal(dX, (dY.double() @ W.double().t()).float().to(dt))
    assert torch.equal(dW, (X.double().t() @ dY.double()).float().to(dt))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_matmul_random(M, K, N, dt):
    print(f"\n[case] matmul random {dt} {M}x{K}x{N}", flush=True)
    g = gen(M * 3 + K + N)
    X = outliers(g, randn(g, M, K)).to(dt)
    W = (randn(g, K, N) * 0.02 * torch.exp2(torch.randint(-3, 3, (K, 1), generator=g).float())).to(dt)
    Wq, s = lm.fp8_quantize_weight_block(W.cuda())
    Y = lm.fp8_matmul_block(X.cuda(), Wq, s)
    xh, what = ref.coded_rows(X)[0], ref.coded_weight(W)[0]
    y, err = ref.product(xh, what.t())
    ref.assert_close(Y, y, err, "Y")
    # far below the bound on the whole: the output's rounding (at most u of the norm), and the
    # dropped bits, which are independent from run to run of 8 products: about 2^-13 of the norm
    assert (Y.double().cpu() - y).norm() <= (ref.U[dt] + 2.0 ** -12) * y.norm()


@pytest.mark.parametrize("dt", DTS)
def test_matmul_rows_do_not_meet(dt):
    """A row that is not finite leaves the others as they were, bit for bit, whatever its place."""
    M, K, N = 37, 400, 264
    g = gen(5)
    X, W = randn(g, M, K).to(dt), (randn(g, K, N) * 0.02).to(dt)
    Wq, s = lm.fp8_quantize_weight_block(W.cuda())
    Y = lm.fp8_matmul_block(X.cuda(), Wq, s).cpu()
    for row, v in ((0, math.nan), (36, math.inf), (16, -math.inf)):
        X2 = X.clone()
        X2[row, 7] = v
        Y2 = lm.fp8_matmul_block(X2.cuda(), Wq, s).cpu()
        keep = torch.arange(M) != row
        assert torch.equal(Y2[keep], Y[keep])
        assert not torch.isfinite(Y2[row].float()).any()


@pytest.mark.parametrize("dt", DTS)
def test_matmul_far_scales(dt):
    """Rows and blocks at the ends of the type's range: the scales are applied without a
    detour through values that overflow or vanish."""
    M, K, N = 20, 256, 136
    g = gen(6)
    lo, hi = (-12, 8) if dt == torch.float16 else (-90, 90)
    X = lattice(g, M, K, dt=torch.float64)
    e = torch.linspace(lo, hi, M).round().double()
    X = (X * torch.exp2(e)[:, None]).to(dt)
    W = (lattice(g, K, N, dt=torch.float64) * 2.0 ** (-4 if dt == torch.float16 else -20)).to(dt)
    Wq, s = lm.fp8_quantize_weight_block(W.cuda())
    Y = lm.fp8_matmul_block(X.cuda(), Wq, s)
    assert torch.equal(Y.cpu(), (X.double() @ W.double()).float().to(dt))


def test_matmul_empty():
    Wq, s = lm.fp8_quantize_weight_block(torch.zeros(0, 64, dtype=torch.float16, device="cuda"))
    Y = lm.fp8_matmul_block(torch.zeros(5, 0, dtype=torch.float16, device="cuda"), Wq, s)
    assert Y.shape == (5, 64) and not Y.any()
    Wq, s = lm.fp8_quantize_weight_block(torch.zeros(64, 8, dtype=torch.float16, device="cuda"))
    assert lm.fp8_matmul_block(torch.zeros(0, 64, dtype=torch.float16, device="cuda"), Wq, s).shape == (0, 8)


def test_matmul_of_very_many_columns():
    """2^29 + 136 columns (64 GiB of codes): more than a few-row kernel's grid can have.  Whole numbers, so
    that pieces of the weight multiplied alone give the same bits."""
    N, K = (1 << 29) + 136, 16
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free device memory")
    print(f"\n[case] matmul very many columns {K}x{N}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    code = torch.arange(-3, 4, device="cuda").float().to(F8).view(torch.uint8)
    Wq = torch.zeros(N, 128, dtype=torch.uint8, device="cuda")
    step = 1 << 24
    for a in range(0, N, step):
        b = min(N, a + step)
        Wq[a:b, :K] = code[torch.randint(0, 7, (b - a, K), generator=g, device="cuda")]
    Wq, s = Wq.view(F8), torch.zeros(-(-N // 128), 4, dtype=torch.uint8, device="cuda")
    s[:, 0] = torch.randint(125, 130, (s.shape[0],), generator=g, device="cuda")
    s = s.view(E8)
    X = torch.randint(-3, 4, (2, K), generator=g, device="cuda").half()
    Y = lm.fp8_matmul_block(X, Wq, s)
    for a in (0, step, N // 2 // 128 * 128, (1 << 29) - 128, N - N % 128 - (1 << 20)):
        b = min(N, a + (1 << 20) + 8)
        part = lm.fp8_matmul_block(X, Wq[a:b], s[a // 128: -(-b // 128)])
        assert part.any() and torch.equal(Y[:, a:b], part), a
    del Wq, s, Y, part
    torch.cuda.empty_cache()


def trits(seed, *shape, dt=torch.float16):
    """-1, 0, 1 at random, on the GPU: sums of up to 2^24 products are exact in fp32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(dt)


# the longest sum, in each kernel; (2056 x 2056: tiles of 256 in parts, against rows of it alone)
@pytest.mark.parametrize("M,N", [(1, 8), (3, 2056), (20, 136), (64, 72), (130, 136), (300, 264), (2056, 2056)])
def test_matmul_longest_sum(M, N):
    K, dt = 1 << 22, torch.bfloat16
    print(f"\n[case] matmul longest sum {M}x{K}x{N}", flush=True)
    X, W = trits(M, M, K, dt=dt), trits(M + N, K, N, dt=dt)
    Wq, s = lm.fp8_quantize_weight_block(W)
    Y = lm.fp8_matmul_block(X, Wq, s)
    if M > 2000:
        want = torch.cat([lm.fp8_matmul_block(X[a: a + 128], Wq, s) for a in range(0, M, 128)])
    else:
        want = sum(X[:, a: a + (1 << 18)].double() @ W[a: a + (1 << 18)].double() for a in range(0, K, 1 << 18)).float().to(dt)
    assert Y.any() and torch.equal(Y, want)
    del X, W, Wq, s, Y, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,N", [(1 << 22, 144, 136), (1 << 22, 16, 8), (40, 1 << 22, 72), (40, 144, 1 << 22)])
def test_longest_sides_of_product_and_gradient(M, K, N):
    print(f"\n[case] longest side {M}x{K}x{N}", flush=True)
    dt = torch.float16
    X, W, dY = trits(1, M, K, dt=dt), trits(2, K, N, dt=dt), trits(3, M, N, dt=dt)
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    step = 1 << 18

    def product(a, b):  # the sum in pieces
        return sum(a[:, i: i + step].double() @ b[i: i + step].double() for i in range(0, a.shape[1], step)).float().to(dt)

    assert torch.equal(lm.fp8_matmul_block(X, Wq, s), product(X, W))
    dX, dW = lm.fp8_matmul_block_backward(dY, X, WqT, sT)
    assert torch.equal(dX, product(dY, W.t().contiguous()))
    assert torch.equal(dW, product(X.t().contiguous(), dY))
    del X, W, dY, Wq, s, WqT, sT, dX, dW
    torch.cuda.empty_cache()


def framed(shape, dt, fill=3.0):
    """(view, whole): a buffer of the shape between canaries."""
    n = math.prod(shape)
    whole = torch.full((n + 512,), fill, dtype=dt, device="cuda")
    return whole[256: 256 + n].view(shape), whole


def frame_untouched(whole, n, fill=3.0):
    return bool((whole[:256] == fill).all()) and bool((whole[256 + n:] == fill).all())


@pytest.mark.parametrize("M,K,N", [(1, 144, 72), (19, 272, 136), (70, 400, 264), (300, 1040, 520)])
def test_matmul_writes_its_output_alone(M, K, N):
    g = gen(7)
    X, W = randn(g, M, K).half().cuda(), randn(g, K, N).half().cuda()
    Wq, s = lm.fp8_quantize_weight_block(W)
    Y, yw = framed((M, N), torch.float16)
    nb = lm.fp8_matmul_block_workspace_bytes(M, K, N)
    ws, wsw = framed((nb,), torch.uint8, 90)
    lm.fp8_matmul_block(X, Wq, s, Y=Y, workspace=ws)
    torch.cuda.synchronize()
    assert frame_untouched(yw, M * N) and frame_untouched(wsw, nb, 90)
    # the workspace's old contents do not matter, and equal calls give equal bits
    ws.fill_(255)
    assert torch.equal(lm.fp8_matmul_block(X, Wq, s, workspace=ws), Y)


# ---- gradient

BACK = [(40, 264 * 16, 136), (2100, 272, 264), (300, 272, 4360), (24, 400, 6152), (1, 16, 8), (5, 144, 136), (128, 256, 128), (130, 272, 264), (333, 1040, 520), (64, 2064, 72), (700, 400, 1288)]


# (as above; the last one's weight gradient splits tiles of 256, the one before splits tiles of 128)
LARGE_BACK = [(200, 2064, 2056), (300, 4112, 4104), (5000, 144, 264), (12300, 2064, 2056)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", BACK + LARGE_BACK)
def test_backward_exact_lattice(M, K, N, dt):
    print(f"\n[case] backward lattice {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K + N)
    X, W, dY = lattice(g, M, K, dt=dt), lattice(g, K, N, dt=dt), lattice(g, M, N, dt=dt)
    _, _, WqT, sT = lm.fp8_quantize_weight_block(W.cuda(), transposed=True)
    dX, dW = lm.fp8_matmul_block_backward(dY.cuda(), X.cuda(), WqT, sT)
    assert torch.equal(dX.cpu(), (dY.double() @ W.double().t()).float().to(dt))
    assert torch.equal(dW.cpu(), (X.double().t() @ dY.double()).float().to(dt))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", BACK)
def test_backward_random(M, K, N, dt):
    print(f"\n[case] backward random {dt} {M}x{K}x{N}", flush=True)
    g = gen(M + K * 2 + N)
    X = outliers(g, randn(g, M, K)).to(dt)
    W = (randn(g, K, N) * 0.02).to(dt)
    dY = (randn(g, M, N) * 0.01 * torch.exp2(torch.randint(-4, 4, (M, 1), generator=g).float())).to(dt)
    _, _, WqT, sT = lm.fp8_quantize_weight_block(W.cuda(), transposed=True)
    dX, dW = lm.fp8_matmul_block_backward(dY.cuda(), X.cuda(), WqT, sT)
    x, err = ref.product(ref.coded_rows(dY)[0], ref.coded_weight(W)[0])
    ref.assert_close(dX, x, err, "dX")
    w, err = ref.product(ref.coded_rows(X.t())[0], ref.coded_rows(dY.t())[0])
    ref.assert_close(dW, w, err, "dW")


def test_backward_against_differences():
    """<dY, Y(X + D) - Y(X)> = <dX, D> and <dY, Y(W + D) - Y(W)> = <dW, D>: on whole numbers
    -1 .. 1 the codes, the outputs and both gradients are exact, and Y is linear."""
    M, K, N, dt = 70, 272, 136, torch.float16
    g = gen(9)

    def trits(*shape):
        return torch.randint(-1, 2, shape, generator=g).to(dt)

    X, W, dY, DX, DW = trits(M, K), trits(K, N), trits(M, N), trits(M, K), trits(K, N)

    def forward(X, W):
        return lm.fp8_matmul_block(X.cuda(), *lm.fp8_quantize_weight_block(W.cuda())).cpu().double()

    _, _, WqT, sT = lm.fp8_quantize_weight_block(W.cuda(), transposed=True)
    dX, dW = (t.cpu().double() for t in lm.fp8_matmul_block_backward(dY.cuda(), X.cuda(), WqT, sT))
    Y = forward(X, W)
    assert (dY.double() * (forward(X + DX, W) - Y)).sum() == (dX * DX.double()).sum()
    assert (dY.double() * (forward(X, W + DW) - Y)).sum() == (dW * DW.double()).sum()


def test_backward_one_of_the_two_and_empty_sums():
    M, K, N = 130, 272, 136
    g = gen(10)
    X, W, dY = randn(g, M, K).half().cuda(), randn(g, K, N).half().cuda(), randn(g, M, N).half().cuda()
    _, _, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    dX, dW = lm.fp8_matmul_block_backward(dY, X, WqT, sT)
    a, none = lm.fp8_matmul_block_backward(dY, None, WqT, sT, need_dw=False)
    assert none is None and torch.equal(a, dX)
    none, b = lm.fp8_matmul_block_backward(dY, X, None, None, need_dx=False)
    assert none is None and torch.equal(b, dW)
    assert lm.fp8_matmul_block_backward(dY, None, None, None, need_dx=False, need_dw=False) == (None, None)
    e, z = lm.fp8_matmul_block_backward(dY[:0], X[:0], WqT, sT)  # no tokens
    assert e.shape == (0, K) and z.shape == (K, N) and not z.any()


def test_product_and_gradient_under_autograd():
    """The calls are not recorded; a torch.autograd.Function of the two is, and its gradients are those of
    the product (exact here: whole numbers)."""
    M, K, N, dt = 40, 272, 136, torch.bfloat16
    g = gen(15)
    X, W, dY = (lattice(g, *sh, dt=dt).cuda() for sh in ((M, K), (K, N), (M, N)))

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W):
            Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
            ctx.save_for_backward(X, WqT, sT)
            return lm.fp8_matmul_block(X, Wq, s)

        @staticmethod
        def backward(ctx, dY):
            X, WqT, sT = ctx.saved_tensors
            return lm.fp8_matmul_block_backward(dY.contiguous(), X, WqT, sT, need_dx=ctx.needs_input_grad[0],
                                                need_dw=ctx.needs_input_grad[1])

    X.requires_grad_()
    W.requires_grad_()
    Y = Product.apply(X, W)
    Y.backward(dY)
    x, w, dy = X.detach().double(), W.detach().double(), dY.double()
    assert torch.equal(Y, (x @ w).float().to(dt))
    assert torch.equal(X.grad, (dy @ w.t()).float().to(dt)) and torch.equal(W.grad, (x.t() @ dy).float().to(dt))
    Wq, s = lm.fp8_quantize_weight_block(W)
    plain = lm.fp8_matmul_block(X, Wq, s)
    assert not plain.requires_grad and torch.equal(plain, Y)


@pytest.mark.parametrize("M,K,N", [(3, 144, 72), (200, 400, 264)])
def test_backward_writes_its_outputs_alone(M, K, N):
    g = gen(11)
    X, W, dY = randn(g, M, K).bfloat16().cuda(), randn(g, K, N).bfloat16().cuda(), randn(g, M, N).bfloat16().cuda()
    _, _, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    dX, xw = framed((M, K), torch.bfloat16)
    dW, ww = framed((K, N), torch.bfloat16)
    nb = lm.fp8_matmul_block_backward_workspace_bytes(M, K, N)
    ws, wsw = framed((nb,), torch.uint8, 90)
    lm.fp8_matmul_block_backward(dY, X, WqT, sT, dX=dX, dW=dW, workspace=ws)
    torch.cuda.synchronize()
    assert frame_untouched(xw, M * K) and frame_untouched(ww, K * N) and frame_untouched(wsw, nb, 90)
    ws.fill_(255)
    a, b = lm.fp8_matmul_block_backward(dY, X, WqT, sT, workspace=ws)
    assert torch.equal(a, dX) and torch.equal(b, dW)


# ---- values that are not finite

NOT_FINITE = [math.nan, math.inf, -math.inf]


def is_nan_code(q):
    return (q.view(torch.uint8) & 0x7f) == 0x7f


def blocks_zeroed(W, at):
    W = W.clone()
    for k, n in at:
        W[k // 128 * 128: k // 128 * 128 + 128, n // 128 * 128: n // 128 * 128 + 128] = 0
    return W


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("v", NOT_FINITE)
def test_quantize_weight_not_finite(v, dt):
    """Its own code is NaN, its block's other values vanish beside it, no other block changes."""
    K, N, at = 400, 264, [(5, 7), (391, 263)]
    g = gen(21)
    W = (randn(g, K, N) * 0.02).to(dt)
    W2 = W.clone()
    for k, n in at:
        W2[k, n] = v
    rest = lm.fp8_quantize_weight_block(blocks_zeroed(W, at).cuda(), transposed=True)
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W2.cuda(), transposed=True)
    nan = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    for k, n in at:
        nan[n, k] = True
    assert torch.equal(is_nan_code(Wq)[:, :K], nan) and torch.equal(is_nan_code(WqT)[:, :N], nan.t())
    assert not is_nan_code(Wq)[:, K:].any() and not is_nan_code(WqT)[:, N:].any()
    for got, want, own in ((Wq, rest[0], nan), (WqT, rest[2], nan.t())):
        keep = torch.ones(got.shape, dtype=torch.bool, device="cuda")
        keep[:, :own.shape[1]] = ~own
        assert torch.equal(got.float()[keep], want.float()[keep])
    for got, want, blocks in ((s, rest[1], [(n, k) for k, n in at]), (sT, rest[3], at)):
        keep = torch.ones(got.shape, dtype=torch.bool)
        for r, c in blocks:
            keep[r // 128, c // 128] = False
        assert torch.equal(u8(got)[keep], u8(want)[keep])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M", [2, 20, 100, 12000, 24000])
def test_matmul_weights_not_finite(M, dt):
    K, N, at = 400, 264, [(5, 7), (391, 263)]
    print(f"\n[case] matmul weights not finite {dt} {M}x{K}x{N}", flush=True)
    g = gen(22)
    X, W = randn(g, M, K).to(dt).cuda(), (randn(g, K, N) * 0.02).to(dt)
    W2 = W.clone()
    for (k, n), v in zip(at, NOT_FINITE):
        W2[k, n] = v
    want = lm.fp8_matmul_block(X, *lm.fp8_quantize_weight_block(blocks_zeroed(W, at).cuda()))
    Y = lm.fp8_matmul_block(X, *lm.fp8_quantize_weight_block(W2.cuda()))
    cols = torch.zeros(N, dtype=torch.bool)
    cols[[n for _, n in at]] = True
    assert not torch.isfinite(Y[:, cols].float()).any() and torch.equal(Y[:, ~cols], want[:, ~cols])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K,N", [(70, 400, 264), (300, 272, 4360), (5000, 144, 264), (4400, 4240, 1040)])
def test_backward_not_finite(M, K, N, dt):
    print(f"\n[case] backward not finite {dt} {M}x{K}x{N}", flush=True)
    g = gen(23)
    X, W, dY = randn(g, M, K).to(dt).cuda(), (randn(g, K, N) * 0.02).to(dt), randn(g, M, N).to(dt).cuda()
    w = lm.fp8_quantize_weight_block(W.cuda(), transposed=True)[2:]
    dX, dW = lm.fp8_matmul_block_backward(dY, X, *w)
    for v in NOT_FINITE:
        m, k, n = M - 1, K - 1, N - 1
        Y2, X2, W2 = dY.clone(), X.clone(), W.clone()
        Y2[m, n] = X2[0, k] = W2[0, n] = v
        a, b = lm.fp8_matmul_block_backward(Y2, X, *w)
        assert not torch.isfinite(a[m].float()).any() and torch.equal(a[:m], dX[:m]), v
        assert not torch.isfinite(b[:, n].float()).any() and torch.equal(b[:, :n], dW[:, :n]), v
        a, b = lm.fp8_matmul_block_backward(dY, X2, *w)
        assert torch.equal(a, dX) and not torch.isfinite(b[k].float()).any() and torch.equal(b[:k], dW[:k]), v
        w2 = lm.fp8_quantize_weight_block(W2.cuda(), transposed=True)[2:]
        zeroed = lm.fp8_quantize_weight_block(blocks_zeroed(W, [(0, n)]).cuda(), transposed=True)[2:]
        a, _ = lm.fp8_matmul_block_backward(dY, None, *w2, need_dw=False)
        want, _ = lm.fp8_matmul_block_backward(dY, None, *zeroed, need_dw=False)
        assert not torch.isfinite(a[:, 0].float()).any() and torch.equal(a[:, 1:], want[:, 1:]), v


# ---- mixture of experts

def experts(g, E, H, I, dt):
    up = [lm.fp8_quantize_weight_block((randn(g, H, 2 * I) * 0.05).to(dt).cuda()) for _ in range(E)]
    down = [lm.fp8_quantize_weight_block((randn(g, I, H) * 0.05).to(dt).cuda()) for _ in range(E)]

    def stacked(ts, t):
        return torch.stack([x.view(torch.uint8) for x in ts]).view(t)

    return (stacked([q for q, _ in up], F8), stacked([s for _, s in up], E8), stacked([q for q, _ in down], F8),
            stacked([s for _, s in down], E8))


def moe_check(X, logits, w, k, renormalize):
    W13q, s13, W2q, s2 = w
    E, I, (T, H) = W13q.shape[0], W13q.shape[1] // 2, X.shape
    Y, ids, p = lm.fp8_moe_block(X.cuda(), logits.cuda(), *w, top_k=k, renormalize=renormalize)
    W13 = torch.stack([ref.weight_values(W13q[e].cpu(), s13[e].cpu(), H) for e in range(E)])
    W2 = torch.stack([ref.weight_values(W2q[e].cpu(), s2[e].cpu(), I) for e in range(E)])
    y, err, rids, rp = ref.moe(X, logits, W13, W2, k, renormalize)
    assert torch.equal(ids.cpu(), rids)
    # exp and a sum of at most 1024 of them, a division: 64 steps are ample for top_k <= 16,
    # and E steps more where all experts are summed
    assert ((p.cpu().double() - rp).abs() <= (64 + (0 if renormalize else E)) * 2.0 ** -24 * rp + 2.0 ** -140).all()
    ref.assert_close(Y, y, err + y.abs() * (64 + E) * 2.0 ** -24, "y")
    return Y, ids, p


MOE = [(1, 4352, 144, 8, 2), (12, 4112, 80, 9, 2), (3, 272, 1040, 600, 4), (70, 272, 144, 64, 5), (128, 144, 272, 16, 2),
       (50, 4128, 64, 6, 2), (20, 144, 80, 3, 2), (2, 64, 33 * 128, 520, 16), (128, 64, 48, 1024, 16),
       (1, 16, 16, 1, 1), (1, 256, 128, 8, 2), (1, 272, 144, 64, 8), (2, 528, 400, 12, 3), (4, 384, 272, 5, 5),
       (9, 256, 144, 70, 4), (17, 272, 208, 6, 2), (40, 144, 272, 9, 4), (64, 256, 128, 130, 8), (128, 128, 144, 4, 2),
       (33, 128, 128, 3, 1), (5, 1040, 64, 20, 16), (30, 528, 4112, 40, 1), (20, 2064, 4112, 8, 1)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,I,E,k", MOE)
def test_moe(T, H, I, E, k, dt):
    for renormalize in (True, False):
        print(f"\n[case] moe {dt} T={T} H={H} I={I} E={E} k={k} renormalize={renormalize}", flush=True)
        g = gen(T + H + I + E + k)
        X = randn(g, T, H).to(dt)
        logits = 2 * randn(g, T, E)
        moe_check(X, logits, experts(g, E, H, I, dt), k, renormalize)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T", [3, 20, 100])
def test_moe_masks_ties_and_odd_logits(T, dt):
    """Closed experts, rows of padding, ties, NaN and infinities in the logits; every token on one
    expert, and an expert without tokens."""
    H, I, E, k = 144, 80, 11, 3
    g = gen(T)
    X = randn(g, T, H).to(dt)
    w = experts(g, E, H, I, dt)
    l = 2 * randn(g, T, E)
    l[torch.rand(T, E, generator=g) < 0.4] = -math.inf
    l[0] = -math.inf           # no expert at all
    l[1] = 0.5                 # all equal
    l[2] = -math.inf
    l[2, 7] = -3.0             # a single one
    l[T - 1] = -math.inf
    if T > 10:
        l[3, 4] = math.nan
        l[4] = math.nan
        l[5, 2] = math.inf
        l[6, 2] = l[6, 5] = math.inf
        l[7] = torch.finfo(torch.float32).min
        l[8] = torch.arange(E).float() * 90
        X[0] = math.nan        # padding may hold anything
    for renormalize in (True, False):
        Y, ids, p = moe_check(X if T <= 10 else torch.where(torch.isnan(X), torch.zeros_like(X), X), l, w, k, renormalize)
        assert not Y[0].any() and (ids[0] == -1).all() and not p[0].any()
        if T > 10:
            Y2, ids2, p2 = lm.fp8_moe_block(X.cuda(), l.cuda(), *w, top_k=k, renormalize=renormalize)
            assert torch.equal(Y2, Y) and torch.equal(ids2, ids) and torch.equal(p2, p)
    one = torch.full((T, E), -1.0)
    one[:, 6] = 1.0
    moe_check(torch.nan_to_num(X), one, w, 1, True)


# many tokens an expert in a large layer: two and four pieces of 16 tokens, up to 64 tokens and more
@pytest.mark.parametrize("T,H,I,E,k,dt", [(60, 4112, 2064, 8, 2, DTS[0]), (64, 4112, 2064, 8, 5, DTS[1]),
                                          (128, 4112, 2064, 8, 2, DTS[0]), (128, 2064, 1040, 30, 6, DTS[1]),
                                          (20, 32768, 2064, 1, 1, DTS[1])])
def test_moe_many_tokens(T, H, I, E, k, dt):
    print(f"\n[case] moe many {dt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    g = gen(T + H + E)
    X = randn(g, T, H).to(dt)
    w = experts(g, E, H, I, dt)
    l = 2 * randn(g, T, E)
    moe_check(X, l, w, k, True)
    l[:, E // 2] += 40  # every token on one expert
    l[torch.rand(T, E, generator=g) < 0.3] = -math.inf
    l[[1, T - 1]] = -math.inf  # rows of padding
    moe_check(X, l, w, k, False)


@pytest.mark.parametrize("seed", range(16))
def test_moe_sweep(seed):
    g = gen(1000 + seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    T, E = rnd(1, 128 if seed % 2 else 12), rnd(1, 40)
    k, H, I, dt = rnd(1, min(E, 8)), 16 * rnd(1, 40), 16 * rnd(1, 30), DTS[seed % 2]
    print(f"\n[case] moe sweep {dt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    l = 2 * randn(g, T, E)
    l[torch.rand(T, E, generator=g) < 0.1 * (seed % 4)] = -math.inf
    moe_check(randn(g, T, H).to(dt), l, experts(g, E, H, I, dt), k, bool(rnd(0, 1)))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T", [0, 1, 40, 128])
def test_moe_without_inner_columns_or_tokens(T, dt):
    """I = 0: the choices stand, the output is zero; T = 0: nothing."""
    H, E, k = 48, 3, 2
    g = gen(T)
    X, l = randn(g, T, H).to(dt).cuda(), randn(g, T, E).cuda()
    empty = [torch.empty(E, 0, 128, dtype=F8, device="cuda"), torch.empty(E, 0, 4, dtype=E8, device="cuda"),
             torch.empty(E, H, 0, dtype=F8, device="cuda"), torch.empty(E, 1, 0, dtype=E8, device="cuda")]
    Y = torch.full((T, H), 7.0, dtype=dt, device="cuda")
    Y, ids, p = lm.fp8_moe_block(X, l, *empty, top_k=k, Y=Y)
    assert Y.shape == (T, H) and not Y.any()
    assert torch.equal(ids.long(), l.topk(k).indices) and torch.allclose(p, torch.softmax(l.topk(k).values, -1), atol=1e-6)


# each pair of forms; H of a number of groups that the light form's four waves do not share evenly
NON_FINITE = [(1, 2064, 144, 64, 8), (3, 272, 1040, 60, 4), (12, 272, 144, 11, 4), (1, 4352, 144, 8, 2), (70, 272, 144, 64, 5),
              (30, 528, 4112, 40, 1), (50, 4128, 64, 6, 2), (128, 144, 272, 16, 2), (40, 144, 272, 9, 4), (128, 144, 48, 700, 16),
              (60, 4112, 2064, 8, 2)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,I,E,k", NON_FINITE)
def test_moe_non_finite_values_stay_where_they_are(T, H, I, E, k, dt):
    """NaN among an expert's weights or a token's values reaches the outputs whose sums it enters;
    every other output keeps its bits."""
    print(f"\n[case] moe non-finite {dt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    g = gen(T + H + I + E + k + 1)
    X, l, w = randn(g, T, H).to(dt).cuda(), 2 * randn(g, T, E), experts(g, E, H, I, dt)
    l[0::2, 0], l[1::2, 0] = -math.inf, 50.0  # the odd tokens alone meet expert 0
    l = l.cuda()
    Y, ids, p = lm.fp8_moe_block(X, l, *w, top_k=k)
    meets = (ids == 0).any(1)
    assert not meets[0::2].any() and meets[1::2].all() and torch.isfinite(Y.float()).all()

    def run(X, w):
        Y2, ids2, p2 = lm.fp8_moe_block(X, l, *w, top_k=k)
        assert torch.equal(ids2, ids) and torch.equal(p2, p)
        return Y2

    def with_nan(q, at):
        q = q.view(torch.uint8).clone()
        q[at] = 0x7f
        return q.view(F8)

    # the first expert's first line of gate weights, and the end of its last up row
    for at in ((0, 0, slice(0, 128)), (0, 2 * I - 1, slice(H - 16, H))):
        Y2 = run(X, (with_nan(w[0], at),) + w[1:])
        assert torch.equal(Y2[~meets], Y[~meets]), at
        assert not torch.isfinite(Y2[meets].float()).any(), at
    # a row of its down weights is an output column of its tokens
    for row in (0, H - 1):
        Y2 = run(X, w[:2] + (with_nan(w[2], (0, row, slice(0, 16))), w[3]))
        keep = torch.ones_like(Y, dtype=torch.bool)
        keep[meets, row] = False
        assert torch.equal(Y2[keep], Y[keep]) and not torch.isfinite(Y2[~keep].float()).any(), row
    # a token's own values
    for t in {0, T - 1}:
        X2 = X.clone()
        X2[t, H - 1] = math.nan
        Y2 = run(X2, w)
        assert torch.equal(Y2[torch.arange(T) != t], Y[torch.arange(T) != t]) and not torch.isfinite(Y2[t].float()).any()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,H,I,E,k", [(8, 16, 128, 2, 2), (8, 272, 272, 16, 16), (7, 144, 2064, 5, 4), (16, 272, 128, 40, 6)])
def test_moe_tokens_of_both_entries_at_once(T, H, I, E, k, dt):
    """The light second launch takes two experts at a time: here their tokens are the same ones, so each
    token's sum is added to from both, in the same step and in neighbouring ones."""
    print(f"\n[case] moe both entries {dt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    g = gen(T * H + I + E)
    l = randn(g, T, E)
    l[:, k:] = -math.inf  # every token on the first k experts
    moe_check(randn(g, T, H).to(dt), l, experts(g, E, H, I, dt), k, True)


@pytest.mark.parametrize("T,H,I,E,k", [(2, 272, 144, 8, 2), (40, 144, 272, 9, 4), (50, 4128, 64, 6, 2), (60, 4112, 2064, 8, 2)])
@pytest.mark.parametrize("which", [0, 2])
def test_moe_smallest_scales(which, T, H, I, E, k):
    """bf16, gate and up (0) or down (2) weights at the smallest scales: converted weights around bf16's
    smallest numbers, and every small code at 2^-124, as exact as anywhere."""
    print(f"\n[case] moe smallest scales {which} T={T} H={H} I={I} E={E} k={k}", flush=True)
    g, dt = gen(T + H + I + which), torch.bfloat16
    X, l, w = randn(g, T, H), 2 * randn(g, T, E), list(experts(g, E, H, I, dt))
    shape = (H, 2 * I) if which == 0 else (I, H)
    tiny = [lm.fp8_quantize_weight_block((randn(g, *shape) * 2.0 ** -127).to(dt).cuda()) for _ in range(E)]
    w[which] = torch.stack([q.view(torch.uint8) for q, _ in tiny]).view(F8)
    w[which + 1] = torch.stack([s.view(torch.uint8) for _, s in tiny]).view(E8)
    assert not w[which + 1].view(torch.uint8).any()  # 2^-127, all of them
    moe_check((X * (2.0 ** 122 if which == 0 else 1)).to(dt), l, w, k, True)
    q = torch.randint(0, 16, w[which].shape, generator=g) + 128 * torch.randint(0, 2, w[which].shape, generator=g)
    q[:, :, shape[0]:] = 0
    w[which] = q.to(torch.uint8).cuda().view(F8)
    s = w[which + 1].view(torch.uint8).clone()
    s[:, :, :-(-shape[0] // 128)] = 127 - 124
    w[which + 1] = s.view(E8)
    moe_check((X * (2.0 ** 122 if which == 0 else 1)).to(dt), l, w, k, False)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 1 << 22, 16, 1, 1), (2, 1 << 22, 16, 5, 2), (20, 1 << 22, 16, 2, 1), (1, 16, 1 << 21, 8, 2),
                                       (70, 48, 1 << 21, 3, 2), (128, 16, 1 << 20, 2, 2), (12, 16, 1 << 20, 9, 2)])
@pytest.mark.parametrize("dt", DTS)
def test_moe_longest_sides(dt, T, H, I, E, k):
    """The longest rows, with values at 48 features and inner columns alone, both ends among them: a sum of
    zeros is exact, so the reference and its bound are those of the 48."""
    print(f"\n[case] moe longest sides {dt} T={T} H={H} I={I} E={E} k={k}", flush=True)
    g = gen(T + H + I + E)

    def some(n):
        at = torch.cat([torch.arange(8), torch.randint(0, n, (32,), generator=g), n - 1 - torch.arange(8)])
        return at.unique()

    def codes(*shape):  # magnitudes 0.5 to 1.875
        return (torch.randint(0x30, 0x40, shape, generator=g) + 128 * torch.randint(0, 2, shape, generator=g)).to(torch.uint8).cuda()

    hs, cs = some(H), some(I)
    x = randn(g, T, len(hs)).to(dt)
    X = torch.zeros(T, H, dtype=dt)
    X[:, hs] = x
    rows = torch.cat([cs, I + cs])
    c13, c2 = codes(E, len(rows), len(hs)), codes(E, H, len(cs))
    W13 = torch.zeros(E, 2 * I, ref.pitch(H), dtype=torch.uint8, device="cuda")
    W2 = torch.zeros(E, H, ref.pitch(I), dtype=torch.uint8, device="cuda")
    for e in range(E):
        W13[e, rows.cuda()[:, None], hs.cuda()] = c13[e]
        W2[e][:, cs.cuda()] = c2[e]
    s13 = torch.zeros(E, -(-2 * I // 128), ref.sp(H), dtype=torch.uint8)
    s2 = torch.zeros(E, -(-H // 128), ref.sp(I), dtype=torch.uint8)
    s13[:, :, : -(-H // 128)] = torch.randint(125, 128, (E, s13.shape[1], -(-H // 128)), generator=g, dtype=torch.uint8)
    s2[:, :, : -(-I // 128)] = torch.randint(125, 128, (E, s2.shape[1], -(-I // 128)), generator=g, dtype=torch.uint8)
    l = 2 * randn(g, T, E)
    Y, ids, p = lm.fp8_moe_block(X.cuda(), l.cuda(), W13.view(F8), s13.cuda().view(E8), W2.view(F8), s2.cuda().view(E8), top_k=k)
    v13 = torch.exp2(s13.double() - 127)[:, rows // 128][:, :, hs // 128] * c13.cpu().view(F8).float().double()
    v2 = torch.exp2(s2.double() - 127)[:, torch.arange(H) // 128][:, :, cs // 128] * c2.cpu().view(F8).float().double()
    y, err, rids, rp = _moe_of(x, l, v13, v2, k)
    assert torch.equal(ids.cpu(), rids)
    assert ((p.cpu().double() - rp).abs() <= 64 * 2.0 ** -24 * rp).all()
    ref.assert_close(Y, y, err + y.abs() * 128 * 2.0 ** -24, "y")
    del W13, W2, c13, c2, Y
    torch.cuda.empty_cache()


def _moe_of(x, l, v13, v2, k):
    """fp8_ref.moe (renormalized), and its bound, for outputs of another width than the inputs."""
    t, I = x.dtype, v2.shape[2]
    ids, p = ref.route(l, k, True)
    y = torch.zeros(x.shape[0], v2.shape[1], dtype=torch.float64)
    err = torch.zeros_like(y)
    for i, j in (ids >= 0).nonzero().tolist():
        e, xi = int(ids[i, j]), x[i].double()
        (g, u), (dg, du) = (v13[e] @ xi).split(I), (x.shape[1] * 2.0 ** -23 * (v13[e].abs() @ xi.abs())).split(I)
        h = g * torch.sigmoid(g) * u
        hr = h.to(torch.float32).to(t).double()
        dh = 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + 16 * 2.0 ** -23 * h.abs()
        dh = dh + (hr - h).abs() + 2 * ref.U[t] * h.abs() + ref.TINY[t]
        y[i] += p[i, j] * (v2[e] @ hr)
        err[i] += p[i, j] * (v2[e].abs() @ dh + (I + 64) * 2.0 ** -23 * (v2[e].abs() @ (hr.abs() + dh)))
    return y, err, ids, p


def test_moe_writes_its_outputs_alone():
    T, H, I, E, k = 7, 272, 144, 6, 2
    g = gen(12)
    X, logits, w = randn(g, T, H).half().cuda(), randn(g, T, E).cuda(), experts(g, E, H, I, torch.float16)
    Y, yw = framed((T, H), torch.float16)
    nb = lm.fp8_moe_block_workspace_bytes(T, H, I, E, k)
    ws, wsw = framed((nb,), torch.uint8, 90)
    lm.fp8_moe_block(X, logits, *w, top_k=k, Y=Y, workspace=ws)
    torch.cuda.synchronize()
    assert frame_untouched(yw, T * H) and frame_untouched(wsw, nb, 90)
    ws.fill_(255)
    assert torch.equal(lm.fp8_moe_block(X, logits, *w, top_k=k, workspace=ws)[0], Y)


# ---- together, captured, and on another stream

def block_forward(X, gate, proj, moe_w, k):
    """A projection, then the expert layer on its output: the operators as a decoding step uses them."""
    Y = lm.fp8_matmul_block(X, *proj)
    return lm.fp8_moe_block(Y, (Y.float() @ gate), *moe_w, top_k=k)


@pytest.mark.parametrize("T", [1, 6, 48])
def test_together_captured_and_replayed(T):
    K, H, I, E, k = 272, 256, 144, 12, 3
    g = gen(T)
    dt = torch.bfloat16
    proj = lm.fp8_quantize_weight_block((randn(g, K, H) * 0.05).to(dt).cuda())
    gate, moe_w = (randn(g, H, E) * 0.2).cuda(), experts(g, E, H, I, dt)
    X = randn(g, T, K).to(dt).cuda()
    block_forward(X, gate, proj, moe_w, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block_forward(X, gate, proj, moe_w, k)
    for r in range(4):
        X.copy_(randn(g, T, K).to(dt))
        want = block_forward(X, gate, proj, moe_w, k)
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), r


def test_two_captured_graphs_and_a_training_step():
    M, K, N = 130, 272, 264
    g = gen(13)
    W = (randn(g, K, N) * 0.05).half().cuda()
    X, dY = randn(g, M, K).half().cuda(), randn(g, M, N).half().cuda()

    def step():
        Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
        Y = lm.fp8_matmul_block(X, Wq, s)
        return (Y,) + lm.fp8_matmul_block_backward(dY, X, WqT, sT)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for r in range(3):
        X.copy_(randn(g, M, K).half())
        W.copy_((randn(g, K, N) * 0.05).half())
        want = step()
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b), r


def test_on_another_stream():
    M, K, N = 40, 272, 264
    g = gen(14)
    X, W = randn(g, M, K).half().cuda(), randn(g, K, N).half().cuda()
    Wq, s = lm.fp8_quantize_weight_block(W)
    want = lm.fp8_matmul_block(X, Wq, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [lm.fp8_matmul_block(X, Wq, s, stream=side if i % 2 else side.cuda_stream) for i in range(8)]
    side.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert torch.cuda.current_stream() != side


# ---- calls whose sums are split over workgroups: what the workspace held before, graphs that share
# one, calls at the same time with one each

def split_call(op, sizes):
    """f(workspace) -> outputs, and the workspace's bytes"""
    g = gen(sum(sizes))
    dt = torch.bfloat16
    if op == "moe":
        T, H, I, E, k = sizes
        X, l, w = randn(g, T, H).to(dt).cuda(), (2 * randn(g, T, E)).cuda(), experts(g, E, H, I, dt)
        return (lambda ws: lm.fp8_moe_block(X, l, *w, top_k=k, workspace=ws)), lm.fp8_moe_block_workspace_bytes(T, H, I, E, k)
    M, K, N = sizes
    X, W = randn(g, M, K).to(dt).cuda(), randn(g, K, N).to(dt).cuda()
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    if op == "matmul":
        return (lambda ws: (lm.fp8_matmul_block(X, Wq, s, workspace=ws),)), lm.fp8_matmul_block_workspace_bytes(M, K, N)
    dY = randn(g, M, N).to(dt).cuda()
    return (lambda ws: lm.fp8_matmul_block_backward(dY, X, WqT, sT, workspace=ws)), lm.fp8_matmul_block_backward_workspace_bytes(M, K, N)


@pytest.mark.parametrize("op,sizes", [
    ("matmul", (16, 4240, 264)), ("matmul", (100, 4240, 264)), ("matmul", (300, 8208, 520)), ("matmul", (1200, 12304, 4104)),
    ("backward", (5000, 144, 264)), ("backward", (130, 272, 8200)), ("moe", (70, 272, 144, 64, 5)), ("moe", (128, 144, 272, 16, 2)),
    ("moe", (2, 64, 4224, 520, 16)), ("moe", (60, 4112, 2064, 8, 2)),
])
def test_split_sums_and_their_workspaces(op, sizes):
    print(f"\n[case] split {op} {sizes}", flush=True)
    f, nb = split_call(op, sizes)
    want = f(None)
    ws, whole = framed((nb,), torch.uint8, 90)
    for fill in (255, 0, 129):
        ws.fill_(fill)
        for a, b in zip(f(ws), want):
            assert torch.equal(a, b), fill
    assert frame_untouched(whole, nb, 90)
    # two graphs with one workspace, replayed in turn
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f(ws)
        graphs.append((graph, out))
    for r in range(3):
        ws.fill_(255)
        for graph, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b), r
    # two streams at once, a workspace each
    sides = [(torch.cuda.Stream(), torch.full((nb,), 255, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for side, own in sides:
            with torch.cuda.stream(side):
                outs.append(f(own))
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# ---- what the binding refuses

def test_refusals_of_gpu_tensors():
    W = torch.zeros(272, 264, dtype=torch.float16, device="cuda")
    X, dY = torch.zeros(5, 272, dtype=torch.float16, device="cuda"), torch.zeros(5, 264, dtype=torch.float16, device="cuda")
    Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
    T, H, I, E = 5, 272, 144, 4
    w = experts(gen(1), E, H, I, torch.float16)
    l = torch.zeros(T, E, device="cuda")
    with pytest.raises(TypeError):
        lm.fp8_quantize_weight_block(W.float())
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(X.float(), Wq, s)
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(X, Wq.view(torch.int8), s)
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(X, Wq, s.cpu())
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(X, Wq, s, Y=dY.bfloat16())
    with pytest.raises(TypeError):
        lm.fp8_moe_block(X, l.half(), *w, top_k=2)
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(X, Wq, s, workspace=torch.zeros(1 << 20, device="cuda"))
    with pytest.raises(ValueError):
        lm.fp8_quantize_weight_block(W.t())
    with pytest.raises(ValueError):
        lm.fp8_matmul_block(X[:, ::2], Wq, s)
    with pytest.raises(ValueError):
        lm.fp8_matmul_block(X[0], Wq, s)
    with pytest.raises(lm.LLMInt8Error):  # 264 features: no multiple of 16
        lm.fp8_matmul_block(dY, Wq, s)
    with pytest.raises(ValueError):
        lm.fp8_matmul_block(X, Wq, s[:1])
    with pytest.raises(ValueError):
        lm.fp8_matmul_block(X, Wq, s, Y=X)
    with pytest.raises(ValueError):
        lm.fp8_matmul_block_backward(dY, X[:4], WqT, sT)
    with pytest.raises(ValueError):
        lm.fp8_matmul_block_backward(dY, X, Wq, sT)
    with pytest.raises(ValueError):
        lm.fp8_moe_block(X, l[:3], *w, top_k=2)
    with pytest.raises(ValueError):
        lm.fp8_moe_block(X, l, *w, top_k=5)
    with pytest.raises(ValueError):
        lm.fp8_moe_block(X, l, *w, top_k=0)
    with pytest.raises(ValueError):
        lm.fp8_moe_block(X, l, w[0][:3], *w[1:], top_k=2)
    with pytest.raises(ValueError):
        lm.fp8_moe_block(X, l, w[0].transpose(1, 2), *w[1:], top_k=2)
    with pytest.raises(lm.LLMInt8Error):
        lm.fp8_moe_block(X, l, *w, top_k=2, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lm.LLMInt8Error):  # the output is an input
        lm.fp8_matmul_block(torch.zeros(264, 272, dtype=torch.float16, device="cuda"), Wq, s,
                            workspace=Wq.view(torch.uint8).view(-1))
    torch.cuda.synchronize()
