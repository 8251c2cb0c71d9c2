"""The root-mean-square norm and its gradient on the GPU against the 64-bit reference (mxfp4_ref), its
codes against the products' own, and a layer's run of them together; captured, in place, on another
stream, in caller-owned buffers between canaries."""
import math

import pytest
import torch

import int8_quantized_matmul_rowwise_amd as lm
from tests import fp8_ref
from tests import mxfp4_ref as ref
from tests.test_fp8_gpu import frame_untouched, framed, gen, outliers, randn, u8

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16]
EPS = 1e-5
# a wave, several, pieces of 8 columns one to four a thread, and rows longer than registers
SHAPES = [(1, 16), (3, 64), (2, 144), (37, 528), (5, 1040), (130, 2064), (1, 4096), (9, 8192), (3, 8208), (2, 16400), (2, 32784), (3, 65536), (2, 65552), (1, 131088)]
BACK = [(1, 16), (3, 64), (70, 144), (333, 1040), (5, 4096), (600, 4112), (9, 8208), (520, 16400), (3, 32768), (3, 32784), (70, 65552)]


def inputs(M, K, dt, seed=0):
    g = gen(M + 7 * K + seed)
    X = outliers(g, randn(g, M, K)) if K > 128 else randn(g, M, K)
    if M > 2:
        X[1] = 0
    R = 2 * randn(g, M, K)
    if M > 4:
        R[1] = 0  # a row of zeros
    w = 1 + 0.2 * randn(g, K)
    return X.to(dt), R.to(dt), w.to(dt), g


def summed(X, R):
    return (X.float() + R.float()).to(X.dtype)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm(M, K, dt):
    print(f"\n[case] rmsnorm {dt} {M}x{K}", flush=True)
    X, R, w, _ = inputs(M, K, dt)
    for res in (None, R):
        Y, H = lm.rmsnorm(X.cuda(), w.cuda(), residual=None if res is None else res.cuda(), eps=EPS)
        h = X if res is None else summed(X, R)
        assert (H is None) == (res is None) and (H is None or torch.equal(H.cpu(), h))
        want, rel = ref.norm(h.double(), w.double(), EPS)
        ref.assert_close(Y, want, rel * want.abs(), "Y")
        if M > 4:
            assert not Y[1].any()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", SHAPES + [(32, 256), (33, 272), (64, 128), (65, 144)])
@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
def test_norm_codes_are_those_of_its_output(M, K, dt, format):
    """The codes and scales of Y in 16 bits, bit for bit, whether Y is kept or not; zeros past the last row."""
    print(f"\n[case] rmsnorm codes {format} {dt} {M}x{K}", flush=True)
    X, R, w, _ = inputs(M, K, dt)
    X, R, w = X.cuda(), R.cuda(), w.cuda()
    plain, H0 = lm.rmsnorm(X, w, residual=R, eps=EPS)
    for keep in (False, True):
        q, s, Y, H = lm.rmsnorm_quantize(X, w, residual=R, eps=EPS, format=format, keep=keep)
        assert torch.equal(H, H0) and (Y is None) == (not keep) and (Y is None or torch.equal(Y, plain))
        if format == "mxfp4":
            q0, s0 = lm.mxfp4_quantize(plain)
            assert torch.equal(q, q0) and torch.equal(u8(s), u8(s0))
        else:
            _, rq, rs = fp8_ref.coded_rows(plain.cpu())
            assert torch.equal(q.cpu().float().double(), rq)
            m = torch.arange(M)
            want = torch.zeros(-(-K // 128), lm.fp8_row_scale_pitch(M), dtype=torch.uint8)
            want[:, m // 64 * 64 + m % 16 * 4 + m // 16 % 4] = rs[:, : want.shape[0]].t()
            assert torch.equal(u8(s), want)
    q, s, Y, H = lm.rmsnorm_quantize(X, w, eps=EPS, format=format, keep=True)  # without a residual
    assert H is None and torch.equal(Y, lm.rmsnorm(X, w, eps=EPS)[0])


# from 2048 rows on: two pieces of 8 columns a thread with one to eight waves a row, four with eight and sixteen
MANY = [(2048, 528), (2051, 1024), (2049, 1040), (2080, 2064), (2050, 4112), (2049, 8192), (2050, 8208), (2048, 16400)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", MANY)
def test_norm_of_many_rows(M, K, dt):
    print(f"\n[case] rmsnorm of many rows {dt} {M}x{K}", flush=True)
    X, R, w, _ = inputs(M, K, dt)
    h = summed(X, R)
    X, R, w = X.cuda(), R.cuda(), w.cuda()
    for res, sum_ in ((None, X.cpu()), (R, h)):
        Y, H = lm.rmsnorm(X, w, residual=res, eps=EPS)
        assert H is None if res is None else torch.equal(H.cpu(), sum_)
        want, rel = ref.norm(sum_.double(), w.cpu().double(), EPS)
        ref.assert_close(Y, want, rel * want.abs(), "Y")
    assert not Y[1].any()
    for keep in (False, True):
        q, s, Y4, H = lm.rmsnorm_quantize(X, w, residual=R, eps=EPS, format="mxfp4", keep=keep)
        q0, s0 = lm.mxfp4_quantize(Y)
        assert torch.equal(q, q0) and torch.equal(u8(s), u8(s0)) and torch.equal(H.cpu(), h) and (Y4 is None or torch.equal(Y4, Y))
        q, s, Y8, H = lm.rmsnorm_quantize(X, w, residual=R, eps=EPS, format="fp8", keep=keep)
        assert torch.equal(H.cpu(), h) and (Y8 is None or torch.equal(Y8, Y))
    _, rq, rs = fp8_ref.coded_rows(Y.cpu())
    assert torch.equal(q.cpu().float().double(), rq)
    m = torch.arange(M)
    want = torch.zeros(-(-K // 128), lm.fp8_row_scale_pitch(M), dtype=torch.uint8)
    want[:, m // 64 * 64 + m % 16 * 4 + m // 16 % 4] = rs[:, : want.shape[0]].t()
    assert torch.equal(u8(s), want)


@pytest.mark.parametrize("M,K,N", [(1, 144, 72), (5, 4096, 264), (20, 272, 136), (30, 8208, 72), (70, 400, 264), (300, 1040, 520), (2400, 272, 4360)])
def test_fp8_product_of_coded_rows(M, K, N):
    """Past 4 rows the same kernels run on the same codes, so the bits are fp8_matmul_block's; up to 4 rows
    another kernel adds the groups in another order."""
    dt = torch.bfloat16
    X, R, w, g = inputs(M, K, dt)
    W = (randn(g, K, N) * 0.02).to(dt)
    Wq, s_w = lm.fp8_quantize_weight_block(W.cuda())
    q, s, Y, _ = lm.rmsnorm_quantize(X.cuda(), w.cuda(), residual=R.cuda(), eps=EPS, format="fp8", keep=True)
    got = lm.fp8_matmul_block_coded(q, s, Wq, s_w, dt)
    if M > 4:
        assert torch.equal(got, lm.fp8_matmul_block(Y, Wq, s_w))
    else:
        want, err = fp8_ref.product(fp8_ref.coded_rows(Y.cpu())[0], fp8_ref.weight_values(Wq.cpu(), s_w.cpu(), K))
        fp8_ref.assert_close(got, want, err, "Y")
    nb = lm.fp8_matmul_block_coded_workspace_bytes(M, K, N)
    out, yw = framed((M, N), dt)
    ws, whole = framed((nb,), torch.uint8, 90)
    for fill in (255, 0):
        ws.fill_(fill)
        lm.fp8_matmul_block_coded(q, s, Wq, s_w, dt, Y=out, workspace=ws)
        assert torch.equal(out, got)
    assert frame_untouched(yw, M * N) and frame_untouched(whole, nb, 90)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = lm.fp8_matmul_block_coded(q, s, Wq, s_w, dt, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, got)


@pytest.mark.parametrize("M", [3, 20, 100, 300])
def test_fp8_scales_of_rows_past_the_last_have_no_effect(M):
    K, N, dt = 272, 136, torch.bfloat16
    X, R, w, g = inputs(M, K, dt)
    Wq, s_w = lm.fp8_quantize_weight_block((randn(g, K, N) * 0.02).to(dt).cuda())
    q, s, _, _ = lm.rmsnorm_quantize(X.cuda(), w.cuda(), residual=R.cuda(), eps=EPS, format="fp8")
    want = lm.fp8_matmul_block_coded(q, s, Wq, s_w, dt)
    m = torch.arange(M, lm.fp8_row_scale_pitch(M))
    s.view(torch.uint8)[:, (m // 64 * 64 + m % 16 * 4 + m // 16 % 4).cuda()] = 255
    assert torch.isfinite(want).all() and torch.equal(lm.fp8_matmul_block_coded(q, s, Wq, s_w, dt), want)


@pytest.mark.parametrize("M,K", [(5, 272), (2050, 1040), (2, 65552)])
def test_the_same_tensor_twice(M, K):
    """One tensor as X and residual, and H in its place; one as all of a gradient's inputs."""
    X, _, w, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in inputs(M, K, torch.bfloat16))
    for format in (None, "fp8", "mxfp4"):
        call = lambda x, r, h: (lm.rmsnorm(x, w, residual=r, eps=EPS, H=h) if format is None else
                                lm.rmsnorm_quantize(x, w, residual=r, eps=EPS, format=format, keep=True, H=h))
        want, x = call(X, X.clone(), None), X.clone()
        for got in (call(X, X, None), call(x, x, x)):
            for a, b in zip(got, want):
                assert torch.equal(u8(a), u8(b))
        assert torch.equal(x, want[-1])
    want = lm.rmsnorm_backward(X, X.clone(), w, dH=X.clone(), eps=EPS)
    for a, b in zip(lm.rmsnorm_backward(X, X, w, dH=X, eps=EPS), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K", [(5, 272), (3, 16400), (2, 65552)])
@pytest.mark.parametrize("format", ["fp8", "mxfp4", None])
def test_norm_in_place(M, K, format):
    """H in the place of X, and of the residual."""
    X, R, w, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in inputs(M, K, torch.bfloat16))

    def call(x, r, h):
        if format is None:
            return lm.rmsnorm(x, w, residual=r, eps=EPS, H=h)
        return lm.rmsnorm_quantize(x, w, residual=r, eps=EPS, format=format, keep=True, H=h)

    want = call(X, R, None)
    x, r = X.clone(), R.clone()
    for got, kept in ((call(x, R, x), x), (call(X, r, r), r)):
        assert got[-1] is kept
        for a, b in zip(got, want):
            assert torch.equal(u8(a), u8(b))
    assert not torch.equal(x, X) and not torch.equal(r, R)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("K", [528, 65552])
def test_rows_that_are_not_finite_stay_alone(K, dt):
    M = 40
    X, R, w, _ = inputs(M, K, dt)
    w = w.cuda()
    Y, _ = lm.rmsnorm(X.cuda(), w, eps=EPS)
    for v in (math.nan, math.inf, -math.inf):
        bad = X.clone()
        bad[7, 3] = bad[39, K - 1] = v
        keep = torch.ones(M, dtype=torch.bool)
        keep[7] = keep[39] = False
        Y2, _ = lm.rmsnorm(bad.cuda(), w, eps=EPS)
        assert torch.equal(Y2.cpu()[keep], Y.cpu()[keep])
        assert torch.isnan(Y2[7, 3]) and torch.isnan(Y2[39, K - 1])
        q, s, _, _ = lm.rmsnorm_quantize(bad.cuda(), w, eps=EPS, format="mxfp4")
        v4, v0 = lm.mxfp4_dequantize(q, s, K, dt).cpu(), lm.mxfp4_dequantize(*lm.mxfp4_quantize(Y), K, dt).cpu()
        assert torch.equal(v4[keep], v0[keep]) and torch.isnan(v4[7, :32]).all() and torch.isnan(v4[39, K - 1])
        dX, _ = lm.rmsnorm_backward(X.cuda(), bad.cuda(), w, eps=EPS, need_dw=False)
        assert torch.equal(dX.cpu()[keep], lm.rmsnorm_backward(X.cuda(), X.cuda(), w, eps=EPS)[0].cpu()[keep])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", [(5, 16), (5, 144), (3, 272), (7, 1040), (2, 4112), (2, 8208), (2, 16400), (2, 32784), (2060, 272), (2060, 528),
                                 (2060, 1040), (2060, 2064), (2060, 4112), (2060, 8208)])
def test_padding_of_rows_that_are_not_finite(M, K, dt):
    """Codes and scales past a row's last value are zeros whatever the row holds, and all of them are the codes of
    Y: every kernel of the norm, at sizes whose rows do not fill the codes' lines."""
    print(f"\n[case] rmsnorm padding {dt} {M}x{K}", flush=True)
    X, _, w, _ = inputs(M, K, dt)
    bad = {0: math.nan, M // 2: math.inf, M - 1: math.nan}
    for r, v in bad.items():
        X[r, K - 1 - 3 * r % K] = v
    X, w = X.cuda(), w.cuda()
    plain, _ = lm.rmsnorm(X, w, eps=EPS)
    q, s, Y, _ = lm.rmsnorm_quantize(X, w, eps=EPS, format="mxfp4", keep=True)
    q0, s0 = lm.mxfp4_quantize(plain)
    assert torch.equal(u8(Y), u8(plain)) and torch.equal(u8(s), u8(s0)) and torch.equal(u8(q), u8(q0))
    assert not q[:, K // 2:].any()
    q, s, Y, _ = lm.rmsnorm_quantize(X, w, eps=EPS, format="fp8", keep=True)
    assert torch.equal(u8(Y), u8(plain)) and not q.view(torch.uint8)[:, K:].any()
    assert torch.isnan(q[0].float()[:K]).all() and torch.isnan(q[M - 1].float()[:K]).all()
    codes, y = q.cpu().float().double(), plain.cpu()
    codes[list(bad)], y[list(bad)] = 0, 0
    assert torch.equal(codes, fp8_ref.coded_rows(y)[1])


def test_norm_of_large_and_small_numbers():
    """Squares stay within fp32 up to a sum of 2^128; below eps a row is as good as divided by its root."""
    dt, K = torch.bfloat16, 256
    w = torch.ones(K, dtype=dt, device="cuda")
    X = torch.stack([torch.full((K,), v) for v in (2.0 ** 59, 2.0 ** -60, 2.0 ** 70, 1.0)]).to(dt).cuda()
    Y, _ = lm.rmsnorm(X, w, eps=1e-6)
    assert torch.equal(Y[0].double(), torch.ones(K, device="cuda").double()) and not Y[2].any()
    assert torch.allclose(Y[1].double(), torch.full((K,), 2.0 ** -60 * 1000.0, device="cuda").double(), rtol=2.0 ** -8)


def test_norm_empty():
    for M, K in ((0, 64), (5, 0)):
        x, w = torch.zeros(M, K, dtype=torch.float16, device="cuda"), torch.zeros(K, dtype=torch.float16, device="cuda")
        assert lm.rmsnorm(x, w)[0].shape == (M, K)
        for f in ("fp8", "mxfp4"):
            assert lm.rmsnorm_quantize(x, w, residual=x, format=f)[3].shape == (M, K)
        dX, dW = lm.rmsnorm_backward(x, x, w)
        assert dX.shape == (M, K) and dW.shape == (K,) and not dW.any()
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    assert not lm.rmsnorm_backward(x, x, w)[1].any()


def test_norm_past_32_bits():
    """More than 2^32 values, more rows than a launch has workgroups, and the longest row."""
    dt = torch.bfloat16
    for M, K in (((1 << 19) + 40, 8208), ((1 << 21) + 3, 16), (3, 1 << 22)):
        print(f"\n[case] rmsnorm past 32 bits {M}x{K}", flush=True)
        X = torch.zeros(M, K, dtype=dt, device="cuda")
        rows = sorted({0, 1, M // 2, M - 1})
        X[rows] = randn(gen(K), len(rows), K).to(dt).cuda()
        w = torch.ones(K, dtype=dt, device="cuda")
        part = X[rows].contiguous()
        Y, _ = lm.rmsnorm(X, w)
        assert torch.equal(Y[rows], lm.rmsnorm(part, w)[0]) and int(Y.count_nonzero()) == int(Y[rows].count_nonzero())
        q, s, _, _ = lm.rmsnorm_quantize(X, w, format="mxfp4")
        q0, s0 = lm.mxfp4_quantize(Y)
        assert torch.equal(q, q0) and torch.equal(u8(s), u8(s0))
        del Y, q, s, q0, s0
        dX, dW = lm.rmsnorm_backward(X, X, w)
        assert torch.equal(dX[rows], lm.rmsnorm_backward(part, part, w)[0])
        h = part.double()
        want, err = (lambda r: (r[2], r[3]))(ref.norm_backward(h.cpu(), h.cpu(), w.double().cpu(), None, 1e-6))
        ref.assert_close(dW, want, err + M * 2.0 ** -23 * want.abs(), "dW")
        del X, dX
        torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K", [(5, 144), (33, 272), (2, 65552)])
@pytest.mark.parametrize("format", [None, "fp8", "mxfp4"])
def test_norm_writes_its_outputs_alone(M, K, format):
    X, R, w, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in inputs(M, K, torch.float16))
    H, hw = framed((M, K), torch.float16)
    Y, yw = framed((M, K), torch.float16)
    pitch, sb = {None: (0, 0), "fp8": (lm.fp8_code_pitch(K), -(-K // 128) * lm.fp8_row_scale_pitch(M)),
                 "mxfp4": (lm.fp4_code_pitch(K), -(-M // 32) * lm.fp4_scale_pitch(K))}[format]
    q, qw = framed((M * pitch,), torch.uint8, 90)
    s, sw = framed((sb,), torch.uint8, 90)
    rc = lm.lib().rmsnorm_forward(X.data_ptr(), R.data_ptr(), w.data_ptr(), M, K, lm.F16, EPS, H.data_ptr(), Y.data_ptr(),
                                  lm._FORMATS[format], q.data_ptr() if format else None, s.data_ptr() if format else None,
                                  torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == lm.OK
    for whole, n, fill in ((hw, M * K, 3.0), (yw, M * K, 3.0), (qw, M * pitch, 90), (sw, sb, 90)):
        assert frame_untouched(whole, n, fill)
    if format:
        q0, s0, Y0, H0 = lm.rmsnorm_quantize(X, w, residual=R, eps=EPS, format=format, keep=True)
        assert torch.equal(u8(q0).view(-1), q.cpu()) and torch.equal(u8(s0).view(-1), s.cpu()) and torch.equal(Y0, Y) and torch.equal(H0, H)


# ---- gradient

@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", BACK)
def test_backward(M, K, dt):
    print(f"\n[case] rmsnorm backward {dt} {M}x{K}", flush=True)
    H, dH, w, g = inputs(M, K, dt)
    dY = (randn(g, M, K) * 0.1).to(dt)
    for extra in (None, dH):
        args = (dY.cuda(), H.cuda(), w.cuda())
        dX, dW = lm.rmsnorm_backward(*args, dH=None if extra is None else extra.cuda(), eps=EPS)
        x, xe, v, ve = ref.norm_backward(dY.double(), H.double(), w.double(), None if extra is None else extra.double(), EPS)
        ref.assert_close(dX, x, xe, "dX")
        ref.assert_close(dW, v, ve, "dW")
        alone, none = lm.rmsnorm_backward(*args, dH=None if extra is None else extra.cuda(), eps=EPS, need_dw=False)
        assert none is None and torch.equal(alone, dX)
        again = lm.rmsnorm_backward(*args, dH=None if extra is None else extra.cuda(), eps=EPS)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


# a workgroup of sixteen waves a row; one, two and four waves a row with two, four and eight rows side by side
BACK_DENSE = [(100, 1024), (100, 8192), (511, 8208), (600, 272), (513, 1024), (520, 1040), (520, 4096), (1030, 272), (1030, 1024), (1100, 1040),
              (1030, 4096), (2050, 272), (2050, 1024), (2100, 1040), (2049, 2064), (5003, 16)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M,K", BACK_DENSE)
def test_backward_of_dense_rows(M, K, dt):
    """Every row and column enters dW."""
    print(f"\n[case] rmsnorm backward, dense {dt} {M}x{K}", flush=True)
    H, dH, w, g = inputs(M, K, dt)
    H[1] = randn(g, K).to(dt)
    dY = (randn(g, M, K) * 0.1).to(dt)
    args = (dY.cuda(), H.cuda(), w.cuda())
    for extra in (None, dH):
        extra_ = None if extra is None else extra.cuda()
        dX, dW = lm.rmsnorm_backward(*args, dH=extra_, eps=EPS)
        x, xe, v, ve = ref.norm_backward(dY.double(), H.double(), w.double(), None if extra is None else extra.double(), EPS)
        ref.assert_close(dX, x, xe, "dX")
        ref.assert_close(dW, v, ve, "dW")
        alone, none = lm.rmsnorm_backward(*args, dH=extra_, eps=EPS, need_dw=False)
        assert none is None and torch.equal(alone, dX)
        again = lm.rmsnorm_backward(*args, dH=extra_, eps=EPS)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


@pytest.mark.parametrize("M,K", [((1 << 19) + 40, 8208), ((1 << 21) + 3, 16)])
def test_backward_past_32_bits_and_most_rows_zero(M, K):
    """A row of zeros adds nothing to dW, without a rounding: the bound is that of the other rows alone."""
    dt = torch.bfloat16
    print(f"\n[case] rmsnorm backward, rows of zeros {M}x{K}", flush=True)
    H, dY = torch.zeros(M, K, dtype=dt, device="cuda"), torch.zeros(M, K, dtype=dt, device="cuda")
    rows = [0, 1, 2, 5, 255, 256, 2047, 2048, M // 2, M - 2, M - 1]
    g = gen(K + 1)
    h, dy, w = randn(g, len(rows), K).to(dt), randn(g, len(rows), K).to(dt), (1 + 0.2 * randn(g, K)).to(dt)
    H[rows], dY[rows] = h.cuda(), dy.cuda()
    dX, dW = lm.rmsnorm_backward(dY, H, w.cuda())
    x, xe, v, ve = ref.norm_backward(dy.double(), h.double(), w.double(), None, 1e-6)
    ref.assert_close(dX[rows], x, xe, "dX")
    ref.assert_close(dW, v, ve, "dW")
    assert int(dX.count_nonzero()) == int(dX[rows].count_nonzero())
    del H, dY, dX
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K", [(3, 256), (3, 8208), (600, 1040), (3, 16400), (3, 32784)])
def test_backward_of_zeros_with_the_smallest_eps(M, K):
    """r = 2^64.. is an fp32 number, its square is not: a row of zeros has the gradient r d."""
    dt, eps = torch.bfloat16, float(torch.tensor(2.0 ** -130))
    H, _, w, g = inputs(M, K, dt)
    H[0] = H[M - 1] = 0
    dY = randn(g, M, K).to(dt)
    dX, dW = lm.rmsnorm_backward(dY.cuda(), H.cuda(), w.cuda(), eps=eps)
    x, xe, v, ve = ref.norm_backward(dY.double(), H.double(), w.double(), None, eps)
    assert float(x[0].abs().max()) > 2.0 ** 64
    ref.assert_close(dX, x, xe, "dX")
    ref.assert_close(dW, v, ve, "dW")


def test_backward_against_differences():
    """sum(dY * y) along a direction, from the reference's own norm in 64 bits; 16-bit gradients are off by
    half a step a value, which over K products of random sign stays far below the sum's size."""
    M, K, dt = 6, 528, torch.float16
    H, _, w, g = inputs(M, K, dt)
    dY = randn(g, M, K).to(dt)
    dX, dW = lm.rmsnorm_backward(dY.cuda(), H.cuda(), w.cuda(), eps=EPS)
    f = lambda h, v: float((ref.norm(h, v, EPS)[0] * dY.double()).sum())
    for i in range(4):
        u, v = randn(g, M, K).double(), randn(g, K).double()
        t = 1e-4
        slope = (f(H.double() + t * u, w.double()) - f(H.double() - t * u, w.double())) / (2 * t)
        mag = float((dX.cpu().double().abs() * u.abs()).sum())
        assert abs(slope - float((dX.cpu().double() * u).sum())) <= 2.0 ** -10 * mag + 1e-5
        slope = (f(H.double(), w.double() + t * v) - f(H.double(), w.double() - t * v)) / (2 * t)
        mag = float((dW.cpu().double().abs() * v.abs()).sum())
        assert abs(slope - float((dW.cpu().double() * v).sum())) <= 2.0 ** -10 * mag + 1e-5


@pytest.mark.parametrize("M,K", [(5, 144), (600, 1040), (70, 65552)])
def test_backward_workspaces_graphs_and_streams(M, K):
    dt = torch.bfloat16
    H, dH, w, g = inputs(M, K, dt)
    dY, H, dH, w = randn(g, M, K).to(dt).cuda(), H.cuda(), dH.cuda(), w.cuda()
    nb = lm.rmsnorm_backward_workspace_bytes(M, K)
    f = lambda ws: lm.rmsnorm_backward(dY, H, w, dH=dH, eps=EPS, workspace=ws)
    want = f(None)
    ws, whole = framed((nb,), torch.uint8, 90)
    for fill in (255, 0):
        ws.fill_(fill)
        for a, b in zip(f(ws), want):
            assert torch.equal(a, b), fill
    assert frame_untouched(whole, nb, 90)
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
    side, own = torch.cuda.Stream(), torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    outs = [lm.rmsnorm_backward(dY, H, w, dH=dH, eps=EPS, workspace=own, stream=side) for _ in range(4)]
    here = [f(ws) for _ in range(4)]
    torch.cuda.synchronize()
    for out in outs + here:
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    dX, xw = framed((M, K), dt)
    lm.rmsnorm_backward(dY, H, w, dH=dH, eps=EPS, dX=dX)
    torch.cuda.synchronize()
    assert frame_untouched(xw, M * K) and torch.equal(dX, want[0])


# ---- together

def layer(X, R, p, format):
    """A feed-forward half of a layer: norm, up product, its activation, down product, and the next norm."""
    if format == "mxfp4":
        q, s, _, H = lm.rmsnorm_quantize(X, p["n1"], residual=R, eps=EPS, format="mxfp4")
        u = lm.mxfp4_matmul_coded(q, s, *p["up4"], X.dtype)
        d = lm.mxfp4_matmul(torch.relu(u), *p["down4"])
    else:
        q, s, _, H = lm.rmsnorm_quantize(X, p["n1"], residual=R, eps=EPS, format="fp8")
        u = lm.fp8_matmul_block_coded(q, s, *p["up8"], X.dtype)
        d = lm.fp8_matmul_block(torch.relu(u), *p["down8"])
    return lm.rmsnorm(d, p["n2"], residual=H, eps=EPS)


def weights(g, K, I, dt):
    up, down = (randn(g, K, I) * 0.05).to(dt).cuda(), (randn(g, I, K) * 0.05).to(dt).cuda()
    return {"n1": (1 + 0.1 * randn(g, K)).to(dt).cuda(), "n2": (1 + 0.1 * randn(g, K)).to(dt).cuda(),
            "up4": lm.mxfp4_quantize(up, columns=True), "down4": lm.mxfp4_quantize(down, columns=True),
            "up8": lm.fp8_quantize_weight_block(up), "down8": lm.fp8_quantize_weight_block(down)}


@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
@pytest.mark.parametrize("M", [20, 40, 150])
def test_layer_equals_its_steps(M, format):
    """The coded way bit for bit the way through 16 bits, past 16 rows, from where both take the same kernels."""
    K, I, dt = 272, 1040, torch.bfloat16
    X, R, _, g = inputs(M, K, dt)
    X, R, p = X.cuda(), R.cuda(), weights(g, K, I, dt)
    Y, H2 = layer(X, R, p, format)
    n, H = lm.rmsnorm(X, p["n1"], residual=R, eps=EPS)
    product = lm.mxfp4_matmul if format == "mxfp4" else lm.fp8_matmul_block
    up, down = ("up4", "down4") if format == "mxfp4" else ("up8", "down8")
    d = product(torch.relu(product(n, *p[up])), *p[down])
    want = lm.rmsnorm(d, p["n2"], residual=H, eps=EPS)
    assert torch.equal(H2, want[1]) and torch.equal(Y, want[0])


@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
@pytest.mark.parametrize("M", [1, 16, 150])
def test_layer_captured_and_replayed(M, format):
    K, I, dt = 272, 1040, torch.bfloat16
    X, R, _, g = inputs(M, K, dt)
    X, R, p = X.cuda(), R.cuda(), weights(g, K, I, dt)
    layer(X, R, p, format)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(X, R, p, format)
    for r in range(4):
        X.copy_(randn(g, M, K).to(dt))
        want = layer(X, R, p, format)
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), r


class NormProduct(torch.autograd.Function):
    """A norm with its residual and an 8-bit product in training."""

    @staticmethod
    def forward(ctx, X, R, weight, W):
        Wq, s, WqT, sT = lm.fp8_quantize_weight_block(W, transposed=True)
        q, sx, Y, H = lm.rmsnorm_quantize(X, weight, residual=R, eps=EPS, format="fp8", keep=True)
        ctx.save_for_backward(Y, H, weight, WqT, sT)
        return lm.fp8_matmul_block_coded(q, sx, Wq, s, X.dtype), H

    @staticmethod
    def backward(ctx, dO, dH):
        Y, H, weight, WqT, sT = ctx.saved_tensors
        dY, dW = lm.fp8_matmul_block_backward(dO.contiguous(), Y, WqT, sT)
        dX, dweight = lm.rmsnorm_backward(dY, H, weight, dH=dH.contiguous(), eps=EPS)
        return dX, dX, dweight, dW


def test_layer_in_training():
    """Gradients under autograd: bit for bit those of the calls themselves, and near the formula's in 64 bits
    (the product's operands have 4 significant bits, so by a few per cent of the norm)."""
    M, K, N, dt = 70, 272, 136, torch.bfloat16
    X, R, w, g = inputs(M, K, dt)
    W = (randn(g, K, N) * 0.05).to(dt)
    leaves = [t.cuda().requires_grad_() for t in (X, R, w, W)]
    O, H = NormProduct.apply(*leaves)
    dO, dH = randn(g, M, N).to(dt).cuda(), randn(g, M, K).to(dt).cuda()
    torch.autograd.backward([O, H], [dO, dH])
    x, r, v, m = (t.detach().cpu().double().requires_grad_() for t in leaves)
    h = x + r
    y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS) * v
    torch.autograd.backward([y @ m, h], [dO.cpu().double(), dH.cpu().double()])
    for got, want in zip(leaves, (x, r, v, m)):
        a, b = got.grad.cpu().double(), want.grad
        assert float((a - b).norm() / b.norm()) < 0.05
    assert torch.equal(leaves[0].grad, leaves[1].grad)
    with torch.no_grad():
        d = [t.detach() for t in leaves]
        Wq, s, WqT, sT = lm.fp8_quantize_weight_block(d[3], transposed=True)
        q, sx, Y, Hn = lm.rmsnorm_quantize(d[0], d[2], residual=d[1], eps=EPS, format="fp8", keep=True)
        dY, dW = lm.fp8_matmul_block_backward(dO, Y, WqT, sT)
        dX, dw = lm.rmsnorm_backward(dY, Hn, d[2], dH=dH, eps=EPS)
    for a, b in zip((t.grad for t in leaves), (dX, dX, dw, dW)):
        assert torch.equal(a, b)
    assert not lm.rmsnorm(leaves[0], leaves[2])[0].requires_grad


def test_refusals_of_gpu_tensors():
    X, w = torch.zeros(5, 272, dtype=torch.float16, device="cuda"), torch.ones(272, dtype=torch.float16, device="cuda")
    for bad in (lambda: lm.rmsnorm(X.float(), w), lambda: lm.rmsnorm(X, w.float()), lambda: lm.rmsnorm(X, w.cpu()), lambda: lm.rmsnorm(X, w, residual=X.bfloat16()),
                lambda: lm.rmsnorm_backward(X, X.bfloat16(), w), lambda: lm.rmsnorm_backward(X, X, w, dH=X.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lm.rmsnorm(X[:, ::2], w), lambda: lm.rmsnorm(X, w[:16]), lambda: lm.rmsnorm(X[0], w), lambda: lm.rmsnorm(X, w, residual=X[:4]),
                lambda: lm.rmsnorm(X, w, H=X), lambda: lm.rmsnorm_quantize(X, w, format="int8"), lambda: lm.rmsnorm_backward(X, X[:4], w),
                lambda: lm.rmsnorm_backward(X, X, w, dX=X[:4])):
        with pytest.raises(ValueError):
            bad()
    both = torch.zeros(6, 272, dtype=torch.float16, device="cuda")
    for bad in (lambda: lm.rmsnorm(X, w, eps=0.0), lambda: lm.rmsnorm(X, w, eps=math.nan), lambda: lm.rmsnorm_backward(X, X, w, eps=-1.0),
                lambda: lm.rmsnorm(both[:5], w, residual=X, H=both[1:]), lambda: lm.rmsnorm_backward(X, X, w, dX=X),
                lambda: lm.rmsnorm_backward(X, X, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                lambda: lm.rmsnorm(X[:, :264].contiguous(), w[:264].contiguous())):
        with pytest.raises(lm.LLMInt8Error):
            bad()
    torch.cuda.synchronize()
