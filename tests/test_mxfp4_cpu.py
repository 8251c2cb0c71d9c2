"""The boundary of the 4-bit floating point operators and of the norm on the CPU: argument checks
(which come before any GPU work), layouts, the stages of a dry run, and the reference's own pins."""
import math
import re

import pytest
import torch

import int8_quantized_matmul_rowwise_amd as lm
from tests import mxfp4_ref as ref

MB = 0x100000
A, B, C, D, E, F, G, H_, W_ = (MB * 4096 * i for i in range(1, 10))  # fake device addresses, never dereferenced
BIG = 1 << 40
NAN, INF = math.nan, math.inf


def quant(**kw):
    a = dict(A=A, R=64, C=72, dt=0, cols=1, q=B, s=C)
    a.update(kw)
    return lm.lib().mxfp4_quantize(a["A"], a["R"], a["C"], a["dt"], a["cols"], a["q"], a["s"], None)


def deq(**kw):
    a = dict(q=A, s=B, R=70, n=64, dt=0, A=C)
    a.update(kw)
    return lm.lib().mxfp4_dequantize(a["q"], a["s"], a["R"], a["n"], a["dt"], a["A"], None)


def mm(**kw):
    a = dict(X=A, M=100, K=64, dt=0, Wq=B, s=C, N=72, Y=D, ws=E, wsb=BIG >> 10)
    a.update(kw)
    return lm.lib().mxfp4_matmul(a["X"], a["M"], a["K"], a["dt"], a["Wq"], a["s"], a["N"], a["Y"], a["ws"], a["wsb"], None)


def mmc(four=True, **kw):
    a = dict(X=A, xs=F, M=100, K=64, dt=0, Wq=B, s=C, N=72, Y=D, ws=E, wsb=BIG >> 10)
    a.update(kw)
    fn = lm.lib().mxfp4_matmul_coded if four else lm.lib().fp8_matmul_block_coded
    return fn(a["X"], a["xs"], a["M"], a["K"], a["dt"], a["Wq"], a["s"], a["N"], a["Y"], a["ws"], a["wsb"], None)


def norm(**kw):
    a = dict(X=A, R=B, w=C, M=3, K=64, dt=0, eps=1e-6, H=D, Y=E, fmt=2, q=F, s=G)
    a.update(kw)
    return lm.lib().rmsnorm_forward(a["X"], a["R"], a["w"], a["M"], a["K"], a["dt"], a["eps"], a["H"], a["Y"], a["fmt"], a["q"], a["s"], None)


def back(**kw):
    a = dict(dY=A, H=B, w=C, dH=D, M=3, K=64, dt=0, eps=1e-6, dX=E, dW=F, ws=G, wsb=MB)
    a.update(kw)
    return lm.lib().rmsnorm_backward(a["dY"], a["H"], a["w"], a["dH"], a["M"], a["K"], a["dt"], a["eps"], a["dX"], a["dW"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), lm.EINVAL), (dict(R=-16), lm.EINVAL), (dict(R=24), lm.EINVAL), (dict(C=12), lm.EINVAL), (dict(cols=0), lm.EINVAL),
    (dict(R=(1 << 22) + 16), lm.ERANGE), (dict(C=(1 << 22) + 8), lm.ERANGE), (dict(R=1 << 22, C=1 << 15), lm.ERANGE),
    (dict(cols=0, R=1 << 15, C=1 << 22), lm.ERANGE),
    (dict(A=None), lm.EINVAL), (dict(A=A + 8), lm.EINVAL), (dict(q=None), lm.EINVAL), (dict(q=B + 8), lm.EINVAL), (dict(s=None), lm.EINVAL),
    (dict(s=C + 2), lm.EINVAL), (dict(q=A), lm.EINVAL), (dict(q=A + 64 * 72 * 2 - 16), lm.EINVAL), (dict(s=B + 128), lm.EINVAL), (dict(s=A + 4), lm.EINVAL),
    (dict(R=0, A=None), lm.OK), (dict(C=0, q=None), lm.OK), (dict(R=0, cols=0, C=32, s=None), lm.OK),
])
def test_quantize_refuses(kw, code):
    assert quant(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), lm.EINVAL), (dict(R=-1), lm.EINVAL), (dict(n=24), lm.EINVAL), (dict(n=(1 << 22) + 16), lm.ERANGE),
    (dict(R=(1 << 22) + 1), lm.ERANGE), (dict(q=None), lm.EINVAL), (dict(q=A + 8), lm.EINVAL), (dict(s=None), lm.EINVAL),
    (dict(s=B + 1), lm.EINVAL), (dict(A=None), lm.EINVAL), (dict(A=C + 2), lm.EINVAL), (dict(A=A), lm.EINVAL), (dict(A=B), lm.EINVAL),
    (dict(R=0, q=None), lm.OK), (dict(n=0, A=None), lm.OK),
])
def test_dequantize_refuses(kw, code):
    assert deq(**kw) == code


PRODUCT = [
    (dict(dt=-1), lm.EINVAL), (dict(M=-1), lm.EINVAL), (dict(K=24), lm.EINVAL), (dict(N=12), lm.EINVAL),
    (dict(K=(1 << 22) + 16), lm.ERANGE), (dict(M=(1 << 22) + 1), lm.ERANGE),
    (dict(X=None), lm.EINVAL), (dict(X=A + 8), lm.EINVAL), (dict(Wq=None), lm.EINVAL), (dict(Wq=B + 8), lm.EINVAL),
    (dict(s=None), lm.EINVAL), (dict(s=C + 1), lm.EINVAL), (dict(Y=None), lm.EINVAL), (dict(Y=D + 2), lm.EINVAL),
    (dict(Y=A), lm.EINVAL), (dict(Y=B), lm.EINVAL), (dict(Y=C), lm.EINVAL),
    (dict(M=0, X=None, ws=None), lm.OK), (dict(N=0, Y=None, Wq=None), lm.OK),
]


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(N=(1 << 22) + 8), lm.ERANGE), (dict(M=1 << 20, N=1 << 18), lm.ERANGE), (dict(M=1 << 22, K=1 << 16), lm.ERANGE),
    (dict(ws=None), lm.EWORKSPACE), (dict(ws=E + 8), lm.EWORKSPACE), (dict(wsb=100), lm.EWORKSPACE),
    (dict(Y=E), lm.EINVAL), (dict(ws=A), lm.EINVAL), (dict(ws=B), lm.EINVAL), (dict(ws=C), lm.EINVAL),
])
def test_matmul_refuses(kw, code):
    assert mm(**kw) == code


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("kw,code", PRODUCT + [(dict(xs=None), lm.EINVAL), (dict(xs=F + 2), lm.EINVAL), (dict(Y=F), lm.EINVAL)])
def test_coded_matmul_refuses(kw, code, four):
    assert mmc(four, **kw) == code


@pytest.mark.parametrize("four", [True, False])
def test_coded_matmul_checks_its_workspace(four):
    kw = dict(M=30, K=8192, N=72)  # a split sum
    bytes_ = (lm.mxfp4_matmul_coded_workspace_bytes if four else lm.fp8_matmul_block_coded_workspace_bytes)(30, 8192, 72)
    assert 0 < bytes_ < MB
    for bad in (dict(ws=None), dict(ws=E + 8), dict(wsb=bytes_ - 1)):
        assert mmc(four, **kw, **bad) == lm.EWORKSPACE
    for bad in (dict(ws=A), dict(ws=B), dict(ws=C), dict(ws=D), dict(ws=F)):
        assert mmc(four, **kw, **bad) == lm.EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), lm.EINVAL), (dict(M=-1), lm.EINVAL), (dict(K=24), lm.EINVAL), (dict(M=(1 << 22) + 1), lm.ERANGE), (dict(K=(1 << 22) + 16), lm.ERANGE),
    (dict(eps=0.0), lm.EINVAL), (dict(eps=-1.0), lm.EINVAL), (dict(eps=NAN), lm.EINVAL), (dict(eps=INF), lm.EINVAL),
    (dict(fmt=3), lm.EINVAL), (dict(fmt=-1), lm.EINVAL), (dict(fmt=0), lm.EINVAL), (dict(fmt=0, s=None), lm.EINVAL),
    (dict(X=None), lm.EINVAL), (dict(X=A + 8), lm.EINVAL), (dict(R=B + 8), lm.EINVAL), (dict(w=None), lm.EINVAL), (dict(w=C + 2), lm.EINVAL),
    (dict(H=D + 8), lm.EINVAL), (dict(Y=E + 8), lm.EINVAL), (dict(q=None), lm.EINVAL), (dict(q=F + 8), lm.EINVAL), (dict(s=None), lm.EINVAL),
    (dict(s=G + 2), lm.EINVAL), (dict(R=None), lm.EINVAL),
    (dict(H=A + 16), lm.EINVAL), (dict(H=B + 16), lm.EINVAL), (dict(Y=A), lm.EINVAL), (dict(Y=B), lm.EINVAL), (dict(Y=D), lm.EINVAL),
    (dict(q=A), lm.EINVAL), (dict(s=F), lm.EINVAL), (dict(q=C), lm.EINVAL), (dict(H=C), lm.EINVAL),
    (dict(M=0, X=None), lm.OK), (dict(K=0, w=None), lm.OK), (dict(fmt=0, q=None, s=None, H=None, Y=None), lm.OK),
])
def test_norm_refuses(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), lm.EINVAL), (dict(M=-1), lm.EINVAL), (dict(K=24), lm.EINVAL), (dict(M=(1 << 22) + 1), lm.ERANGE), (dict(K=(1 << 22) + 16), lm.ERANGE),
    (dict(eps=0.0), lm.EINVAL), (dict(eps=NAN), lm.EINVAL), (dict(dY=None), lm.EINVAL), (dict(dY=A + 8), lm.EINVAL), (dict(H=None), lm.EINVAL),
    (dict(w=None), lm.EINVAL), (dict(w=C + 8), lm.EINVAL), (dict(dH=D + 8), lm.EINVAL), (dict(dX=None), lm.EINVAL), (dict(dX=E + 8), lm.EINVAL),
    (dict(dW=F + 8), lm.EINVAL), (dict(ws=None), lm.EWORKSPACE), (dict(ws=G + 4), lm.EWORKSPACE), (dict(wsb=64), lm.EWORKSPACE),
    (dict(dX=A), lm.EINVAL), (dict(dX=B), lm.EINVAL), (dict(dX=D), lm.EINVAL), (dict(dW=C), lm.EINVAL), (dict(dW=E), lm.EINVAL),
    (dict(ws=A), lm.EINVAL), (dict(ws=E), lm.EINVAL),
    (dict(K=0, dY=None), lm.OK), (dict(M=0, dW=None, dY=None, ws=None), lm.OK),
])
def test_norm_backward_refuses(kw, code):
    assert back(**kw) == code


def _calls():
    return {
        "quantize": (lambda: quant(), ["mxfp4_columns"]),
        "quantize_rows": (lambda: quant(cols=0, C=80), ["mxfp4_rows"]),
        "dequantize": (lambda: deq(), ["mxfp4_values"]),
        "matmul": (lambda: mm(M=300, K=1024, N=520), ["mxfp4_rows", "mxfp4_gemm"]),
        "matmul_fused": (lambda: mm(M=2, K=1024, N=520, ws=None, wsb=0), ["mxfp4_gemm"]),
        "matmul_k0": (lambda: mm(K=0), ["fill_zero"]),
        "coded": (lambda: mmc(M=3000, K=1024, N=5200), ["mxfp4_gemm"]),
        "coded_split": (lambda: mmc(M=30, K=8192, N=72), ["fill_zero", "mxfp4_gemm"]),
        "coded_fp8": (lambda: mmc(False, M=3000, K=1024, N=5200), ["fp8_gemm"]),
        "coded_fp8_split": (lambda: mmc(False, M=30, K=8192, N=72), ["fill_zero", "fp8_gemm"]),
        "norm": (lambda: norm(), ["rmsnorm"]),
        "norm_in_place": (lambda: norm(H=A), ["rmsnorm"]),
        "norm_in_place_of_the_residual": (lambda: norm(H=B, fmt=1), ["rmsnorm"]),
        "norm_backward": (lambda: back(), ["rmsnorm_backward"]),
        "norm_backward_no_rows": (lambda: back(M=0, ws=None), ["fill_zero"]),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_stages_and_their_failures(name, monkeypatch, capfd):
    fn, want = _calls()[name]
    monkeypatch.setenv("LLMINT8_LOG", "1")

    def run(fault):
        monkeypatch.setenv("LLMINT8_FAULT", fault)
        capfd.readouterr()
        rc = fn()
        return rc, re.findall(r"^\[llmint8\]   stage (\w+)", capfd.readouterr().err, flags=re.M)

    assert run("no_such_stage") == (lm.OK, want)
    for i, st in enumerate(want):
        assert run(st) == (lm.EHIP, want[: i + 1])


@pytest.mark.parametrize("M,K,N,path,coded", [
    (1, 16, 8, "mxfp4_small_fused", "mxfp4_small"), (4, 8192, 16384, "mxfp4_small_fused", "mxfp4_small"), (4, 8192, 16392, "mxfp4_small", "mxfp4_small"),
    (8, 8192, 8192, "mxfp4_small_fused", "mxfp4_small"), (9, 8192, 8192, "mxfp4_small", "mxfp4_small"), (16, 4096, 4096, "mxfp4_small_fused", "mxfp4_small"),
    (17, 4096, 4096, "mxfp4_small", "mxfp4_small"), (16, 4096, 28672, "mxfp4_small", "mxfp4_small"), (1, 16384, 1024, "mxfp4_small_split", "mxfp4_small_split"),
    (64, 8192, 8192, "mxfp4_small", "mxfp4_small"), (64, 4096, 16384, "mxfp4_single", "mxfp4_single"), (65, 256, 8, "mxfp4_single", "mxfp4_single"),
    (128, 16384, 4096, "mxfp4_single_split", "mxfp4_single_split"), (2048, 4096, 4096, "mxfp4_tile128", "mxfp4_tile128"),
    (2048, 16384, 4096, "mxfp4_tile128", "mxfp4_tile128"), (4096, 16384, 2056, "mxfp4_tile256", "mxfp4_tile256"),
])
def test_routes(M, K, N, path, coded, monkeypatch, capfd):
    monkeypatch.setenv("LLMINT8_LOG", "1")
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")
    far = 1 << 44  # addresses that nothing reads
    for name, call in ((path, lambda: mm(X=far, M=M, K=K, Wq=2 * far, s=3 * far, N=N, Y=4 * far, ws=5 * far, wsb=1 << 40)),
                       (coded, lambda: mmc(X=far, xs=6 * far, M=M, K=K, Wq=2 * far, s=3 * far, N=N, Y=4 * far, ws=5 * far, wsb=1 << 40))):
        capfd.readouterr()
        assert call() == lm.OK
        assert re.findall(r"path=(\w+)", capfd.readouterr().err) == [name]
    assert lm.mxfp4_matmul_workspace_bytes(M, K, N) < 1 << 30


def test_sizes():
    for n in (0, 1, 16, 255, 256, 257, 4096, 12288):
        assert lm.lib().fp4_code_pitch(n) == lm.fp4_code_pitch(n) == ref.code_pitch(n)
        assert lm.lib().fp4_scale_pitch(n) == lm.fp4_scale_pitch(n) == ref.scale_pitch(n)
        assert lm.lib().fp8_row_scale_pitch(n) == lm.fp8_row_scale_pitch(n) == -(-n // 64) * 64
    assert lm.lib().fp4_code_pitch(-1) == lm.lib().fp4_scale_pitch(-1) == lm.lib().fp8_row_scale_pitch(-1) == 0
    assert lm.mxfp4_matmul_workspace_bytes(-1, 16, 8) == lm.mxfp4_matmul_coded_workspace_bytes(4, 24, 8) == 0
    assert lm.mxfp4_matmul_workspace_bytes(0, 272, 136) == lm.mxfp4_matmul_workspace_bytes(130, 0, 136) == 0
    assert lm.mxfp4_matmul_workspace_bytes(130, 272, 136) >= 130 * 256 + 5 * 512
    assert lm.rmsnorm_backward_workspace_bytes(3, 64, False) == lm.rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert lm.rmsnorm_backward_workspace_bytes(3, 64) >= 3 * 64 * 4
    for M in (1, 100, 1 << 22):
        for K in (16, 8192, 32768, 32784, 1 << 22):
            assert K * 4 <= lm.rmsnorm_backward_workspace_bytes(M, K) <= 1024 * K * 4 + M * 4 + 1024


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.float16)
    for call in (lambda: lm.mxfp4_quantize(x), lambda: lm.mxfp4_dequantize(x, x, 64), lambda: lm.mxfp4_matmul(x, x, x),
                 lambda: lm.mxfp4_matmul_coded(x, x, x, x), lambda: lm.fp8_matmul_block_coded(x, x, x, x),
                 lambda: lm.rmsnorm(x, x), lambda: lm.rmsnorm_quantize(x, x), lambda: lm.rmsnorm_backward(x, x, x)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        lm.rmsnorm_quantize(x, x, format="int8")


# ---- the reference's own pins

def test_reference_codes():
    v = torch.tensor([0.0, 0.25, 0.26, 0.5, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7.0, 100.0], dtype=torch.float64)
    assert ref.nearest_code(v).tolist() == [0, 0, 1, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 7]
    assert ref.nearest_code(-v).tolist() == ref.nearest_code(v).tolist()


def test_reference_scales():
    a = torch.tensor([7.0, 7.0001, 6.9, 3.5, 3.6, 0.0, 2.0 ** -140, 1.0, 7 * 2.0 ** 20, 65504.0, INF], dtype=torch.float64)
    assert (ref.scale_byte(a) - 127).tolist() == [0, 1, 0, -1, 0, -127, -127, -2, 20, 14, 128]


def test_reference_on_a_case_by_hand():
    """1 and 100 in a group: 7 * 2^3 = 56 < 100 <= 7 * 2^4, so the scale is 16; 100 / 16 = 6.25 is nearest to 6,
    1 / 16 to 0, -9 / 16 to -0.5; the next group is another scale's."""
    x = torch.zeros(33, 48, dtype=torch.float64)
    x[32, 0], x[32, 1], x[32, 2], x[32, 33] = 1.0, 100.0, -9.0, 3.0
    v, q, s = ref.coded(x)
    assert v[32, :3].tolist() == [0.0, 96.0, -8.0] and v[32, 33] == 3.0
    assert q[32, 0] == 0x70 and q[32, 1] == 0x09 and q[32, 16] == 0x70  # (3 = 6 * 2^-1)
    assert s.shape == (2, 256) and s[1, 0] == 127 + 4 and s[1, 64] == 127 - 1 and int(s.long().sum()) == 127 + 4 + 127 - 1
    assert torch.equal(ref.values(q, s, 48), v)
