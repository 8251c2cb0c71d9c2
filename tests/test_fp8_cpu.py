"""The boundary of the e4m3 block-scaled operators on the CPU: argument checks (which come before
any GPU work), layouts, the stages of a dry run, and the reference's own pins."""
import re

import pytest
import torch

import int8_quantized_matmul_rowwise_amd as lm
from tests import fp8_ref as ref

MB = 0x100000
A, B, C, D, E, F, G, H_, W_ = (MB * 4096 * i for i in range(1, 10))  # fake device addresses, never dereferenced
BIG = 1 << 40


def quant(**kw):
    a = dict(W=A, K=64, N=72, dt=0, Wq=B, s=C, WqT=D, sT=E)
    a.update(kw)
    return lm.lib().fp8_quantize_weight_block(a["W"], a["K"], a["N"], a["dt"], a["Wq"], a["s"], a["WqT"], a["sT"], None)


def mm(**kw):
    a = dict(X=A, M=100, K=64, dt=0, Wq=B, s=C, N=72, Y=D, ws=E, wsb=BIG >> 10)
    a.update(kw)
    return lm.lib().fp8_matmul_block(a["X"], a["M"], a["K"], a["dt"], a["Wq"], a["s"], a["N"], a["Y"], a["ws"], a["wsb"], None)


def back(**kw):
    a = dict(dY=A, X=B, M=4, K=64, N=72, dt=0, WqT=C, sT=D, dX=E, dW=F, ws=G, wsb=BIG >> 10)
    a.update(kw)
    return lm.lib().fp8_matmul_block_backward(a["dY"], a["X"], a["M"], a["K"], a["N"], a["dt"], a["WqT"], a["sT"],
                                              a["dX"], a["dW"], a["ws"], a["wsb"], None)


def moe(**kw):
    a = dict(X=A, T=3, H=64, dt=0, l=A + MB, E=4, k=2, W13=B, s13=C, W2=D, s2=E, I=48, Y=F, ids=G, p=G + MB, ws=H_, wsb=MB)
    a.update(kw)
    return lm.lib().fp8_moe_block(a["X"], a["T"], a["H"], a["dt"], a["l"], a["E"], a["k"], 1, a["W13"], a["s13"],
                                  a["W2"], a["s2"], a["I"], a["Y"], a["ids"], a["p"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), lm.EINVAL), (dict(K=-16), lm.EINVAL), (dict(K=24), lm.EINVAL), (dict(N=12), lm.EINVAL),
    (dict(K=(1 << 22) + 16), lm.ERANGE), (dict(N=(1 << 22) + 8), lm.ERANGE), (dict(W=None), lm.EINVAL),
    (dict(N=(1 << 22) + 8, WqT=None, sT=None), lm.ERANGE),
    (dict(W=A + 8), lm.EINVAL), (dict(Wq=None), lm.EINVAL), (dict(Wq=B + 4), lm.EINVAL), (dict(s=None), lm.EINVAL),
    (dict(s=C + 2), lm.EINVAL), (dict(WqT=None), lm.EINVAL), (dict(sT=None), lm.EINVAL), (dict(WqT=D + 8), lm.EINVAL),
    (dict(Wq=A), lm.EINVAL), (dict(WqT=B + 128), lm.EINVAL), (dict(s=B), lm.EINVAL), (dict(sT=C), lm.EINVAL),
    (dict(K=0, W=None, Wq=None), lm.OK), (dict(N=0, W=None), lm.OK),
])
def test_quantize_refuses(kw, code):
    assert quant(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), lm.EINVAL), (dict(M=-1), lm.EINVAL), (dict(K=24), lm.EINVAL), (dict(N=12), lm.EINVAL),
    (dict(K=(1 << 22) + 16), lm.ERANGE), (dict(M=1 << 31), lm.EINVAL), (dict(M=(1 << 22) + 1), lm.ERANGE),
    (dict(X=None), lm.EINVAL), (dict(X=A + 8), lm.EINVAL), (dict(Wq=None), lm.EINVAL), (dict(Wq=B + 8), lm.EINVAL),
    (dict(s=None), lm.EINVAL), (dict(s=C + 1), lm.EINVAL), (dict(Y=None), lm.EINVAL), (dict(Y=D + 2), lm.EINVAL),
    (dict(ws=None), lm.EWORKSPACE), (dict(ws=E + 8), lm.EWORKSPACE), (dict(wsb=100), lm.EWORKSPACE),
    (dict(Y=A), lm.EINVAL), (dict(Y=B), lm.EINVAL), (dict(Y=E), lm.EINVAL), (dict(ws=A), lm.EINVAL), (dict(ws=B), lm.EINVAL),
    (dict(M=0, X=None, ws=None), lm.OK), (dict(N=0, Y=None, Wq=None), lm.OK),
])
def test_matmul_refuses(kw, code):
    assert mm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), lm.EINVAL), (dict(K=8), lm.EINVAL), (dict(N=4), lm.EINVAL), (dict(M=(1 << 22) + 1), lm.ERANGE),
    (dict(N=(1 << 22) + 8), lm.ERANGE), (dict(K=(1 << 22) + 16), lm.ERANGE), (dict(dY=None), lm.EINVAL),
    (dict(dY=A + 8), lm.EINVAL), (dict(X=None), lm.EINVAL), (dict(WqT=None), lm.EINVAL), (dict(sT=None), lm.EINVAL),
    (dict(dX=E + 8), lm.EINVAL), (dict(dW=F + 8), lm.EINVAL), (dict(ws=None), lm.EWORKSPACE), (dict(wsb=64), lm.EWORKSPACE),
    (dict(dX=F), lm.EINVAL), (dict(dX=A), lm.EINVAL), (dict(dW=B), lm.EINVAL), (dict(ws=C), lm.EINVAL), (dict(dW=G), lm.EINVAL),
    (dict(dX=None, dW=None, dY=None, ws=None), lm.OK),
])
def test_backward_refuses(kw, code):
    assert back(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), lm.EINVAL), (dict(T=-1), lm.EINVAL), (dict(H=24), lm.EINVAL), (dict(I=8), lm.EINVAL), (dict(E=0), lm.EINVAL),
    (dict(k=0), lm.EINVAL), (dict(k=5), lm.EINVAL), (dict(T=129), lm.ERANGE), (dict(E=1025), lm.ERANGE),
    (dict(E=32, k=17), lm.ERANGE), (dict(H=(1 << 22) + 16), lm.ERANGE), (dict(l=None), lm.EINVAL), (dict(l=A + MB + 2), lm.EINVAL),
    (dict(X=None), lm.EINVAL), (dict(X=A + 8), lm.EINVAL), (dict(W13=None), lm.EINVAL), (dict(W2=D + 8), lm.EINVAL),
    (dict(s13=None), lm.EINVAL), (dict(s2=None), lm.EINVAL), (dict(Y=None), lm.EINVAL), (dict(ids=None), lm.EINVAL),
    (dict(p=None), lm.EINVAL), (dict(ws=None), lm.EWORKSPACE), (dict(wsb=16), lm.EWORKSPACE), (dict(Y=A), lm.EINVAL),
    (dict(ids=F), lm.EINVAL), (dict(p=G), lm.EINVAL), (dict(ws=D), lm.EINVAL), (dict(Y=B), lm.EINVAL),
    (dict(T=0, X=None, ws=None), lm.OK), (dict(H=0, X=None), lm.OK),
])
def test_moe_refuses(kw, code):
    assert moe(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(I=1 << 21), lm.OK), (dict(I=(1 << 21) + 16), lm.ERANGE),
    (dict(T=73, E=7, k=7, I=1 << 21), lm.OK), (dict(T=128, E=4, k=4, I=1 << 21), lm.ERANGE),
    (dict(T=128, E=16, k=16, I=524160), lm.OK), (dict(T=128, E=16, k=16, I=524176), lm.ERANGE), (dict(T=64, E=16, k=16, I=524288), lm.OK),
    (dict(H=1 << 22, I=16), lm.OK), (dict(H=(1 << 22) + 16, I=16), lm.ERANGE),
])
def test_moe_bounds_of_the_columns(kw, code, monkeypatch):
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")  # a dry run
    far = 1 << 44  # addresses that nothing reads
    a = dict(X=far, l=2 * far, W13=3 * far, s13=4 * far, W2=5 * far, s2=6 * far, Y=7 * far, ids=8 * far, p=9 * far, ws=10 * far,
             wsb=1 << 40)
    assert moe(**{**a, **kw}) == code
    n = lm.fp8_moe_block_workspace_bytes(kw.get("T", 3), kw.get("H", 64), kw["I"], kw.get("E", 4), kw.get("k", 2))
    assert (n > 0) == (code == lm.OK)


def test_sizes():
    for n in (0, 1, 16, 127, 128, 129, 512, 513, 4096, 12288):
        assert lm.lib().fp8_code_pitch(n) == lm.fp8_code_pitch(n) == ref.pitch(n)
        assert lm.lib().fp8_scale_pitch(n) == lm.fp8_scale_pitch(n) == ref.sp(n)
    assert lm.lib().fp8_code_pitch(-1) == 0 and lm.lib().fp8_scale_pitch(-1) == 0
    assert lm.fp8_matmul_block_workspace_bytes(-1, 16, 8) == 0
    assert lm.fp8_matmul_block_backward_workspace_bytes(4, -16, 8) == 0
    assert lm.fp8_moe_block_workspace_bytes(1, 64, 64, 4, 5) == 0
    for dx in (False, True):
        for dw in (False, True):
            assert lm.fp8_matmul_block_backward_workspace_bytes(130, 272, 136, dx, dw) >= dx * 130 * 256 + dw * (136 + 272) * 256
    assert lm.fp8_matmul_block_workspace_bytes(130, 272, 136) >= 130 * 384
    assert lm.fp8_matmul_block_workspace_bytes(0, 272, 136) == lm.fp8_matmul_block_workspace_bytes(130, 0, 136) == 0


def _calls():
    return {
        "quantize": (lambda: quant(), ["fp8_weight"]),
        "matmul": (lambda: mm(M=300, K=1024, N=520), ["fp8_rows", "fp8_gemm"]),
        "matmul_fused": (lambda: mm(M=2, K=1024, N=520, ws=None, wsb=0), ["fp8_gemm"]),
        "matmul_k0": (lambda: mm(K=0), ["fill_zero"]),
        "backward": (lambda: back(M=300, K=1024, N=520), ["fp8_cols", "fp8_gemm_dx", "fp8_gemm_dw"]),
        "backward_dx": (lambda: back(M=300, dW=None), ["fp8_rows", "fp8_gemm_dx"]),
        "backward_dw": (lambda: back(M=300, dX=None), ["fp8_cols", "fp8_gemm_dw"]),
        "backward_no_tokens": (lambda: back(M=0, ws=None), ["fill_zero"]),
        "backward_n0": (lambda: back(N=0, ws=None, dY=None), ["fill_zero"]),
        "moe": (lambda: moe(), ["fp8_moe"]),
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


@pytest.mark.parametrize("M,K,N,path", [
    (1, 16, 8, "fp8_small_fused"), (4, 4096, 8192, "fp8_small_fused"), (4, 8192, 8192, "fp8_small_fused"), (4, 8192, 8200, "fp8_small"), (5, 4096, 8192, "fp8_small"),
    (1, 16384, 1024, "fp8_small_split"), (32, 4096, 4096, "fp8_small"), (33, 4096, 4096, "fp8_small"),
    (33, 8192, 4096, "fp8_single_split"), (65, 128, 8, "fp8_single"), (100, 4240, 264, "fp8_single_split"),
    (2048, 2048, 2048, "fp8_single"), (2048, 272, 2056, "fp8_tile128"), (4096, 4096, 2048, "fp8_tile128"),
    (4104, 4096, 2048, "fp8_tile256"), (1200, 12304, 4104, "fp8_tile256_split"), (1200, 12160, 4104, "fp8_tile128"),
])
def test_routes(M, K, N, path, monkeypatch, capfd):
    monkeypatch.setenv("LLMINT8_LOG", "1")
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")
    capfd.readouterr()
    far = 1 << 44  # addresses that nothing reads
    assert lm.lib().fp8_matmul_block(far, M, K, 0, 2 * far, 3 * far, N, 4 * far, 5 * far, 1 << 40, None) == lm.OK
    assert re.findall(r"path=(\w+)", capfd.readouterr().err) == [path]
    assert lm.fp8_matmul_block_workspace_bytes(M, K, N) < 1 << 30


@pytest.mark.parametrize("M,N,path", [(1, (1 << 29) - 8, "fp8_small"), (32, (1 << 29) - 8, "fp8_small"), (1, 1 << 29, "fp8_tile256"),
                                      (32, (1 << 31) - 8, "fp8_tile256")])
def test_routes_of_very_many_columns(M, N, path, monkeypatch, capfd):
    """The few-row kernels have a workgroup for some columns each: 2^32 threads would be too many for a launch."""
    monkeypatch.setenv("LLMINT8_LOG", "1")
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")
    capfd.readouterr()
    far = 1 << 50  # addresses that nothing reads
    assert lm.lib().fp8_matmul_block(far, M, 16, 0, 2 * far, 3 * far, N, 4 * far, 5 * far, 1 << 40, None) == lm.OK
    assert re.findall(r"path=(\w+)", capfd.readouterr().err) == [path]


@pytest.mark.parametrize("T,H,I,E,k,path", [
    (1, 2048, 768, 64, 8, "fp8_moe_light"), (3, 272, 1040, 600, 4, "fp8_moe_light_split"),
    (1, 4352, 144, 8, 2, "fp8_moe_light_wide"), (70, 272, 144, 64, 5, "fp8_moe_light_wide_split"),
    (8, 4096, 14336, 8, 2, "fp8_moe_wide_many_split"), (8, 2048, 768, 128, 8, "fp8_moe_wide_light"), (30, 528, 4112, 40, 1, "fp8_moe_wide_light_split"),
    (20, 2064, 4112, 8, 1, "fp8_moe_wide_light_split"), (50, 4128, 64, 6, 2, "fp8_moe_wide"),
    (128, 144, 272, 16, 2, "fp8_moe_many_wide_split"), (40, 144, 272, 9, 4, "fp8_moe_many_wide"),
    (128, 64, 48, 1024, 16, "fp8_moe_many_light_split"), (16, 2048, 768, 64, 4, "fp8_moe_many_light"),
    (60, 4112, 2064, 8, 2, "fp8_moe_many_split"), (20, 32768, 2064, 1, 1, "fp8_moe_wide_many"),
    (64, 4096, 1024, 140, 16, "fp8_moe_wide"), (128, 4096, 1024, 128, 16, "fp8_moe_many_split"),
])
def test_moe_routes(T, H, I, E, k, path, monkeypatch, capfd):
    monkeypatch.setenv("LLMINT8_LOG", "1")
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")
    capfd.readouterr()
    far = 1 << 44  # addresses that nothing reads
    assert lm.lib().fp8_moe_block(far, T, H, 0, 2 * far, E, k, 1, 3 * far, 4 * far, 5 * far, 6 * far, I, 7 * far,
                                  8 * far, 9 * far, 10 * far, 1 << 40, None) == lm.OK
    assert re.findall(r"path=(\w+)", capfd.readouterr().err) == [path]


def test_moe_workspace_of_every_size():
    for T in (0, 1, 2, 16, 17, 33, 128):
        for E, k in ((1, 1), (2, 2), (8, 2), (16, 16), (1024, 16)):
            for H, I in ((0, 16), (16, 0), (16, 16), (4112, 2064), (1 << 22, 16)):
                n = lm.fp8_moe_block_workspace_bytes(T, H, I, E, k)
                assert 0 <= n <= 16 * T * k * (I + 256) + 64 * T * (H + 256) + 64 * H + (1 << 20), (T, H, I, E, k)


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        lm.fp8_matmul_block(x, x, x)
    with pytest.raises(TypeError):
        lm.fp8_quantize_weight_block(x)
    with pytest.raises(TypeError):
        lm.fp8_matmul_block_backward(x, x, x, x)
    with pytest.raises(TypeError):
        lm.fp8_moe_block(x, x, x, x, x, x, top_k=1)


def test_reference_rounds_as_the_type_does():
    """The reference's e4m3 against torch's conversion, over every code, the midpoints between
    neighbours and their surroundings."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    v = torch.cat([v, -v])
    assert torch.equal(ref.e4m3(v), v.float().to(torch.float8_e4m3fn).double())


def test_reference_scales():
    a = torch.tensor([448.0, 448.0001, 447.9, 1.75, 1.7500001, 0.0, 2.0 ** -140, 224.0, 224.0001], dtype=torch.float64)
    e = ref.power_of(a)
    assert e.tolist() == [0, 1, 0, -8, -7, -127, -127, -1, 0]
    assert (a <= 448 * torch.exp2(e.double())).all()


def test_reference_on_a_case_by_hand():
    """One group: 448 * 2^-2 = 112 >= 100, so the scale is 2^-2; 100 / 2^-2 = 400 lies between the
    codes 384 and 416, at their middle: the even one is taken."""
    v, q, b = ref.coded_rows(torch.tensor([[1.0, 100.0]]))
    assert b[0, 0] == 127 - 2 and q[0, :2].tolist() == [4.0, 384.0] and v[0].tolist() == [1.0, 96.0]
