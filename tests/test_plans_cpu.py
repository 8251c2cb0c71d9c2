"""Every form of a kernel that some size takes is run by a GPU test: the forms that dry runs report over a
sweep of sizes (LLMINT8_FAULT naming no stage: nothing is enqueued, no GPU) against those of the sizes
that the GPU tests use."""
import re

import pytest

import int8_quantized_matmul_rowwise_amd as lm
from tests import test_mxfp4_gpu as mx
from tests import test_rmsnorm_gpu as rn

FAR = [i << 44 for i in range(1, 9)]  # addresses that nothing reads
NAMES = {0: None, 1: "fp8", 2: "mxfp4"}


@pytest.fixture
def plan(monkeypatch, capfd):
    monkeypatch.setenv("LLMINT8_LOG", "1")
    monkeypatch.setenv("LLMINT8_FAULT", "no_such_stage")

    def of(name, *args):
        capfd.readouterr()
        assert getattr(lm.lib(), name)(*args) == lm.OK
        err = capfd.readouterr().err
        path, = re.findall(r"path=(\w+)", err)
        values, = re.findall(r"^\[llmint8\]   plan (.*)$", err, flags=re.M)
        return (path,) + tuple(int(v) for v in re.findall(r"=(-?\d+)", values))

    return of


def edges(*borders):
    """Multiples of 16 on either side of borders."""
    return sorted({max(16, b + d) for b in borders for d in (-16, 0, 16)})


def test_norm_forms_are_tested(plan):
    x, r, w, h, y, q, s, _ = FAR

    def form(M, K, f):
        return plan("rmsnorm_forward", x, r, w, M, K, 0, 1e-6, h, y, f, q if f else None, s if f else None, None)

    taken = {form(M, K, f) for M in (1, 2, 100, 2047, 2048, 4096, 100000) for f in NAMES
             for K in edges(16, 256, 512, 768, 1024, 2048, 4096, 8192, 16384, 32768, 65536)}
    tested = {form(M, K, f) for f in NAMES for M, K in rn.SHAPES + rn.MANY}
    assert taken <= tested, sorted(taken - tested)
    assert len(taken) == 3 * 13


def test_norm_gradient_forms_are_tested(plan):
    dy, h, w, dh, dx, dw, ws, _ = FAR

    def form(M, K):
        return plan("rmsnorm_backward", dy, h, w, dh, M, K, 0, 1e-6, dx, dw, ws, 1 << 42, None)

    taken = {form(M, K) for M in (1, 100, 512, 513, 767, 768, 1023, 1024, 2047, 2048, 100000)
             for K in edges(16, 512, 1024, 2048, 4096, 8192, 16384, 32768)}
    tested = {form(M, K) for M, K in rn.BACK + rn.BACK_DENSE}
    assert taken <= tested, sorted(taken - tested)


@pytest.mark.parametrize("coded", [False, True])
def test_product_forms_are_tested(plan, coded):
    x, xs, w, ws, y, buf, _, _ = FAR

    def form(M, K, N):
        p = (plan("mxfp4_matmul_coded", x, xs, M, K, 1, w, ws, N, y, buf, 1 << 42, None) if coded else
             plan("mxfp4_matmul", x, M, K, 1, w, ws, N, y, buf, 1 << 42, None))
        # (parts of a sum or not; the fused kernel has fewer waves from 12288 columns on)
        return p[:3] + (p[3] > 1, "fused" in p[0] and N >= 12288)

    taken = {form(M, K, N) for M in (1, 3, 4, 5, 8, 9, 16, 17, 32, 33, 48, 64, 65, 128, 300, 1000, 2048, 4100)
             for K in (16, 256, 1024, 4096, 8192, 16384, 65536)
             for N in (8, 128, 1024, 2040, 2048, 4096, 8184, 8192, 12280, 12288, 16384, 24568, 24576, 32768)}
    tested = {form(*c) for c in mx.SHAPES + mx.LARGE + mx.WIDE}
    assert taken <= tested, sorted(taken - tested)
