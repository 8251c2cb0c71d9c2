"""64-bit reference of the e4m3 block-scaled operators (test infrastructure), written from the
format's definition and sharing no code with the library.

Bounds (derived, not fitted).  Let S be a sum's products in magnitude, added up.
  matrix unit, e4m3    it adds each run of 8 products aligned to the largest of them, dropping
                       what lies below 2^-13 of that one's binade: at most 8 * 2^-13 = 2^-10 of
                       the largest, so 2^-10 S over the sum; the run sums are added in fp32,
                       each addition off by at most one step 2^-23 of a partial sum <= S;
  16-bit products      exact in fp32; K additions, each at most 2^-23 S;
  output               one rounding, half a step u = finfo.eps / 2 of the value, or half the
                       smallest subnormal.
"""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def pitch(n):
    return -(-n // 128) * 128


def sp(n):
    return -(-n // 512) * 4


def power_of(a):
    """The exponent e of the scale of each group with largest magnitude a (64 bits)."""
    m, e = torch.frexp(a)  # a = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(a > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def e4m3(v):
    """The nearest e4m3 value, ties to even, of 64-bit values of magnitude up to 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step


def coded_rows(x):
    """(values as coded, codes padded to the pitch, scale bytes padded) of x (R x C) in groups
    of 128 along its rows; 64 bits."""
    R, C = x.shape
    w = torch.zeros(R, pitch(C), dtype=torch.float64)
    w[:, :C] = x.double()
    w = w.view(R, pitch(C) // 128, 128)
    e = power_of(w.abs().amax(dim=2))
    s = torch.exp2(e.double())[:, :, None]
    q = e4m3(w / s)
    b = torch.zeros(R, sp(C), dtype=torch.uint8)
    b[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return (q * s).view(R, -1)[:, :C], q.view(R, -1), b


def coded_weight(W):
    """(What K x N, Wq N x pitch(K), s_w bytes, WqT K x pitch(N), s_wT bytes) of W (K x N)."""
    K, N = W.shape
    w = torch.zeros(pitch(K), pitch(N), dtype=torch.float64)
    w[:K, :N] = W.double()
    w = w.view(pitch(K) // 128, 128, pitch(N) // 128, 128)
    e = power_of(w.abs().amax(dim=(1, 3)))
    s = torch.exp2(e.double())
    q = e4m3(w / s[:, None, :, None])
    what = (q * s[:, None, :, None]).reshape(pitch(K), pitch(N))[:K, :N]
    q = q.reshape(pitch(K), pitch(N))
    sw = torch.zeros(e.shape[1], sp(K), dtype=torch.uint8)
    sw[:, :e.shape[0]] = (e + 127).t().to(torch.uint8)
    swt = torch.zeros(e.shape[0], sp(N), dtype=torch.uint8)
    swt[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return what, q[:, :N].t(), sw, q[:K], swt


def weight_values(Wq, s, K):
    """The values of a weight held as codes (N x pitch(K)) with block scales, N x K, 64 bits."""
    b = s.view(torch.uint8).double()
    wide = torch.exp2(b - 127).repeat_interleave(128, 0)[: Wq.shape[0]].repeat_interleave(128, 1)[:, :K]
    return Wq.view(torch.float8_e4m3fn).float().double()[:, :K] * wide


def product(a, b):
    """(a b^T, its bound before the output's rounding) for 64-bit a (M x K), b (N x K)."""
    S = a.abs() @ b.abs().t()
    K = a.shape[1]
    return a @ b.t(), (2.0 ** -10 + (K / 8 + 32) * 2.0 ** -23) * S


def assert_close(got, ref, err, what=""):
    """got (16-bit) within err (before rounding) and one rounding of ref (64-bit)."""
    t = got.dtype
    lim = err + U[t] * (ref.abs() + err) + TINY[t]
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= lim)  # NaN is bad too
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}, worst {float((d / lim).nan_to_num(math.inf).max()):.3g} of the bound")


def route(logits, k, renormalize):
    """(ids, p) of one layer's gate, on the host in 64 bits."""
    T, E = logits.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    p = torch.zeros(T, k, dtype=torch.float64)
    big = torch.finfo(torch.float32).max
    for t in range(T):
        l = [(-math.inf if math.isnan(v) else min(v, big)) for v in logits[t].tolist()]
        best = [e for e in sorted(range(E), key=lambda e: (-l[e], e)) if l[e] > -math.inf][:k]
        if not best:
            continue
        top = l[best[0]]
        z = math.fsum(math.exp(l[e] - top) for e in (best if renormalize else range(E)))
        for j, e in enumerate(best):
            ids[t, j] = e
            p[t, j] = math.exp(l[e] - top) / z
    return ids, p


def moe(X, logits, W13, W2, k, renormalize):
    """(y, its bound before rounding, ids, p): W13 E x 2I x H, W2 E x H x I, 64-bit values."""
    t = X.dtype
    x = X.double()
    T, H = x.shape
    E, I = W13.shape[0], W13.shape[1] // 2
    ids, p = route(logits.cpu(), k, renormalize)
    y = torch.zeros(T, H, dtype=torch.float64)
    err = torch.zeros_like(y)
    for i in range(T):
        for j in range(k):
            e = int(ids[i, j])
            if e < 0:
                continue
            gu, S = W13[e] @ x[i], W13[e].abs() @ x[i].abs()
            d = H * 2.0 ** -23 * S
            g, u = gu[:I], gu[I:]
            silu = g * torch.sigmoid(g)
            h = silu * u
            # |silu'| <= 1.1; exp, division and the two products: a few steps each
            dh = 1.1 * d[:I] * (u.abs() + d[I:]) + silu.abs() * d[I:] + 16 * 2.0 ** -23 * h.abs()
            hr = h.to(torch.float32).to(t).double()
            dh = dh + (hr - h).abs() + 2 * U[t] * h.abs() + TINY[t]
            y[i] += p[i, j] * (W2[e] @ hr)
            mag = W2[e].abs() @ (hr.abs() + dh)
            err[i] += p[i, j] * (W2[e].abs() @ dh + (I + 64) * 2.0 ** -23 * mag)
    return y, err, ids, p
