"""64-bit reference of the 4-bit floating point operators and of the root-mean-square norm (test
infrastructure), written from their definitions and sharing no code with the library.

Bounds (derived, not fitted).  u = finfo.eps / 2 of the output's type, S a sum's terms in magnitude,
added up.
  product    a group's 32 products are whole multiples of a quarter of its scales, at most 36, and so
             is their sum: exact.  The K / 32 groups, the parts of the waves (at most 8) and those of
             the workgroups (at most 64) meet in fp32, each addition off by at most one step 2^-23 of a
             partial sum <= S: (K / 32 + 72) 2^-23 S.
  norm       the sum of K squares in fp32, each fma and each addition off by at most 2^-23 of it: a row
             of n values is added by a thread (at most K / 64 of them or 64 in turn, whichever is more),
             6 steps over lanes and at most 16 over waves; r takes half of that relative error, and a
             division, an addition of eps, a square root and a reciprocal, half a step each; y two
             products more.  Relative: (K / 64 + 64 + 22) 2^-24 + 6 * 2^-24.
  gradient   as derived in norm_backward below.
"""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def code_pitch(n):
    return -(-n // 256) * 128


def scale_pitch(n):
    return -(-n // 256) * 256


def nearest_code(v):
    """Codes 0 .. 7 of the nearest e2m1 magnitudes to |v| (64 bits), ties to the even code."""
    d = (v.abs()[..., None] - torch.tensor(E2M1, dtype=torch.float64)).abs()
    least = d.amin(dim=-1, keepdim=True)
    at = torch.arange(8)
    tied = torch.where(d == least, at, torch.full_like(at, 99))
    even = torch.where((d == least) & (at % 2 == 0), at, torch.full_like(at, 99)).amin(dim=-1)
    return torch.where(even < 99, even, tied.amin(dim=-1))


def scale_byte(a):
    """The byte of a group with the largest magnitude a: the least e >= -127 with a <= 7 2^e, found by
    trying; not finite: 255."""
    e = torch.full(a.shape, -127, dtype=torch.int64)
    for k in range(-126, 128):
        e = torch.where(a > 7 * torch.exp2((e.double())), torch.full_like(e, k), e)
    return torch.where(torch.isfinite(a), e + 127, torch.full_like(e, 255))


def coded(x):
    """(values as coded R x n, codes R x pitch bytes, scale bytes in their tiles) of x (R x n), 64 bits."""
    R, n = x.shape
    P = -(-n // 256) * 256
    w = torch.zeros(R, P, dtype=torch.float64)
    w[:, :n] = x.double()
    g = w.view(R, P // 32, 32)
    mag = torch.where(torch.isnan(g), torch.full_like(g, math.inf), g.abs()).amax(dim=2)
    b = scale_byte(mag)
    s = torch.where(b < 255, torch.exp2(b.double() - 127), torch.full_like(mag, math.nan))[:, :, None]
    c = nearest_code(torch.where(torch.isnan(s), torch.zeros_like(g), g / s))
    neg = torch.signbit(g)
    v = torch.tensor(E2M1, dtype=torch.float64)[c] * torch.where(neg, -1.0, 1.0) * s
    nib = (c + 8 * neg.long()).view(R, P)
    q = (nib[:, 0::2] + 16 * nib[:, 1::2]).to(torch.uint8)
    return v.view(R, P)[:, :n], q, tiles(b)


def tiles(b):
    """Scale bytes (R x groups, groups a multiple of 8) where the format keeps them, one at a time."""
    R, G = b.shape
    out = torch.zeros(-(-R // 32), G * 32, dtype=torch.uint8)
    r, g = torch.meshgrid(torch.arange(R), torch.arange(G), indexing="ij")
    out[r // 32, (g // 8) * 256 + (g % 4) * 64 + (r % 16) * 4 + (g % 8 // 4) * 2 + r % 32 // 16] = b.to(torch.uint8)
    return out


def values(q, s, n):
    """The values of codes (R x pitch bytes) with scales: R x n, 64 bits."""
    R = q.shape[0]
    q = q.long()
    nib = torch.stack((q & 15, q >> 4), dim=2).view(R, -1)
    v = torch.tensor(E2M1, dtype=torch.float64)[nib & 7] * torch.where(nib > 7, -1.0, 1.0)
    r, g = torch.meshgrid(torch.arange(R), torch.arange(q.shape[1] // 16), indexing="ij")
    b = s[r // 32, (g // 8) * 256 + (g % 4) * 64 + (r % 16) * 4 + (g % 8 // 4) * 2 + r % 32 // 16].double()
    w = torch.where(b < 255, torch.exp2(b - 127), torch.full_like(b, math.nan))
    return (v * w.repeat_interleave(32, dim=1))[:, :n]


def product(a, b):
    """(a b^T, its bound before the output's rounding) for 64-bit a (M x K), b (N x K)."""
    S = a.abs() @ b.abs().t()
    return a @ b.t(), (a.shape[1] / 32 + 72) * 2.0 ** -23 * S


def assert_close(got, ref, err, what=""):
    """got (16-bit) within err (before rounding) and one rounding of ref (64-bit)."""
    t = got.dtype
    lim = err + U[t] * (ref.abs() + err) + TINY[t]
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= lim)  # NaN is bad too
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}, worst {float((d / lim).nan_to_num(math.inf).max()):.3g} of the bound")


# ---- norm

def rounded(x, t):
    """64-bit x to the 16-bit type and back, one rounding (the sum of two 16-bit numbers in fp32 is exact
    or off by a step 2^-24 of it, which matters only next to a tie: such values are left to the bound)."""
    return x.float().to(t).double()


def norm(h, w, eps):
    """(y, its relative bound before rounding) of 64-bit h (M x K), already the rounded sum."""
    K = h.shape[1]
    y = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / K + eps) * w
    return y, ((K / 64 + 64 + 22) + 6) * 2.0 ** -24


def norm_backward(dy, h, w, dh, eps):
    """(dx, bound, dw, bound), both bounds before rounding, of 64-bit operands.  With e = (K / 64 + 86 + 6)
    2^-23 the relative error of either of a row's sums (against its terms in magnitude): r is off by e r / 2,
    r^3 mean(d h) h by 2 e of r^3 mean|d h| |h|, r d by e r |d|, and a few steps of each term; dw's terms dy h r
    by e, their sum over M rows in fp32 by M + 16 steps of the sum of their magnitudes."""
    M, K = h.shape
    e = (K / 64 + 92) * 2.0 ** -23
    r = 1 / torch.sqrt((h * h).sum(dim=1, keepdim=True) / K + eps)
    d = dy * w
    c, C = (d * h).sum(dim=1, keepdim=True) / K, (d * h).abs().sum(dim=1, keepdim=True) / K
    dx = r * (d - h * r * r * c)
    err = 2 * e * (r * d.abs() + h.abs() * r ** 3 * C)
    if dh is not None:
        dx = dx + dh
        err = err + 2.0 ** -23 * (dh.abs() + dx.abs())
    t = dy * h * r
    return dx, err, t.sum(dim=0), (e + (M + 16) * 2.0 ** -23) * t.abs().sum(dim=0)
