"""Cases of the 4-bit floating point operators and of the norm that feeds the products, with their
plain forms.

  codec          mxfp4_quantize, mxfp4_dequantize: a 16-bit matrix to e2m1 codes with a power-of-two
                 scale per 32 values (microscaled 4-bit floating point), and back
  matmul         mxfp4_matmul: Y = X W on such a weight, X coded per row inside the call
  norm           rmsnorm, rmsnorm_quantize: residual addition and root-mean-square norm, its output
                 in 16 bits or as e4m3 codes with a scale per 128 features
  norm_matmul    rmsnorm_quantize and mxfp4_matmul_coded: the norm's output as e2m1 codes, and the
                 product that takes them
  norm_backward  rmsnorm_backward: the norm's gradients

A group of 32 values with the largest magnitude a has the smallest scale s = 2^e, e >= -127, with
a <= 7 s; its codes are the nearest e2m1 values (ties to even, magnitudes above 6 to 6) of x / s.
A row of codes over n values is padded with zeros to a multiple of 256 values, two codes to a byte,
the first in the low half.  Scales lie in tiles of 32 rows x 256 values (256 bytes, zero past the
last row and group): the byte of row r and group g of a tile is at
  64 (g % 4) + 4 (r % 16) + 2 (g / 4) + r / 16.
e4m3 codes: a <= 448 s in groups of 128 features, rows of codes padded with zeros to a multiple of
128, and the byte of row r and group g at g R + (r / 64) 64 + 4 (r % 16) + (r / 16) % 4, R being the
rows rounded up to a multiple of 64.
"""
import math

import torch

own = False  # True: run() makes the framework's calls

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


def up(n, m):
    return -(-n // m) * m


# ---- cases

def listed():
    return [
        # a projection of a small model, converted while it is loaded
        {"name": "codec_ragged", "op": "codec", "R": 2064, "C": 7424, "columns": True, "dtype": "bf16"},
        # a large layer's weight in a checkpoint's order, one row per output
        {"name": "codec_ffn_down", "op": "codec", "R": 8192, "C": 28672, "columns": False, "dtype": "fp16"},
        # a generated token of a single sequence
        {"name": "one_token", "op": "matmul", "M": 1, "K": 4096, "N": 4096, "dtype": "bf16"},
        # a batch of sequences, one new token each
        {"name": "decode", "op": "matmul", "M": 16, "K": 8192, "N": 8192, "dtype": "bf16"},
        # a prompt of odd length on sizes that fill no tile
        {"name": "ragged", "op": "matmul", "M": 1000, "K": 2064, "N": 7424, "dtype": "fp16"},
        # prompts through an up-projection
        {"name": "ffn_up", "op": "matmul", "M": 2048, "K": 4096, "N": 16384, "dtype": "fp16"},
        # a large prompt batch through the joint projection of a large model
        {"name": "qkv_175b", "op": "matmul", "M": 4096, "K": 12288, "N": 36864, "dtype": "fp16"},
        # the norm before the first layer of a single sequence's new token
        {"name": "norm_token", "op": "norm", "M": 1, "K": 4096, "dtype": "bf16", "residual": False, "out": "16"},
        # prompts between two layers, coded for the 8-bit product
        {"name": "norm_prompt", "op": "norm", "M": 2048, "K": 4096, "dtype": "fp16", "residual": True, "out": "fp8"},
        # the end of one layer and the start of the next, for a batch of new tokens
        {"name": "norm_matmul_decode", "op": "norm_matmul", "M": 16, "K": 8192, "N": 8192, "dtype": "bf16"},
        # a small odd micro-batch in training
        {"name": "norm_backward_ragged", "op": "norm_backward", "M": 333, "K": 1040, "dtype": "fp16", "residual": False},
        # a training step's rows between two layers of a large model
        {"name": "norm_backward_large", "op": "norm_backward", "M": 8192, "K": 8192, "dtype": "bf16", "residual": True},
    ]


def draw(rng):
    def size(lo, hi, step):  # spread over the logarithm, multiples of step
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    c = {"op": rng.choice(("codec", "matmul", "matmul", "matmul", "norm", "norm", "norm_matmul", "norm_backward")),
         "dtype": rng.choice(("bf16", "fp16"))}
    if c["op"] == "codec":
        c["columns"] = rng.random() < 0.5
        c["R"], c["C"] = (size(256, 16384, 16), size(256, 28672, 8)) if c["columns"] else (size(1, 16384, 1), size(256, 28672, 16))
        while c["R"] * c["C"] > 8192 * 28672:
            c["R"] = max(16, c["R"] // 32 * 16)
        return c
    c["M"], c["K"] = size(1, 16384, 1), size(256, 16384, 16)
    if c["op"] in ("norm", "norm_backward"):
        while c["M"] * c["K"] > 8192 * 8192:
            c["M"] //= 2
        c["residual"] = rng.random() < 0.6
        if c["op"] == "norm":
            c["out"] = rng.choice(("16", "fp8"))
        return c
    c["N"] = size(256, 32768, 8)
    c["M"] = min(c["M"], 4096) if c["op"] == "matmul" else size(1, 256, 1)
    while c["M"] * c["K"] * c["N"] > 4096 * 12288 * 36864:
        c["M"] //= 2
    return c


def codes_bytes(rows, n):
    return rows * n // 2 + rows * -(-n // 32)


def work(case):
    c = case
    if c["op"] == "codec":
        rows, n = (c["C"], c["R"]) if c["columns"] else (c["R"], c["C"])
        return {"bytes": 4 * rows * n + 2 * codes_bytes(rows, n), "flops": 4 * rows * n}
    M, K = c["M"], c["K"]
    x = 2 * M * K
    if c["op"] == "matmul":
        return {"bytes": x + codes_bytes(c["N"], K) + 2 * M * c["N"], "flops": 2 * M * K * c["N"]}
    if c["op"] == "norm_matmul":
        return {"bytes": 3 * x + 2 * K + codes_bytes(c["N"], K) + 2 * M * c["N"], "flops": 2 * M * K * c["N"]}
    if c["op"] == "norm":
        out = x if c["out"] == "16" else M * K + M * -(-K // 128)
        return {"bytes": x * (3 if c["residual"] else 1) + 2 * K + out, "flops": 5 * M * K}
    return {"bytes": x * (4 if c["residual"] else 3) + 4 * K, "flops": 10 * M * K}


# ---- inputs

def _weight(g, rows, n, sigma):
    """Random codes and scales of a weight ~ N(0, sigma), rows x n."""
    q = torch.randint(0, 256, (rows, n // 2), generator=g, device=g.device, dtype=torch.uint8)
    out = torch.zeros(rows, up(n, 256) // 2, dtype=torch.uint8, device=g.device)
    out[:, :n // 2] = q
    most = int(math.floor(math.log2(sigma * 2.5 / 6))) + 127
    s = torch.randint(most - 1, most + 1, (rows, -(-n // 32)), generator=g, device=g.device, dtype=torch.uint8)
    return out, _tiles(s)


def _acts(g, M, K):
    """Activations ~ N(0, 1), a few features of every row far larger."""
    x = torch.randn(M, K, generator=g, device=g.device)
    cols = torch.randint(0, K, (6,), generator=g, device=g.device)
    x[:, cols] *= 20.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(int(seed))
    c, t = case, DT[case["dtype"]]
    s = {"case": case}
    if c["op"] == "codec":
        s["X"] = torch.randn(c["R"], c["C"], generator=g, device=g.device).mul_(0.02).to(t)
        return s
    M, K = c["M"], c["K"]
    if c["op"] == "norm_backward":
        s["H"] = (2.0 * _acts(g, M, K)).to(t)
        s["dY"] = torch.randn(M, K, generator=g, device=g.device).mul_(1e-2).to(t)
        if c["residual"]:
            s["dH"] = torch.randn(M, K, generator=g, device=g.device).mul_(1e-2).to(t)
    else:
        s["X"] = _acts(g, M, K).to(t)
    if c["op"] != "matmul":
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device=g.device)).to(t)
        if c.get("residual", c["op"] == "norm_matmul") and c["op"] != "norm_backward":
            s["residual"] = (2.0 * _acts(g, M, K)).to(t)
    if c["op"] in ("matmul", "norm_matmul"):
        s["Wq"], s["w_scale"] = _weight(g, c["N"], K, 0.02)
    return s


# ---- one pass

def run(state):
    c = state["case"]
    if own:
        import int8_quantized_matmul_rowwise_amd as lm

        if c["op"] == "codec":
            q, scale = lm.mxfp4_quantize(state["X"], columns=c["columns"])
            values = lm.mxfp4_dequantize(q, scale, c["R"] if c["columns"] else c["C"], state["X"].dtype)
            return values, scale.view(E8)
        if c["op"] == "matmul":
            return lm.mxfp4_matmul(state["X"], state["Wq"], state["w_scale"])
        if c["op"] == "norm_backward":
            return lm.rmsnorm_backward(state["dY"], state["H"], state["weight"], dH=state.get("dH"), eps=EPS)
        if c["op"] == "norm_matmul":
            q, scale, _, H = lm.rmsnorm_quantize(state["X"], state["weight"], residual=state["residual"], eps=EPS, format="mxfp4")
            return lm.mxfp4_matmul_coded(q, scale, state["Wq"], state["w_scale"], state["X"].dtype), H
        if c["out"] == "16":
            return lm.rmsnorm(state["X"], state["weight"], residual=state.get("residual"), eps=EPS)
        q, scale, _, H = lm.rmsnorm_quantize(state["X"], state["weight"], residual=state.get("residual"), eps=EPS, format="fp8")
        return q, scale, H
    if c["op"] == "codec":
        v, b = _coded4(state["X"].t() if c["columns"] else state["X"])
        return v.to(state["X"].dtype), _tiles(b).view(E8)
    if c["op"] == "norm_backward":
        return _plain_backward(state)
    if c["op"] == "matmul":
        X = state["X"]
        return (_coded4(X)[0] @ _values(state["Wq"], state["w_scale"], c["K"]).t()).to(X.dtype)
    Y, H = _plain_norm(state["X"], state["weight"], state.get("residual"))
    if c["op"] == "norm_matmul":
        return (_coded4(Y)[0] @ _values(state["Wq"], state["w_scale"], c["K"]).t()).to(Y.dtype), H
    if c["out"] == "16":
        return Y, H
    q, scale = _coded8(Y)
    return q, scale, H


def _tiles(b):
    """Scale bytes (rows x groups of 32) in tiles of 32 rows x 8 groups."""
    R, G = b.shape
    out = torch.zeros(up(R, 32), up(G, 8), dtype=torch.uint8, device=b.device)
    out[:R, :G] = b
    out = out.view(up(R, 32) // 32, 2, 16, up(G, 8) // 8, 2, 4)  # tile, r / 16, r % 16; tile, g / 4, g % 4
    return out.permute(0, 3, 5, 2, 4, 1).reshape(up(R, 32) // 32, up(G, 8) * 32)


def _untiled(s, rows, groups):
    """The scale bytes (rows x groups) of such tiles."""
    T = s.shape[0]
    b = s.view(T, s.shape[1] // 256, 4, 16, 2, 2).permute(0, 5, 3, 1, 4, 2)
    return b.reshape(T * 32, s.shape[1] // 32)[:rows, :groups]


def _bytes(a, most):
    """The e8m0 bytes (2^(byte - 127)) of groups with the largest magnitudes a, most = 1.75 * 2^n the
    largest quotient."""
    m, e = torch.frexp(a)
    e = e + (m > 0.875).to(e.dtype) - int(math.log2(most / 0.875)) + 127
    return torch.where(a > 0, e, torch.zeros_like(e)).clamp_(min=0)


def _power(b):
    return b.to(torch.uint8).view(E8).float()


def _coded4(X):
    """(X's values after coding in groups of 32 along each row, fp32; the scales' bytes)"""
    M, K = X.shape
    x = torch.zeros(M, up(K, 32), dtype=torch.float32, device=X.device)
    x[:, :K] = X
    x = x.view(M, up(K, 32) // 32, 32)
    b = _bytes(x.abs().amax(dim=2), 7.0)
    s = _power(b)[:, :, None]
    v = x / s
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    v = torch.copysign((torch.round(m / step) * step).clamp_(max=6.0), v)
    return (v * s).view(M, up(K, 32))[:, :K], b


def _values(q, scale, n):
    """The values that codes (rows x pitch bytes) with scales stand for: rows x n, fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=q.device)
    q = q[:, :n // 2].int()
    v = torch.stack((table[q & 15], table[q >> 4]), dim=2).view(q.shape[0], n)
    return v * _power(_untiled(scale, q.shape[0], -(-n // 32))).repeat_interleave(32, dim=1)[:, :n]


def _coded8(X):
    """e4m3 codes (rows padded to a multiple of 128) and scales of X in groups of 128 along each row."""
    M, K = X.shape
    x = torch.zeros(M, up(K, 128), dtype=torch.float32, device=X.device)
    x[:, :K] = X
    x = x.view(M, up(K, 128) // 128, 128)
    b = _bytes(x.abs().amax(dim=2), 448.0)
    q = (x / _power(b)[:, :, None]).view(M, up(K, 128)).to(F8)
    s = torch.zeros(up(M, 64), b.shape[1], dtype=torch.uint8, device=X.device)
    s[:M] = b
    return q, s.view(up(M, 64) // 64, 4, 16, b.shape[1]).permute(3, 0, 2, 1).reshape(b.shape[1], up(M, 64)).view(E8)


def _plain_norm(X, weight, residual):
    """(the norm of X + residual, that sum): both rounded once to X's type, the norm taken of the rounded sum."""
    H = X if residual is None else (X.float() + residual.float()).to(X.dtype)
    h = H.float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * weight.float()
    return y.to(X.dtype), None if residual is None else H


def _plain_backward(state):
    h, w, dy = state["H"].float(), state["weight"].float(), state["dY"].float()
    r = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    dw = (dy * h * r).sum(dim=0)
    d = dy * w
    dx = r * (d - h * (r * r * (d * h).mean(dim=1, keepdim=True)))
    if "dH" in state:
        dx = dx + state["dH"].float()
    return dx.to(state["H"].dtype), dw.to(state["H"].dtype)


# ---- the definition in 64 bits

def _nearest(v, bits, least, most):
    """The nearest value (ties to even) with `bits` bits after the first, exponents from `least` on, to v in 64 bits."""
    e = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=least) - bits)
    return (torch.round(v / step) * step).clamp(-most, most)


def _scales(a, most):
    """The scales of groups with the largest magnitudes a."""
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / most))
    return torch.exp2(torch.where(a > 0, e, torch.full_like(e, -127)).clamp(min=-127))


def _group(x, size, bits, least, most, top):
    """(codes, scales) of 64-bit x in groups along its rows: lists over the groups."""
    q, s = [], []
    for part in x.split(size, dim=1):
        s.append(_scales(part.abs().amax(dim=1, keepdim=True), top))
        q.append(_nearest(part / s[-1], bits, least, most))
    return q, s


def _four(x):
    q, s = _group(x, 32, 1, 0, 6.0, 7.0)
    return torch.cat([a * b for a, b in zip(q, s)], dim=1), torch.cat(s, dim=1)


def _decoded(q, scale, n):
    """The values of a coded weight, a nibble and a scale byte at a time."""
    rows = torch.arange(q.shape[0], device=q.device)[:, None]
    at = torch.arange(n, device=q.device)[None, :]
    code = (q.long().gather(1, (at // 2).expand(q.shape[0], n)) >> (4 * (at % 2))) & 15
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2) * (1 - 2 * (code >> 3).double())
    g = torch.arange(-(-n // 32), device=q.device)[None, :]
    place = (g // 8) * 256 + 64 * (g % 4) + 4 * (rows % 16) + 2 * (g % 8 // 4) + rows % 32 // 16
    e = scale[rows // 32, place].double() - 127
    return v * torch.exp2(e).repeat_interleave(32, dim=1)[:, :n]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    t = DT[c["dtype"]]
    if c["op"] == "codec":
        x = (s["X"].t() if c["columns"] else s["X"]).double()
        v, sc = _four(x)
        R, G = sc.shape
        out = torch.full((up(R, 32) // 32, up(G, 8) * 32), 2.0 ** -127, dtype=torch.float64, device=x.device)
        r = torch.arange(R, device=x.device)[:, None]
        g = torch.arange(G, device=x.device)[None, :]
        out[r // 32, (g // 8) * 256 + 64 * (g % 4) + 4 * (r % 16) + 2 * (g % 8 // 4) + r % 32 // 16] = sc
        return v, out
    if c["op"] == "matmul":
        return _four(s["X"].double())[0] @ _decoded(s["Wq"], s["w_scale"], c["K"]).t()
    w = s["weight"].double()
    if c["op"] == "norm_backward":
        h, dy = s["H"].double(), s["dY"].double()
        rms = (h.pow(2).sum(dim=1) / c["K"] + EPS).sqrt()[:, None]
        n = h / rms
        g = dy * w
        dx = (g - n * ((g * n).sum(dim=1) / c["K"])[:, None]) / rms
        return dx + s["dH"].double() if c["residual"] else dx, (dy * n).sum(dim=0)
    H = None
    h = s["X"].double()
    if "residual" in s:
        H = h + s["residual"].double()
        h = H.to(t).double()
    y = h / (h.pow(2).sum(dim=1, keepdim=True) / c["K"] + EPS).sqrt() * w
    if c["op"] == "norm_matmul":
        return _four(y.to(t).double())[0] @ _decoded(s["Wq"], s["w_scale"], c["K"]).t(), H
    if c["out"] == "16":
        return y, H
    M, K = c["M"], c["K"]
    q, sc = _group(y.to(t).double(), 128, 3, -6, 448.0, 448.0)
    codes = torch.zeros(M, up(K, 128), dtype=torch.float64, device=y.device)
    codes[:, :K] = torch.cat(q, dim=1)
    scales = torch.full((len(sc), up(M, 64)), 2.0 ** -127, dtype=torch.float64, device=y.device)
    r = torch.arange(M, device=y.device)
    scales[:, r // 64 * 64 + 4 * (r % 16) + r // 16 % 4] = torch.cat(sc, dim=1).t()
    return codes, scales, H
