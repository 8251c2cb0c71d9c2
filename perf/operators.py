"""Cases of the 8-bit floating point block-scaled operators, with their plain forms.

The operators share one weight format: e4m3 codes with one power-of-two scale (e8m0) per
128 x 128 block.
  quantize  fp8_quantize_weight_block: a 16-bit weight to codes and scales (and both transposed)
  matmul    fp8_matmul_block: Y = X W, X coded per row in groups of 128 features
  backward  fp8_matmul_block_backward: dX and dW of that product
  moe       fp8_moe_block: a mixture-of-experts layer for few tokens on 16-bit activations

A group of values with the largest magnitude a has the smallest scale s = 2^e, e >= -127, with
a <= 448 s; its codes are the nearest e4m3 values (ties to even) of x / s.  The last group of
an axis may be short.  Rows of codes are padded with zeros to a multiple of 128, rows of scales
to a multiple of 4 with 2^-127 (the byte 0).
"""
import math

import torch

own = False  # True: run() makes the framework's calls

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
B = 128  # values of a group along each axis


def ceil_div(a, b):
    return -(-a // b)


def padded(n):
    return ceil_div(n, B) * B


def groups(n):
    return ceil_div(ceil_div(n, B), 4) * 4


# ---- cases

def listed():
    return [
        # a projection of a small model, converted while it is loaded
        {"name": "quantize_ragged", "op": "quantize", "K": 2064, "N": 7424, "dtype": "bf16", "transposed": False},
        # a training step's weight, needed in both orders
        {"name": "quantize_ffn_down", "op": "quantize", "K": 28672, "N": 8192, "dtype": "bf16", "transposed": True},
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
        # a small odd micro-batch in training
        {"name": "backward_ragged", "op": "backward", "M": 333, "K": 1040, "N": 2056, "dtype": "fp16"},
        # an up-projection in training
        {"name": "backward_ffn_up", "op": "backward", "M": 2048, "K": 4096, "N": 16384, "dtype": "bf16"},
        # many small experts, a single sequence
        {"name": "moe_one_token", "op": "moe", "T": 1, "H": 2048, "I": 768, "E": 64, "k": 8, "dtype": "bf16", "renormalize": True, "masked": False},
        # a padded batch (rows without any expert), odd sizes
        {"name": "moe_ragged", "op": "moe", "T": 37, "H": 2064, "I": 1424, "E": 60, "k": 4, "dtype": "fp16", "renormalize": False, "masked": True},
        # few large experts, a small batch
        {"name": "moe_large", "op": "moe", "T": 8, "H": 4096, "I": 14336, "E": 8, "k": 2, "dtype": "bf16", "renormalize": True, "masked": False},
    ]


def draw(rng):
    def size(lo, hi, step):  # spread over the logarithm, multiples of step
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(("quantize", "matmul", "matmul", "matmul", "backward", "moe", "moe"))
    c = {"op": op, "dtype": rng.choice(("bf16", "fp16"))}
    if op == "moe":
        c["T"], c["E"] = size(1, 64, 1), size(4, 128, 1)
        c["k"] = rng.randint(1, min(8, c["E"]))
        c["H"] = size(512, 4096, 16)
        c["I"] = size(256, 4096, 16)
        while c["E"] * c["H"] * c["I"] > 8 * 4096 * 14336:
            c["E"] = max(c["k"], c["E"] // 2)
            c["I"] = max(256, c["I"] // 32 * 16)
        c["renormalize"], c["masked"] = rng.random() < 0.5, rng.random() < 0.5
        return c
    c["K"], c["N"] = size(256, 16384, 16), size(256, 32768, 8)
    if op == "quantize":
        c["transposed"] = rng.random() < 0.5
    else:
        c["M"] = size(1, 4096, 1) if op == "matmul" else size(64, 4096, 1)
        while c["M"] * c["K"] * c["N"] > (4096 * 12288 * 36864 if op == "matmul" else 4096 * 4096 * 16384):
            c["M"] = c["M"] // 2
    return c


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["K"] * c["N"]
        return {"bytes": 2 * n + n * (2 if c["transposed"] else 1) + ceil_div(c["K"], B) * ceil_div(c["N"], B), "flops": 2 * n}
    if c["op"] == "moe":
        # the experts that T tokens with k choices each are expected to meet
        met = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
        return {"bytes": int(met * 3 * c["H"] * c["I"] * (1 + 1 / (B * B))) + c["T"] * (4 * c["H"] + 4 * c["E"] + 8 * c["k"]),
                "flops": 6 * c["T"] * c["k"] * c["H"] * c["I"]}
    M, K, N = c["M"], c["K"], c["N"]
    scales = ceil_div(K, B) * ceil_div(N, B)
    if c["op"] == "matmul":
        return {"bytes": 2 * M * K + K * N + scales + 2 * M * N, "flops": 2 * M * K * N}
    return {"bytes": 2 * M * N + 2 * M * K + K * N + scales + 2 * M * K + 2 * K * N, "flops": 4 * M * K * N}


# ---- inputs

def _codes(g, rows, cols, sigma, transposed=False):
    """Random codes (rows x cols, pitch padded with zeros) and block scales of a weight ~ N(0, sigma)."""
    q = torch.randn(rows, cols, generator=g, device=g.device, dtype=torch.float32).mul_(448 / 4.5).clamp_(-448, 448).to(F8)
    most = int(math.floor(math.log2(sigma * 4.5 / 448))) + 127
    s = torch.zeros(ceil_div(rows, B), groups(cols), dtype=torch.uint8, device=g.device)
    s[:, :ceil_div(cols, B)] = torch.randint(most - 1, most + 1, (ceil_div(rows, B), ceil_div(cols, B)), generator=g, device=g.device)
    out = torch.zeros(rows, padded(cols), dtype=torch.uint8, device=g.device)
    out[:, :cols] = q.view(torch.uint8)
    if not transposed:
        return out.view(F8), s.view(E8)
    st = torch.zeros(ceil_div(cols, B), groups(rows), dtype=torch.uint8, device=g.device)
    st[:, :ceil_div(rows, B)] = s[:, :ceil_div(cols, B)].t()
    turned = torch.zeros(cols, padded(rows), dtype=torch.uint8, device=g.device)
    turned[:, :rows] = q.view(torch.uint8).t()
    return turned.view(F8), st.view(E8)


def _acts(g, M, K, dtype):
    """Activations ~ N(0, 1), a few features of every row far larger."""
    x = torch.randn(M, K, generator=g, device=g.device)
    cols = torch.randint(0, K, (6,), generator=g, device=g.device)
    x[:, cols] *= 20.0
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(int(seed))
    c, t = case, DT[case["dtype"]]
    s = {"case": case}
    if c["op"] == "quantize":
        s["W"] = torch.randn(c["K"], c["N"], generator=g, device=g.device).mul_(0.02).to(t)
    elif c["op"] == "matmul":
        s["X"] = _acts(g, c["M"], c["K"], t)
        s["Wq"], s["s_w"] = _codes(g, c["N"], c["K"], 0.02)
    elif c["op"] == "backward":
        s["X"] = _acts(g, c["M"], c["K"], t)
        s["dY"] = torch.randn(c["M"], c["N"], generator=g, device=g.device).mul_(1e-2).to(t)
        s["WqT"], s["s_wT"] = _codes(g, c["N"], c["K"], 0.02, transposed=True)
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        s["X"] = torch.randn(T, H, generator=g, device=g.device).to(t)
        s["logits"] = 2.0 * torch.randn(T, E, generator=g, device=g.device)
        if c["masked"]:  # some experts closed to some tokens, and rows of padding at the end
            s["logits"][torch.rand(T, E, generator=g, device=g.device) < 0.1] = -math.inf
            s["logits"][T - T // 8:] = -math.inf
        up = [_codes(g, 2 * I, H, 0.03) for _ in range(E)]
        down = [_codes(g, H, I, 0.03) for _ in range(E)]
        s["W13q"] = torch.stack([q.view(torch.uint8) for q, _ in up]).view(F8)
        s["W2q"] = torch.stack([q.view(torch.uint8) for q, _ in down]).view(F8)
        s["s_w13"] = torch.stack([v.view(torch.uint8) for _, v in up]).view(E8)
        s["s_w2"] = torch.stack([v.view(torch.uint8) for _, v in down]).view(E8)
    return s


# ---- one pass

def run(state):
    c = state["case"]
    if own:
        import int8_quantized_matmul_rowwise_amd as lm

        if c["op"] == "quantize":
            return lm.fp8_quantize_weight_block(state["W"], transposed=c["transposed"])
        if c["op"] == "matmul":
            return lm.fp8_matmul_block(state["X"], state["Wq"], state["s_w"])
        if c["op"] == "backward":
            return lm.fp8_matmul_block_backward(state["dY"], state["X"], state["WqT"], state["s_wT"])
        return lm.fp8_moe_block(state["X"], state["logits"], state["W13q"], state["s_w13"], state["W2q"], state["s_w2"],
                                top_k=c["k"], renormalize=c["renormalize"])
    if c["op"] == "quantize":
        return _plain_quantize(state["W"], c["transposed"])
    if c["op"] == "matmul":
        X = state["X"]
        return (_rows(X) @ _weight(state["Wq"], state["s_w"], X.shape[1]).t()).to(X.dtype)
    if c["op"] == "backward":
        X, dY = state["X"], state["dY"]
        dX = _rows(dY) @ _weight(state["WqT"], state["s_wT"], dY.shape[1]).t()
        dW = _rows(X.t()) @ _rows(dY.t()).t()
        return dX.to(X.dtype), dW.to(X.dtype)
    return _plain_moe(state)


def _bytes(a):
    """The e8m0 bytes (2^(byte - 127)) of groups with the largest magnitudes a: 448 = 0.875 * 2^9."""
    m, e = torch.frexp(a)
    e = e + (m > 0.875).to(e.dtype) - 9 + 127
    return torch.where(a > 0, e, torch.zeros_like(e)).clamp_(min=0)


def _power(b):
    return b.to(torch.uint8).view(E8).float()


def _plain_quantize(W, transposed):
    K, N = W.shape
    w = torch.zeros(padded(N), padded(K), dtype=torch.float32, device=W.device)
    w[:N, :K] = W.t()
    w = w.view(padded(N) // B, B, padded(K) // B, B)
    b = _bytes(w.abs().amax(dim=(1, 3)))
    q = (w / _power(b)[:, None, :, None]).view(padded(N), padded(K)).to(F8)

    def laid(b):
        out = torch.zeros(b.shape[0], groups(b.shape[1] * B), dtype=torch.uint8, device=W.device)
        out[:, :b.shape[1]] = b
        return out.view(E8)

    if not transposed:
        return q[:N], laid(b)
    return q[:N], laid(b), q[:, :K].view(torch.uint8).t().contiguous().view(F8), laid(b.t())


def _rows(X):
    """X's values after coding, in fp32: groups of 128 along each row."""
    M, K = X.shape
    x = torch.zeros(M, padded(K), dtype=torch.float32, device=X.device)
    x[:, :K] = X
    x = x.view(M, padded(K) // B, B)
    s = _power(_bytes(x.abs().amax(dim=2)))[:, :, None]
    return ((x / s).to(F8).float() * s).view(M, padded(K))[:, :K]


def _weight(q, s, cols):
    """The values that codes (R x pitch) with block scales stand for: R x cols, fp32."""
    R = q.shape[-2]
    wide = s.float().repeat_interleave(B, dim=-1)[..., :cols].repeat_interleave(B, dim=-2)[..., :R, :]
    return q[..., :cols].float() * wide


def _plain_moe(state):
    c, X = state["case"], state["X"]
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    l, order = torch.sort(state["logits"], dim=1, descending=True, stable=True)
    l, ids = l[:, :k], order[:, :k]
    open_ = l > -math.inf
    top = torch.where(open_[:, :1], l[:, :1], torch.zeros_like(l[:, :1]))
    e = torch.where(open_, torch.exp(l - top), torch.zeros_like(l))
    total = (e if c["renormalize"] else torch.exp(state["logits"] - top)).sum(dim=1, keepdim=True)
    p = torch.where(open_, e / total, torch.zeros_like(e))
    if T * k <= E:  # the chosen experts' weights alone
        at, x = ids.reshape(-1), X.float().repeat_interleave(k, dim=0)[:, :, None]
        gu = torch.bmm(_weight(state["W13q"].view(torch.uint8)[at].view(F8), state["s_w13"].view(torch.uint8)[at].view(E8), H), x)
        h = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).to(X.dtype).float()
        y = torch.bmm(_weight(state["W2q"].view(torch.uint8)[at].view(F8), state["s_w2"].view(torch.uint8)[at].view(E8), I), h).view(T, k, H)
        y = (y * p[:, :, None]).sum(dim=1)
    else:  # every expert on every token
        gu = torch.matmul(_weight(state["W13q"], state["s_w13"], H), X.float().t())
        h = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).to(X.dtype).float()
        y = torch.bmm(_weight(state["W2q"], state["s_w2"], I), h.contiguous())
        gate = torch.zeros(T, E, device=X.device).scatter_(1, ids, p)
        y = (y * gate.t()[:, None, :]).sum(dim=0).t()
    ids = torch.where(open_, ids, torch.full_like(ids, -1))
    return y.to(X.dtype), ids.to(torch.int32), p


# ---- the definition in 64 bits

def _e4m3(v):
    """The nearest e4m3 value (ties to even) of 64-bit values up to 448 in magnitude."""
    e = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _scale(a):
    """The scales of groups with the largest magnitudes a."""
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448.0))
    return torch.exp2(torch.where(a > 0, e, torch.full_like(e, -127)).clamp(min=-127))


def _coded(x, dim):
    """The values of 64-bit x after coding in groups of 128 along dim."""
    parts = []
    for part in x.split(B, dim=dim):
        s = _scale(part.abs().amax(dim=dim, keepdim=True))
        parts.append(_e4m3(part / s) * s)
    return torch.cat(parts, dim=dim)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        W = s["W"]
        K, N = c["K"], c["N"]
        q = torch.zeros(N, padded(K), dtype=F8, device=W.device)
        sw = torch.full((ceil_div(N, B), groups(K)), 2.0 ** -127, dtype=torch.float64, device=W.device)
        for b in range(ceil_div(K, B)):
            w = torch.zeros(B, padded(N), dtype=torch.float64, device=W.device)
            w[: min(B, K - b * B), :N] = W[b * B:(b + 1) * B]
            w = w.view(B, padded(N) // B, B)
            sw[:, b] = _scale(w.abs().amax(dim=(0, 2)))
            codes = _e4m3(w / sw[:, b][None, :, None])
            q[:, b * B:(b + 1) * B] = codes.view(B, padded(N))[:, :N].t().float().to(F8)
        if not c["transposed"]:
            return q, sw
        t = torch.zeros(K, padded(N), dtype=torch.uint8, device=W.device)
        t[:, :N] = q.view(torch.uint8)[:, :K].t()
        swt = torch.full((ceil_div(K, B), groups(N)), 2.0 ** -127, dtype=torch.float64, device=W.device)
        swt[:, :ceil_div(N, B)] = sw[:, :ceil_div(K, B)].t()
        return q, sw, t.view(F8), swt

    def weight(q, sc, cols):
        at_r = torch.arange(q.shape[0], device=q.device) // B
        at_c = torch.arange(cols, device=q.device) // B
        return q[:, :cols].float().double() * sc.float().double()[at_r][:, at_c]

    if c["op"] == "matmul":
        return _coded(s["X"].double(), 1) @ weight(s["Wq"], s["s_w"], c["K"]).t()
    if c["op"] == "backward":
        x, dy = s["X"].double(), s["dY"].double()
        dx = _coded(dy, 1) @ weight(s["WqT"], s["s_wT"], c["N"]).t()
        dw = _coded(x, 0).t().contiguous() @ _coded(dy, 0)
        return dx, dw
    T, I, k = c["T"], c["I"], c["k"]
    x, logits = s["X"].double(), s["logits"].double()
    order = sorted  # of each row on the host: highest first, the lowest expert among equals
    y = torch.zeros(T, c["H"], dtype=torch.float64, device=x.device)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    p = torch.zeros(T, k, dtype=torch.float64)
    for t, row in enumerate(logits.tolist()):
        best = [e for e in order(range(len(row)), key=lambda e: (-row[e], e)) if row[e] > -math.inf][:k]
        if not best:
            continue
        among = [row[e] for e in best] if c["renormalize"] else row
        total = math.fsum(math.exp(v - row[best[0]]) for v in among)
        for j, e in enumerate(best):
            ids[t, j], p[t, j] = e, math.exp(row[e] - row[best[0]]) / total
    for e in range(c["E"]):
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        if not len(rows):
            continue
        gu = weight(s["W13q"][e], s["s_w13"][e], c["H"]) @ x[rows.to(x.device)].t()
        h = (gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]).to(DT[c["dtype"]]).double()
        out = weight(s["W2q"][e], s["s_w2"][e], I) @ h
        y[rows.to(x.device)] += out.t() * p[rows, slots].to(x.device)[:, None]
    return y, ids, p
