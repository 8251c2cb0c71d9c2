"""LLM.int8() matmul for AMD Instinct MI355X: Python binding of the llmint8 C library.

The functions here carry the C-ABI names and only marshal arguments (torch tensors ->
device pointers, the current HIP stream, workspace allocation when the caller passes
none).  Every step of the computation runs in the HIP kernels of libllmint8.so; there
is no fallback, and importing fails loudly when the library has not been built
(``python -m int8_quantized_matmul_rowwise_amd.build``).

    Wq, s_w = int8_quantize_weight(W)                  # offline, W: K x N
    Y = int8_matmul(X, Wq, s_w, threshold=6.0)          # X: M x K -> Y: M x N
    n_outliers, cols = int8_matmul_stats(X, 6.0)

8-bit floating point with a power-of-two scale per block of 128 (codes float8_e4m3fn, scales
float8_e8m0fnu): a product, its gradient, and a mixture-of-experts layer for few tokens

    Wq, s_w = fp8_quantize_weight_block(W)              # W: K x N
    Y = fp8_matmul_block(X, Wq, s_w)
    Wq, s_w, WqT, s_wT = fp8_quantize_weight_block(W, transposed=True)
    dX, dW = fp8_matmul_block_backward(dY, X, WqT, s_wT)
    Y, ids, p = fp8_moe_block(X, logits, W13q, s_w13, W2q, s_w2, top_k=8)

No call is recorded for autograd: outputs do not require a gradient, whatever the inputs do.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# LLMINT8_LIB: another build of the same sources (the host-sanitized test build)
LIB_PATH = os.environ.get("LLMINT8_LIB") or os.path.join(HERE, "libllmint8.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "llmint8.h")

F16, BF16 = 0, 1
_DT = {torch.float16: F16, torch.bfloat16: BF16}
OK, EINVAL, EWORKSPACE, EHIP, ERANGE = 0, -1, -2, -3, -4

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_I = ctypes.c_int


class LLMInt8Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, _SZ) for n in ("xq", "xq_pitch", "s_x", "n_outliers", "outliers", "xo", "xo_pitch", "wo",
                                   "scratch", "total", "small_batch")]


_SIGNATURES = {
    "llmint8_status_string": (ctypes.c_char_p, [_I]),
    "int8_quantize_weight": (_I, [_P, _I64, _I64, _I, _P, _P, _P]),
    "int8_matmul_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "int8_matmul": (_I, [_P, _I64, _I64, _I, _P, _P, _I64, _F, _P, _P, _SZ, _P]),
    "int8_matmul_noalloc": (_I, [_P, _I64, _I64, _I, _P, _P, _I64, _F, _P, _P]),
    "int8_matmul_stats": (_I, [_P, _I64, _I64, _I, _F, _P, _P, _P, _SZ, _P]),
    "int8_matmul_workspace_layout": (_I, [_I64, _I64, _I64, ctypes.POINTER(WorkspaceLayout)]),
    "int8_matmul_accumulators": (_I, [_P, _I64, _I64, _I, _P, _I64, _F, _P, _P, _P, _SZ, _P]),
    "int8_matmul_prepare": (_I, [_P, _I64, _I64, _I, _P, _I64, _F, _P, _SZ, _P]),
    "int8_matmul_products": (_I, [_I64, _I64, _I, _P, _P, _I64, _P, _P, _SZ, _P]),
    "int8_quantize_weight_fixed_workspace_bytes": (_SZ, [_I64]),
    "int8_quantize_weight_fixed": (_I, [_P, _I64, _I64, _I, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "int8_matmul_fixed": (_I, [_P, _I64, _I64, _I, _P, _I64, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "int8_blockwise_quantize": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "int8_blockwise_dequantize": (_I, [_P, _P, _I64, _I64, _P, _P]),
    "int8_quantize_weight_group": (_I, [_P, _I64, _I64, _I, _I64, _P, _P, _P]),
    "int8_matmul_group_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "int8_matmul_group_small_batch": (_I, [_I64, _I64, _I64, _I64]),
    "int8_matmul_group": (_I, [_P, _I64, _I64, _I, _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "int8_matmul_group_prepare": (_I, [_P, _I64, _I64, _I, _I64, _P, _SZ, _P]),
    "int8_matmul_group_products": (_I, [_I64, _I64, _I, _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "fp8_code_pitch": (_I64, [_I64]),
    "fp8_scale_pitch": (_I64, [_I64]),
    "fp8_quantize_weight_block": (_I, [_P, _I64, _I64, _I, _P, _P, _P, _P, _P]),
    "fp8_matmul_block_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8_matmul_block": (_I, [_P, _I64, _I64, _I, _P, _P, _I64, _P, _P, _SZ, _P]),
    "fp8_matmul_block_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "fp8_matmul_block_backward": (_I, [_P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "fp8_moe_block_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "fp8_moe_block": (_I, [_P, _I64, _I64, _I, _P, _I64, _I64, _I, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libllmint8.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with python -m int8_quantized_matmul_rowwise_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().llmint8_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise LLMInt8Error(status, f"{what}: {status_string(status)}")


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return int(getattr(stream, "cuda_stream", stream) or 0)


def _dev_tensor(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def int8_matmul_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().int8_matmul_workspace_bytes(M, K, N))


def int8_matmul_workspace_layout(M: int, K: int, N: int) -> dict:
    out = WorkspaceLayout()
    _check(lib().int8_matmul_workspace_layout(M, K, N, ctypes.byref(out)), "int8_matmul_workspace_layout")
    return {n: int(getattr(out, n)) for n, _ in WorkspaceLayout._fields_}


def _workspace(ws: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    return _dev_tensor(ws, "workspace")


def int8_quantize_weight(W: torch.Tensor, Wq: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """W (K x N, fp16/bf16) -> (Wq N x K int8, w_scale fp32[N])."""
    _dev_tensor(W, "W")
    if W.dtype not in _DT or W.dim() != 2:
        raise TypeError("W must be a 2-D fp16 or bf16 tensor")
    K, N = W.shape
    if Wq is None:
        Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if w_scale is None:
        w_scale = torch.empty((N,), dtype=torch.float32, device=W.device)
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    if tuple(Wq.shape) != (N, K) or tuple(w_scale.shape) != (N,):
        raise ValueError("Wq must be N x K and w_scale N")
    _check(lib().int8_quantize_weight(_ptr(W), K, N, _DT[W.dtype], _ptr(Wq), _ptr(w_scale), _stream(W, stream)),
           "int8_quantize_weight")
    return Wq, w_scale


def int8_matmul(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, threshold: float = 6.0,
                Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = LLM.int8() product of X (M x K, fp16/bf16) with the converted weight (Wq, w_scale)."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    M, K = X.shape
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    N = Wq.shape[0]
    if Wq.dim() != 2 or Wq.shape[1] != K or tuple(w_scale.shape) != (N,):
        raise ValueError("Wq must be N x K and w_scale N")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _dev_tensor(Y, "Y", X.dtype)
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be M x N")
    nbytes = int8_matmul_workspace_bytes(M, K, N)
    ws = _workspace(workspace, nbytes, X.device)
    _check(lib().int8_matmul(_ptr(X), M, K, _DT[X.dtype], _ptr(Wq), _ptr(w_scale), N, float(threshold), _ptr(Y),
                             _ptr(ws), ws.numel(), _stream(X, stream)), "int8_matmul")
    return Y


NOALLOC_SCRATCH_BYTES = 64 << 20  # LLMINT8_NOALLOC_SCRATCH_BYTES


def int8_matmul_noalloc(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, threshold: float = 6.0,
                        Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """int8_matmul on the library's own device scratch (no workspace; the library call
    allocates nothing -- pass Y to keep the binding from allocating it either)."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    M, K = X.shape
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    N = Wq.shape[0]
    if Wq.dim() != 2 or Wq.shape[1] != K or tuple(w_scale.shape) != (N,):
        raise ValueError("Wq must be N x K and w_scale N")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _dev_tensor(Y, "Y", X.dtype)
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be M x N")
    _check(lib().int8_matmul_noalloc(_ptr(X), M, K, _DT[X.dtype], _ptr(Wq), _ptr(w_scale), N, float(threshold),
                                     _ptr(Y), _stream(X, stream)), "int8_matmul_noalloc")
    return Y


def int8_matmul_prepare(X: torch.Tensor, Wq: torch.Tensor, threshold: float = 6.0,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Stage 1 of int8_matmul (the X pass) into a workspace, which is returned."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    M, K = X.shape
    _dev_tensor(Wq, "Wq", torch.int8)
    N = Wq.shape[0]
    ws = _workspace(workspace, int8_matmul_workspace_bytes(M, K, N), X.device)
    _check(lib().int8_matmul_prepare(_ptr(X), M, K, _DT[X.dtype], _ptr(Wq), N, float(threshold), _ptr(ws),
                                     ws.numel(), _stream(X, stream)), "int8_matmul_prepare")
    return ws


def int8_matmul_products(M: int, K: int, dtype: torch.dtype, Wq: torch.Tensor, w_scale: torch.Tensor,
                         workspace: torch.Tensor, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Stage 2 of int8_matmul: the products and the epilogue from a prepared workspace."""
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    _dev_tensor(workspace, "workspace")
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=dtype, device=Wq.device)
    _dev_tensor(Y, "Y", dtype)
    _check(lib().int8_matmul_products(M, K, _DT[dtype], _ptr(Wq), _ptr(w_scale), N, _ptr(Y), _ptr(workspace),
                                      workspace.numel(), _stream(Wq, stream)), "int8_matmul_products")
    return Y


def int8_matmul_stats(X: torch.Tensor, threshold: float = 6.0, outlier_cols: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[int, torch.Tensor]:
    """(n_O, O[:n_O]) -- the outlier feature dimensions of X (synchronizes the stream)."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    M, K = X.shape
    if outlier_cols is None:
        outlier_cols = torch.empty((max(K, 1),), dtype=torch.int32, device=X.device)
    _dev_tensor(outlier_cols, "outlier_cols", torch.int32)
    nbytes = int8_matmul_workspace_bytes(M, K, 0)
    ws = _workspace(workspace, nbytes, X.device)
    n = ctypes.c_int32(0)
    _check(lib().int8_matmul_stats(_ptr(X), M, K, _DT[X.dtype], float(threshold), ctypes.byref(n),
                                   outlier_cols.data_ptr(), _ptr(ws), ws.numel(), _stream(X, stream)),
           "int8_matmul_stats")
    return int(n.value), outlier_cols[: n.value]


def int8_matmul_accumulators(X: torch.Tensor, Wq: torch.Tensor, threshold: float = 6.0,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """Test hook: (C int32 M x N, F fp32 M x N, workspace) from the product kernels."""
    _dev_tensor(X, "X")
    M, K = X.shape
    N = Wq.shape[0]
    C = torch.empty((M, N), dtype=torch.int32, device=X.device)
    F = torch.empty((M, N), dtype=torch.float32, device=X.device)
    ws = _workspace(workspace, int8_matmul_workspace_bytes(M, K, N), X.device)
    _check(lib().int8_matmul_accumulators(_ptr(X), M, K, _DT[X.dtype], _ptr(Wq), N, float(threshold), _ptr(C),
                                          _ptr(F), _ptr(ws), ws.numel(), _stream(X, stream)),
           "int8_matmul_accumulators")
    return C, F, ws


def workspace_views(ws: torch.Tensor, M: int, K: int, N: int, dtype: torch.dtype) -> dict:
    """Views of the X pass's products left in an int8_matmul workspace (see the header)."""
    L = int8_matmul_workspace_layout(M, K, N)
    b = ws.view(torch.uint8)
    n_o = int(b[L["n_outliers"]: L["n_outliers"] + 4].view(torch.int32).item())
    P = int(math.ceil(n_o / 32) * 32)
    xq = b[L["xq"]: L["xq"] + M * L["xq_pitch"]].view(torch.int8).view(M, L["xq_pitch"]) if L["xq_pitch"] else None
    xo = b[L["xo"]: L["xo"] + 2 * M * L["xo_pitch"]].view(dtype).view(M, L["xo_pitch"]) if L["xo_pitch"] else None
    # the small-batch path has no W_O region (its product kernel gathers Wq[:,O] itself)
    wo = (b[L["wo"]: L["wo"] + 2 * N * L["xo_pitch"]].view(dtype).view(N, L["xo_pitch"])
          if L["xo_pitch"] and not L["small_batch"] else None)
    return {
        "n_outliers": n_o,
        "outliers": b[L["outliers"]: L["outliers"] + 4 * n_o].view(torch.int32),
        "Xq": None if xq is None else xq[:, :K],
        "Xq_pad": None if xq is None else xq[:, K:],
        "s_x": b[L["s_x"]: L["s_x"] + 4 * M].view(torch.float32),
        "XO": None if xo is None else xo[:, :P],
        "WO": None if wo is None else wo[:, :P],
    }


def _fixed_pitch(n_o: int) -> int:
    return (n_o + 31) // 32 * 32


def int8_quantize_weight_fixed(W: torch.Tensor, outlier_cols: torch.Tensor, stream=None):
    """Weight conversion with a fixed outlier set (device int32, ascending):
    (Wq N x K int8, w_scale fp32[N], W_O N x P 16-bit exact rows)."""
    _dev_tensor(W, "W")
    if W.dtype not in _DT or W.dim() != 2:
        raise TypeError("W must be a 2-D fp16 or bf16 tensor")
    _dev_tensor(outlier_cols, "outlier_cols", torch.int32)
    K, N = W.shape
    n_o = outlier_cols.numel()
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    s_w = torch.empty(N, dtype=torch.float32, device=W.device)
    W_O = torch.empty((N, _fixed_pitch(n_o)), dtype=W.dtype, device=W.device)
    ws = torch.empty(max(int(lib().int8_quantize_weight_fixed_workspace_bytes(K)), 1), dtype=torch.uint8,
                     device=W.device)
    _check(lib().int8_quantize_weight_fixed(_ptr(W), K, N, _DT[W.dtype], _ptr(outlier_cols), n_o, _ptr(Wq), _ptr(s_w),
                                            _ptr(W_O), _ptr(ws), ws.numel(), _stream(W, stream)),
           "int8_quantize_weight_fixed")
    return Wq, s_w, W_O


def int8_matmul_fixed(X: torch.Tensor, outlier_cols: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                      W_O: torch.Tensor, Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y = X W with the fixed outlier set (no detection; exact 16-bit W rows on the set)."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    _dev_tensor(outlier_cols, "outlier_cols", torch.int32)
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    _dev_tensor(W_O, "W_O", X.dtype)
    M, K = X.shape
    N = Wq.shape[0]
    n_o = outlier_cols.numel()
    if W_O.shape != (N, _fixed_pitch(n_o)):
        raise ValueError("W_O must be N x (n_O rounded up to 32)")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    ws = _workspace(workspace, int8_matmul_workspace_bytes(M, K, N), X.device)
    _check(lib().int8_matmul_fixed(_ptr(X), M, K, _DT[X.dtype], _ptr(outlier_cols), n_o, _ptr(Wq), _ptr(w_scale),
                                   _ptr(W_O), N, _ptr(Y), _ptr(ws), ws.numel(), _stream(X, stream)),
           "int8_matmul_fixed")
    return Y


def int8_blockwise_quantize(x: torch.Tensor, block: int = 2048, q: Optional[torch.Tensor] = None,
                            absmax: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Block-wise absmax int8 code of an fp32 tensor, taken flat: (q int8 of x's shape,
    absmax fp32[ceil(numel / block)])."""
    _dev_tensor(x, "x", torch.float32)
    n = x.numel()
    nb = -(-n // block) if block > 0 else 0
    if q is None:
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if absmax is None:
        absmax = torch.empty(nb, dtype=torch.float32, device=x.device)
    _dev_tensor(q, "q", torch.int8)
    _dev_tensor(absmax, "absmax", torch.float32)
    if q.numel() != n or absmax.numel() != nb:
        raise ValueError("q must hold numel(x) codes and absmax ceil(numel / block) scales")
    _check(lib().int8_blockwise_quantize(_ptr(x), n, int(block), _ptr(q), _ptr(absmax), _stream(x, stream)),
           "int8_blockwise_quantize")
    return q, absmax


def int8_blockwise_dequantize(q: torch.Tensor, absmax: torch.Tensor, block: int = 2048,
                              x: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode of int8_blockwise_quantize: fp32 of q's shape."""
    _dev_tensor(q, "q", torch.int8)
    _dev_tensor(absmax, "absmax", torch.float32)
    n = q.numel()
    if x is None:
        x = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _dev_tensor(x, "x", torch.float32)
    if x.numel() != n or absmax.numel() != (-(-n // block) if block > 0 else 0):
        raise ValueError("x must hold numel(q) values and absmax ceil(numel / block) scales")
    _check(lib().int8_blockwise_dequantize(_ptr(q), _ptr(absmax), n, int(block), _ptr(x), _stream(q, stream)),
           "int8_blockwise_dequantize")
    return x


def int8_quantize_weight_group(W: torch.Tensor, group: int = 1024, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """W (K x N, fp16/bf16) -> (Wq N x K int8, w_scale fp32 N x K/group): one scale per
    output column and group of `group` consecutive rows of W."""
    _dev_tensor(W, "W")
    if W.dtype not in _DT or W.dim() != 2:
        raise TypeError("W must be a 2-D fp16 or bf16 tensor")
    K, N = W.shape
    if group <= 0 or K % group:
        raise ValueError("group must divide K")
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    s_w = torch.empty((N, K // group), dtype=torch.float32, device=W.device)
    _check(lib().int8_quantize_weight_group(_ptr(W), K, N, _DT[W.dtype], int(group), _ptr(Wq), _ptr(s_w),
                                            _stream(W, stream)), "int8_quantize_weight_group")
    return Wq, s_w


def int8_matmul_group_workspace_bytes(M: int, K: int, group: int) -> int:
    return int(lib().int8_matmul_group_workspace_bytes(M, K, group))


def int8_matmul_group_small_batch(M: int, K: int, N: int, group: int) -> bool:
    """True when int8_matmul_group takes the small-batch product kernel for these sizes."""
    r = int(lib().int8_matmul_group_small_batch(M, K, N, group))
    _check(min(r, 0), "int8_matmul_group_small_batch")
    return r == 1


def int8_matmul_group(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, group: int = 1024,
                      Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y = X W with group-wise scales along K on both operands (no outlier decomposition)."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    M, K = X.shape
    N = Wq.shape[0]
    if group <= 0 or K % group or Wq.dim() != 2 or Wq.shape[1] != K or tuple(w_scale.shape) != (N, K // group):
        raise ValueError("Wq must be N x K and w_scale N x K/group, with group dividing K")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _dev_tensor(Y, "Y", X.dtype)
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be M x N")
    ws = _workspace(workspace, int8_matmul_group_workspace_bytes(M, K, group), X.device)
    _check(lib().int8_matmul_group(_ptr(X), M, K, _DT[X.dtype], int(group), _ptr(Wq), _ptr(w_scale), N, _ptr(Y),
                                   _ptr(ws), ws.numel(), _stream(X, stream)), "int8_matmul_group")
    return Y


def int8_matmul_group_prepare(X: torch.Tensor, group: int, workspace: torch.Tensor, stream=None) -> None:
    """The X pass of int8_matmul_group into `workspace`."""
    _dev_tensor(X, "X")
    if X.dtype not in _DT or X.dim() != 2:
        raise TypeError("X must be a 2-D fp16 or bf16 tensor")
    _dev_tensor(workspace, "workspace")
    M, K = X.shape
    _check(lib().int8_matmul_group_prepare(_ptr(X), M, K, _DT[X.dtype], int(group), _ptr(workspace),
                                           workspace.numel(), _stream(X, stream)), "int8_matmul_group_prepare")


def int8_matmul_group_products(M: int, K: int, dtype: torch.dtype, group: int, Wq: torch.Tensor,
                               w_scale: torch.Tensor, workspace: torch.Tensor, Y: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """The products of int8_matmul_group from a workspace filled by int8_matmul_group_prepare."""
    _dev_tensor(Wq, "Wq", torch.int8)
    _dev_tensor(w_scale, "w_scale", torch.float32)
    _dev_tensor(workspace, "workspace")
    N = Wq.shape[0]
    if group <= 0 or K % group or Wq.dim() != 2 or Wq.shape[1] != K or tuple(w_scale.shape) != (N, K // group):
        raise ValueError("Wq must be N x K and w_scale N x K/group, with group dividing K")
    if Y is None:
        Y = torch.empty((M, N), dtype=dtype, device=Wq.device)
    _dev_tensor(Y, "Y", dtype)
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be M x N")
    _check(lib().int8_matmul_group_products(M, K, _DT[dtype], int(group), _ptr(Wq), _ptr(w_scale), N, _ptr(Y),
                                            _ptr(workspace), workspace.numel(), _stream(Wq, stream)),
           "int8_matmul_group_products")
    return Y


def group_workspace_views(ws: torch.Tensor, M: int, K: int, group: int) -> dict:
    """The X pass's products left in an int8_matmul_group workspace (see the header)."""
    ng = K // group
    b = ws.view(torch.uint8)
    o_s = (M * K + 255) // 256 * 256
    o_r = (o_s + 4 * M * ng + 255) // 256 * 256
    return {
        "Xq": b[: M * K].view(torch.int8).view(M, K),
        "s_x": b[o_s: o_s + 4 * M * ng].view(torch.float32).view(M, ng),
        "r": b[o_r: o_r + 4 * M * ng].view(torch.float32).view(ng, M),
    }


# ---- 8-bit floating point with a power-of-two scale per block of 128

_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_E8M0 = (torch.float8_e8m0fnu, torch.uint8)
_T16 = (torch.float16, torch.bfloat16)


def fp8_code_pitch(n: int) -> int:
    """Bytes of a row of codes over n values: n rounded up to a multiple of 128."""
    return -(-n // 128) * 128


def fp8_scale_pitch(n: int) -> int:
    """Bytes of a row of scales over n values: a byte per 128, rounded up to a multiple of 4."""
    return -(-n // 512) * 4


def _fp8_arg(t, name: str, dtypes, shape=None, device=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _fp8_on(device: torch.device, stream):
    """None where a call allocates and enqueues as things stand (the current device, its current
    stream), else the context to do it in: the tensors' device, and the given stream (what is
    allocated then belongs to it)."""
    if stream is None:
        return None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(getattr(stream, "cuda_stream", stream) or 0)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _fp8_workspace(ws, nbytes: int, device):
    """(the workspace, its address, its bytes)"""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        _fp8_arg(ws, "workspace", (torch.uint8,), device=device)
    return ws, ws.data_ptr(), ws.numel()


def fp8_quantize_weight_block(W: torch.Tensor, transposed: bool = False, stream=None) -> Tuple[torch.Tensor, ...]:
    """W (K x N, fp16/bf16) -> (Wq N x code_pitch(K) e4m3, w_scale ceil(N/128) x scale_pitch(K)
    e8m0); with transposed also (WqT K x code_pitch(N), wT_scale ceil(K/128) x scale_pitch(N))."""
    if _fp8_arg(W, "W", _T16).dim() != 2:
        raise ValueError("W must be 2-D")
    K, N = W.shape
    dev = W.device
    on = _fp8_on(dev, stream)
    if on is not None:
        with on:
            return fp8_quantize_weight_block(W, transposed)
    out = [torch.empty((N, fp8_code_pitch(K)), dtype=_E4M3[0], device=dev),
           torch.empty((-(-N // 128), fp8_scale_pitch(K)), dtype=_E8M0[0], device=dev)]
    if transposed:
        out += [torch.empty((K, fp8_code_pitch(N)), dtype=_E4M3[0], device=dev),
                torch.empty((-(-K // 128), fp8_scale_pitch(N)), dtype=_E8M0[0], device=dev)]
    ptrs = [t.data_ptr() for t in out] + [None] * (4 - len(out))
    _check(lib().fp8_quantize_weight_block(W.data_ptr(), K, N, _DT[W.dtype], *ptrs,
                                           torch._C._cuda_getCurrentRawStream(dev.index)), "fp8_quantize_weight_block")
    return tuple(out)


def fp8_matmul_block_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().fp8_matmul_block_workspace_bytes(M, K, N))


def fp8_matmul_block(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, Y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W (M x N) of X (M x K, fp16/bf16), coded per row in groups of 128, with a converted weight.

    Like every call here it is not recorded for autograd: Y does not require a gradient, whatever X does.  A
    training step calls fp8_matmul_block_backward itself, or both from a torch.autograd.Function."""
    if _fp8_arg(X, "X", _T16).dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    dev = X.device
    on = _fp8_on(dev, stream)
    if on is not None:
        with on:
            return fp8_matmul_block(X, Wq, w_scale, Y, workspace)
    if _fp8_arg(Wq, "Wq", _E4M3, device=dev).dim() != 2 or Wq.shape[1] != fp8_code_pitch(K):
        raise ValueError(f"Wq must be N x {fp8_code_pitch(K)} for K = {K}, got {tuple(Wq.shape)}")
    N = Wq.shape[0]
    _fp8_arg(w_scale, "w_scale", _E8M0, (-(-N // 128), fp8_scale_pitch(K)), dev)
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=dev)
    else:
        _fp8_arg(Y, "Y", (X.dtype,), (M, N), dev)
    L = lib()
    ws, at, size = _fp8_workspace(workspace, L.fp8_matmul_block_workspace_bytes(M, K, N), dev)
    rc = L.fp8_matmul_block(X.data_ptr(), M, K, _DT[X.dtype], Wq.data_ptr(), w_scale.data_ptr(), N, Y.data_ptr(),
                            at, size, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc:
        _check(rc, "fp8_matmul_block")
    return Y


def fp8_matmul_block_backward_workspace_bytes(M: int, K: int, N: int, need_dx: bool = True, need_dw: bool = True) -> int:
    return int(lib().fp8_matmul_block_backward_workspace_bytes(M, K, N, int(need_dx), int(need_dw)))


def fp8_matmul_block_backward(dY: torch.Tensor, X: Optional[torch.Tensor], WqT: Optional[torch.Tensor],
                              wT_scale: Optional[torch.Tensor], need_dx: bool = True, need_dw: bool = True,
                              dX: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None):
    """(dX M x K, dW K x N) of fp8_matmul_block; one that is not needed is None, and its operands
    (WqT and wT_scale for dX, X for dW) may be None then."""
    if _fp8_arg(dY, "dY", _T16).dim() != 2:
        raise ValueError("dY must be 2-D")
    M, N = dY.shape
    dev, t = dY.device, dY.dtype
    on = _fp8_on(dev, stream)
    if on is not None:
        with on:
            return fp8_matmul_block_backward(dY, X, WqT, wT_scale, need_dx, need_dw, dX, dW, workspace)
    if not need_dx and not need_dw:
        return None, None
    if need_dw:
        if _fp8_arg(X, "X", (t,), device=dev).dim() != 2 or X.shape[0] != M:
            raise ValueError(f"X must be {M} x K, got {tuple(X.shape)}")
        K = X.shape[1]
    if need_dx:
        if _fp8_arg(WqT, "WqT", _E4M3, device=dev).dim() != 2 or WqT.shape[1] != fp8_code_pitch(N):
            raise ValueError(f"WqT must be K x {fp8_code_pitch(N)} for N = {N}, got {tuple(WqT.shape)}")
        if need_dw and WqT.shape[0] != K:
            raise ValueError(f"WqT must have {K} rows, got {WqT.shape[0]}")
        K = WqT.shape[0]
        _fp8_arg(wT_scale, "wT_scale", _E8M0, (-(-K // 128), fp8_scale_pitch(N)), dev)
    L = lib()
    if not need_dx:
        dX = None
    elif dX is None:
        dX = torch.empty((M, K), dtype=t, device=dev)
    else:
        _fp8_arg(dX, "dX", (t,), (M, K), dev)
    if not need_dw:
        dW = None
    elif dW is None:
        dW = torch.empty((K, N), dtype=t, device=dev)
    else:
        _fp8_arg(dW, "dW", (t,), (K, N), dev)
    ws, at, size = _fp8_workspace(workspace, L.fp8_matmul_block_backward_workspace_bytes(M, K, N, int(need_dx), int(need_dw)), dev)
    _check(L.fp8_matmul_block_backward(dY.data_ptr(), X.data_ptr() if need_dw else None, M, K, N, _DT[t],
                                       WqT.data_ptr() if need_dx else None, wT_scale.data_ptr() if need_dx else None,
                                       dX.data_ptr() if need_dx else None, dW.data_ptr() if need_dw else None,
                                       at, size, torch._C._cuda_getCurrentRawStream(dev.index)), "fp8_matmul_block_backward")
    return dX, dW


def fp8_moe_block_workspace_bytes(T: int, H: int, I: int, E: int, top_k: int) -> int:
    return int(lib().fp8_moe_block_workspace_bytes(T, H, I, E, top_k))


def fp8_moe_block(X: torch.Tensor, logits: torch.Tensor, W13q: torch.Tensor, w13_scale: torch.Tensor,
                  W2q: torch.Tensor, w2_scale: torch.Tensor, top_k: int, renormalize: bool = True,
                  Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y T x H, topk_ids T x top_k int32, topk_weights T x top_k fp32) of a mixture-of-experts
    layer on X (T x H, at most 128 tokens) with gate logits (T x E fp32); W13q E x 2I x
    code_pitch(H) (gate rows first) and W2q E x H x code_pitch(I) with their scales: E conversions
    by fp8_quantize_weight_block, stacked.  I is W13q.shape[1] / 2."""
    if _fp8_arg(X, "X", _T16).dim() != 2:
        raise ValueError("X must be 2-D")
    T, H = X.shape
    dev = X.device
    on = _fp8_on(dev, stream)
    if on is not None:
        with on:
            return fp8_moe_block(X, logits, W13q, w13_scale, W2q, w2_scale, top_k, renormalize, Y, workspace)
    if _fp8_arg(logits, "logits", (torch.float32,), device=dev).dim() != 2 or logits.shape[0] != T:
        raise ValueError(f"logits must be {T} x E, got {tuple(logits.shape)}")
    E = logits.shape[1]
    if not isinstance(W13q, torch.Tensor) or W13q.dim() != 3 or W13q.shape[1] % 2:
        raise ValueError("W13q must be E x 2I x code_pitch(H)")
    I = W13q.shape[1] // 2
    _fp8_arg(W13q, "W13q", _E4M3, (E, 2 * I, fp8_code_pitch(H)), dev)
    _fp8_arg(w13_scale, "w13_scale", _E8M0, (E, -(-2 * I // 128), fp8_scale_pitch(H)), dev)
    _fp8_arg(W2q, "W2q", _E4M3, (E, H, fp8_code_pitch(I)), dev)
    _fp8_arg(w2_scale, "w2_scale", _E8M0, (E, -(-H // 128), fp8_scale_pitch(I)), dev)
    if Y is None:
        Y = torch.empty((T, H), dtype=X.dtype, device=dev)
    else:
        _fp8_arg(Y, "Y", (X.dtype,), (T, H), dev)
    top_k = int(top_k)
    if not 0 < top_k <= E:
        raise ValueError(f"top_k must be in 1 .. {E}, got {top_k}")
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    p = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    L = lib()
    ws, at, size = _fp8_workspace(workspace, L.fp8_moe_block_workspace_bytes(T, H, I, E, top_k), dev)
    rc = L.fp8_moe_block(X.data_ptr(), T, H, _DT[X.dtype], logits.data_ptr(), E, top_k, int(renormalize),
                         W13q.data_ptr(), w13_scale.data_ptr(), W2q.data_ptr(), w2_scale.data_ptr(), I,
                         Y.data_ptr(), ids.data_ptr(), p.data_ptr(), at, size,
                         torch._C._cuda_getCurrentRawStream(dev.index))
    if rc:
        _check(rc, "fp8_moe_block")
    return Y, ids, p


__all__ = [
    "int8_quantize_weight", "int8_matmul", "int8_matmul_noalloc", "int8_matmul_stats", "int8_matmul_prepare", "int8_matmul_products", "int8_matmul_workspace_bytes",
    "int8_matmul_workspace_layout", "int8_matmul_accumulators", "workspace_views", "LLMInt8Error", "lib",
    "int8_blockwise_quantize", "int8_blockwise_dequantize", "int8_quantize_weight_fixed", "int8_matmul_fixed",
    "status_string", "int8_quantize_weight_group", "int8_matmul_group", "int8_matmul_group_workspace_bytes",
    "group_workspace_views", "int8_matmul_group_small_batch", "int8_matmul_group_prepare", "int8_matmul_group_products",
    "fp8_code_pitch", "fp8_scale_pitch", "fp8_quantize_weight_block", "fp8_matmul_block",
    "fp8_matmul_block_workspace_bytes", "fp8_matmul_block_backward", "fp8_matmul_block_backward_workspace_bytes",
    "fp8_moe_block", "fp8_moe_block_workspace_bytes",
]
