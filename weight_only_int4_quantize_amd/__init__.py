"""Python binding of libawq_mi355x.so, the MI355X (gfx950) W4A16 library.

Argument marshalling only: every step runs in the library's HIP kernels.
PyTorch supplies device memory and the current stream. The binding raises
if the library has not been built or a tensor is not a GPU tensor; there is
no CPU fallback.

Entry points (same names as the C ABI in include/awq.h):
    awq_quantize(w, group_size=128, channel_scale=None)  -> qweight, scales, zeros
    awq_gemm(x, qweight, scales, zeros, group_size=128, path=0, workspace=None) -> y
        (awq_gemm_ex when a workspace from gemm_workspace(M, N, K) is given)
    awq_activation_absmean(x) -> m
    awq_scale_search(w, x, group_size=128, alphas=None) -> losses, best_index, best_scales
    awq_gemm_fused(x, qweight, scales, zeros, group_size=128, bias=None, activation="none", mul=None,
        residual=None) -> y
    awq_kv_write(cache, seqs, k, v), awq_kv_read(cache, seqs) -> k, v
    awq_kv_attention(q, cache, seqs) -> out
        (a paged 8-bit cache, KVCache, and a batch of sequences over it, KVSeqs)
"""

from __future__ import annotations

import ctypes
import os
import re
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libawq_mi355x.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "awq.h")

AWQ_OK = 0
STATUS_NAMES = {
    0: "AWQ_OK", 1: "AWQ_ERR_NULL", 2: "AWQ_ERR_SHAPE", 3: "AWQ_ERR_ALIGN",
    4: "AWQ_ERR_CONFIG", 5: "AWQ_ERR_WORKSPACE", 6: "AWQ_ERR_HIP",
}
PATH_AUTO, PATH_GEMV, PATH_GEMM, PATH_SKINNY, PATH_COLTILE = 0, 1, 2, 3, 4
QUANT_ASYMMETRIC, QUANT_SYMMETRIC = 0, 1

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
KV_FORMATS = {"int8": 0, "e4m3": 1}

_lib = None


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int)]


class _KVSeqsStruct(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("cu_tokens", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("max_tokens", ctypes.c_int64), ("max_len", ctypes.c_int64)]


class AwqError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed: {message}")
        self.status = status


def lib_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Loads the built library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m weight_only_int4_quantize_amd.build` "
            "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    c_i64, c_int, c_vp, c_sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.awq_status_string.restype = ctypes.c_char_p
    L.awq_status_string.argtypes = [c_int]
    L.awq_version.restype = c_int
    L.awq_version.argtypes = []
    L.awq_quantize.restype = c_int
    L.awq_quantize.argtypes = [c_vp, c_vp, c_i64, c_i64, c_int, c_vp, c_vp, c_vp, c_vp]
    L.awq_quantize_ex.restype = c_int
    L.awq_quantize_ex.argtypes = [c_vp, c_vp, c_i64, c_i64, c_int, c_int, ctypes.c_double, c_vp, c_vp, c_vp, c_vp]
    L.awq_clip_search_workspace_bytes.restype = c_sz
    L.awq_clip_search_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, c_int]
    L.awq_clip_search.restype = c_int
    L.awq_clip_search.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_vp, c_int, c_vp, c_sz,
                                  c_vp, c_vp, c_vp]
    L.awq_gemm.restype = c_int
    L.awq_gemm.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_vp]
    L.awq_gemm_path.restype = c_int
    L.awq_gemm_path.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_int, c_vp]
    L.awq_gemm_workspace_bytes.restype = c_sz
    L.awq_gemm_workspace_bytes.argtypes = [c_i64, c_i64, c_i64]
    L.awq_gemm_ex.restype = c_int
    L.awq_gemm_ex.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_int, c_vp, c_sz, c_vp]
    L.awq_gemm_kernel.restype = c_int
    L.awq_gemm_kernel.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, c_int]
    L.awq_gemm_noalloc.restype = c_int
    L.awq_gemm_noalloc.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_int, c_vp]
    L.awq_gemm_grouped.restype = c_int
    L.awq_gemm_grouped.argtypes = [c_vp, c_int, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_int, c_vp, c_vp]
    L.awq_activation_absmean_workspace_bytes.restype = c_sz
    L.awq_activation_absmean_workspace_bytes.argtypes = [c_i64, c_i64]
    L.awq_activation_absmean.restype = c_int
    L.awq_activation_absmean.argtypes = [c_vp, c_i64, c_i64, c_vp, c_vp, c_sz, c_vp]
    L.awq_scale_search_workspace_bytes.restype = c_sz
    L.awq_scale_search_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_int, c_int]
    L.awq_scale_search.restype = c_int
    L.awq_scale_search.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_int, c_vp, c_sz,
                                   c_vp, c_vp, c_vp, c_vp]
    L.awq_select_salient.restype = c_int
    L.awq_select_salient.argtypes = [c_vp, c_i64, c_int, c_vp, c_vp]
    L.awq_quantize_salient.restype = c_int
    L.awq_quantize_salient.argtypes = [c_vp, c_i64, c_i64, c_int, c_int, c_vp, c_int, c_vp, c_vp, c_vp, c_vp, c_vp]
    L.awq_salient_apply.restype = c_int
    L.awq_salient_apply.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_vp]
    L.awq_salient_count.restype = c_i64
    L.awq_salient_count.argtypes = [c_i64]
    L.awq_salient_loss_workspace_bytes.restype = c_sz
    L.awq_salient_loss_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_int, c_int]
    L.awq_salient_loss.restype = c_int
    L.awq_salient_loss.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_int, c_vp, c_sz, c_vp, c_vp,
                                   c_vp, c_vp]
    L.awq_quantize_w8.restype = c_int
    L.awq_quantize_w8.argtypes = [c_vp, c_vp, c_i64, c_i64, c_int, c_int, c_vp, c_vp, c_vp, c_vp]
    L.awq_gemm_w8.restype = c_int
    L.awq_gemm_w8.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_int, c_vp, c_sz, c_vp]
    L.awq_gemm_fused_kernel.restype = c_int
    L.awq_gemm_fused_kernel.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, c_int, c_int]
    L.awq_gemm_fused.restype = c_int
    L.awq_gemm_fused.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_vp, c_int, c_vp, c_i64,
                                 c_vp, c_i64, c_vp, c_int, c_vp, c_sz, c_vp]
    L.awq_kv_write.restype = c_int
    L.awq_kv_write.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp]
    L.awq_kv_read.restype = c_int
    L.awq_kv_read.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]
    L.awq_kv_attention_workspace_bytes.restype = c_sz
    L.awq_kv_attention_workspace_bytes.argtypes = [c_vp, c_vp, c_int]
    L.awq_kv_attention.restype = c_int
    L.awq_kv_attention.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, ctypes.c_float, c_int, c_i64,
                                   c_vp, c_i64, c_i64, c_vp, c_vp, c_sz, c_vp]
    _lib = L
    return L


def header_functions() -> list:
    """Names of the functions include/awq.h declares."""
    with open(HEADER, encoding="utf-8") as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(awq_[a-z0-9_]+)\s*\(", text)))


def _check(fn: str, status: int) -> None:
    if status != AWQ_OK:
        msg = load().awq_status_string(status).decode()
        raise AwqError(fn, status, msg)


def _torch():
    import torch
    return torch


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _need_gpu(name: str, t, dtype=None) -> None:
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_out(qweight, scales, zeros, q_shape, sz_shape, device) -> None:
    """Caller-given quantize outputs: int32 qweight and fp16 scales / zeros of
    exactly the shapes the call writes, contiguous, on the input's device."""
    torch = _torch()
    for name, t, dtype, shape in (("qweight", qweight, torch.int32, q_shape), ("scales", scales, torch.float16, sz_shape),
                                  ("zeros", zeros, torch.float16, sz_shape)):
        _need_gpu(name, t, dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}")


def awq_quantize(w, group_size: int = 128, channel_scale=None, out=None, symmetric: bool = False,
                 clip_fraction: float = 0.0):
    """Group-wise INT4 quantization of w[N, K] (fp16), asymmetric by default
    (awq_quantize); symmetric=True or clip_fraction > 0 go to
    awq_quantize_ex (symmetric map; percentile clip of each group).

    Returns (qweight int32 [N, K/8] holding the uint32 words, scales fp16
    [N, K/G], zeros fp16 [N, K/G]). channel_scale: optional fp32 [K]."""
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    if w.dim() != 2:
        raise ValueError("w must be 2-D [N, K]")
    N, K = w.shape
    if channel_scale is not None:
        _need_gpu("channel_scale", channel_scale, torch.float32)
        if channel_scale.numel() != K:
            raise ValueError("channel_scale must have K elements")
    ng = K // group_size if group_size > 0 else 0
    if out is None:
        dev = w.device
        qweight = torch.empty((N, max(K // 8, 0)), dtype=torch.int32, device=dev)
        scales = torch.empty((N, ng), dtype=torch.float16, device=dev)
        zeros = torch.empty((N, ng), dtype=torch.float16, device=dev)
    else:
        qweight, scales, zeros = out
        _need_out(qweight, scales, zeros, (N, K // 8), (N, ng), w.device)
    if symmetric or clip_fraction != 0.0:
        mode = QUANT_SYMMETRIC if symmetric else QUANT_ASYMMETRIC
        st = load().awq_quantize_ex(_ptr(w), _ptr(channel_scale), N, K, group_size, mode, float(clip_fraction),
                                    _ptr(qweight), _ptr(scales), _ptr(zeros), _stream(w.device))
        _check("awq_quantize_ex", st)
    else:
        st = load().awq_quantize(_ptr(w), _ptr(channel_scale), N, K, group_size, _ptr(qweight),
                                 _ptr(scales), _ptr(zeros), _stream(w.device))
        _check("awq_quantize", st)
    return qweight, scales, zeros


KERNEL_NAMES = {1: "gemv", 2: "gemm", 3: "skinny", 4: "coltile", 5: "gemm_small"}


def gemm_kernel(M: int, N: int, K: int, group_size: int = 128, path: int = PATH_AUTO,
                workspace: bool = False) -> str:
    """Name of the kernel awq_gemm runs for this shape (awq_gemm_kernel)."""
    k = int(load().awq_gemm_kernel(M, N, K, group_size, path, int(workspace)))
    if k < 0:
        raise AwqError("awq_gemm_kernel", 4, "the path cannot take this shape")
    return KERNEL_NAMES[k]


def gemm_fused_kernel(M: int, N: int, K: int, group_size: int = 128, bits: int = 4, path: int = PATH_AUTO,
                      workspace: bool = False) -> str:
    """Name of the kernel awq_gemm_fused runs for this shape where it has
    something to fuse (awq_gemm_fused_kernel)."""
    k = int(load().awq_gemm_fused_kernel(M, N, K, group_size, bits, path, int(workspace)))
    if k < 0:
        raise AwqError("awq_gemm_fused_kernel", 4, "the path cannot take this shape")
    return KERNEL_NAMES[k]


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().awq_gemm_workspace_bytes(M, N, K))


def gemm_workspace(M: int, N: int, K: int, device=None):
    """A zero-filled uint8 GPU tensor of awq_gemm_workspace_bytes(M, N, K)
    bytes: awq_gemm_ex's workspace for this shape and for any other whose
    awq_gemm_workspace_bytes is no larger (today the size depends on M
    only). Each call leaves it ready for the next, without clearing."""
    torch = _torch()
    nbytes = gemm_workspace_bytes(M, N, K)
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device or "cuda")


def awq_gemm(x, qweight, scales, zeros, group_size: int = 128, path: int = PATH_AUTO, out=None,
             workspace=None):
    """y[M, N] = x[M, K] . dequant(Wq)^T in fp16 (fp32 accumulation).

    With a workspace (see gemm_workspace) the call goes to awq_gemm_ex,
    which may split output tiles' K loops across blocks (stream-K)."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    _need_gpu("qweight", qweight, torch.int32)
    _need_gpu("scales", scales, torch.float16)
    _need_gpu("zeros", zeros, torch.float16)
    if x.dim() != 2 or qweight.dim() != 2:
        raise ValueError("x and qweight must be 2-D")
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 8 != K:
        raise ValueError(f"qweight has {qweight.shape[1]} words per row, K={K} needs {K // 8}")
    if scales.shape != (N, K // group_size) or zeros.shape != scales.shape:
        raise ValueError("scales/zeros must be [N, K/group_size]")
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=x.device)
    if out is not None:
        _need_gpu("out", y, torch.float16)
        if tuple(y.shape) != (M, N):
            raise ValueError("out must be [M, N]")
    if workspace is None:
        st = load().awq_gemm_path(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), M, N, K, group_size,
                                  _ptr(y), int(path), _stream(x.device))
        _check("awq_gemm", st)
    else:
        _need_gpu("workspace", workspace, torch.uint8)
        st = load().awq_gemm_ex(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), M, N, K, group_size,
                                _ptr(y), int(path), _ptr(workspace), workspace.numel(), _stream(x.device))
        _check("awq_gemm_ex", st)
    return y


def awq_gemm_noalloc(x, qweight, scales, zeros, group_size: int = 128, path: int = PATH_AUTO, out=None):
    """awq_gemm_noalloc: awq_gemm with the skinny kernel's K-split scratch
    held by the library (no workspace, no device allocation in the call;
    calls on one device must not overlap). Pass `out` to keep the binding
    from allocating y."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    _need_gpu("qweight", qweight, torch.int32)
    _need_gpu("scales", scales, torch.float16)
    _need_gpu("zeros", zeros, torch.float16)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape != (N, K // 8) or K % 8:
        raise ValueError(f"qweight must be [N, K/8] = [{N}, {K // 8}]")
    if scales.shape != (N, K // group_size) or zeros.shape != scales.shape:
        raise ValueError("scales/zeros must be [N, K/group_size]")
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=x.device)
    _need_gpu("out", y, torch.float16)
    if tuple(y.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    st = load().awq_gemm_noalloc(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), M, N, K, group_size, _ptr(y),
                                 int(path), _stream(x.device))
    _check("awq_gemm_noalloc", st)
    return y


def awq_gemm_grouped(x, layers, group_size: int = 128, outs=None):
    """y_i = x . dequant(Wq_i)^T for layers [(qweight, scales, zeros), ...]
    (1 to 4) that share x: one GEMV or column-tile launch over their
    stacked rows where awq_gemm would take that kernel, else one awq_gemm
    per layer. Returns the list of y_i (`outs`, when given, receives them)."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    n = len(layers)
    ys = list(outs) if outs is not None else [None] * n
    if len(ys) != n:
        raise ValueError("outs must hold one tensor per layer")
    Ns = []
    for i, (qw, sc, zr) in enumerate(layers):
        _need_gpu("qweight", qw, torch.int32)
        _need_gpu("scales", sc, torch.float16)
        _need_gpu("zeros", zr, torch.float16)
        N = qw.shape[0]
        if qw.dim() != 2 or qw.shape[1] * 8 != K:
            raise ValueError(f"layer {i}: qweight must be [N, K/8] with K = {K}")
        if sc.shape != (N, K // group_size) or zr.shape != sc.shape:
            raise ValueError(f"layer {i}: scales/zeros must be [N, K/group_size]")
        if ys[i] is None:
            ys[i] = torch.empty((M, N), dtype=torch.float16, device=x.device)
        _need_gpu("out", ys[i], torch.float16)
        if tuple(ys[i].shape) != (M, N):
            raise ValueError(f"layer {i}: out must be [M, N]")
        Ns.append(N)
    arr = ctypes.c_void_p * max(n, 1)
    st = load().awq_gemm_grouped(
        _ptr(x), n, arr(*[_ptr(l[0]) for l in layers]), arr(*[_ptr(l[1]) for l in layers]),
        arr(*[_ptr(l[2]) for l in layers]), (ctypes.c_int64 * max(n, 1))(*Ns), M, K, group_size,
        arr(*[_ptr(y) for y in ys]), _stream(x.device))
    _check("awq_gemm_grouped", st)
    return ys


def awq_activation_absmean(x):
    """m[k] = max(mean_t |x[t, k]|, 1e-8) in fp64, x fp16 [T, K]."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    T, K = x.shape
    L = load()
    m = torch.empty(K, dtype=torch.float64, device=x.device)
    nbytes = L.awq_activation_absmean_workspace_bytes(T, K)
    ws = torch.empty(max(nbytes, 8), dtype=torch.uint8, device=x.device)
    st = L.awq_activation_absmean(_ptr(x), T, K, _ptr(m), _ptr(ws), nbytes, _stream(x.device))
    _check("awq_activation_absmean", st)
    return m


def scale_search_workspace_bytes(N: int, K: int, T: int, group_size: int = 128, n_alpha: int = 20) -> int:
    return int(load().awq_scale_search_workspace_bytes(N, K, T, group_size, n_alpha))


def awq_scale_search(w, x, group_size: int = 128, alphas=None, workspace=None, n_alpha: int = 20):
    """AWQ scale search over an alpha grid.

    Returns (losses: numpy float64 [n_alpha], best_index: int,
    best_scales: fp32 GPU tensor [K])."""
    import numpy as np
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    _need_gpu("x", x, torch.float16)
    N, K = w.shape
    T = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x must be [T, K] with the K of w")
    # no grid given: the library's default grid of n_alpha points
    if alphas is not None:
        alphas = np.ascontiguousarray(alphas, dtype=np.float64)
    n_alpha = int(alphas.size) if alphas is not None else int(n_alpha)
    L = load()
    nbytes = L.awq_scale_search_workspace_bytes(N, K, T, group_size, n_alpha)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=w.device)
    losses = np.zeros(n_alpha, dtype=np.float64)
    best = ctypes.c_int(-1)
    best_scales = torch.empty(K, dtype=torch.float32, device=w.device)
    st = L.awq_scale_search(_ptr(w), _ptr(x), N, K, T, group_size,
                            None if alphas is None else alphas.ctypes.data_as(ctypes.c_void_p), n_alpha,
                            _ptr(workspace), workspace.numel(),
                            losses.ctypes.data_as(ctypes.c_void_p), ctypes.addressof(best),
                            _ptr(best_scales), _stream(w.device))
    _check("awq_scale_search", st)
    return losses, int(best.value), best_scales


def awq_clip_search(w, x, fractions, group_size: int = 128, channel_scale=None, symmetric: bool = False,
                    workspace=None):
    """Clip-fraction search (awq_clip_search). Returns (losses: numpy float64
    [n], best_index: int)."""
    import numpy as np
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    _need_gpu("x", x, torch.float16)
    N, K = w.shape
    T = x.shape[0]
    if channel_scale is not None:
        _need_gpu("channel_scale", channel_scale, torch.float32)
        if channel_scale.numel() != K:
            raise ValueError("channel_scale must have K elements")
    fr = np.ascontiguousarray(fractions, dtype=np.float64)
    n = int(fr.size)
    L = load()
    nbytes = L.awq_clip_search_workspace_bytes(N, K, T, group_size, n, int(channel_scale is not None))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=w.device)
    losses = np.zeros(n, dtype=np.float64)
    best = ctypes.c_int(-1)
    mode = QUANT_SYMMETRIC if symmetric else QUANT_ASYMMETRIC
    st = L.awq_clip_search(_ptr(w), _ptr(x), _ptr(channel_scale), N, K, T, group_size, mode,
                           fr.ctypes.data_as(ctypes.c_void_p), n, _ptr(workspace), workspace.numel(),
                           losses.ctypes.data_as(ctypes.c_void_p), ctypes.addressof(best), _stream(w.device))
    _check("awq_clip_search", st)
    return losses, int(best.value)


# ---------------------------------------------------------------- mixed precision (fp16 salient channels)

def select_salient(m, n_salient: int):
    """awq_select_salient: int32 [n_salient] channel indices, largest m first
    (m: fp64 GPU tensor [K], e.g. awq_activation_absmean's)."""
    torch = _torch()
    _need_gpu("m", m, torch.float64)
    idx = torch.empty(max(n_salient, 1), dtype=torch.int32, device=m.device)[:n_salient]
    _check("awq_select_salient", load().awq_select_salient(_ptr(m), m.numel(), n_salient, _ptr(idx),
                                                           _stream(m.device)))
    return idx


def awq_quantize_salient(w, group_size: int, idx, symmetric: bool = False):
    """awq_quantize_salient: (qweight, scales, zeros, w_salient fp16
    [n_salient, N]) for the channels idx (int32 GPU tensor)."""
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    _need_gpu("idx", idx, torch.int32)
    N, K = w.shape
    n = idx.numel()
    dev = w.device
    qweight = torch.empty((N, max(K // 8, 0)), dtype=torch.int32, device=dev)
    ng = K // group_size if group_size > 0 else 0
    scales = torch.empty((N, ng), dtype=torch.float16, device=dev)
    zeros = torch.empty((N, ng), dtype=torch.float16, device=dev)
    w_sal = torch.empty((n, N), dtype=torch.float16, device=dev)
    mode = QUANT_SYMMETRIC if symmetric else QUANT_ASYMMETRIC
    st = load().awq_quantize_salient(_ptr(w), N, K, group_size, mode, _ptr(idx), n, _ptr(qweight), _ptr(scales),
                                     _ptr(zeros), _ptr(w_sal), _stream(dev))
    _check("awq_quantize_salient", st)
    return qweight, scales, zeros, w_sal


def awq_salient_apply(x, idx, w_salient, y):
    """awq_salient_apply: y (fp16 [M, N]) += x[:, idx] . w_salient, in place."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    _need_gpu("idx", idx, torch.int32)
    _need_gpu("w_salient", w_salient, torch.float16)
    _need_gpu("y", y, torch.float16)
    M, K = x.shape
    n, N = w_salient.shape
    if idx.numel() != n or y.shape != (M, N):
        raise ValueError("shapes: idx [n], w_salient [n, N], y [M, N]")
    _check("awq_salient_apply", load().awq_salient_apply(_ptr(x), _ptr(idx), _ptr(w_salient), M, N, K, n, _ptr(y),
                                                         _stream(x.device)))
    return y


def awq_gemm_salient(x, qweight, scales, zeros, idx, w_salient, group_size: int = 128, path: int = PATH_AUTO,
                     out=None, workspace=None):
    """The mixed layer: awq_gemm then awq_salient_apply on the same stream."""
    y = awq_gemm(x, qweight, scales, zeros, group_size, path=path, out=out, workspace=workspace)
    return awq_salient_apply(x, idx, w_salient, y)


def awq_salient_loss(w, x, group_size: int = 128, n_salient: int | None = None, symmetric: bool = False,
                     workspace=None):
    """awq_salient_loss: (loss_rtn, loss_salient, idx int32 GPU tensor).
    n_salient defaults to the library's awq_salient_count(K), the pages' 1 %."""
    import numpy as np
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    _need_gpu("x", x, torch.float16)
    N, K = w.shape
    T = x.shape[0]
    L = load()
    n = int(L.awq_salient_count(K)) if n_salient is None else int(n_salient)
    nbytes = L.awq_salient_loss_workspace_bytes(N, K, T, group_size, n)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=w.device)
    idx = torch.empty(max(n, 1), dtype=torch.int32, device=w.device)[:n]
    lr, ls = np.zeros(1), np.zeros(1)
    mode = QUANT_SYMMETRIC if symmetric else QUANT_ASYMMETRIC
    st = L.awq_salient_loss(_ptr(w), _ptr(x), N, K, T, group_size, mode, n, _ptr(workspace), workspace.numel(),
                            lr.ctypes.data_as(ctypes.c_void_p), ls.ctypes.data_as(ctypes.c_void_p), _ptr(idx),
                            _stream(w.device))
    _check("awq_salient_loss", st)
    return float(lr[0]), float(ls[0]), idx


# ---------------------------------------------------------------- W8A16

def awq_quantize_w8(w, group_size: int = 128, channel_scale=None, symmetric: bool = False, out=None):
    """awq_quantize_w8: (qweight int32 [N, K/4] holding the uint32 words,
    scales fp16 [N, K/G], zeros fp16 [N, K/G])."""
    torch = _torch()
    _need_gpu("w", w, torch.float16)
    N, K = w.shape
    if channel_scale is not None:
        _need_gpu("channel_scale", channel_scale, torch.float32)
        if channel_scale.numel() != K:
            raise ValueError("channel_scale must have K elements")
    ng = K // group_size if group_size > 0 else 0
    if out is None:
        out = (torch.empty((N, max(K // 4, 0)), dtype=torch.int32, device=w.device),
               torch.empty((N, ng), dtype=torch.float16, device=w.device),
               torch.empty((N, ng), dtype=torch.float16, device=w.device))
    qweight, scales, zeros = out
    _need_out(qweight, scales, zeros, (N, K // 4), (N, ng), w.device)
    mode = QUANT_SYMMETRIC if symmetric else QUANT_ASYMMETRIC
    st = load().awq_quantize_w8(_ptr(w), _ptr(channel_scale), N, K, group_size, mode, _ptr(qweight), _ptr(scales),
                                _ptr(zeros), _stream(w.device))
    _check("awq_quantize_w8", st)
    return qweight, scales, zeros


def awq_gemm_w8(x, qweight, scales, zeros, group_size: int = 128, path: int = PATH_AUTO, out=None, workspace=None):
    """awq_gemm_w8: y = x . dequant(Wq)^T for the W8 form (path 0 auto,
    1 GEMV, 2 GEMM)."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    _need_gpu("qweight", qweight, torch.int32)
    _need_gpu("scales", scales, torch.float16)
    _need_gpu("zeros", zeros, torch.float16)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape != (N, K // 4) or K % 4:
        raise ValueError("qweight must be [N, K/4]")
    if scales.shape != (N, K // group_size) or zeros.shape != scales.shape:
        raise ValueError("scales/zeros must be [N, K/group_size]")
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=x.device)
    _need_gpu("out", y, torch.float16)
    if tuple(y.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    if workspace is not None:
        _need_gpu("workspace", workspace, torch.uint8)
    nbytes = workspace.numel() if workspace is not None else 0
    st = load().awq_gemm_w8(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), M, N, K, group_size, _ptr(y), path,
                            _ptr(workspace), nbytes, _stream(x.device))
    _check("awq_gemm_w8", st)
    return y


# ---------------------------------------------------------------- the linear layer with its epilogue

def _need_on(name: str, t, dtype, index: int) -> None:
    _need_gpu(name, t, dtype)
    if t.get_device() != index:
        raise ValueError(f"{name} must be on GPU {index}")


def _workspace(t, index: int):
    """Address and bytes of a uint8 workspace on GPU `index`, or of none."""
    if t is None:
        return None, 0
    _need_on("workspace", t, _torch().uint8, index)
    return t.data_ptr(), t.numel()


def _rows(name: str, t, shape, dtype, index: int):
    """Address and row stride of fp16 [M, N] with contiguous rows, or of none."""
    if t is None:
        return None, 0
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on GPU {index}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    row, col = t.stride()
    if shape[1] > 1 and col != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _explain_layer(x, qweight, scales, zeros, group_size) -> None:
    """Raises what is wrong with a linear layer's tensors."""
    torch = _torch()
    _need_gpu("x", x, torch.float16)
    index = x.get_device()
    _need_on("qweight", qweight, torch.int32, index)
    _need_on("scales", scales, torch.float16, index)
    _need_on("zeros", zeros, torch.float16, index)
    if x.dim() != 2 or qweight.dim() != 2:
        raise ValueError("x and qweight must be 2-D")
    if not isinstance(group_size, int) or group_size < 1:
        raise ValueError("group_size must be a positive integer")
    raise ValueError("scales/zeros must be [N, K/group_size]")


def awq_gemm_fused(x, qweight, scales, zeros, group_size: int = 128, bias=None, activation: str = "none", mul=None,
                   residual=None, path: int = PATH_AUTO, out=None, workspace=None):
    """awq_gemm_fused: y = act(x . dequant(Wq)^T + bias) * mul + residual in
    one launch, INT4 or W8 weights by qweight's width (K / 8 or K / 4 words).

    bias fp16 [N]; mul and residual fp16 [M, N], rows N halves or more apart;
    activation one of ACTIVATIONS. out may be residual or mul itself (when
    packed). workspace: gemm_workspace(M, N, K)."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    ext, entry, *_ = _fast or _fast_calls()
    if ext is not None:
        try:
            index = x.get_device()
            y = x.new_empty((x.shape[0], qweight.shape[0])) if out is None else out
            stream = _stream_on(index)
        except (AttributeError, IndexError, TypeError, ValueError):
            stream = None
        if stream is not None:
            st = ext.gemm_fused(entry, stream, index, x, qweight, scales, zeros, group_size, bias, act, mul, residual,
                                path, y, workspace)
            if st == AWQ_OK:
                return y
            if st is not None:
                _check("awq_gemm_fused", st)
    torch = _torch()
    half = torch.float16
    try:
        (M, K), (N, words), index = x.shape, qweight.shape, x.get_device()
        layer = (N, K // group_size)
        ok = x.dtype is half and x.is_contiguous() and qweight.dtype is torch.int32 and qweight.is_contiguous() and \
            scales.dtype is half and scales.is_contiguous() and zeros.dtype is half and zeros.is_contiguous() and \
            scales.shape == layer and zeros.shape == layer and \
            index == qweight.get_device() == scales.get_device() == zeros.get_device() and index >= 0
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ok = False
    if not ok:
        _explain_layer(x, qweight, scales, zeros, group_size)
    bits = 4 if words * 8 == K else 8
    if words * 32 != K * bits:
        raise ValueError(f"qweight has {words} words per row, K={K} needs {K // 8} (INT4) or {K // 4} (W8)")
    bias_p = None
    if bias is not None:
        _need_on("bias", bias, half, index)
        if bias.shape != (N,):
            raise ValueError(f"bias must be [{N}]")
        bias_p = bias.data_ptr()
    shape = (M, N)
    mul_p, mul_stride = _rows("mul", mul, shape, half, index)
    res_p, res_stride = _rows("residual", residual, shape, half, index)
    if out is None:
        out = torch.empty(shape, dtype=half, device=x.device)
    elif out.dtype is not half or out.shape != shape or not out.is_contiguous() or out.get_device() != index:
        _need_on("out", out, half, index)
        raise ValueError(f"out must be [{M}, {N}]")
    ws, nbytes = _workspace(workspace, index)
    st = _on_device(index, (_lib or load()).awq_gemm_fused, x.data_ptr(), qweight.data_ptr(), scales.data_ptr(),
                    zeros.data_ptr(), M, N, K, group_size, bits, bias_p, act, mul_p, mul_stride, res_p, res_stride,
                    out.data_ptr(), path, ws, nbytes)
    if st != AWQ_OK:
        _check("awq_gemm_fused", st)
    return out


# ---------------------------------------------------------------- the paged 8-bit key / value cache

class KVCache:
    """A paged 8-bit key / value cache (awq_kv_cache): the caller's tensors
    k_codes uint8 [pages, heads, D / 16, page, 16], v_codes uint8 [pages,
    heads, page / 16, D, 16], k_scales and v_scales fp32 [pages, heads];
    fmt "int8" or "e4m3". KVCache.empty allocates them."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales, fmt: str = "int8"):
        torch = _torch()
        if fmt not in KV_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(KV_FORMATS)}")
        _need_gpu("k_codes", k_codes, torch.uint8)
        _need_gpu("v_codes", v_codes, torch.uint8)
        _need_gpu("k_scales", k_scales, torch.float32)
        _need_gpu("v_scales", v_scales, torch.float32)
        if k_codes.dim() != 5 or k_codes.shape[4] != 16:
            raise ValueError("k_codes must be [pages, heads, D / 16, page, 16]")
        pages, heads, dc, page, _ = k_codes.shape
        if tuple(v_codes.shape) != (pages, heads, page // 16, dc * 16, 16) or page % 16:
            raise ValueError(f"v_codes must be [{pages}, {heads}, page / 16, {dc * 16}, 16]")
        if tuple(k_scales.shape) != (pages, heads) or tuple(v_scales.shape) != (pages, heads):
            raise ValueError(f"k_scales and v_scales must be [{pages}, {heads}]")
        if len({t.device for t in (k_codes, v_codes, k_scales, v_scales)}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales, self.fmt = k_codes, v_codes, k_scales, v_scales, fmt
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = pages, heads, page, dc * 16
        self.device, self.index, self.half = k_codes.device, k_codes.get_device(), torch.float16
        self._struct = _KVCacheStruct(_ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), pages, heads, page,
                                      dc * 16, KV_FORMATS[fmt])
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, page_size: int = 64, fmt: str = "int8", device=None):
        """A cache of n_pages pages that hold nothing yet."""
        torch = _torch()
        dev = device or "cuda"
        return cls(torch.empty((n_pages, n_kv_heads, head_dim // 16, page_size, 16), dtype=torch.uint8, device=dev),
                   torch.empty((n_pages, n_kv_heads, page_size // 16, head_dim, 16), dtype=torch.uint8, device=dev),
                   torch.zeros((n_pages, n_kv_heads), dtype=torch.float32, device=dev),
                   torch.zeros((n_pages, n_kv_heads), dtype=torch.float32, device=dev), fmt)


class KVSeqs:
    """A batch of sequences over a cache (awq_kv_seqs): block_table int32
    [B, pages], cu_tokens int32 [B + 1], kv_len int32 [B] on the GPU.
    max_tokens and max_len bound the new tokens and the length of any
    sequence; without them they are read from the tensors (a
    synchronisation). The tensors may be changed in place between calls,
    within those bounds."""

    def __init__(self, block_table, cu_tokens, kv_len, max_tokens: int | None = None, max_len: int | None = None):
        torch = _torch()
        for name, t in (("block_table", block_table), ("cu_tokens", cu_tokens), ("kv_len", kv_len)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.device.type != "cuda":
                raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
        n = kv_len.numel()
        if kv_len.dim() != 1 or cu_tokens.dim() != 1 or cu_tokens.numel() != n + 1:
            raise ValueError("kv_len must be [B] and cu_tokens [B + 1]")
        if block_table.dim() != 2 or block_table.shape[0] != n:
            raise ValueError("block_table must be [B, pages]")
        if not kv_len.is_contiguous() or not cu_tokens.is_contiguous() or \
                (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("kv_len, cu_tokens and the rows of block_table must be contiguous")
        if not (block_table.device == cu_tokens.device == kv_len.device):
            raise ValueError("the batch's tensors must be on one device")
        if max_tokens is None:
            max_tokens = int((cu_tokens[1:] - cu_tokens[:-1]).max()) if n else 0
        if max_len is None:
            max_len = int(kv_len.max()) if n else 0
        self.block_table, self.cu_tokens, self.kv_len = block_table, cu_tokens, kv_len
        self.max_tokens, self.max_len, self.n_seqs = int(max_tokens), int(max_len), n
        self.device, self.index = kv_len.device, kv_len.get_device()
        stride = block_table.stride(0) if n > 1 else block_table.shape[1]
        self._struct = _KVSeqsStruct(_ptr(block_table), _ptr(cu_tokens), _ptr(kv_len), stride, block_table.shape[1], n,
                                     self.max_tokens, self.max_len)
        self._ref = ctypes.addressof(self._struct)


_torch_c = None        # (current device index, raw current stream of an index)


def _torch_calls():
    """torch's current device and the raw handle of a device's current stream,
    by its C entry points where this torch has them: the public Stream object
    costs 2 us a call, a third of a small launch."""
    global _torch_c
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    get = getattr(torch._C, "_cuda_getDevice", None)
    _torch_c = (get or torch.cuda.current_device,
                raw or (lambda i: torch.cuda.current_stream(i).cuda_stream))
    return _torch_c


_fast = None           # (extension or None, addresses of the library's entry points)


def _fast_calls():
    """The call extension (csrc/calls.cpp) and the entry points it calls; the
    wrappers below marshal in Python where it has not been built, or not for
    this interpreter and this torch."""
    global _fast
    _torch()
    entries = {n: ctypes.cast(getattr(load(), "awq_" + n), ctypes.c_void_p).value
               for n in ("gemm_fused", "kv_write", "kv_read", "kv_attention")}
    ext = None
    path = os.path.join(HERE, "_calls.so")
    if os.path.exists(path):
        import importlib.machinery
        import importlib.util
        loader = importlib.machinery.ExtensionFileLoader("_calls", path)
        try:
            ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
            loader.exec_module(ext)
        except ImportError as e:
            warnings.warn(f"{path} is of another build and is left out, calls take some 4 us longer; run "
                          f"`python -m weight_only_int4_quantize_amd.build` ({e})", RuntimeWarning, stacklevel=3)
            ext = None
    _fast = (ext, *entries.values())
    return _fast


def _stream_on(index) -> int | None:
    """The current stream of GPU `index` if that is the current device, else None."""
    if index < 0:       # a CPU tensor
        return None
    current, raw = _torch_c or _torch_calls()
    return raw(index) if current() == index else None


def _on_device(index: int, fn, *args) -> int:
    """fn(*args, stream) with GPU `index` current, on its current stream."""
    current, raw = _torch_c or _torch_calls()
    if current() == index:
        return fn(*args, raw(index))
    with _torch().cuda.device(index):
        return fn(*args, raw(index))


def _need_tokens(name: str, t, cache, heads: int | None) -> None:
    """Raises what is wrong with t as fp16 [T, heads, D] with contiguous
    channels on the cache's device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    if t.get_device() != cache.index:
        raise ValueError(f"{name} must be on {cache.device}")
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {cache.head_dim}]")
    if t.stride(2) != 1:
        raise ValueError(f"{name}'s channels must be contiguous")


def _tokens(name: str, t, cache, heads: int | None):
    """Checks t (see _need_tokens); its tokens, heads, and the strides of
    both (0 where there is one)."""
    try:
        T, h, D = t.shape
        st, sh, sd = t.stride()
        ok = sd == 1 and D == cache.head_dim and (heads is None or h == heads) and t.dtype is cache.half and \
            t.get_device() == cache.index
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        _need_tokens(name, t, cache, heads)
    return T, h, st if T > 1 else 0, sh if h > 1 else 0


def _need_seqs(cache, seqs) -> None:
    if seqs.index != cache.index:
        raise ValueError(f"seqs must be on {cache.device}")


def awq_kv_write(cache: KVCache, seqs: KVSeqs, k, v) -> None:
    """awq_kv_write: quantizes the batch's new tokens k, v (fp16 [T, heads, D],
    any token and head strides that are multiples of 8) into the cache."""
    _need_seqs(cache, seqs)
    ext, _, entry, *_ = _fast or _fast_calls()
    stream = _stream_on(cache.index) if ext is not None else None
    if stream is not None:
        st = ext.kv_write(entry, stream, cache.index, cache._ref, seqs._ref, cache.n_kv_heads, cache.head_dim, k, v)
        if st == AWQ_OK:
            return
        if st is not None:
            _check("awq_kv_write", st)
    T, _, k_token, k_head = _tokens("k", k, cache, cache.n_kv_heads)
    T2, _, v_token, v_head = _tokens("v", v, cache, cache.n_kv_heads)
    if T2 != T:
        raise ValueError("k and v must hold the same tokens")
    st = _on_device(cache.index, (_lib or load()).awq_kv_write, cache._ref, seqs._ref, k.data_ptr(), k_token, k_head,
                    v.data_ptr(), v_token, v_head, T)
    if st != AWQ_OK:
        _check("awq_kv_write", st)


def awq_kv_read(cache: KVCache, seqs: KVSeqs, n_tokens: int | None = None, out=None):
    """awq_kv_read: the sequences' newest tokens as (k, v), fp16
    [n_tokens, heads, D] each, rows as seqs.cu_tokens says (n_tokens defaults
    to its last entry, read with a synchronisation). out: the two tensors to
    fill, either of them None to leave it out; rows of no sequence stay."""
    torch = _torch()
    _need_seqs(cache, seqs)
    if out is None:
        T = int(seqs.cu_tokens[-1]) if n_tokens is None else int(n_tokens)
        out = tuple(torch.zeros((T, cache.n_kv_heads, cache.head_dim), dtype=torch.float16, device=cache.device)
                    for _ in range(2))
    k, v = out
    ext, _, _, entry, _ = _fast or _fast_calls()
    stream = _stream_on(cache.index) if ext is not None and n_tokens is None else None
    if stream is not None:
        st = ext.kv_read(entry, stream, cache.index, cache._ref, seqs._ref, cache.n_kv_heads, cache.head_dim, k, v)
        if st == AWQ_OK:
            return k, v
        if st is not None:
            _check("awq_kv_read", st)
    T = None
    for name, t in (("k", k), ("v", v)):
        if t is None:
            continue
        rows = _tokens(name, t, cache, cache.n_kv_heads)[0]
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if T is not None and rows != T:
            raise ValueError("k and v must hold the same tokens")
        T = rows
    if T is None:
        return k, v
    if n_tokens is not None and n_tokens != T:
        raise ValueError(f"out must hold {n_tokens} tokens")
    st = _on_device(cache.index, (_lib or load()).awq_kv_read, cache._ref, seqs._ref, _ptr(k), _ptr(v), T)
    if st != AWQ_OK:
        _check("awq_kv_read", st)
    return k, v


def kv_attention_workspace_bytes(cache: KVCache, seqs: KVSeqs, n_heads: int) -> int:
    return int(load().awq_kv_attention_workspace_bytes(cache._ref, seqs._ref, n_heads))


def kv_attention_workspace(cache: KVCache, seqs: KVSeqs, n_heads: int):
    """A zero-filled uint8 GPU tensor for awq_kv_attention calls of these
    bounds (max_tokens, max_len) and heads, and of any that need no more.
    Each call leaves it ready for the next, without clearing."""
    torch = _torch()
    nbytes = kv_attention_workspace_bytes(cache, seqs, n_heads)
    if nbytes == 0:
        raise AwqError("awq_kv_attention_workspace_bytes", 4, "the call cannot take these arguments")
    return torch.zeros(nbytes, dtype=torch.uint8, device=cache.device)


def awq_kv_attention(q, cache: KVCache, seqs: KVSeqs, scale: float | None = None, causal: bool = True, window: int = 0,
                     out=None, lse=None, workspace=None):
    """awq_kv_attention: softmax attention of the batch's newest tokens q (fp16
    [T, heads, D], heads a multiple of the cache's) over the cache. scale
    defaults to D ** -0.5; lse, when given, is fp32 [T, heads] and receives
    the softmax denominators' logarithms. Without `out` the rows of no
    sequence are 0."""
    torch = _torch()
    _need_seqs(cache, seqs)
    if scale is None:
        scale = cache.head_dim ** -0.5
    ext, *_, entry = _fast or _fast_calls()
    stream = _stream_on(cache.index) if ext is not None and out is not None else None
    if stream is not None:
        st = ext.kv_attention(entry, stream, cache.index, cache._ref, seqs._ref, cache.head_dim, q, scale, causal,
                              window, out, lse, workspace)
        if st == AWQ_OK:
            return out
        if st is not None:
            _check("awq_kv_attention", st)
    T, heads, q_token, q_head = _tokens("q", q, cache, None)
    if out is None:
        out = torch.zeros((T, heads, cache.head_dim), dtype=torch.float16, device=q.device)
    T2, _, out_token, out_head = _tokens("out", out, cache, heads)
    if T2 != T:
        raise ValueError(f"out must be [{T}, {heads}, {cache.head_dim}]")
    if lse is not None:
        _need_gpu("lse", lse, torch.float32)
        if tuple(lse.shape) != (T, heads) or lse.device != q.device:
            raise ValueError(f"lse must be [{T}, {heads}] on {q.device}")
    ws, nbytes = _workspace(workspace, cache.index)
    st = _on_device(cache.index, (_lib or load()).awq_kv_attention, cache._ref, seqs._ref, q.data_ptr(), q_token, q_head,
                    T, heads, scale, 1 if causal else 0, window,
                    out.data_ptr(), out_token, out_head, _ptr(lse), ws, nbytes)
    if st != AWQ_OK:
        _check("awq_kv_attention", st)
    return out
