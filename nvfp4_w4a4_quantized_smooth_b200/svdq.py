"""Thin ctypes binding of libsvdq.so (include/svdq.h), same call names.

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch supplies device
memory and streams); each wrapper checks dtypes / contiguity, passes raw
device pointers and the current stream, and raises ``SvdqError`` on a
non-OK status.  There is no CPU fallback: if the library cannot be loaded
the import of this module fails.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvdq.so")

SVDQ_OK = 0
SVDQ_ERR_INVALID_ARG = 1
SVDQ_ERR_SHAPE = 2
SVDQ_ERR_ALIGNMENT = 3
SVDQ_ERR_UNSUPPORTED = 4
SVDQ_ERR_ARCH = 5
SVDQ_ERR_CUDA = 6
SVDQ_ERR_TIMEOUT = 7

# Constants of include/svdq.h.
ABI_VERSION = 11
SCALES_ACT = 0
SCALES_WEIGHT = 1
GEMM_TOKEN_MAJOR = 0
GEMM_FEW_TOKENS = 1
GEMM_PAIRS = 2
BF16 = 0
FP16 = 1
NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2
GATE_NONE = 0
GATE_LINEAR = 1
GATE_TANH = 2

# Every symbol include/svdq.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_L = ctypes.c_int64
_F = ctypes.c_float
_D = ctypes.c_double
SIGNATURES = {
    "svdq_status_string": (ctypes.c_char_p, [_I]),
    "svdq_abi_version": (_I, []),
    "svdq_ascales_tiled_bytes": (_SZ, [_I, _I]),
    "svdq_wscales_tiled_bytes": (_SZ, [_I, _I]),
    "svdq_lowrank_bytes": (_SZ, [_I, _I]),
    "svdq_repack_weights": (_I, [_P, _I, _I, _P, _P]),
    "svdq_quantize_act": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P]),
    "svdq_w4a4_linear": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I,
                              _P]),
    "svdq_fold_proj_up": (_I, [_P, _P, _P, _I, _I, _P, _P, _P]),
    "svdq_silu_mul_quantize_act": (_I, [_P, _P, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P]),
    "svdq_quantize_plan": (_I, [_I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "svdq_linear_plan": (_I, [_I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I),
                              ctypes.POINTER(_I)]),
    "svdq_unpack_scales": (_I, [_P, _I, _I, _I, _P, _P]),
    "svdq_silu_mul": (_I, [_P, _P, _P, _SZ, _P]),
    "svdq_weight_workspace_bytes": (_SZ, [_I]),
    "svdq_quantize_weights": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "svdq_quantize_weights_noalloc": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P]),
    "svdq_norm_gate_residual": (_I, [_I, _P, _L, _P, _L, _I, _I, _P, _I, _I, _P, _I, _P, _L, _F,
                                     _I, _P, _P, _L, _P, _L, _F, _P, _L, _P, _L, _P]),
    "svdq_rope_turns": (_I, [_P, _I, _D, _P]),
    "svdq_rope_qk": (_I, [_I, _P, _L, _L, _I, _P, _L, _L, _I, _I, _I, _P, _L, _P, _I, _P, _I, _P,
                          _P, _F, _P, _L, _L, _P, _L, _L, _P]),
    "svdq_attention": (_I, [_I, _P, _L, _L, _P, _L, _L, _P, _L, _L, _I, _I, _I, _I, _P, _I, _I,
                            _F, _P, _L, _L, _P, _SZ, _P]),
    "svdq_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "svdq_check_device_error": (_I, [_P]),
    "svdq_set_wait_timeout_ns": (_I, [ctypes.c_uint64]),
    "svdq_wait_probe": (_I, [_I, _P]),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python -m nvfp4_w4a4_quantized_smooth_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.svdq_abi_version() != ABI_VERSION:
        raise ImportError(f"{path} has ABI version {lib.svdq_abi_version()}, this binding "
                          f"expects {ABI_VERSION}: rebuild it")
    return lib


_lib = load_library()


class SvdqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.svdq_status_string(status).decode()
        super().__init__(f"{where}: {msg}")


def _check(status: int, where: str) -> None:
    if status != SVDQ_OK:
        raise SvdqError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str, dim: Optional[int] = None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims")


def abi_version() -> int:
    return _lib.svdq_abi_version()


def ascales_tiled_bytes(M: int, K: int) -> int:
    return _lib.svdq_ascales_tiled_bytes(M, K)


def wscales_tiled_bytes(N: int, K: int) -> int:
    return _lib.svdq_wscales_tiled_bytes(N, K)


def lowrank_bytes(M: int, R: int) -> int:
    return _lib.svdq_lowrank_bytes(M, R)


def repack_weights(wscales: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """wscales [K/16, N] uint8 (e4m3 codes) -> tiled scale buffer (uint8)."""
    _need(wscales, torch.uint8, "wscales", 2)
    wscales = wscales.contiguous()
    K = wscales.shape[0] * 16
    N = wscales.shape[1]
    nbytes = wscales_tiled_bytes(N, K)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=wscales.device)
    _check(_lib.svdq_repack_weights(_ptr(wscales), N, K, _ptr(out), _stream(stream)),
           "svdq_repack_weights")
    return out


def quantize_act(x: torch.Tensor, smooth: Optional[torch.Tensor],
                 proj_down: Optional[torch.Tensor],
                 qact: Optional[torch.Tensor] = None,
                 ascales_tiled: Optional[torch.Tensor] = None,
                 lowrank: Optional[torch.Tensor] = None, stream=None):
    """x [M, K] bf16 (row stride may exceed K) -> (qact, ascales_tiled, lowrank).

    smooth None: no smoothing.  proj_down None: the plain NVFP4 layer
    (R = 0); lowrank is then None."""
    _need(x, torch.bfloat16, "x", 2)
    if smooth is not None:
        _need(smooth, torch.bfloat16, "smooth", 1)
        smooth = smooth.contiguous()
    if proj_down is not None:
        _need(proj_down, torch.bfloat16, "proj_down", 2)
        proj_down = proj_down.contiguous()
    if x.stride(1) != 1:
        raise ValueError("x must have unit stride along K")
    M, K = x.shape
    R = 0 if proj_down is None else proj_down.shape[1]
    dev = x.device
    if qact is None:
        qact = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if ascales_tiled is None:
        ascales_tiled = torch.empty(max(ascales_tiled_bytes(M, K), 1), dtype=torch.uint8,
                                    device=dev)
    if lowrank is None and R:
        lowrank = torch.empty(M, R, dtype=torch.bfloat16, device=dev)
    _check(_lib.svdq_quantize_act(_ptr(x), M, K, x.stride(0), _ptr(smooth), _ptr(proj_down), R,
                                  _ptr(qact), _ptr(ascales_tiled), _ptr(lowrank if R else None),
                                  _stream(stream)),
           "svdq_quantize_act")
    return qact, ascales_tiled, (lowrank if R else None)


def silu_mul_quantize_act(a: torch.Tensor, b: torch.Tensor, smooth: Optional[torch.Tensor],
                          proj_down: Optional[torch.Tensor],
                          qact: Optional[torch.Tensor] = None,
                          ascales_tiled: Optional[torch.Tensor] = None,
                          lowrank: Optional[torch.Tensor] = None, stream=None):
    """quantize_act of x = silu(a) * b (the w2 input of a DiT feed-forward
    block), formed on the device without writing x -> (qact, ascales_tiled,
    lowrank)."""
    _need(a, torch.bfloat16, "a", 2)
    _need(b, torch.bfloat16, "b", 2)
    if a.shape != b.shape or a.stride() != b.stride() or a.stride(1) != 1:
        raise ValueError("a and b must have the same shape and strides, unit stride along K")
    if smooth is not None:
        _need(smooth, torch.bfloat16, "smooth", 1)
        smooth = smooth.contiguous()
    if proj_down is not None:
        _need(proj_down, torch.bfloat16, "proj_down", 2)
        proj_down = proj_down.contiguous()
    M, K = a.shape
    R = 0 if proj_down is None else proj_down.shape[1]
    dev = a.device
    if qact is None:
        qact = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if ascales_tiled is None:
        ascales_tiled = torch.empty(max(ascales_tiled_bytes(M, K), 1), dtype=torch.uint8,
                                    device=dev)
    if lowrank is None and R:
        lowrank = torch.empty(M, R, dtype=torch.bfloat16, device=dev)
    _check(_lib.svdq_silu_mul_quantize_act(_ptr(a), _ptr(b), M, K, a.stride(0), _ptr(smooth),
                                           _ptr(proj_down), R, _ptr(qact), _ptr(ascales_tiled),
                                           _ptr(lowrank if R else None), _stream(stream)),
           "svdq_silu_mul_quantize_act")
    return qact, ascales_tiled, (lowrank if R else None)


def w4a4_linear(qact: torch.Tensor, ascales_tiled: torch.Tensor,
                lowrank: Optional[torch.Tensor], qweight: torch.Tensor,
                wscales_tiled: torch.Tensor, wcscales: torch.Tensor, wtscale: torch.Tensor,
                proj_up: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                y: Optional[torch.Tensor] = None, stream=None,
                proj_up_folded: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The block-scaled FP4 GEMM with the fused epilogue -> y [M, N] bf16.

    lowrank and proj_up None: the plain NVFP4 layer (R = 0).  proj_up_folded:
    fold_proj_up's factor for these proj_up / wcscales / wtscale (the GEMM
    for M > 128 then adds the low-rank product inside its accumulator)."""
    _need(qact, torch.uint8, "qact", 2)
    _need(qweight, torch.uint8, "qweight", 2)
    if (lowrank is None) != (proj_up is None):
        raise ValueError("lowrank and proj_up go together (both None for R = 0)")
    if lowrank is not None:
        _need(lowrank, torch.bfloat16, "lowrank", 2)
        _need(proj_up, torch.bfloat16, "proj_up", 2)
    if proj_up_folded is not None:
        _need(proj_up_folded, torch.bfloat16, "proj_up_folded", 2)
        if proj_up is None or proj_up_folded.shape != proj_up.shape:
            raise ValueError("proj_up_folded needs proj_up of the same shape")
    M = qact.shape[0]
    K = qact.shape[1] * 2
    N = qweight.shape[0]
    R = 0 if proj_up is None else proj_up.shape[1]
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=qact.device)
    _check(_lib.svdq_w4a4_linear(_ptr(qact), _ptr(ascales_tiled), _ptr(lowrank),
                                 _ptr(qweight), _ptr(wscales_tiled), _ptr(wcscales),
                                 _ptr(wtscale), _ptr(proj_up), _ptr(proj_up_folded), _ptr(bias),
                                 M, N, K, R, _ptr(y), y.stride(0), _stream(stream)),
           "svdq_w4a4_linear")
    return y


def fold_proj_up(proj_up: torch.Tensor, wcscales: torch.Tensor, wtscale: torch.Tensor,
                 stream=None):
    """svdq_fold_proj_up -> (proj_up_folded [N, R] bf16, number of elements
    that cannot be folded).  Reads the count back (synchronizes the
    stream); pass the factor to w4a4_linear only when the count is 0."""
    _need(proj_up, torch.bfloat16, "proj_up", 2)
    N, R = proj_up.shape
    out = torch.empty_like(proj_up)
    count = torch.empty(1, dtype=torch.int32, device=proj_up.device)
    _check(_lib.svdq_fold_proj_up(_ptr(proj_up), _ptr(wcscales), _ptr(wtscale), N, R, _ptr(out),
                                  _ptr(count), _stream(stream)),
           "svdq_fold_proj_up")
    if stream is not None:
        stream.synchronize()
    else:
        torch.cuda.current_stream(proj_up.device).synchronize()
    return out, int(count.item())


def quantize_plan(M: int, K: int):
    """(rows per CTA, K split) svdq_quantize_act uses for [M, K] on this device."""
    bm, split = _I(), _I()
    _check(_lib.svdq_quantize_plan(M, K, ctypes.byref(bm), ctypes.byref(split)),
           "svdq_quantize_plan")
    return bm.value, split.value


def linear_plan(M: int, N: int, K: int):
    """(kernel, K split, grid) svdq_w4a4_linear uses for M x N x K on this
    device; kernel is GEMM_PAIRS, GEMM_TOKEN_MAJOR or GEMM_FEW_TOKENS."""
    kernel, split, grid = _I(), _I(), _I()
    _check(_lib.svdq_linear_plan(M, N, K, ctypes.byref(kernel), ctypes.byref(split),
                                 ctypes.byref(grid)),
           "svdq_linear_plan")
    return kernel.value, split.value, grid.value


def unpack_scales(scales_tiled: torch.Tensor, rows: int, K: int, kind: str = "act",
                  stream=None) -> torch.Tensor:
    """Tiled scales -> logical [rows, K/16] uint8 (test / inspection helper).

    kind: "act" for svdq_quantize_act's order, "weight" for
    svdq_repack_weights' order."""
    code = {"act": SCALES_ACT, "weight": SCALES_WEIGHT}[kind]
    out = torch.empty(rows, K // 16, dtype=torch.uint8, device=scales_tiled.device)
    _check(_lib.svdq_unpack_scales(_ptr(scales_tiled), rows, K, code, _ptr(out),
                                   _stream(stream)),
           "svdq_unpack_scales")
    return out


def silu_mul(a: torch.Tensor, b: torch.Tensor, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """silu(a) * b elementwise, bf16 (the w2 input of a DiT FFN block)."""
    _need(a, torch.bfloat16, "a")
    _need(b, torch.bfloat16, "b")
    if a.shape != b.shape or not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("a and b must be contiguous with the same shape")
    if out is None:
        out = torch.empty_like(a)
    _check(_lib.svdq_silu_mul(_ptr(a), _ptr(b), _ptr(out), a.numel(), _stream(stream)),
           "svdq_silu_mul")
    return out


def quantize_weights_residual(W: torch.Tensor, smooth: torch.Tensor,
                              lowrank: Optional[torch.Tensor] = None, stream=None):
    """NVFP4 encoding of (W - lowrank) / smooth (svdq_quantize_weights) ->
    (qweight [N, K/2] uint8, wscales [K/16, N] uint8 e4m3 codes, wcscales
    [N] bf16, wtscale [1] bf16)."""
    _need(W, torch.bfloat16, "W", 2)
    _need(smooth, torch.bfloat16, "smooth", 1)
    W = W.contiguous()
    smooth = smooth.contiguous()
    if lowrank is not None:
        _need(lowrank, torch.float32, "lowrank", 2)
        lowrank = lowrank.contiguous()
    N, K = W.shape
    dev = W.device
    qweight = torch.empty(N, K // 2, dtype=torch.uint8, device=dev)
    wscales = torch.empty(K // 16, N, dtype=torch.uint8, device=dev)
    wcscales = torch.empty(N, dtype=torch.bfloat16, device=dev)
    wtscale = torch.empty(1, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(_lib.svdq_weight_workspace_bytes(N), dtype=torch.uint8, device=dev)
    _check(_lib.svdq_quantize_weights(_ptr(W), _ptr(smooth), _ptr(lowrank), N, K, _ptr(qweight),
                                      _ptr(wscales), _ptr(wcscales), _ptr(wtscale), _ptr(ws),
                                      _stream(stream)),
           "svdq_quantize_weights")
    return qweight, wscales, wcscales, wtscale


def quantize_weights(W: torch.Tensor, smooth: torch.Tensor, R: int = 128, stream=None,
                     return_lowrank: bool = False):
    """Offline weight side of the layer: a bf16 weight [N, K] and its
    smoothing factor [K] -> the stored operands (a dict: qweight, wscales,
    wcscales, wtscale, proj_down [K, R], proj_up [N, R]).

    The low-rank factors are the rank-R truncated SVD of W / smooth
    (proj_up = U_R S_R^1/2, proj_down = diag(smooth) V_R S_R^1/2, bf16),
    computed with torch's linear algebra on the device (a library SVD and
    GEMM: this runs once per layer at load time, not on the layer's path);
    the residual and its NVFP4 encoding run in svdq_quantize_weights.
    return_lowrank adds the float32 proj_up @ proj_down^T the encoding
    used (for tests)."""
    _need(W, torch.bfloat16, "W", 2)
    _need(smooth, torch.bfloat16, "smooth", 1)
    N, K = W.shape
    if R > min(N, K):
        raise ValueError("R exceeds the weight's rank bound")
    s = smooth.float()
    if R > 0:
        U, S, Vh = torch.linalg.svd(W.float() / s[None, :], full_matrices=False)
        sq = S[:R].sqrt()
        proj_up = (U[:, :R] * sq[None, :]).to(torch.bfloat16).contiguous()
        proj_down = (Vh[:R].T * sq[None, :] * s[:, None]).to(torch.bfloat16).contiguous()
        lowrank = proj_up.float() @ proj_down.float().T
    else:
        proj_up = torch.zeros(N, 0, dtype=torch.bfloat16, device=W.device)
        proj_down = torch.zeros(K, 0, dtype=torch.bfloat16, device=W.device)
        lowrank = None
    qweight, wscales, wcscales, wtscale = quantize_weights_residual(W, smooth, lowrank,
                                                                    stream=stream)
    out = dict(qweight=qweight, wscales=wscales, wcscales=wcscales, wtscale=wtscale,
               proj_down=proj_down, proj_up=proj_up)
    if return_lowrank:
        out["lowrank"] = lowrank
    return out


# ---- between the linears of a block -----------------------------------------

_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16}
_NORMS = {None: NORM_NONE, "rms": NORM_RMS, "layer": NORM_LAYER}


_current_device = torch.cuda.current_device


def _raw_stream(index: int) -> int:
    """The handle of the device's current stream (1.2 us less than through a
    Stream object).  Looked up at the call: a torch built without CUDA does not
    have it, and this module imports there."""
    return torch._C._cuda_getCurrentRawStream(index)


def _on(index: int, stream: Optional[torch.cuda.Stream]):
    """A context in which the stream (or, without one, the device of that
    index) is the current one.  A call on another stream or device than the
    current ones enters it and calls itself: its launch and the outputs it
    allocates then belong there."""
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return torch.cuda.stream(stream)


def _need_like(t: torch.Tensor, dtype: torch.dtype, index: int, shape, name: str):
    """Check an operand against the call's type, device and shape; its
    strides, with a last one of 1."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on cuda:{index}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return strides


def _need_16bit(t: torch.Tensor, name: str, dim: int) -> int:
    code = _DTYPES.get(t.dtype)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims")
    return code


def _need_cu(cu: torch.Tensor, index: int) -> int:
    """The number of sequences of cu_seqlens."""
    if (cu.dtype is not torch.int32 or cu.get_device() != index or cu.dim() != 1
            or cu.shape[0] < 2):
        raise ValueError(f"cu_seqlens must be an int32 vector of at least 2 on cuda:{index}")
    if not cu.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous")
    return cu.shape[0] - 1


def norm_gate_residual(x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                       gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                       shift: Optional[torch.Tensor] = None,
                       post_weight: Optional[torch.Tensor] = None,
                       pre_weight: Optional[torch.Tensor] = None, post: Optional[str] = None,
                       pre: Optional[str] = "rms", eps: float = 1e-6, gate_tanh: bool = False,
                       residual_scale: float = 1.0, cu_seqlens: Optional[torch.Tensor] = None,
                       h: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None,
                       stream=None):
    """The norms before and after a block with its gate and residual scale:

        h = residual_scale * x + gate * post(y)
        n = pre(h) * (1 + scale) + shift

    x, y [T, C] bf16 or fp16; gate, scale, shift [n_seqs, C] (tanh(gate) with
    gate_tanh), rows by cu_seqlens [n_seqs + 1] int32; post, pre: None, "rms"
    or "layer" with their weights [C] -> (h, n).  y None (the first norm of a
    stack): h is x itself.  pre None without scale and shift: n is None.
    h and n may be given, also exactly x or y; rows in no sequence are left
    as they are."""
    code = _need_16bit(x, "x", 2)
    index = x.get_device()
    if stream is not None or index != _current_device():
        with _on(index, stream):
            return norm_gate_residual(x, y, gate=gate, scale=scale, shift=shift,
                                      post_weight=post_weight, pre_weight=pre_weight, post=post,
                                      pre=pre, eps=eps, gate_tanh=gate_tanh,
                                      residual_scale=residual_scale, cu_seqlens=cu_seqlens, h=h,
                                      n=n)
    if post not in _NORMS or pre not in _NORMS:
        raise ValueError('post and pre must be None, "rms" or "layer"')
    shape, dtype = x.shape, x.dtype
    T, C = shape
    S, cu = 1, None
    if cu_seqlens is not None:
        S, cu = _need_cu(cu_seqlens, index), cu_seqlens.data_ptr()
    ldx = _need_like(x, dtype, index, shape, "x")[0]
    py = pg = ps = pb = pw = qw = pn = ph = None
    ldy = ldg = lds = ldb = ldh = ldn = 0
    if y is not None:
        ldy = _need_like(y, dtype, index, shape, "y")[0]
        py = y.data_ptr()
        if h is None:
            h = torch.empty_like(x, memory_format=torch.contiguous_format)
            ldh = C
        else:
            ldh = _need_like(h, dtype, index, shape, "h")[0]
        ph = h.data_ptr()
    elif h is not None:
        raise ValueError("h needs y (without y it is x itself)")
    kind = GATE_NONE
    if gate is not None:
        kind = GATE_TANH if gate_tanh else GATE_LINEAR
        ldg = _need_like(gate, dtype, index, (S, C), "gate")[0]
        pg = gate.data_ptr()
    if scale is not None:
        lds = _need_like(scale, dtype, index, (S, C), "scale")[0]
        ps = scale.data_ptr()
    if shift is not None:
        ldb = _need_like(shift, dtype, index, (S, C), "shift")[0]
        pb = shift.data_ptr()
    if S == 1:                     # the stride of a dimension of one means nothing
        ldg = lds = ldb = 0
    if post_weight is not None:
        _need_like(post_weight, dtype, index, (C,), "post_weight")
        pw = post_weight.data_ptr()
    if pre_weight is not None:
        _need_like(pre_weight, dtype, index, (C,), "pre_weight")
        qw = pre_weight.data_ptr()
    if n is not None:
        ldn = _need_like(n, dtype, index, shape, "n")[0]
        pn = n.data_ptr()
    elif pre is not None or scale is not None or shift is not None:
        n = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldn, pn = C, n.data_ptr()
    if T == 1:
        ldx = ldy = ldh = ldn = C
    st = _lib.svdq_norm_gate_residual(
        code, x.data_ptr(), ldx, py, ldy, T, C, cu, S, _NORMS[post], pw, kind, pg, ldg,
        residual_scale, _NORMS[pre], qw, ps, lds, pb, ldb, eps, ph, ldh, pn, ldn,
        _raw_stream(index))
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_norm_gate_residual")
    return (x if y is None else h), n


class RopePlan:
    """Frequencies of rope_qk, computed once: axes are the even widths of the
    rotated dimensions of each position axis, sum(axes) <= head_dim; pairs are
    (2p, 2p + 1), or (p, p + sum(axes) / 2) with interleaved False."""

    def __init__(self, axes, theta: float, head_dim: int, interleaved: bool = True):
        self.axes = tuple(int(a) for a in axes)
        self.theta = float(theta)
        self.head_dim = int(head_dim)
        self.interleaved = bool(interleaved)
        if sum(self.axes) > self.head_dim:
            raise ValueError(f"axes {self.axes} exceed the head's {self.head_dim}")
        self._axes = (ctypes.c_int * max(1, len(self.axes)))(*self.axes)
        self._pairs = 1 if self.interleaved else 0
        self._turns = (ctypes.c_double * max(1, sum(max(0, a) for a in self.axes) // 2))()
        _check(_lib.svdq_rope_turns(self._axes, len(self.axes), self.theta, self._turns),
               "svdq_rope_turns")


def rope_qk(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
            plan: RopePlan, q_weight: Optional[torch.Tensor] = None,
            k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
            q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
            stream=None):
    """Rotary positions with several axes on q [T, Hq, D] and k [T, Hk, D]
    (bf16 or fp16, strided views allowed, either may be None), after their
    per-head RMS norm where a weight [D] is given -> (q_out, k_out).

    positions [T, len(plan.axes)] int32.  In place: q_out=q, k_out=k."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("rope_qk needs q or k")
    code = _need_16bit(first, "q" if q is not None else "k", 3)
    index = first.get_device()
    if stream is not None or index != _current_device():
        with _on(index, stream):
            return rope_qk(q, k, positions, plan, q_weight, k_weight, eps, q_out, k_out)
    dtype = first.dtype
    T, _, D = first.shape
    if D != plan.head_dim:
        raise ValueError(f"heads of {D}, the plan is for {plan.head_dim}")
    A = len(plan.axes)
    if (positions.dtype is not torch.int32 or positions.get_device() != index
            or positions.shape != (T, A)):
        raise ValueError(f"positions must be int32 [{T}, {A}] on cuda:{index}")
    ldp, one = positions.stride()
    if one != 1 and A > 1:
        raise ValueError("positions must have unit stride along the axes")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    Hq = Hk = 0
    pq = pk = pqo = pko = wq = wk = None
    qs = ks = qos = kos = (0, 0)
    if q is not None:
        Hq = q.shape[1]
        qs = _need_like(q, dtype, index, (T, Hq, D), "q")
        if q_out is None:
            q_out = q.new_empty((T, Hq, D))
        qos = _need_like(q_out, dtype, index, (T, Hq, D), "q_out")
        pq, pqo = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must have 3 dims")
        Hk = k.shape[1]
        ks = _need_like(k, dtype, index, (T, Hk, D), "k")
        if k_out is None:
            k_out = k.new_empty((T, Hk, D))
        kos = _need_like(k_out, dtype, index, (T, Hk, D), "k_out")
        pk, pko = k.data_ptr(), k_out.data_ptr()
    if q_weight is not None:
        _need_like(q_weight, dtype, index, (D,), "q_weight")
        wq = q_weight.data_ptr()
    if k_weight is not None:
        _need_like(k_weight, dtype, index, (D,), "k_weight")
        wk = k_weight.data_ptr()
    st = _lib.svdq_rope_qk(code, pq, qs[0], qs[1], Hq, pk, ks[0], ks[1], Hk, T, D,
                           positions.data_ptr(), ldp if T > 1 else A, plan._axes, A, plan._turns,
                           plan._pairs, wq, wk, eps, pqo, qos[0], qos[1], pko, kos[0], kos[1],
                           _raw_stream(index))
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_rope_qk")
    return q_out, k_out


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              cu_seqlens: Optional[torch.Tensor] = None, causal: bool = False,
              scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Attention over whole packed sequences -> out [T, Hq, D].

    q [T, Hq, D], k, v [T, Hk, D] bf16 or fp16 (strided views allowed),
    Hq a multiple of Hk; the sequences are the row ranges of cu_seqlens
    [n_seqs + 1] int32 on the device (None: one), each attending within
    itself, only backwards with causal.  scale None: 1 / sqrt(D).  Rows in
    no sequence are left as they are in out."""
    code = _need_16bit(q, "q", 3)
    index = q.get_device()
    if stream is not None or index != _current_device():
        with _on(index, stream):
            return attention(q, k, v, cu_seqlens, causal, scale, out)
    if k.dim() != 3:
        raise ValueError("k must have 3 dims")
    dtype, shape = q.dtype, q.shape
    T, Hq, D = shape
    kv_shape = k.shape
    Hk = kv_shape[1]
    if kv_shape != (T, Hk, D):
        raise ValueError(f"k must have shape {[T, Hk, D]}, got {list(kv_shape)}")
    qs = _need_like(q, dtype, index, shape, "q")
    ks = _need_like(k, dtype, index, kv_shape, "k")
    vs = _need_like(v, dtype, index, kv_shape, "v")
    S, cu = 1, None
    if cu_seqlens is not None:
        S, cu = _need_cu(cu_seqlens, index), cu_seqlens.data_ptr()
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    if out is None:
        out = q.new_empty((T, Hq, D))
        so, sh = Hq * D, D
    else:
        so, sh, _ = _need_like(out, dtype, index, shape, "out")
    pw, size = None, 0
    if T > 2048:                     # no workspace is of use to fewer rows
        size = _lib.svdq_attention_workspace_bytes(T, S, Hq, D, 1 if causal else 0)
        if size:
            ws = torch.empty(size, dtype=torch.uint8, device=q.device)
            pw = ws.data_ptr()
    st = _lib.svdq_attention(code, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
                             v.data_ptr(), vs[0], vs[1], T, Hq, Hk, D, cu, S, 1 if causal else 0,
                             scale, out.data_ptr(), so, sh, pw, size, _raw_stream(index))
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_attention")
    return out


def check_device_error(stream=None) -> None:
    """Synchronize the stream and raise if a kernel recorded an error."""
    _check(_lib.svdq_check_device_error(_stream(stream)), "svdq_check_device_error")


def set_wait_timeout_ns(ns: int) -> None:
    _check(_lib.svdq_set_wait_timeout_ns(ns), "svdq_set_wait_timeout_ns")


def wait_probe(arrive: bool, stream=None) -> None:
    """Enqueue one bounded wait that completes only if ``arrive``; without
    it the wait runs out and the next check_device_error raises."""
    _check(_lib.svdq_wait_probe(1 if arrive else 0, _stream(stream)), "svdq_wait_probe")


class PreparedWeights:
    """One layer's device weights with the scales already repacked and (fold
    True, R > 0) the up-projection folded where every element folds."""

    def __init__(self, qweight, wscales, wcscales, wtscale, smooth, proj_down, proj_up,
                 bias=None, stream=None, fold=True):
        self.qweight = qweight
        self.wscales_tiled = repack_weights(wscales, stream=stream)
        self.proj_up_folded = None
        if fold and proj_up is not None and proj_up.shape[1] > 0:
            folded, bad = fold_proj_up(proj_up, wcscales, wtscale, stream=stream)
            self.proj_up_folded = folded if bad == 0 else None
        self.wcscales = wcscales
        self.wtscale = wtscale
        self.smooth = smooth
        self.proj_down = proj_down
        self.proj_up = proj_up
        self.bias = bias
        self.N = qweight.shape[0]
        self.K = qweight.shape[1] * 2


def svdq_linear(x: torch.Tensor, w: PreparedWeights, y: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Whole layer on device tensors: svdq_quantize_act then svdq_w4a4_linear."""
    qact, asc, lr = quantize_act(x, w.smooth, w.proj_down, stream=stream)
    return w4a4_linear(qact, asc, lr, w.qweight, w.wscales_tiled, w.wcscales, w.wtscale,
                       w.proj_up, w.bias, y=y, stream=stream, proj_up_folded=w.proj_up_folded)


class DitBlock:
    """One transformer block: its five linears (PreparedWeights) and the bf16
    vectors of its norms.

    qkv [C -> 3 heads head_dim] (q, then k, then v, head by head), out, w1, w3,
    w2; attn_pre, attn_post, ffn_pre, ffn_post: RMS norm weights [C] in front
    of and behind the attention and the feed-forward; q_norm, k_norm: per-head
    RMS norm weights [head_dim]."""

    def __init__(self, qkv: PreparedWeights, out: PreparedWeights, w1: PreparedWeights,
                 w3: PreparedWeights, w2: PreparedWeights, *, heads: int, attn_pre, attn_post,
                 ffn_pre, ffn_post, q_norm, k_norm, eps: float = 1e-6):
        C, F = qkv.K, w1.N
        if heads < 1 or qkv.N % (3 * heads) or out.K * 3 != qkv.N:
            raise ValueError(f"qkv makes {qkv.N} and out takes {out.K}: not 3 x {heads} heads")
        if (out.N, w1.K, w3.K, w3.N, w2.K, w2.N) != (C, C, C, F, F, C):
            raise ValueError(f"the linears do not fit a width of {C} and a feed-forward of {F}")
        self.qkv, self.out, self.w1, self.w3, self.w2 = qkv, out, w1, w3, w2
        self.heads, self.head_dim = heads, qkv.N // (3 * heads)
        self.attn_pre, self.attn_post = attn_pre, attn_post
        self.ffn_pre, self.ffn_post = ffn_pre, ffn_post
        self.q_norm, self.k_norm = q_norm, k_norm
        self.eps = eps


def dit_block(x: torch.Tensor, w: DitBlock, modulation, positions: torch.Tensor, plan: RopePlan,
              cu_seqlens: Optional[torch.Tensor] = None, causal: bool = False) -> torch.Tensor:
    """One block on x [T, C] bf16 on its device's current stream -> the new x:

        x = x + tanh(gate_attn) * norm(out(attention(rope(qkv(norm(x) (1 + scale_attn))))))
        x = x + tanh(gate_ffn) * norm(w2(silu(w1 n) * w3 n)),  n = norm(x) (1 + scale_ffn)

    modulation: (scale_attn, gate_attn, scale_ffn, gate_ffn), each [n_seqs, C];
    rows by cu_seqlens (None: one sequence).  Rows in no sequence come back
    undefined and reach no other row.  T >= 1, as for the linears."""
    if x.is_cuda and x.get_device() != _current_device():
        with _on(x.get_device(), None):
            return dit_block(x, w, modulation, positions, plan, cu_seqlens, causal)
    scale_attn, gate_attn, scale_ffn, gate_ffn = modulation
    T, H, D, eps = x.shape[0], w.heads, w.head_dim, w.eps
    _, n = norm_gate_residual(x, scale=scale_attn, pre_weight=w.attn_pre, eps=eps,
                              cu_seqlens=cu_seqlens)
    qkv = svdq_linear(n, w.qkv).view(T, 3 * H, D)
    q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
    rope_qk(q, k, positions, plan, w.q_norm, w.k_norm, eps, q_out=q, k_out=k)
    a = attention(q, k, v, cu_seqlens, causal)
    y = svdq_linear(a.view(T, H * D), w.out)
    x, n = norm_gate_residual(x, y, gate=gate_attn, gate_tanh=True, post="rms",
                              post_weight=w.attn_post, pre_weight=w.ffn_pre, scale=scale_ffn,
                              eps=eps, cu_seqlens=cu_seqlens)
    w2 = w.w2
    qact, asc, lr = silu_mul_quantize_act(svdq_linear(n, w.w1), svdq_linear(n, w.w3), w2.smooth,
                                          w2.proj_down)
    y = w4a4_linear(qact, asc, lr, w2.qweight, w2.wscales_tiled, w2.wcscales, w2.wtscale,
                    w2.proj_up, w2.bias, proj_up_folded=w2.proj_up_folded)
    x, _ = norm_gate_residual(x, y, gate=gate_ffn, gate_tanh=True, post="rms",
                              post_weight=w.ffn_post, pre=None, eps=eps, cu_seqlens=cu_seqlens)
    return x
