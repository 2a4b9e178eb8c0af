"""Python binding of the CUDA library's C ABI (include/fp4attn.h).

Argument marshalling only: every step of the path runs in the library's
kernels.  torch supplies device memory and the current stream.  Importing
this module loads ``libfp4attn.so`` and raises if it is missing, the first
call of a linear layer or norm does the same with their extension -- there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
# FP4ATTN_BOUNDS_CHECK=1 selects the bounds-checked build of the same library
# (build.py --checked): every kernel checks its global stores, atomics and tile
# coordinates and reports FP4ATTN_ERR_RANGE instead of an out-of-range access.
LIB_PATH = os.path.join(_PKG, "libfp4attn_checked.so" if os.environ.get("FP4ATTN_BOUNDS_CHECK") == "1"
                        else "libfp4attn.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_RANGE = 4
ERR_TIMEOUT = 5
ERR_WORKSPACE = 6
NO_SMOOTH_K = 1
NO_HADAMARD = 2
DYNAMIC_GSCALE = 4
LAYER_NORM = 8
BF16, F32 = 0, 1

EXPORTS = (
    "fp4attn_workspace_bytes", "fp4attn_quantize_qk", "fp4attn_quantize_qk_ex", "fp4attn_quantize_qk_noalloc",
    "fp4attn_forward", "fp4attn_forward_ex", "fp4attn_forward_bf16qk", "fp4attn_forward_bf16qk_ex",
    "fp4attn_dequant", "fp4attn_dequant_bf16", "fp4attn_backward", "fp4attn_backward_ex",
    "fp4attn_backward_workspace_bytes",
    "fp4attn_scale_tile_bytes", "fp4attn_linear_workspace_bytes", "fp4attn_quantize_rows", "fp4attn_dequant_rows",
    "fp4attn_gemm", "fp4attn_linear", "fp4attn_linear_backward_workspace_bytes", "fp4attn_linear_backward",
    "fp4attn_norm_gate", "fp4attn_norm_gate_backward_workspace_bytes", "fp4attn_norm_gate_backward",
    "fp4attn_read_status", "fp4attn_reset_status", "fp4attn_status_string", "fp4attn_encode_f32",
    "fp4attn_probe_qk_tile", "fp4attn_probe_pv_tile", "fp4attn_probe_wait_timeout", "fp4attn_probe_div6",
    "fp4attn_probe_withheld_key_sums", "fp4attn_probe_mma_rate",
)


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("D", ctypes.c_int32)]


class Strides(ctypes.Structure):
    """Element strides (b, h, n) of a [B,H,N,128] tensor whose channels are contiguous."""
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class NormVectors(ctypes.Structure):
    _fields_ = [("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("scale_stride", ctypes.c_int64),
                ("shift", ctypes.c_void_p), ("shift_stride", ctypes.c_int64)]


class Fp4AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"CUDA library {LIB_PATH} is missing; build it with "
                          f"`python -m nvfp4_precision_b200.build` (there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, U32, U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
    L.fp4attn_workspace_bytes.restype = ctypes.c_size_t
    L.fp4attn_workspace_bytes.argtypes = [Shape]
    L.fp4attn_quantize_qk.restype = ctypes.c_int
    L.fp4attn_quantize_qk.argtypes = [P, P, Shape, P, P, U32, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.fp4attn_quantize_qk_ex.restype = ctypes.c_int
    L.fp4attn_quantize_qk_ex.argtypes = [P, Strides, P, Strides, Shape, P, P, U32, P, P, P, P, P, P,
                                         ctypes.c_size_t, P]
    L.fp4attn_forward_ex.restype = ctypes.c_int
    L.fp4attn_forward_ex.argtypes = [P, P, P, P, P, P, P, Strides, Shape, ctypes.c_float, P, Strides, P, P,
                                     ctypes.c_size_t, P]
    L.fp4attn_forward_bf16qk_ex.restype = ctypes.c_int
    L.fp4attn_forward_bf16qk_ex.argtypes = [P, Strides, P, Strides, P, Strides, Shape, ctypes.c_float, P, Strides,
                                            P, P, ctypes.c_size_t, P]
    L.fp4attn_quantize_qk_noalloc.restype = ctypes.c_int
    L.fp4attn_quantize_qk_noalloc.argtypes = [P, P, Shape, P, P, U32, P, P, P, P, P, P, P]
    L.fp4attn_forward.restype = ctypes.c_int
    L.fp4attn_forward.argtypes = [P, P, P, P, P, P, P, Shape, ctypes.c_float, P, P, P, ctypes.c_size_t, P]
    L.fp4attn_forward_bf16qk.restype = ctypes.c_int
    L.fp4attn_forward_bf16qk.argtypes = [P, P, P, Shape, ctypes.c_float, P, P, P, ctypes.c_size_t, P]
    L.fp4attn_dequant_bf16.restype = ctypes.c_int
    L.fp4attn_dequant_bf16.argtypes = [P, P, P, Shape, P, P]
    L.fp4attn_backward_workspace_bytes.restype = ctypes.c_size_t
    L.fp4attn_backward_workspace_bytes.argtypes = [Shape]
    L.fp4attn_backward.restype = ctypes.c_int
    L.fp4attn_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, Shape, ctypes.c_float, U32, P, P, P, P,
                                   ctypes.c_size_t, P]
    L.fp4attn_backward_ex.restype = ctypes.c_int
    L.fp4attn_backward_ex.argtypes = [P, P, P, P, P, P, P, P, P, Strides, P, Shape, ctypes.c_float, U32, P, P, P,
                                      P, ctypes.c_size_t, P]
    L.fp4attn_dequant.restype = ctypes.c_int
    L.fp4attn_dequant.argtypes = [P, P, P, Shape, P, P]
    I32, SZ = ctypes.c_int, ctypes.c_size_t
    L.fp4attn_scale_tile_bytes.restype = SZ
    L.fp4attn_scale_tile_bytes.argtypes = [I64, I64]
    L.fp4attn_linear_workspace_bytes.restype = SZ
    L.fp4attn_linear_workspace_bytes.argtypes = [I64, I64, I64]
    L.fp4attn_quantize_rows.restype = I32
    L.fp4attn_quantize_rows.argtypes = [P, I32, I64, I64, I64, P, U32, P, P, P, SZ, P]
    L.fp4attn_dequant_rows.restype = I32
    L.fp4attn_dequant_rows.argtypes = [P, P, P, I64, I64, P, I32, P]
    L.fp4attn_gemm.restype = I32
    L.fp4attn_gemm.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, P, I64, P, SZ, P]
    L.fp4attn_linear.restype = I32
    L.fp4attn_linear.argtypes = [P, I64, P, U32, P, P, P, P, I64, I64, I64, P, I64, P, SZ, P]
    L.fp4attn_linear_backward_workspace_bytes.restype = SZ
    L.fp4attn_linear_backward_workspace_bytes.argtypes = [I64, I64, I64]
    L.fp4attn_linear_backward.restype = I32
    L.fp4attn_linear_backward.argtypes = [P, I64, P, P, P, P, P, P, I64, I64, I64, P, I64, P, P, P, SZ, P]
    VEC = ctypes.POINTER(NormVectors)
    L.fp4attn_norm_gate.restype = I32
    L.fp4attn_norm_gate.argtypes = [P, I32, I64, P, I64, VEC, I64, I64, I64, ctypes.c_float, U32, P, I64, P, I64, P, P,
                                    P, P, SZ, P]
    L.fp4attn_norm_gate_backward_workspace_bytes.restype = SZ
    L.fp4attn_norm_gate_backward_workspace_bytes.argtypes = [I64, I64, I64]
    L.fp4attn_norm_gate_backward.restype = I32
    L.fp4attn_norm_gate_backward.argtypes = [P, I64, P, I64, P, I64, I32, P, I64, VEC, I64, I64, I64, ctypes.c_float,
                                             U32, P, I64, P, I64, P, P, P, P, P, P, SZ, P]
    L.fp4attn_read_status.restype = ctypes.c_int
    L.fp4attn_read_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int)]
    L.fp4attn_reset_status.restype = ctypes.c_int
    L.fp4attn_reset_status.argtypes = [P, P]
    L.fp4attn_status_string.restype = ctypes.c_char_p
    L.fp4attn_status_string.argtypes = [ctypes.c_int]
    L.fp4attn_encode_f32.restype = ctypes.c_int
    L.fp4attn_encode_f32.argtypes = [P, I64, P, P, P]
    L.fp4attn_probe_qk_tile.restype = ctypes.c_int
    L.fp4attn_probe_qk_tile.argtypes = [P, P, P, P, P, P]
    L.fp4attn_probe_pv_tile.restype = ctypes.c_int
    L.fp4attn_probe_pv_tile.argtypes = [P, P, P, P]
    L.fp4attn_probe_div6.restype = ctypes.c_int
    L.fp4attn_probe_mma_rate.restype = ctypes.c_int
    L.fp4attn_probe_mma_rate.argtypes = [ctypes.c_int, ctypes.c_int, P, P, P]
    L.fp4attn_probe_div6.argtypes = [P, P]
    L.fp4attn_probe_wait_timeout.restype = ctypes.c_int
    L.fp4attn_probe_wait_timeout.argtypes = [P, U64, P]
    L.fp4attn_probe_withheld_key_sums.restype = ctypes.c_int
    L.fp4attn_probe_withheld_key_sums.argtypes = [P, P, Shape, P, P, P, P, P, ctypes.c_size_t, U64, P]
    return L


lib = _load()


def status_string(code: int) -> str:
    return lib.fp4attn_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != OK:
        raise Fp4AttnError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def shape_of(t: torch.Tensor) -> Shape:
    B, H, N, D = t.shape
    return Shape(B, H, N, D)


def strides_of(t: torch.Tensor) -> Strides:
    """Strides of a [B,H,N,128] tensor or view (e.g. ``x.transpose(1, 2)`` of a
    [B,N,H,128] tensor); the channels must be contiguous.  The library checks
    the rest (positive multiples of 8)."""
    assert t.dim() == 4 and t.stride(3) == 1, "the channel dimension must be contiguous"
    return Strides(t.stride(0), t.stride(1), t.stride(2))


def fp4attn_workspace_bytes(B: int, H: int, N: int, D: int = 128) -> int:
    return int(lib.fp4attn_workspace_bytes(Shape(B, H, N, D)))


def new_workspace(B: int, H: int, N: int, device="cuda") -> torch.Tensor:
    n = fp4attn_workspace_bytes(B, H, N)
    return torch.empty(n, dtype=torch.uint8, device=device)


def fp4attn_quantize_qk(q: torch.Tensor, k: torch.Tensor, q_gscale: Optional[torch.Tensor] = None,
                        k_gscale: Optional[torch.Tensor] = None, flags: int = 0, out: Optional[dict] = None,
                        k_mean: bool = True, workspace: Optional[torch.Tensor] = None, stream=None,
                        dynamic_gscale: bool = False) -> dict:
    """Smooth K + Hadamard + NVFP4 pack of bf16 [B,H,N,128] Q and K (any
    strides with contiguous channels).  dynamic_gscale=True computes each
    tensor's global scale from its transformed amax into q_gscale / k_gscale
    (allocated when None) instead of reading them.

    Returns dict(q_codes, q_scales, k_codes, k_scales, k_mean, workspace) and,
    with dynamic_gscale, q_gscale and k_gscale (fp32 device scalars to pass to
    fp4attn_forward)."""
    assert q.dtype == torch.bfloat16 and k.dtype == torch.bfloat16 and q.shape == k.shape
    B, H, N, D = q.shape
    dev = q.device
    if out is None:
        out = dict(q_codes=torch.empty((B, H, N, D // 2), dtype=torch.uint8, device=dev),
                   q_scales=torch.empty((B, H, N, D // 16), dtype=torch.uint8, device=dev),
                   k_codes=torch.empty((B, H, N, D // 2), dtype=torch.uint8, device=dev),
                   k_scales=torch.empty((B, H, N, D // 16), dtype=torch.uint8, device=dev),
                   k_mean=torch.empty((B, H, D), dtype=torch.float32, device=dev) if k_mean else None)
    if workspace is None:
        workspace = new_workspace(B, H, N, dev)
    if dynamic_gscale:
        flags = int(flags) | DYNAMIC_GSCALE
        q_gscale = torch.empty(1, dtype=torch.float32, device=dev) if q_gscale is None else q_gscale
        k_gscale = torch.empty(1, dtype=torch.float32, device=dev) if k_gscale is None else k_gscale
    rc = lib.fp4attn_quantize_qk_ex(_ptr(q), strides_of(q), _ptr(k), strides_of(k), Shape(B, H, N, D),
                                    _ptr(q_gscale), _ptr(k_gscale), int(flags), _ptr(out["q_codes"]),
                                    _ptr(out["q_scales"]), _ptr(out["k_codes"]), _ptr(out["k_scales"]),
                                    _ptr(out.get("k_mean")), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "fp4attn_quantize_qk_ex")
    out["workspace"] = workspace
    if dynamic_gscale:
        out["q_gscale"], out["k_gscale"] = q_gscale, k_gscale
    return out


def fp4attn_quantize_qk_noalloc(q: torch.Tensor, k: torch.Tensor, q_gscale: Optional[torch.Tensor] = None,
                                k_gscale: Optional[torch.Tensor] = None, flags: int = 0, out: Optional[dict] = None,
                                k_mean: bool = True, status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """fp4attn_quantize_qk for callers that cannot allocate a workspace: the
    library's fixed scratch array is used instead (B*H <= 1024).  The outputs
    (and the optional int32 ``status`` tensor receiving the device status)
    are the caller's.  Returns dict(q_codes, q_scales, k_codes, k_scales,
    k_mean, status)."""
    assert q.dtype == torch.bfloat16 and k.dtype == torch.bfloat16 and q.shape == k.shape
    assert q.is_contiguous() and k.is_contiguous()
    B, H, N, D = q.shape
    dev = q.device
    if out is None:
        out = dict(q_codes=torch.empty((B, H, N, D // 2), dtype=torch.uint8, device=dev),
                   q_scales=torch.empty((B, H, N, D // 16), dtype=torch.uint8, device=dev),
                   k_codes=torch.empty((B, H, N, D // 2), dtype=torch.uint8, device=dev),
                   k_scales=torch.empty((B, H, N, D // 16), dtype=torch.uint8, device=dev),
                   k_mean=torch.empty((B, H, D), dtype=torch.float32, device=dev) if k_mean else None)
    rc = lib.fp4attn_quantize_qk_noalloc(_ptr(q), _ptr(k), Shape(B, H, N, D), _ptr(q_gscale), _ptr(k_gscale),
                                         int(flags), _ptr(out["q_codes"]), _ptr(out["q_scales"]),
                                         _ptr(out["k_codes"]), _ptr(out["k_scales"]), _ptr(out.get("k_mean")),
                                         _ptr(status), _stream(stream))
    _check(rc, "fp4attn_quantize_qk_noalloc")
    out["status"] = status
    return out


def fp4attn_forward(q_codes, q_scales, k_codes, k_scales, v: torch.Tensor, q_gscale=None, k_gscale=None,
                    softmax_scale: float = 0.0, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    want_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Non-causal attention over NVFP4 Q/K and bf16 V [B,H,N,128] (any strides
    with contiguous channels; so may a caller-supplied O be).  Returns
    (O, lse or None); a new O is contiguous [B,H,N,128]."""
    assert v.dtype == torch.bfloat16
    B, H, N, D = v.shape
    if o is None:
        o = torch.empty((B, H, N, D), dtype=torch.bfloat16, device=v.device)
    assert o.shape == v.shape and o.dtype == torch.bfloat16
    if want_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = new_workspace(B, H, N, v.device)
        workspace.zero_()
    rc = lib.fp4attn_forward_ex(_ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales), _ptr(q_gscale),
                                _ptr(k_gscale), _ptr(v), strides_of(v), Shape(B, H, N, D), float(softmax_scale),
                                _ptr(o), strides_of(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                _stream(stream))
    _check(rc, "fp4attn_forward_ex")
    return o, lse


def fp4attn_forward_bf16qk(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float = 0.0,
                           o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           want_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Non-causal attention with bf16 Q, K, V [B,H,N,128] (no quantisation; any
    strides with contiguous channels): the BF16 counterpart of fp4attn_forward.
    Returns (O, lse or None); a new O is contiguous [B,H,N,128]."""
    for t in (q, k, v):
        assert t.dtype == torch.bfloat16 and t.shape == v.shape
    B, H, N, D = v.shape
    if o is None:
        o = torch.empty((B, H, N, D), dtype=torch.bfloat16, device=v.device)
    assert o.shape == v.shape and o.dtype == torch.bfloat16
    if want_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = new_workspace(B, H, N, v.device)
        workspace.zero_()
    rc = lib.fp4attn_forward_bf16qk_ex(_ptr(q), strides_of(q), _ptr(k), strides_of(k), _ptr(v), strides_of(v),
                                       Shape(B, H, N, D), float(softmax_scale), _ptr(o), strides_of(o), _ptr(lse),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "fp4attn_forward_bf16qk_ex")
    return o, lse


def fp4attn_dequant(codes: torch.Tensor, scales: torch.Tensor, gscale: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    B, H, N, C = codes.shape  # C = D / 2 code bytes per row
    out = torch.empty((B, H, N, 2 * C), dtype=torch.float32, device=codes.device)
    rc = lib.fp4attn_dequant(_ptr(codes), _ptr(scales), _ptr(gscale), Shape(B, H, N, 2 * C), _ptr(out),
                             _stream(stream))
    _check(rc, "fp4attn_dequant")
    return out


def fp4attn_dequant_bf16(codes: torch.Tensor, scales: torch.Tensor, gscale: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """NVFP4 [B,H,N,D/2] codes + [B,H,N,D/16] scales -> bf16 [B,H,N,D] values."""
    B, H, N, C = codes.shape
    out = torch.empty((B, H, N, 2 * C), dtype=torch.bfloat16, device=codes.device)
    rc = lib.fp4attn_dequant_bf16(_ptr(codes), _ptr(scales), _ptr(gscale), Shape(B, H, N, 2 * C), _ptr(out),
                                  _stream(stream))
    _check(rc, "fp4attn_dequant_bf16")
    return out


def fp4attn_backward_workspace_bytes(B: int, H: int, N: int, D: int = 128) -> int:
    return int(lib.fp4attn_backward_workspace_bytes(Shape(B, H, N, D)))


def fp4attn_backward(q_codes, q_scales, k_codes, k_scales, v, o, dout, lse, softmax_scale: float = 0.0,
                     flags: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                     q_gscale: Optional[torch.Tensor] = None, k_gscale: Optional[torch.Tensor] = None):
    """Straight-through backward of the FP4 attention (see include/fp4attn.h):
    the forward's NVFP4 Q and K (codes and scales from fp4attn_quantize_qk)
    and global scales (device scalars, None for 1), V, the forward's O, dL/dO
    (one layout of any strides with contiguous channels, e.g. views of
    [B,N,H,128] tensors) and fp32 lse [B,H,N].  Returns (dq, dk, dv,
    workspace): bf16 gradients of the bf16 Q, K, V inputs of the forward, in
    the layout of V."""
    st = strides_of(v)
    for t in (o, dout):
        assert t.dtype == torch.bfloat16 and t.shape == v.shape and t.stride() == v.stride(), \
            "v, o and dout must share one layout"
    assert v.dtype == torch.bfloat16
    assert lse.dtype == torch.float32 and lse.is_contiguous()
    B, H, N, D = v.shape
    assert q_codes.shape == (B, H, N, 64) and k_codes.shape == (B, H, N, 64)
    if workspace is None:
        workspace = torch.empty(fp4attn_backward_workspace_bytes(B, H, N), dtype=torch.uint8, device=v.device)
    dq, dk, dv = (torch.empty_strided(v.shape, v.stride(), dtype=torch.bfloat16, device=v.device) for _ in range(3))
    rc = lib.fp4attn_backward_ex(_ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales), _ptr(q_gscale),
                                 _ptr(k_gscale), _ptr(v), _ptr(o), _ptr(dout), st, _ptr(lse), Shape(B, H, N, D),
                                 float(softmax_scale), int(flags), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(rc, "fp4attn_backward_ex")
    return dq, dk, dv, workspace


class FP4AttentionSTE(torch.autograd.Function):
    """Training-time FP4 attention: the inference path forward (quantise,
    FP4 attention), straight-through backward (fp4attn_backward).  The device
    status words of both halves are checked on the host."""

    @staticmethod
    def forward(ctx, q, k, v, softmax_scale=0.0, flags=0, dynamic_gscale=False):
        # any layout with contiguous channels is used as it is (no copies);
        # O is allocated in V's layout, which the backward then uses throughout
        q, k, v = (t if t.stride(3) == 1 and t.stride(0) > 0 else t.contiguous() for t in (q, k, v))
        out = fp4attn_quantize_qk(q, k, flags=flags, k_mean=False, dynamic_gscale=dynamic_gscale)
        gq, gk = out.get("q_gscale"), out.get("k_gscale")
        o = torch.empty_strided(v.shape, v.stride(), dtype=torch.bfloat16, device=v.device)
        o, lse = fp4attn_forward(out["q_codes"], out["q_scales"], out["k_codes"], out["k_scales"], v, gq, gk,
                                 softmax_scale=softmax_scale, o=o, want_lse=True, workspace=out["workspace"])
        codes = (out["q_codes"], out["q_scales"], out["k_codes"], out["k_scales"])
        st = fp4attn_read_status(out["workspace"])
        if st != OK:
            raise Fp4AttnError(st, "FP4AttentionSTE.forward (device)")
        ctx.save_for_backward(*codes, v, o, lse, gq, gk)
        ctx.softmax_scale, ctx.flags = softmax_scale, flags
        return o

    @staticmethod
    def backward(ctx, do):
        qc, qs, kc, ks, v, o, lse, gq, gk = ctx.saved_tensors
        do = do.to(torch.bfloat16)
        if do.stride() != v.stride():
            do = torch.empty_strided(v.shape, v.stride(), dtype=torch.bfloat16, device=v.device).copy_(do)
        dq, dk, dv, ws = fp4attn_backward(qc, qs, kc, ks, v, o, do, lse, ctx.softmax_scale, ctx.flags,
                                          q_gscale=gq, k_gscale=gk)
        st = fp4attn_read_status(ws)
        if st != OK:
            raise Fp4AttnError(st, "FP4AttentionSTE.backward (device)")
        return dq, dk, dv, None, None, None


def fp4_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float = 0.0,
                  flags: int = 0, dynamic_gscale: bool = False) -> torch.Tensor:
    """Differentiable FP4 attention of bf16 [B,H,N,128] Q, K, V (fake
    quantisation with a straight-through backward); dynamic_gscale selects the
    amax-derived per-tensor scales."""
    return FP4AttentionSTE.apply(q, k, v, softmax_scale, flags, dynamic_gscale)


# ------------------------------------------------- linear layers in NVFP4 --

# The calls below take a few microseconds on the device for one row.  Their
# checks, outputs and library calls are made in native code (csrc/calls.cpp).
# Errors found on the device (a non-finite input, a bad scale, a wait that ran
# out) are in the status word of the workspace: a caller that wants to see them
# passes one and reads it with fp4attn_read_status.

def _load_calls():
    path = build.calls_path()
    if not os.path.exists(path):
        raise ImportError(f"extension {path} is missing; build it with `python -m nvfp4_precision_b200.build`")
    name = __package__ + "._calls"
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(name, path, loader=loader))
    loader.exec_module(module)
    module.bind(Fp4AttnError, torch.OutOfMemoryError,
                *(ctypes.cast(getattr(lib, "fp4attn_" + n), ctypes.c_void_p).value
                  for n in ("quantize_rows", "dequant_rows", "gemm", "linear", "linear_backward", "norm_gate",
                            "norm_gate_backward")))
    return module


class _Unloaded:
    """Stands for the extension until its first call: the attention does without it."""

    def __getattr__(self, name):
        global _calls
        _calls = _load_calls()
        return getattr(_calls, name)


_calls = _Unloaded()


def _on_stream(stream, fn, *args, **kwargs):
    """fn(*args, **kwargs) with the given stream as the current one, so that
    what it allocates (outputs, a workspace) is ordered there too."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def fp4attn_scale_tile_bytes(rows: int, K: int) -> int:
    return int(lib.fp4attn_scale_tile_bytes(rows, K))


def fp4attn_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.fp4attn_linear_workspace_bytes(M, N, K))


def _status_workspace(nbytes: int, device) -> torch.Tensor:
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def new_linear_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace of fp4attn_quantize_rows, fp4attn_gemm, fp4attn_linear and
    fp4attn_norm_gate with a cleared status word; reusable for any call it is
    large enough for."""
    return _status_workspace(fp4attn_linear_workspace_bytes(M, N, K), device)


def new_linear_backward_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    return _status_workspace(int(lib.fp4attn_linear_backward_workspace_bytes(M, N, K)), device)


def new_norm_backward_workspace(rows: int, C: int, groups: int = 1, device="cuda") -> torch.Tensor:
    return _status_workspace(int(lib.fp4attn_norm_gate_backward_workspace_bytes(rows, C, groups)), device)


def tile_scales(scales: torch.Tensor) -> torch.Tensor:
    """Row-major UE4M3 scales [rows, K/16] in the tile order of the linear
    layers (a change of layout, done once for a weight)."""
    rows, nb = scales.shape
    R, C = -(-rows // 128), -(-nb // 4)
    t = torch.zeros((R * 128, C * 4), dtype=torch.uint8, device=scales.device)
    t[:rows, :nb] = scales
    return t.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def untile_scales(scales: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    """The inverse of tile_scales: [rows, K/16]."""
    R, C = -(-rows // 128), -(-K // 64)
    t = scales.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)
    return t[:rows, :K // 16].contiguous()


def fp4attn_quantize_rows(x: torch.Tensor, gscale: Optional[torch.Tensor] = None, dynamic_gscale: bool = False,
                          codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """NVFP4 rows of a bf16 or fp32 [rows, K] matrix (contiguous rows of any
    stride that is a multiple of 8, or 4 for fp32).  dynamic_gscale=True
    computes the per-tensor scale into gscale (allocated when None) instead of
    reading it.  Returns dict(codes, scales, gscale, workspace)."""
    if stream is not None:
        return _on_stream(stream, fp4attn_quantize_rows, x, gscale, dynamic_gscale, codes, scales, workspace)
    if workspace is None:
        workspace = new_linear_workspace(0, 0, 32, x.device)
    codes, scales, gscale = _calls.quantize_rows(x, gscale, dynamic_gscale, codes, scales, workspace)
    return dict(codes=codes, scales=scales, gscale=gscale, workspace=workspace)


def fp4attn_dequant_rows(codes: torch.Tensor, scales: torch.Tensor, gscale: Optional[torch.Tensor] = None,
                         dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of packed NVFP4 rows, bf16 or fp32 [rows, K]."""
    if stream is not None:
        return _on_stream(stream, fp4attn_dequant_rows, codes, scales, gscale, dtype)
    assert dtype is torch.bfloat16 or dtype is torch.float32, "rows are bf16 or fp32"
    return _calls.dequant_rows(codes, scales, gscale, dtype is torch.float32)


def fp4attn_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                 x_gscale: Optional[torch.Tensor] = None, w_gscale: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = g_x g_w x w^T + bias of packed NVFP4 x [M, K] and w [N, K]: bf16
    [M, N] (y may have any row stride)."""
    if stream is not None:
        return _on_stream(stream, fp4attn_gemm, x_codes, x_scales, w_codes, w_scales, x_gscale, w_gscale, bias, y, workspace)
    if workspace is None:
        workspace = new_linear_workspace(0, 0, 32, x_codes.device)
    return _calls.gemm(x_codes, x_scales, w_codes, w_scales, x_gscale, w_gscale, bias, y, workspace)


def fp4attn_linear(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                   w_gscale: Optional[torch.Tensor] = None, x_gscale: Optional[torch.Tensor] = None,
                   dynamic_gscale: bool = False, bias: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The NVFP4 linear layer of bf16 x [M, K]: quantises x (per-tensor scale
    x_gscale, None for 1, or computed with dynamic_gscale) and multiplies by
    the packed weight [N, K].  bf16 [M, N]."""
    if stream is not None:
        return _on_stream(stream, fp4attn_linear, x, w_codes, w_scales, w_gscale, x_gscale, dynamic_gscale, bias, y, workspace)
    if workspace is None:
        workspace = new_linear_workspace(x.shape[0], w_codes.shape[0], x.shape[1], x.device)
    return _calls.linear(x, w_codes, w_scales, w_gscale, x_gscale, dynamic_gscale, bias, y, workspace)


def fp4attn_linear_backward(dy: torch.Tensor, x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor,
                            w_scales: torch.Tensor, x_gscale: Optional[torch.Tensor] = None,
                            w_gscale: Optional[torch.Tensor] = None, want_dx: bool = True, want_dw: bool = True,
                            want_dbias: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
    """Straight-through gradients of fp4attn_linear for bf16 dy [M, N] and the
    packed operands of the forward: (dx bf16 [M, K], dw bf16 [N, K], dbias
    fp32 [N]), None in the place of one not wanted."""
    if stream is not None:
        return _on_stream(stream, fp4attn_linear_backward, dy, x_codes, x_scales, w_codes, w_scales, x_gscale, w_gscale, want_dx, want_dw,
                          want_dbias, workspace)
    if workspace is None:
        workspace = new_linear_backward_workspace(*dy.shape, 2 * x_codes.shape[1], dy.device)
    return _calls.linear_backward(dy, x_codes, x_scales, w_codes, w_scales, x_gscale, w_gscale, want_dx, want_dw, want_dbias,
                                  workspace)


# -------------------------------------------- the norms around a branch --

def fp4attn_norm_gate(x: torch.Tensor, h: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      flags: int = 0, groups: Optional[int] = None, want_y: bool = True, want_z: bool = True,
                      quantize: bool = False, z_gscale: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                      z: Optional[torch.Tensor] = None) -> dict:
    """y = x + gate * (post_weight * norm(h)) and z = norm(y) * pre_weight *
    (1 + scale) + shift, on bf16 or fp32 rows x [rows, C] and bf16 h (None for
    y = x).  RMS norms, or layer norms with flags=LAYER_NORM.  gate, scale and
    shift are bf16 [groups, C], one row for each of `groups` equal samples.
    quantize=True returns z as NVFP4 rows under the static scale z_gscale
    (None for 1), ready for fp4attn_gemm.  y may be given (x itself for an
    update in place), and z where it is not quantised.  Returns dict(y, z) or
    dict(y, z_codes, z_scales, workspace)."""
    if stream is not None:
        return _on_stream(stream, fp4attn_norm_gate, x, h, post_weight, gate, pre_weight, scale, shift, eps, flags, groups, want_y,
                          want_z, quantize, z_gscale, y, workspace, z=z)
    if not quantize:
        y, z = _calls.norm_gate(x, h, post_weight, gate, pre_weight, scale, shift, eps, flags, groups, want_y, want_z, False,
                                None, y, z, workspace)
        return {"y": y, "z": z}
    if workspace is None:
        workspace = new_linear_workspace(0, 0, 32, x.device)
    y, codes, scales = _calls.norm_gate(x, h, post_weight, gate, pre_weight, scale, shift, eps, flags, groups, want_y, False,
                                        True, z_gscale, y, z, workspace)
    return dict(y=y, z_codes=codes, z_scales=scales, workspace=workspace)


def fp4attn_norm_gate_backward(dz: torch.Tensor, dy: Optional[torch.Tensor], y: torch.Tensor,
                               h: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                               gate: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
                               scale: Optional[torch.Tensor] = None, eps: float = 1e-6, flags: int = 0,
                               groups: Optional[int] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of fp4attn_norm_gate for bf16 dz and dy (y's type, None for 0)
    from the forward's y and h: dict(dx, dh, dshift, dscale, dgate,
    dpre_weight, dpost_weight); dh, dgate and dpost_weight are None without h.
    Those of the vectors are fp32."""
    if stream is not None:
        return _on_stream(stream, fp4attn_norm_gate_backward, dz, dy, y, h, post_weight, gate, pre_weight, scale, eps, flags, groups,
                          workspace)
    if workspace is None:
        samples = next((t.shape[0] for t in (gate, scale) if t is not None and t.dim() == 2), 1)
        workspace = new_norm_backward_workspace(*y.shape, samples if groups is None else groups, device=y.device)
    dx, dh, dshift, dscale, dgate, dpre, dpost = _calls.norm_gate_backward(dz, dy, y, h, post_weight, gate, pre_weight, scale,
                                                                           eps, flags, groups, workspace)
    return {"dx": dx, "dh": dh, "dshift": dshift, "dscale": dscale, "dgate": dgate, "dpre_weight": dpre,
            "dpost_weight": dpost}


# ------------------------------------------------------ differentiable --

def _refuse_capture(name: str):
    """The differentiable forms read the device status on the host, which a
    graph capture cannot; the fp4attn_* calls under them can be captured."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name} cannot be captured into a CUDA graph (it reads the device status on the host); "
                           "capture the fp4attn_* calls instead")


def _raise_status(workspace: torch.Tensor, where: str):
    st = fp4attn_read_status(workspace)
    if st != OK:
        raise Fp4AttnError(st, where + " (device)")


def _aligned_rows(t: torch.Tensor, unit: int = 8) -> torch.Tensor:
    """t [rows, cols] itself, or a copy, with contiguous rows that start on 16 bytes."""
    if (t.shape[1] <= 1 or t.stride(1) == 1) and t.data_ptr() % 16 == 0 and \
            (t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % unit == 0)):
        return t
    rows, cols = t.shape
    out = t.new_empty((rows, -(-cols // unit) * unit))[:, :cols]
    return out.copy_(t)


def _aligned_vector(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t [n] itself, or a copy, contiguous and starting on 16 bytes (a slice of a fused bias may not)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class FP4LinearSTE(torch.autograd.Function):
    """Training-time NVFP4 linear layer: input and weight quantised under their
    computed scales, straight-through backward."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        _refuse_capture("FP4LinearSTE")
        K = weight.shape[1]
        rows = _aligned_rows(x.reshape(-1, K))
        w = _aligned_rows(weight, 4 if weight.dtype is torch.float32 else 8)
        ws = new_linear_workspace(0, 0, 32, x.device)
        # what is returned is no view, so that operations in place are allowed on it
        y = x.new_empty((*x.shape[:-1], weight.shape[0]))
        qx = fp4attn_quantize_rows(rows, dynamic_gscale=True, workspace=ws)
        qw = fp4attn_quantize_rows(w, dynamic_gscale=True, workspace=ws)
        fp4attn_gemm(qx["codes"], qx["scales"], qw["codes"], qw["scales"], qx["gscale"], qw["gscale"],
                     _aligned_vector(None if bias is None else bias.to(torch.bfloat16)), y=y.view(rows.shape[0], weight.shape[0]),
                     workspace=ws)
        _raise_status(ws, "FP4LinearSTE.forward")
        ctx.save_for_backward(qx["codes"], qx["scales"], qx["gscale"], qw["codes"], qw["scales"], qw["gscale"])
        ctx.x_shape, ctx.w_dtype, ctx.b_dtype = x.shape, weight.dtype, None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _refuse_capture("FP4LinearSTE")
        xc, xs, gx, wc, wsc, gw = ctx.saved_tensors
        rows = _aligned_rows(dy.to(torch.bfloat16).reshape(xc.shape[0], wc.shape[0]))
        ws = new_linear_backward_workspace(xc.shape[0], wc.shape[0], 2 * wc.shape[1], dy.device)
        dx, dw, db = fp4attn_linear_backward(rows, xc, xs, wc, wsc, gx, gw, want_dx=ctx.needs_input_grad[0],
                                             want_dw=ctx.needs_input_grad[1], want_dbias=ctx.needs_input_grad[2],
                                             workspace=ws)
        _raise_status(ws, "FP4LinearSTE.backward")
        return (None if dx is None else dx.view(ctx.x_shape), None if dw is None else dw.to(ctx.w_dtype),
                None if db is None else db.to(ctx.b_dtype))


def fp4_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable NVFP4 linear layer of bf16 x [..., K] with a bf16 or fp32
    weight [N, K] (fake quantisation of both under their computed scales, a
    straight-through backward); K a multiple of 32.  The weight's gradient is
    rounded to bf16, then widened for an fp32 weight; a bias is rounded to bf16.
    Forward and backward read the device status on the host and so wait for the
    GPU.  The training-time counterpart of fp4attn_linear, next to
    fp4_attention."""
    assert x.dtype is torch.bfloat16 and weight.dim() == 2 and x.shape[-1] == weight.shape[1], "x [..., K], weight [N, K]"
    return FP4LinearSTE.apply(x, weight, bias)


class NormGate(torch.autograd.Function):
    """fp4attn_norm_gate with fp4attn_norm_gate_backward as its gradient."""

    @staticmethod
    def forward(ctx, x, h, post_weight, gate, pre_weight, scale, shift, eps, flags, groups):
        _refuse_capture("NormGate")
        ctx.set_materialize_grads(False)
        C = x.shape[-1]
        unit = 4 if x.dtype is torch.float32 else 8
        xr = _aligned_rows(x.reshape(-1, C), unit)
        hr = None if h is None else _aligned_rows(h.reshape(-1, C))
        vec = [None if t is None else _aligned_rows(t.reshape(-1, C)) for t in (gate, scale, shift)]
        one = [_aligned_vector(t) for t in (post_weight, pre_weight)]
        ws = new_linear_workspace(0, 0, 32, x.device)
        # what is returned is no view, so that operations in place are allowed on it
        y, z = x.new_empty(x.shape), x.new_empty(x.shape, dtype=torch.bfloat16)
        fp4attn_norm_gate(xr, hr, one[0], vec[0], one[1], vec[1], vec[2], eps=eps, flags=flags, groups=groups,
                          y=y.view(xr.shape), z=z.view(xr.shape), workspace=ws)
        _raise_status(ws, "NormGate.forward")
        ctx.save_for_backward(y, hr, one[0], vec[0], one[1], vec[1])
        ctx.args = (eps, flags, groups if groups is not None else next((t.shape[0] for t in vec if t is not None), 1))
        ctx.like = tuple(None if t is None else (t.shape, t.dtype) for t in (x, h, post_weight, gate, pre_weight, scale, shift))
        return y, z

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dz):
        _refuse_capture("NormGate")
        y, h, post_weight, gate, pre_weight, scale = ctx.saved_tensors
        y = y.view(-1, y.shape[-1])
        eps, flags, groups = ctx.args
        dzr = torch.zeros(y.shape, dtype=torch.bfloat16, device=y.device) if dz is None else \
            _aligned_rows(dz.to(torch.bfloat16).reshape(y.shape))
        dyr = None if dy is None else _aligned_rows(dy.to(y.dtype).reshape(y.shape), 4 if y.dtype is torch.float32 else 8)
        ws = new_norm_backward_workspace(*y.shape, groups, device=y.device)
        g = fp4attn_norm_gate_backward(dzr, dyr, y, h, post_weight, gate, pre_weight, scale, eps=eps, flags=flags,
                                       groups=groups, workspace=ws)
        _raise_status(ws, "NormGate.backward")
        names = ("dx", "dh", "dpost_weight", "dgate", "dpre_weight", "dscale", "dshift")
        grads = [None if like is None else g[k].to(like[1]).reshape(like[0]) for k, like in zip(names, ctx.like)]
        # without a branch the gate and the branch's weight have no part in the result
        return (*grads, None, None, None)


def norm_gate(x: torch.Tensor, h: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
              scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None, eps: float = 1e-6,
              layer_norm: bool = False, groups: Optional[int] = None):
    """Differentiable (y, z) of fp4attn_norm_gate for x [..., C] and h of x's
    shape; the rows are `groups` equal samples one after the other (as many as
    gate, scale and shift [groups, C] have).  The backward reads y, so that y is
    not to be changed in place before it (autograd reports that).  Forward and
    backward read the device status on the host and so wait for the GPU."""
    assert h is not None or (gate is None and post_weight is None), "gate and post_weight belong to a branch h"
    return NormGate.apply(x, h, post_weight, gate, pre_weight, scale, shift, eps, LAYER_NORM if layer_norm else 0, groups)


def fp4attn_read_status(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int(-1)
    _check(lib.fp4attn_read_status(_ptr(workspace), _stream(stream), ctypes.byref(v)), "fp4attn_read_status")
    return v.value


def fp4attn_reset_status(workspace: torch.Tensor, stream=None):
    _check(lib.fp4attn_reset_status(_ptr(workspace), _stream(stream)), "fp4attn_reset_status")


def fp4attn_encode_f32(x: torch.Tensor, stream=None):
    assert x.dtype == torch.float32 and x.is_contiguous()
    e2m1 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    e4m3 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib.fp4attn_encode_f32(_ptr(x), x.numel(), _ptr(e2m1), _ptr(e4m3), _stream(stream)), "fp4attn_encode_f32")
    return e2m1, e4m3


def fp4attn_probe_qk_tile(q_codes, q_scales, k_codes, k_scales, stream=None) -> torch.Tensor:
    s = torch.empty((128, 128), dtype=torch.float32, device=q_codes.device)
    _check(lib.fp4attn_probe_qk_tile(_ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales), _ptr(s),
                                     _stream(stream)), "fp4attn_probe_qk_tile")
    return s


def fp4attn_probe_pv_tile(p: torch.Tensor, v: torch.Tensor, stream=None) -> torch.Tensor:
    o = torch.empty((128, 128), dtype=torch.float32, device=p.device)
    _check(lib.fp4attn_probe_pv_tile(_ptr(p), _ptr(v), _ptr(o), _stream(stream)), "fp4attn_probe_pv_tile")
    return o


def fp4attn_probe_div6(stream=None):
    """(number of mismatches, smallest mismatching bit pattern) of the device
    amax / 6 against the IEEE quotient over every non-negative finite fp32."""
    res = torch.zeros(2, dtype=torch.int32, device="cuda")
    _check(lib.fp4attn_probe_div6(_ptr(res), _stream(stream)), "fp4attn_probe_div6")
    r = res.cpu().numpy().view("uint32")
    return int(r[0]), int(r[1])


MMA_RATE_FLOPS_PER_GROUP = {0: 2 * 2 * 128 * 256 * 64, 1: 8 * 2 * 128 * 256 * 16}


def fp4attn_probe_mma_rate(mode: int, reps: int = 40000, stream=None) -> dict:
    """Back-to-back tcgen05 MMA throughput on every SM (mode 0: block-scaled
    FP4 M128 N256 K64; mode 1: BF16 M128 N256 K16), timed by CUDA events on
    the stream, with the SM clock CTA 0 saw: dict(ms, tflops, flop_per_clk_sm,
    sm_mhz)."""
    cycles = torch.zeros(1, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = stream if stream is not None else torch.cuda.current_stream()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record(st)
    _check(lib.fp4attn_probe_mma_rate(mode, reps, _ptr(cycles), _ptr(status), _stream(st)), "fp4attn_probe_mma_rate")
    e1.record(st)
    e1.synchronize()
    ms = e0.elapsed_time(e1)
    cyc = int(cycles.item())
    if int(status.item()) != 0 or cyc <= 0:
        raise RuntimeError(f"fp4attn_probe_mma_rate: status {int(status.item())}, cycles {cyc}")
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    flops = MMA_RATE_FLOPS_PER_GROUP[mode] * reps
    return {"ms": ms, "tflops": flops * sms / (ms * 1e-3) / 1e12, "flop_per_clk_sm": flops / cyc,
            "sm_mhz": cyc / (ms * 1e3)}


def fp4attn_probe_wait_timeout(limit_ns: int, stream=None) -> int:
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(lib.fp4attn_probe_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)), "fp4attn_probe_wait_timeout")
    return int(status.item())


def fp4attn_probe_withheld_key_sums(q: torch.Tensor, k: torch.Tensor, limit_ns: int, stream=None) -> int:
    """The prologue with its key-sum tiles withheld: returns the device status
    after the run (FP4ATTN_ERR_TIMEOUT when the K tiles' bounded wait gave up)."""
    assert q.dtype == torch.bfloat16 and k.dtype == torch.bfloat16 and q.shape == k.shape
    assert q.is_contiguous() and k.is_contiguous()
    B, H, N, D = q.shape
    dev = q.device
    qc = torch.empty((B, H, N, 64), dtype=torch.uint8, device=dev)
    qs = torch.empty((B, H, N, 8), dtype=torch.uint8, device=dev)
    kc = torch.empty_like(qc)
    ks = torch.empty_like(qs)
    ws = new_workspace(B, H, N)
    _check(lib.fp4attn_probe_withheld_key_sums(_ptr(q), _ptr(k), Shape(B, H, N, D), _ptr(qc), _ptr(qs), _ptr(kc),
                                               _ptr(ks), _ptr(ws), ws.numel(), int(limit_ns), _stream(stream)),
           "fp4attn_probe_withheld_key_sums")
    return fp4attn_read_status(ws)
