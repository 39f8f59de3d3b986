"""MI355X-native W4A8 linear / MoE-expert library: thin Python binding of libw4a8.so.

Every function here only marshals arguments to the C ABI declared in include/w4a8.h (same
names); all arithmetic runs in the library (host pack) or its gfx950 kernels.  PyTorch is
used for device memory and streams only.  There is no CPU fallback: if the library is not
built, or the GPU path is asked for without a GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw4a8.so")

W4A8_OK, W4A8_EINVAL, W4A8_ESIZE, W4A8_EUNSUPPORTED, W4A8_EHIP = 0, -1, -2, -3, -4
W4A8_OUT_BF16, W4A8_OUT_F32 = 0, 1
W4A8_BF16, W4A8_F32, W4A8_F16 = 0, 1, 2
W4A8_ROUTE_SOFTMAX, W4A8_ROUTE_SIGMOID = 0, 1
W4A8_MX_FP4, W4A8_MX_FP8, W4A8_QUANT_INT8 = 0, 1, 2
HEADER_BYTES = 256

EXPORTED = [
    "w4a8_packed_size", "w4a8_pack", "w4a8_pack_codes", "w4a8_unpack_codes", "w4a8_blob_check",
    "w4a8_quant_act", "w4a8_quant_act_smooth", "w4a8_gemm", "w4a8_linear", "w4a8_gemm_partials", "w4a8_moe_align",
    "w4a8_moe_gemm",
    "w4a8_moe_gemm_silu_static",
    "w4a8_silu_mul_quant", "w4a8_moe_combine", "w4a8_moe_workspace_size", "w4a8_moe_forward",
    "w4a8_quant_act_static", "w4a8_moe_quant_static", "w4a8_silu_mul_quant_static",
    "w4a8_moe_static_workspace_size", "w4a8_moe_forward_static", "w4a8_moe_forward_sets", "w4a8_moe_forward_noalloc",
    "w4a16_gemm", "w4a16_kernel_name",
    "w4a8_moe_route", "w4a8_moe_gemm_w8a8", "w4a8_moe_gemm_w16a16", "w4a8_moe_gemm_silu_w16a16",
    "w4a8_moe_forward_w8a8", "w4a8_moe_w16a16_workspace_size", "w4a8_moe_forward_w16a16",
    "w4a8_mx_quant", "w4a8_mx_dequant", "w4a8_mx_packed_size", "w4a8_mx_pack", "w4a8_mx_pack_codes", "w4a8_mx_unpack_codes",
    "w4a8_mx_gemm", "w4a8_moe_gemm_mx", "w4a8_moe_gemm_silu_mx", "w4a8_moe_gemm_silu_mx_quant",
    "w4a8_moe_mx_workspace_size", "w4a8_moe_forward_mx", "w4a8_norm_residual", "w4a8_norm_residual_quant",
    "w4a8_kernel_name", "w4a8_status_string", "w4a8_version",
]


class W4A8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class WDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("asymmetric", ctypes.c_int32), ("weight_bits", ctypes.c_int32), ("scale_bits", ctypes.c_int32)]

    def __repr__(self):
        return (f"WDesc(K={self.K}, N={self.N}, group_size={self.group_size}, asymmetric={self.asymmetric}, "
                f"weight_bits={self.weight_bits}, scale_bits={self.scale_bits})")


class ExpertSet(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("gu_blobs", ctypes.c_void_p), ("gu_stride", ctypes.c_size_t),
                ("gu_desc", ctypes.POINTER(WDesc)), ("d_blobs", ctypes.c_void_p), ("d_stride", ctypes.c_size_t),
                ("d_desc", ctypes.POINTER(WDesc))]


class RouteDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32), ("scale", ctypes.c_float)]


class NormDesc(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("eps_post", ctypes.c_float), ("alpha", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libw4a8.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m moe_token_int8_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, SZ, VP = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        DP = ctypes.POINTER(WDesc)
        sig = {
            "w4a8_packed_size": (SZ, [DP]),
            "w4a8_pack": (I, [DP, P, P, SZ]),
            "w4a8_pack_codes": (I, [DP, P, P, P, P, SZ]),
            "w4a8_unpack_codes": (I, [P, SZ, DP, P, P, P]),
            "w4a8_blob_check": (I, [P, SZ, DP]),
            "w4a8_quant_act": (I, [P, I, I, I, P, P, VP]),
            "w4a8_quant_act_smooth": (I, [P, I, I, I, P, P, P, VP]),
            "w4a8_gemm": (I, [P, P, I, P, DP, P, I, I, VP]),
            "w4a8_linear": (I, [P, I, I, I, P, DP, P, I, I, P, P, VP]),
            "w4a8_gemm_partials": (I, [P, I, P, DP, P, VP]),
            "w4a8_moe_align": (I, [P, I, I, I, P, P, P, VP]),
            "w4a8_moe_gemm": (I, [P, P, P, I, P, I, I, I, P, SZ, DP, P, I, VP]),
            "w4a8_moe_gemm_silu_static": (I, [P, P, P, I, P, I, I, I, P, SZ, DP, P, P, P, VP]),
            "w4a8_silu_mul_quant": (I, [P, I, I, P, P, VP]),
            "w4a8_moe_combine": (I, [P, P, P, I, I, I, P, VP]),
            "w4a8_moe_workspace_size": (SZ, [I, I, I, I, I]),
            "w4a8_moe_forward": (I, [P, P, P, I, I, I, P, SZ, DP, P, SZ, DP, P, SZ, P, VP]),
            "w4a8_quant_act_static": (I, [P, I, I, I, P, P, P, VP]),
            "w4a8_moe_quant_static": (I, [P, I, I, I, P, I, P, I, P, P, P, VP]),
            "w4a8_silu_mul_quant_static": (I, [P, I, I, P, I, P, P, P, VP]),
            "w4a8_moe_static_workspace_size": (SZ, [I, I, I, I, I]),
            "w4a8_moe_forward_static": (I, [P, P, P, I, I, I, P, SZ, DP, P, SZ, DP, P, P, P, SZ, P, VP]),
            "w4a8_moe_forward_sets": (I, [P, P, P, I, I, ctypes.POINTER(ExpertSet), I, P, SZ, P, VP]),
            "w4a8_moe_forward_noalloc": (I, [P, P, P, I, I, I, P, SZ, DP, P, SZ, DP, P, VP]),
            "w4a8_moe_route": (I, [P, I, I, I, P, ctypes.POINTER(RouteDesc), P, P, VP]),
            "w4a8_moe_gemm_w8a8": (I, [P, P, P, I, P, I, I, I, P, SZ, DP, P, I, VP]),
            "w4a8_moe_gemm_w16a16": (I, [P, I, I, P, I, P, I, I, I, P, SZ, I, I, I, P, I, I, VP]),
            "w4a8_moe_gemm_silu_w16a16": (I, [P, I, I, P, I, P, I, I, I, P, SZ, I, I, I, P, I, VP]),
            "w4a8_moe_forward_w8a8": (I, [P, P, P, I, I, I, P, SZ, DP, P, SZ, DP, P, SZ, P, VP]),
            "w4a8_moe_w16a16_workspace_size": (SZ, [I, I, I, I, I]),
            "w4a8_moe_forward_w16a16": (I, [P, P, P, I, I, I, P, SZ, P, SZ, I, I, P, SZ, P, VP]),
            "w4a8_mx_quant": (I, [P, I, I, I, I, I, P, P, VP]),
            "w4a8_mx_dequant": (I, [P, P, I, I, I, P, I, I, VP]),
            "w4a8_mx_packed_size": (SZ, [I, I]),
            "w4a8_mx_pack": (I, [P, I, I, I, I, I, SZ, P, SZ, VP]),
            "w4a8_mx_pack_codes": (I, [P, P, I, I, I, I, P, VP]),
            "w4a8_mx_unpack_codes": (I, [P, I, I, P, P, VP]),
            "w4a8_mx_gemm": (I, [P, P, I, I, P, I, I, P, I, I, VP]),
            "w4a8_moe_gemm_mx": (I, [P, P, I, P, I, P, I, I, I, P, SZ, I, I, P, I, I, VP]),
            "w4a8_moe_gemm_silu_mx": (I, [P, P, I, P, I, P, I, I, I, P, SZ, I, I, P, I, I, VP]),
            "w4a8_moe_gemm_silu_mx_quant": (I, [P, P, I, P, I, P, I, I, I, P, SZ, I, I, I, P, P, VP]),
            "w4a8_moe_mx_workspace_size": (SZ, [I, I, I, I, I, I]),
            "w4a8_moe_forward_mx": (I, [P, P, P, I, I, I, I, P, SZ, P, SZ, I, I, P, SZ, P, VP]),
            "w4a8_norm_residual": (I, [P, I, I, P, I, I, P, I, P, P, ctypes.POINTER(NormDesc), I, I, P, I, P, I, VP]),
            "w4a8_norm_residual_quant": (I, [P, I, I, P, I, I, P, I, P, P, ctypes.POINTER(NormDesc), I, I, P, I, I, P, P, VP]),
            "w4a8_kernel_name": (ctypes.c_char_p, [DP, I]),
            "w4a16_gemm": (I, [P, I, I, P, DP, P, I, I, VP]),
            "w4a16_kernel_name": (ctypes.c_char_p, [DP, I]),
            "w4a8_status_string": (ctypes.c_char_p, [I]),
            "w4a8_version": (I, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().w4a8_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != W4A8_OK:
        raise W4A8Error(status, where)


def desc(K: int, N: int, group_size: int, asymmetric: bool, bits: int = 4, scale_bits: int = 32) -> WDesc:
    """Weight descriptor; bits = 8 selects the symmetric INT8-weight (W8A8) form, scale_bits = 16
    binary16 group scales."""
    return WDesc(int(K), int(N), int(group_size), int(bool(asymmetric)), int(bits), int(scale_bits))


def route_desc(E: int, k: int, score: int = W4A8_ROUTE_SOFTMAX, renormalize: bool = False, scale: float = 1.0,
               n_group: int = 1, topk_group: int = 1) -> RouteDesc:
    """How a router chooses: see w4a8_route_desc."""
    return RouteDesc(int(E), int(k), int(score), int(bool(renormalize)), int(n_group), int(topk_group), float(scale))


def norm_desc(eps: float = 1e-6, eps_post: float = 1e-6, alpha: float = 1.0) -> NormDesc:
    """Constants of the norm around a block: see w4a8_norm_desc."""
    return NormDesc(float(eps), float(eps_post), float(alpha))


def _dtype(t) -> int:
    """w4a8_dtype of a tensor."""
    try:
        return _torch().types[t.dtype]
    except KeyError:
        raise ValueError(f"{t.dtype} is not an element type of this call") from None


def _require_current(tensors, int32=(), float32=(), int8=()):
    """Device tensors, those of the keywords of that type, on the current device, whose stream the call uses."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -1
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("GPU entry points take device tensors")
        if t.get_device() != dev:
            raise ValueError("the tensors are not on the current device")
    for want, typed in ((torch.int32, int32), (torch.float32, float32), (torch.int8, int8)):
        for t in typed:
            if t is None:
                continue
            if t.dtype is not want:
                raise ValueError(f"expected {want}, got {t.dtype}")
            if t.get_device() != dev or dev < 0:
                raise ValueError("GPU entry points take device tensors, on the current device")


class _Torch:
    """What the calls below need of torch, looked up once: their host time is most of a small call's."""

    def __init__(self):
        import torch
        self.int32, self.int8, self.float32 = torch.int32, torch.int8, torch.float32
        self.uint8, self.bfloat16 = torch.uint8, torch.bfloat16
        self.initialized, self.device = torch.cuda.is_initialized, torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.types = {torch.bfloat16: W4A8_BF16, torch.float32: W4A8_F32, torch.float16: W4A8_F16}

    def current(self) -> int:
        return self.device() if self.initialized() else -2      # a CPU tensor's device is -1


_torch_of_calls = None


def _torch() -> _Torch:
    global _torch_of_calls
    if _torch_of_calls is None:
        _torch_of_calls = _Torch()
    return _torch_of_calls


_INT_MAX = 0x7fffffff


def _check_int32(*sizes) -> None:
    """The library's int arguments: ctypes would hand on the low 32 bits of anything larger.  (Calls of a few us test the OR of
    their sizes, none negative, before they call this: 0.1 us in place of 0.4.)"""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX:
        raise ValueError("a size or a stride does not fit in 32 bits")


def _ptr(x) -> int | None:
    """Data pointer of a torch tensor or numpy array (None passes NULL)."""
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return int(stream)
    import torch
    # the handle of torch.cuda.current_stream(), without the object around it (2.8 us of a 10 us call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _require_cuda(*tensors):
    for t in tensors:
        if t is not None and not (hasattr(t, "is_cuda") and t.is_cuda):
            raise ValueError("GPU entry points take device tensors")


# ------------------------------------------------------------------------------ host side
def w4a8_packed_size(d: WDesc) -> int:
    return int(lib().w4a8_packed_size(ctypes.byref(d)))


def w4a8_pack(d: WDesc, W: np.ndarray) -> np.ndarray:
    """RTN-quantize and pack float32 W[K, N] on the host; returns the blob (uint8)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    if W.shape != (d.K, d.N):
        raise ValueError(f"W shape {W.shape} does not match {d}")
    n = w4a8_packed_size(d)
    if n == 0:
        raise W4A8Error(W4A8_EINVAL, "w4a8_packed_size")
    blob = np.empty(n, dtype=np.uint8)
    _check(lib().w4a8_pack(ctypes.byref(d), _ptr(W), _ptr(blob), n), "w4a8_pack")
    return blob


def w4a8_pack_codes(d: WDesc, codes: np.ndarray, scales: np.ndarray, zeros: np.ndarray | None) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.int8)
    scales = np.ascontiguousarray(scales, dtype=np.float32)
    if zeros is not None:
        zeros = np.ascontiguousarray(zeros, dtype=np.uint8)
    n = w4a8_packed_size(d)
    if n == 0:
        raise W4A8Error(W4A8_EINVAL, "w4a8_packed_size")
    blob = np.empty(n, dtype=np.uint8)
    _check(lib().w4a8_pack_codes(ctypes.byref(d), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(blob), n),
           "w4a8_pack_codes")
    return blob


def w4a8_unpack_codes(blob: np.ndarray):
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    d = WDesc()
    st = lib().w4a8_unpack_codes(_ptr(blob), blob.nbytes, ctypes.byref(d), None, None, None)
    _check(st, "w4a8_unpack_codes")
    G = d.K // d.group_size
    codes = np.empty((d.K, d.N), np.int8)
    scales = np.empty((G, d.N), np.float32)
    zeros = np.empty((G, d.N), np.uint8) if d.asymmetric else None
    _check(lib().w4a8_unpack_codes(_ptr(blob), blob.nbytes, ctypes.byref(d), _ptr(codes), _ptr(scales),
                                   _ptr(zeros)), "w4a8_unpack_codes")
    return d, codes, scales, zeros


def w4a8_blob_check(blob: np.ndarray, d: WDesc) -> None:
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    _check(lib().w4a8_blob_check(_ptr(blob), blob.nbytes, ctypes.byref(d)), "w4a8_blob_check")


def w4a8_kernel_name(d: WDesc, M: int) -> str:
    return lib().w4a8_kernel_name(ctypes.byref(d), int(M)).decode()


def w4a8_moe_workspace_size(T: int, k: int, H: int, I: int, E: int) -> int:
    return int(lib().w4a8_moe_workspace_size(T, k, H, I, E))


def w4a8_moe_static_workspace_size(T: int, k: int, H: int, I: int, E: int) -> int:
    return int(lib().w4a8_moe_static_workspace_size(T, k, H, I, E))


def w4a8_version() -> int:
    return int(lib().w4a8_version())


# ------------------------------------------------------------------------------ GPU side
def w4a8_quant_act(X, Xq, sx, stream=None) -> None:
    """X: bf16 [M, K] (row stride X.stride(0)); Xq: int8 [M, K]; sx: float32 [M]."""
    _require_cuda(X, Xq, sx)
    M, K = X.shape
    _check(lib().w4a8_quant_act(_ptr(X), M, K, X.stride(0), _ptr(Xq), _ptr(sx), _stream(stream)),
           "w4a8_quant_act")


def w4a8_quant_act_smooth(X, inv_alpha, Xq, sx, stream=None) -> None:
    """w4a8_quant_act of X diag(alpha)^-1; inv_alpha: float32 [K] on the device."""
    _require_cuda(X, inv_alpha, Xq, sx)
    M, K = X.shape
    _check(lib().w4a8_quant_act_smooth(_ptr(X), M, K, X.stride(0), _ptr(inv_alpha), _ptr(Xq), _ptr(sx),
                                       _stream(stream)), "w4a8_quant_act_smooth")


def w4a8_quant_act_static(X, s, Xq, sx, stream=None) -> None:
    """Quantize every row of X (bf16 [M, K]) with the one calibrated scale s (float32 [1] on
    the device); sx[m] receives s."""
    _require_cuda(X, s, Xq, sx)
    M, K = X.shape
    _check(lib().w4a8_quant_act_static(_ptr(X), M, K, X.stride(0), _ptr(s), _ptr(Xq), _ptr(sx), _stream(stream)),
           "w4a8_quant_act_static")


def w4a8_moe_quant_static(X, k: int, sorted_rows, expert_offsets, E: int, s, Xq, sx, stream=None) -> None:
    """Routed rows in expert-sorted order: row r quantizes token sorted_rows[r] // k of X with the
    scale s[e] of its expert; Xq int8 [T*k, H], sx float32 [T*k]."""
    _require_cuda(X, sorted_rows, expert_offsets, s, Xq, sx)
    T, H = X.shape
    _check(lib().w4a8_moe_quant_static(_ptr(X), T, H, X.stride(0), _ptr(sorted_rows), int(k), _ptr(expert_offsets),
                                       int(E), _ptr(s), _ptr(Xq), _ptr(sx), _stream(stream)), "w4a8_moe_quant_static")


def w4a8_gemm(Xq, sx, blob_dev, d: WDesc, Y, out_dtype: int = W4A8_OUT_BF16, stream=None) -> None:
    _require_cuda(Xq, sx, blob_dev, Y)
    _check(lib().w4a8_gemm(_ptr(Xq), _ptr(sx), Xq.shape[0], _ptr(blob_dev), ctypes.byref(d), _ptr(Y),
                           Y.stride(0), int(out_dtype), _stream(stream)), "w4a8_gemm")


def w4a8_linear(X, blob_dev, d: WDesc, Y, Xq, sx, out_dtype: int = W4A8_OUT_BF16, stream=None) -> None:
    """Quantize X (bf16 [M, K]) per token and multiply: Y = GEMM(quant(X)); Xq/sx receive the
    activation codes and scales."""
    _require_cuda(X, blob_dev, Y, Xq, sx)
    M, K = X.shape
    _check(lib().w4a8_linear(_ptr(X), M, K, X.stride(0), _ptr(blob_dev), ctypes.byref(d), _ptr(Y), Y.stride(0),
                             int(out_dtype), _ptr(Xq), _ptr(sx), _stream(stream)), "w4a8_linear")


def w4a16_gemm(X, blob_dev, d: WDesc, Y, out_dtype: int = W4A8_OUT_BF16, stream=None) -> None:
    """W4A16 sibling: Y = X W with bfloat16 activations and the blob's 4-bit weights dequantized in
    the kernel (no activation quantization)."""
    _require_cuda(X, blob_dev, Y)
    M = X.shape[0]
    _check(lib().w4a16_gemm(_ptr(X), int(M), int(X.stride(0)), _ptr(blob_dev), ctypes.byref(d), _ptr(Y),
                            int(Y.stride(0)), int(out_dtype), _stream(stream)), "w4a16_gemm")


def w4a16_kernel_name(d: WDesc, M: int) -> str:
    return lib().w4a16_kernel_name(ctypes.byref(d), int(M)).decode()


def w4a8_gemm_partials(Xq, blob_dev, d: WDesc, P, stream=None) -> None:
    _require_cuda(Xq, blob_dev, P)
    _check(lib().w4a8_gemm_partials(_ptr(Xq), Xq.shape[0], _ptr(blob_dev), ctypes.byref(d), _ptr(P),
                                    _stream(stream)), "w4a8_gemm_partials")


def w4a8_moe_align(topk_ids, E: int, sorted_rows, expert_offsets, inv, stream=None) -> None:
    _require_cuda(topk_ids, sorted_rows, expert_offsets, inv)
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_align(_ptr(topk_ids), T, k, int(E), _ptr(sorted_rows), _ptr(expert_offsets),
                                _ptr(inv), _stream(stream)), "w4a8_moe_align")


def w4a8_moe_gemm(Xq, sx, gather, k: int, expert_offsets, E: int, rows: int, blobs_dev, expert_stride: int,
                  d: WDesc, Y, out_dtype: int = W4A8_OUT_BF16, stream=None) -> None:
    _require_cuda(Xq, sx, gather, expert_offsets, blobs_dev, Y)
    src_rows = int(Xq.shape[0])
    if sx.numel() < src_rows:
        raise ValueError("sx must hold one scale per row of Xq")
    _check(lib().w4a8_moe_gemm(_ptr(Xq), _ptr(sx), _ptr(gather), int(k), _ptr(expert_offsets), int(E), int(rows),
                               src_rows, _ptr(blobs_dev), int(expert_stride), ctypes.byref(d), _ptr(Y),
                               int(out_dtype), _stream(stream)), "w4a8_moe_gemm")


def w4a8_moe_gemm_silu_static(Xq, sx, gather, k: int, expert_offsets, E: int, rows: int, blobs_dev,
                              expert_stride: int, d: WDesc, s, Hq, sh, stream=None) -> None:
    """Grouped gate/up GEMM with the static SiLU-requant in its epilogue: Hq [rows, N/2], sh [rows]."""
    _require_cuda(Xq, sx, gather, expert_offsets, blobs_dev, s, Hq, sh)
    src_rows = int(Xq.shape[0])
    if sx.numel() < src_rows:
        raise ValueError("sx must hold one scale per row of Xq")
    _check(lib().w4a8_moe_gemm_silu_static(_ptr(Xq), _ptr(sx), _ptr(gather), int(k), _ptr(expert_offsets), int(E),
                                           int(rows), src_rows, _ptr(blobs_dev), int(expert_stride), ctypes.byref(d),
                                           _ptr(s), _ptr(Hq), _ptr(sh), _stream(stream)),
           "w4a8_moe_gemm_silu_static")


def w4a8_silu_mul_quant(GU, Hq, sh, stream=None) -> None:
    _require_cuda(GU, Hq, sh)
    R, I2 = GU.shape
    _check(lib().w4a8_silu_mul_quant(_ptr(GU), R, I2 // 2, _ptr(Hq), _ptr(sh), _stream(stream)),
           "w4a8_silu_mul_quant")


def w4a8_silu_mul_quant_static(GU, expert_offsets, E: int, s, Hq, sh, stream=None) -> None:
    _require_cuda(GU, expert_offsets, s, Hq, sh)
    R, I2 = GU.shape
    _check(lib().w4a8_silu_mul_quant_static(_ptr(GU), R, I2 // 2, _ptr(expert_offsets), int(E), _ptr(s), _ptr(Hq),
                                            _ptr(sh), _stream(stream)), "w4a8_silu_mul_quant_static")


def w4a8_moe_combine(Yd, inv, topk_w, out, stream=None) -> None:
    _require_cuda(Yd, inv, topk_w, out)
    T, k = inv.shape
    H = Yd.shape[1]
    _check(lib().w4a8_moe_combine(_ptr(Yd), _ptr(inv), _ptr(topk_w), T, k, H, _ptr(out), _stream(stream)),
           "w4a8_moe_combine")


def w4a8_moe_forward(X, topk_ids, topk_w, E: int, gu_blobs, gu_stride: int, gu_desc: WDesc, d_blobs,
                     d_stride: int, d_desc: WDesc, workspace, out, stream=None) -> None:
    _require_cuda(X, topk_ids, topk_w, gu_blobs, d_blobs, workspace, out)
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_forward(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, int(E), _ptr(gu_blobs),
                                  int(gu_stride), ctypes.byref(gu_desc), _ptr(d_blobs), int(d_stride),
                                  ctypes.byref(d_desc), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _ptr(out), _stream(stream)), "w4a8_moe_forward")


def w4a8_moe_forward_noalloc(X, topk_ids, topk_w, E: int, gu_blobs, gu_stride: int, gu_desc: WDesc, d_blobs,
                             d_stride: int, d_desc: WDesc, out, stream=None) -> None:
    """w4a8_moe_forward on the library's own device scratch (no workspace argument; the call
    allocates nothing).  Calls that overlap on one GPU race: serialize them."""
    _require_cuda(X, topk_ids, topk_w, gu_blobs, d_blobs, out)
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_forward_noalloc(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, int(E), _ptr(gu_blobs),
                                          int(gu_stride), ctypes.byref(gu_desc), _ptr(d_blobs), int(d_stride),
                                          ctypes.byref(d_desc), _ptr(out), _stream(stream)),
           "w4a8_moe_forward_noalloc")


def w4a8_moe_forward_static(X, topk_ids, topk_w, E: int, gu_blobs, gu_stride: int, gu_desc: WDesc, d_blobs,
                            d_stride: int, d_desc: WDesc, s_gu, s_dn, workspace, out, stream=None) -> None:
    """w4a8_moe_forward with static per-expert activation scales s_gu, s_dn (float32 [E] on the
    device); workspace of w4a8_moe_static_workspace_size bytes."""
    _require_cuda(X, topk_ids, topk_w, gu_blobs, d_blobs, s_gu, s_dn, workspace, out)
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_forward_static(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, int(E), _ptr(gu_blobs),
                                         int(gu_stride), ctypes.byref(gu_desc), _ptr(d_blobs), int(d_stride),
                                         ctypes.byref(d_desc), _ptr(s_gu), _ptr(s_dn), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
           "w4a8_moe_forward_static")


def w4a8_moe_forward_sets(X, topk_ids, topk_w, sets, workspace, out, stream=None) -> None:
    """One MoE layer whose experts come in format classes: `sets` is a list of
    (DeviceWeights gate/up, DeviceWeights down) pairs, experts numbered set by set."""
    _require_cuda(X, topk_ids, topk_w, workspace, out)
    T, k = topk_ids.shape
    arr = (ExpertSet * len(sets))()
    keep = []
    for i, (gu, dn) in enumerate(sets):
        if gu.experts != dn.experts:
            raise ValueError("gate/up and down sets must hold the same experts")
        gd, dd = WDesc(*[getattr(gu.desc, f) for f, _ in WDesc._fields_]), \
            WDesc(*[getattr(dn.desc, f) for f, _ in WDesc._fields_])
        keep += [gd, dd]
        arr[i] = ExpertSet(gu.experts, _ptr(gu.blob), gu.stride, ctypes.pointer(gd), _ptr(dn.blob), dn.stride,
                           ctypes.pointer(dd))
    _check(lib().w4a8_moe_forward_sets(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, arr, len(sets), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
           "w4a8_moe_forward_sets")


def w4a8_moe_route(logits, d: RouteDesc, topk_ids, topk_w, bias=None, stream=None) -> None:
    """Top-k routing: logits [T, E] (float32, bfloat16 or float16; rows may be further apart than E) -> topk_ids int32 [T, k],
    topk_w float32 [T, k]; bias: float32 [E] for the choice only."""
    t = _torch()
    dev = t.current()
    if not (logits.get_device() == dev and topk_ids.get_device() == dev and topk_ids.dtype is t.int32 and
            topk_w.get_device() == dev and topk_w.dtype is t.float32 and
            (bias is None or bias.get_device() == dev and bias.dtype is t.float32)):
        _require_current((logits,), int32=(topk_ids,), float32=(topk_w, bias))      # says which
    T, E = logits.shape
    ldl, step = logits.stride()
    if T <= 1:
        ldl = E                                                 # the stride of a single row says nothing
    if E != d.E or (step != 1 and E > 1) or ldl < E:
        raise ValueError("logits must be [T, E] with contiguous rows that do not overlap")
    if T | ldl > _INT_MAX:
        _check_int32(T, ldl)
    want = (T, d.k)
    if topk_ids.shape != want or topk_w.shape != want or not topk_ids.is_contiguous() or not topk_w.is_contiguous():
        raise ValueError("topk_ids and topk_w must be contiguous [T, k]")
    if bias is not None and (bias.numel() != E or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous [E]")
    _check(lib().w4a8_moe_route(logits.data_ptr(), _dtype(logits), T, ldl,
                                None if bias is None else bias.data_ptr(), d, topk_ids.data_ptr(), topk_w.data_ptr(),
                                t.raw_stream(dev) if stream is None else int(stream)), "w4a8_moe_route")


_packed_sizes: dict = {}


def _packed_size(d: WDesc) -> int:
    """w4a8_packed_size, a function of the descriptor's bytes alone."""
    key = bytes(d)
    size = _packed_sizes.get(key)
    if size is None:
        size = _packed_sizes[key] = w4a8_packed_size(d)
    return size


def _check_rows(gather, expert_offsets, E: int, rows: int) -> None:
    """The index arrays of the grouped products: read from their first entry on, one after another."""
    if expert_offsets.numel() != E + 1 or not expert_offsets.is_contiguous():
        raise ValueError("expert_offsets must be a contiguous [E + 1]")
    if gather is not None and (gather.numel() < rows or not gather.is_contiguous()):
        raise ValueError("gather must be contiguous, with an entry for each routed row")


def _check_blobs(blobs, E: int, stride: int, d: WDesc) -> None:
    if stride < 0 or blobs.numel() * blobs.element_size() < (E - 1) * stride + _packed_size(d) or not blobs.is_contiguous():
        raise ValueError("the packed weights must be contiguous and hold E blobs at their stride")


def w4a8_moe_gemm_w8a8(Xq, sx, gather, k: int, expert_offsets, E: int, rows: int, blobs_dev, expert_stride: int,
                       d: WDesc, Y, out_dtype: int = W4A8_OUT_BF16, stream=None) -> None:
    """Grouped W8A8 GEMM: w4a8_moe_gemm for 8-bit blobs with one scale per output channel (group_size = K)."""
    t = _torch()
    dev = t.current()
    if not (Xq.get_device() == dev and Xq.dtype is t.int8 and sx.get_device() == dev and sx.dtype is t.float32 and
            expert_offsets.get_device() == dev and expert_offsets.dtype is t.int32 and blobs_dev.get_device() == dev and
            Y.get_device() == dev and (gather is None or gather.get_device() == dev and gather.dtype is t.int32)):
        _require_current((blobs_dev, Y), int8=(Xq,), float32=(sx,), int32=(gather, expert_offsets))     # says which
    src_rows, K = Xq.shape
    if K != d.K or not Xq.is_contiguous() or sx.numel() < src_rows or not sx.is_contiguous():
        raise ValueError("Xq must be a contiguous [src_rows, K] with one scale in sx for each row")
    if src_rows > _INT_MAX or not (-_INT_MAX <= k <= _INT_MAX and -_INT_MAX <= E <= _INT_MAX and -_INT_MAX <= rows <= _INT_MAX):
        _check_int32(k, E, rows, src_rows)
    _check_rows(gather, expert_offsets, E, rows)
    if t.types.get(Y.dtype) != out_dtype or out_dtype == W4A8_F16 or Y.numel() < rows * d.N or not Y.is_contiguous():
        raise ValueError("Y must be a contiguous [rows, N] of out_dtype, bfloat16 or float32")
    _check_blobs(blobs_dev, E, expert_stride, d)
    _check(lib().w4a8_moe_gemm_w8a8(Xq.data_ptr(), sx.data_ptr(), None if gather is None else gather.data_ptr(), int(k),
                                    expert_offsets.data_ptr(), int(E), int(rows), src_rows, blobs_dev.data_ptr(),
                                    int(expert_stride), d, Y.data_ptr(), int(out_dtype),
                                    t.raw_stream(dev) if stream is None else int(stream)), "w4a8_moe_gemm_w8a8")


def _w16_args(X, gather, k, expert_offsets, W, Y, width: int, stream):
    """Checked arguments of the unquantized grouped products, up to and including the row stride of Y; the stream."""
    t = _torch()
    dev = t.current()
    if not (X.get_device() == dev and W.get_device() == dev and Y.get_device() == dev and
            expert_offsets.get_device() == dev and expert_offsets.dtype is t.int32 and
            (gather is None or gather.get_device() == dev and gather.dtype is t.int32)):
        _require_current((X, W, Y), int32=(gather, expert_offsets))                 # says which
    (E, N, K), (src_rows, Kx), (rows, I) = W.shape, X.shape, Y.shape
    (stride, ldw, w1), (ldx, x1), (ldy, y1) = W.stride(), X.stride(), Y.stride()
    if X.dtype is not W.dtype or Kx != K or N != width * I:
        raise ValueError("X [src_rows, K], W [E, N, K] and Y do not match")
    if x1 != 1 or w1 != 1 or (y1 != 1 and I > 1):
        raise ValueError("the last dimension of X, W and Y must be contiguous")
    _check_rows(gather, expert_offsets, E, rows)
    # the stride of a dimension of one entry says nothing
    ldx, ldy = K if src_rows == 1 else ldx, I if rows == 1 else ldy
    ldw = K if N == 1 else ldw
    stride = N * ldw if E == 1 else stride
    if ldx | ldw | ldy | E | N | K | rows | src_rows > _INT_MAX or not -_INT_MAX <= k <= _INT_MAX:
        _check_int32(ldx, k, E, rows, src_rows, ldw, K, N, ldy)
    return (X.data_ptr(), _dtype(X), ldx, None if gather is None else gather.data_ptr(), int(k), expert_offsets.data_ptr(), E,
            rows, src_rows, W.data_ptr(), stride, ldw, K, I, Y.data_ptr(), ldy), (t.raw_stream(dev) if stream is None else int(stream))


def w4a8_moe_gemm_w16a16(X, gather, k: int, expert_offsets, W, Y, stream=None) -> None:
    """Grouped unquantized GEMM: X [src_rows, K] and W [E, N, K] in bfloat16 or float16, Y [rows, N] in the same type
    or float32; rows may be strided."""
    args, s = _w16_args(X, gather, k, expert_offsets, W, Y, 1, stream)
    _check(lib().w4a8_moe_gemm_w16a16(*args, _dtype(Y), s), "w4a8_moe_gemm_w16a16")


def w4a8_moe_gemm_silu_w16a16(X, gather, k: int, expert_offsets, W, H, stream=None) -> None:
    """Grouped unquantized gate/up GEMM with silu(gate) * up in its epilogue: W [E, 2I, K], H [rows, I] of X's type."""
    args, s = _w16_args(X, gather, k, expert_offsets, W, H, 2, stream)
    if H.dtype is not X.dtype:
        raise ValueError("H must have the type of X")
    _check(lib().w4a8_moe_gemm_silu_w16a16(*args, s), "w4a8_moe_gemm_silu_w16a16")


def w4a8_moe_w16a16_workspace_size(T: int, k: int, H: int, I: int, E: int) -> int:
    _check_int32(T, k, H, I, E)
    return int(lib().w4a8_moe_w16a16_workspace_size(T, k, H, I, E))


def _check_layer(X, topk_ids, topk_w, workspace, out, *weights) -> None:
    _require_current((X, workspace, out) + weights, int32=(topk_ids,), float32=(topk_w,))
    if str(X.dtype) != "torch.bfloat16" or X.dtype != out.dtype or X.shape != out.shape or X.dim() != 2:
        raise ValueError("X and out must be bfloat16 [T, H]")
    if topk_ids.dim() != 2 or topk_ids.shape != topk_w.shape or topk_ids.shape[0] != X.shape[0]:
        raise ValueError("topk_ids and topk_w must be [T, k]")
    _check_int32(*X.shape, *topk_ids.shape)
    if not all(t.is_contiguous() for t in (X, topk_ids, topk_w, workspace, out)):
        raise ValueError("the layer's tensors must be contiguous")


def w4a8_moe_forward_w8a8(X, topk_ids, topk_w, E: int, gu_blobs, gu_stride: int, gu_desc: WDesc, d_blobs, d_stride: int,
                          d_desc: WDesc, workspace, out, stream=None) -> None:
    """w4a8_moe_forward on 8-bit per-channel experts; workspace of w4a8_moe_workspace_size bytes."""
    _check_layer(X, topk_ids, topk_w, workspace, out, gu_blobs, d_blobs)
    if X.shape[1] != gu_desc.K:
        raise ValueError("X must be [T, K of the gate/up weights]")
    _check_int32(E)
    _check_blobs(gu_blobs, E, gu_stride, gu_desc)
    _check_blobs(d_blobs, E, d_stride, d_desc)
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_forward_w8a8(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, int(E), _ptr(gu_blobs), int(gu_stride),
                                       gu_desc, _ptr(d_blobs), int(d_stride), d_desc, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
           "w4a8_moe_forward_w8a8")


def w4a8_moe_forward_w16a16(X, topk_ids, topk_w, Wgu, Wd, workspace, out, stream=None) -> None:
    """One MoE layer on unquantized bfloat16 experts: Wgu [E, 2I, H], Wd [E, H, I]; workspace of
    w4a8_moe_w16a16_workspace_size bytes."""
    _check_layer(X, topk_ids, topk_w, workspace, out, Wgu, Wd)
    E, I2, H = Wgu.shape
    if Wd.shape != (E, H, I2 // 2) or X.shape[1] != H or I2 % 2 or Wgu.dtype != X.dtype or Wd.dtype != X.dtype:
        raise ValueError("Wgu [E, 2I, H] and Wd [E, H, I] must be bfloat16 and match X")
    _check_int32(E, I2)
    if E == 0 or not Wgu[0].is_contiguous() or not Wd[0].is_contiguous():
        raise ValueError("each expert's weights must be dense")
    T, k = topk_ids.shape
    _check(lib().w4a8_moe_forward_w16a16(_ptr(X), _ptr(topk_ids), _ptr(topk_w), T, k, E, _ptr(Wgu), Wgu.stride(0), _ptr(Wd),
                                         Wd.stride(0), H, I2 // 2, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
           "w4a8_moe_forward_w16a16")


# ------------------------------------------------------------------------------ microscaled formats
def mx_row_bytes(fmt: int, K: int) -> int:
    """Bytes of a row of codes: K rounded up to 128, two E2M1 codes to a byte."""
    Kp = -(-K // 128) * 128
    return Kp // 2 if fmt == W4A8_MX_FP4 else Kp


def mx_empty(fmt: int, M: int, K: int, device="cuda"):
    """Uninitialized codes and scales of M rows of K, as the quantizing calls take them."""
    import torch
    return (torch.empty((M, mx_row_bytes(fmt, K)), dtype=torch.uint8, device=device),
            torch.empty((M, -(-K // 128) * 4), dtype=torch.uint8, device=device))


def _row_stride(x, what: str) -> int:
    """Elements between the rows of a matrix whose rows are contiguous; that of a single row says nothing."""
    (M, N), (ld, step) = x.shape, x.stride()
    if M <= 1:
        ld = N
    if (step != 1 and N > 1) or ld < N:
        raise ValueError(f"{what} must be a matrix with contiguous rows that do not overlap")
    if M | N | ld > _INT_MAX:
        _check_int32(M, N, ld)
    return ld


def _ld(x, N: int, what: str) -> int:
    """_row_stride of a matrix of N columns, which is N if it is contiguous."""
    return N if x.is_contiguous() else _row_stride(x, what)


def _kind(t, x) -> int:
    """_dtype, without the calls in between."""
    kind = t.types.get(x.dtype)
    return _dtype(x) if kind is None else kind


# The calls below test all of their arguments in one expression, cheapest first (half of a small call's host time otherwise), and
# say what is wrong with them only where it is false.
def _mx_rows(t, dev: int, Xq, sx, fmt: int, M: int, K: int) -> bool:
    """Whether Xq and sx are codes and scales of M rows of K as w4a8_mx_quant leaves them, on device dev."""
    Kp = (K + 127) & -128
    return (Xq.get_device() == dev and sx.get_device() == dev and Xq.dtype is t.uint8 and sx.dtype is t.uint8 and
            (fmt == W4A8_MX_FP8 and Xq.numel() == M * Kp or fmt == W4A8_MX_FP4 and 2 * Xq.numel() == M * Kp) and
            32 * sx.numel() == M * Kp and Xq.is_contiguous() and sx.is_contiguous() and 0 < K <= _INT_MAX and M <= _INT_MAX)


def _refuse(tensors, mx=(), what: str = "the tensors do not match") -> None:
    """Raises for a call whose test failed: tensors elsewhere, codes (Xq, sx, fmt, M, K) of another shape, or `what`."""
    _require_current([x for x in tensors if x is not None])
    t = _torch()
    for Xq, sx, fmt, M, K in mx:
        if fmt != W4A8_MX_FP4 and fmt != W4A8_MX_FP8:
            raise ValueError("fmt must be W4A8_MX_FP4 or W4A8_MX_FP8")
        if not 0 < K <= _INT_MAX or M > _INT_MAX:
            raise ValueError("K must be positive, and it and the rows fit in 32 bits")
        if not _mx_rows(t, t.current(), Xq, sx, fmt, M, K):
            raise ValueError("the codes and scales must be contiguous uint8 [M, K rounded up to 128 (MXFP4: / 2)] and "
                             "[M, the same / 32]")
    raise ValueError(what)


_mx_packed_sizes: dict = {}


def w4a8_mx_packed_size(K: int, N: int) -> int:
    """Bytes of packed MXFP4 weights [N, K]; 0 if there are none of that size."""
    size = _mx_packed_sizes.get((K, N))
    if size is None:
        _check_int32(K, N)
        size = int(lib().w4a8_mx_packed_size(int(K), int(N)))
        if len(_mx_packed_sizes) < 4096:
            _mx_packed_sizes[K, N] = size
    return size


def _mx_blobs(t, dev: int, blobs, E: int, stride: int, K: int, N: int) -> bool:
    """Whether blobs holds E packed [N, K], stride bytes apart, on device dev."""
    size = _mx_packed_sizes.get((K, N)) or w4a8_mx_packed_size(K, N)
    if size == 0:
        raise W4A8Error(W4A8_EUNSUPPORTED if K > 0 and N > 0 else W4A8_EINVAL, "w4a8_mx_packed_size")
    return (blobs.get_device() == dev and blobs.dtype is t.uint8 and 0 < E <= _INT_MAX and stride >= 0 and
            blobs.numel() >= (E - 1) * stride + size and blobs.is_contiguous())


_NO_BLOBS = "the packed weights must be contiguous uint8 and hold the matrices at their stride"


def w4a8_mx_quant(X, fmt: int, Xq, sx, stream=None) -> None:
    """X [M, K] (bfloat16, float16 or float32, rows may be strided) -> MX codes and scales (mx_empty)."""
    t = _torch_of_calls or _torch()
    dev = X.get_device()
    M, K = X.shape
    if dev != (t.device() if dev >= 0 else t.current()) or not _mx_rows(t, dev, Xq, sx, fmt, M, K):
        _refuse((X, Xq, sx), ((Xq, sx, fmt, M, K),))
    st = lib().w4a8_mx_quant(X.data_ptr(), _kind(t, X), M, K, _ld(X, K, "X"), fmt, Xq.data_ptr(), sx.data_ptr(),
                             t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_mx_quant")


def w4a8_mx_dequant(Xq, sx, fmt: int, Y, stream=None) -> None:
    """The values of MX codes and scales: Y [M, K] in bfloat16, float16 or float32, rows may be strided."""
    t = _torch_of_calls or _torch()
    dev = Y.get_device()
    M, K = Y.shape
    if dev != (t.device() if dev >= 0 else t.current()) or not _mx_rows(t, dev, Xq, sx, fmt, M, K):
        _refuse((Y, Xq, sx), ((Xq, sx, fmt, M, K),))
    st = lib().w4a8_mx_dequant(Xq.data_ptr(), sx.data_ptr(), fmt, M, K, Y.data_ptr(), _kind(t, Y), _ld(Y, K, "Y"),
                               t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_mx_dequant")


def w4a8_mx_pack(W, blobs, stream=None) -> None:
    """Quantize W [N, K] or [E, N, K] to MXFP4 and pack it into blobs, uint8 [w4a8_mx_packed_size] or [E, stride]."""
    t = _torch()
    dev = t.current()
    if W.dim() not in (2, 3) or blobs.dim() != W.dim() - 1:
        raise ValueError("W must be [N, K] or [E, N, K], and blobs uint8 [bytes] or [E, bytes]")
    one = W.dim() == 2
    E, (N, K) = 1 if one else W.shape[0], W.shape[-2:]
    if E == 0:
        return
    if not one and blobs.shape[0] != E:
        raise ValueError("W and blobs must have the same experts")
    ldw = _row_stride(W if one else W[0], "W")
    expert, stride = (0, 0) if E == 1 else (W.stride(0), blobs.stride(0))
    if W.get_device() != dev or expert < 0 or not _mx_blobs(t, dev, blobs, E, stride, K, N):
        _refuse((W, blobs), what=_NO_BLOBS)
    _check(lib().w4a8_mx_pack(W.data_ptr(), _dtype(W), E, N, K, ldw, expert, blobs.data_ptr(), stride,
                              t.raw_stream(dev) if stream is None else int(stream)), "w4a8_mx_pack")


def w4a8_mx_pack_codes(codes, scales, blob, stream=None) -> None:
    """Pack existing MXFP4 codes uint8 [N, K / 2] (row stride a multiple of 16) and scales uint8 [N, K / 32], K % 32 == 0."""
    t = _torch()
    dev = t.current()
    N, K = codes.shape[0], 2 * codes.shape[1]
    if codes.dtype is not t.uint8 or scales.dtype is not t.uint8 or scales.shape != (N, K // 32) or K % 32:
        raise ValueError("codes and scales must be uint8 [N, K / 2] and [N, K / 32]")
    ldc, lds = _row_stride(codes, "codes"), _row_stride(scales, "scales")
    if codes.get_device() != dev or scales.get_device() != dev or not _mx_blobs(t, dev, blob, 1, 0, K, N):
        _refuse((codes, scales, blob), what=_NO_BLOBS)
    _check(lib().w4a8_mx_pack_codes(codes.data_ptr(), scales.data_ptr(), N, K, ldc, lds, blob.data_ptr(),
                                    t.raw_stream(dev) if stream is None else int(stream)), "w4a8_mx_pack_codes")


def w4a8_mx_unpack_codes(blob, N: int, K: int, codes, scales, stream=None) -> None:
    """The inverse, into the layout of activations: codes and scales of mx_empty(W4A8_MX_FP4, N, K)."""
    t = _torch()
    dev = t.current()
    if not _mx_rows(t, dev, codes, scales, W4A8_MX_FP4, N, K) or not _mx_blobs(t, dev, blob, 1, 0, K, N):
        _refuse((codes, scales, blob), ((codes, scales, W4A8_MX_FP4, N, K),), _NO_BLOBS)
    _check(lib().w4a8_mx_unpack_codes(blob.data_ptr(), N, K, codes.data_ptr(), scales.data_ptr(),
                                      t.raw_stream(dev) if stream is None else int(stream)), "w4a8_mx_unpack_codes")


def w4a8_mx_gemm(Xq, sx, fmt: int, blob, K: int, N: int, Y, stream=None) -> None:
    """Y [M, N] (bfloat16, float16 or float32, rows may be strided) = MX activations times packed MXFP4 weights [N, K]."""
    t = _torch_of_calls or _torch()
    dev = Y.get_device()
    M, width = Y.shape
    if (width != N or dev != (t.device() if dev >= 0 else t.current()) or not _mx_rows(t, dev, Xq, sx, fmt, M, K) or
            not _mx_blobs(t, dev, blob, 1, 0, K, N)):
        _refuse((Xq, sx, blob, Y), ((Xq, sx, fmt, M, K),), _NO_BLOBS if width == N else "Y must be [M, N]")
    st = lib().w4a8_mx_gemm(Xq.data_ptr(), sx.data_ptr(), fmt, M, blob.data_ptr(), K, N, Y.data_ptr(), _ld(Y, N, "Y"),
                            _kind(t, Y), t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_mx_gemm")


def _mx_moe_args(t, dev: int, Xq, sx, fmt, gather, k, expert_offsets, E, blobs, expert_stride, K, rows, N, other):
    """Checked arguments of the grouped MX products, up to and including K.  dev: where `other`, an output, is."""
    src_rows = Xq.shape[0]
    if not (dev == (t.device() if dev >= 0 else t.current()) and _mx_rows(t, dev, Xq, sx, fmt, src_rows, K) and
            _mx_blobs(t, dev, blobs, E, expert_stride, K, N) and expert_offsets.get_device() == dev and
            expert_offsets.dtype is t.int32 and expert_offsets.numel() == E + 1 and expert_offsets.is_contiguous() and
            (gather is None or gather.get_device() == dev and gather.dtype is t.int32 and gather.numel() >= rows and
             gather.is_contiguous()) and -_INT_MAX <= k <= _INT_MAX and rows <= _INT_MAX):
        _require_current((Xq, sx, blobs, other), int32=(gather, expert_offsets))
        _check_rows(gather, expert_offsets, E, rows)
        _check_int32(k, E, rows)
        _refuse((), ((Xq, sx, fmt, src_rows, K),), _NO_BLOBS)
    return (Xq.data_ptr(), sx.data_ptr(), fmt, None if gather is None else gather.data_ptr(), k, expert_offsets.data_ptr(),
            E, rows, src_rows, blobs.data_ptr(), expert_stride, K)


def w4a8_moe_gemm_mx(Xq, sx, fmt: int, gather, k: int, expert_offsets, E: int, blobs, expert_stride: int, K: int, Y,
                     stream=None) -> None:
    """Grouped product of MX activations with E packed MXFP4 matrices [N, K]; Y [rows, N]."""
    t = _torch_of_calls or _torch()
    dev = Y.get_device()
    rows, N = Y.shape
    args = _mx_moe_args(t, dev, Xq, sx, fmt, gather, k, expert_offsets, E, blobs, expert_stride, K, rows, N, Y)
    st = lib().w4a8_moe_gemm_mx(*args, N, Y.data_ptr(), _ld(Y, N, "Y"), _kind(t, Y),
                                t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_moe_gemm_mx")


def w4a8_moe_gemm_silu_mx(Xq, sx, fmt: int, gather, k: int, expert_offsets, E: int, blobs, expert_stride: int, K: int, H,
                          stream=None) -> None:
    """Grouped gate/up product with silu(gate) * up in its epilogue: E packed [2I, K], H [rows, I] in bfloat16 or float16."""
    t = _torch_of_calls or _torch()
    dev = H.get_device()
    rows, I = H.shape
    args = _mx_moe_args(t, dev, Xq, sx, fmt, gather, k, expert_offsets, E, blobs, expert_stride, K, rows, 2 * I, H)
    st = lib().w4a8_moe_gemm_silu_mx(*args, I, H.data_ptr(), _ld(H, I, "H"), _kind(t, H),
                                     t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_moe_gemm_silu_mx")


def w4a8_moe_gemm_silu_mx_quant(Xq, sx, fmt: int, gather, k: int, expert_offsets, E: int, blobs, expert_stride: int, K: int, I: int,
                                h_fmt: int, Hq, sh, stream=None) -> None:
    """The same with H quantized to h_fmt: codes and scales of mx_empty(h_fmt, rows, I)."""
    t = _torch_of_calls or _torch()
    dev = Hq.get_device()
    rows = Hq.shape[0]
    if not _mx_rows(t, dev, Hq, sh, h_fmt, rows, I):
        _refuse((Hq, sh), ((Hq, sh, h_fmt, rows, I),))
    args = _mx_moe_args(t, dev, Xq, sx, fmt, gather, k, expert_offsets, E, blobs, expert_stride, K, rows, 2 * I, Hq)
    st = lib().w4a8_moe_gemm_silu_mx_quant(*args, I, h_fmt, Hq.data_ptr(), sh.data_ptr(),
                                           t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_moe_gemm_silu_mx_quant")


def w4a8_moe_mx_workspace_size(T: int, k: int, H: int, I: int, E: int, fmt: int) -> int:
    _check_int32(T, k, H, I, E, fmt)
    return int(lib().w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt))


def w4a8_moe_forward_mx(X, topk_ids, topk_w, E: int, fmt: int, gu_blobs, gu_stride: int, d_blobs, d_stride: int, I: int, workspace,
                        out, stream=None) -> None:
    """One MoE layer on MXFP4 experts: gu_blobs E packed [2I, H], d_blobs E packed [H, I]; workspace of
    w4a8_moe_mx_workspace_size bytes, or less (the experts' outputs are then made by slices of columns)."""
    t = _torch_of_calls or _torch()
    dev = X.get_device()
    (T, H), (rows, k) = X.shape, topk_ids.shape
    if not (dev == (t.device() if dev >= 0 else t.current()) and topk_ids.get_device() == dev and topk_w.get_device() == dev and
            workspace.get_device() == dev and out.get_device() == dev and _mx_blobs(t, dev, gu_blobs, E, gu_stride, H, 2 * I) and
            _mx_blobs(t, dev, d_blobs, E, d_stride, I, H) and T | H | k <= _INT_MAX):
        _check_layer(X, topk_ids, topk_w, workspace, out, gu_blobs, d_blobs)
        _check_int32(E, I, T, H, k)
        raise ValueError(_NO_BLOBS)
    if not (X.dtype is t.bfloat16 and out.dtype is t.bfloat16 and topk_ids.dtype is t.int32 and topk_w.dtype is t.float32 and
            rows == T and topk_w.shape == (T, k) and out.shape == (T, H) and X.is_contiguous() and out.is_contiguous() and
            topk_ids.is_contiguous() and topk_w.is_contiguous() and workspace.is_contiguous()):
        _check_layer(X, topk_ids, topk_w, workspace, out, gu_blobs, d_blobs)
    st = lib().w4a8_moe_forward_mx(X.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(), T, k, E, fmt, gu_blobs.data_ptr(),
                                   gu_stride, d_blobs.data_ptr(), d_stride, H, I, workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), out.data_ptr(),
                                   t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_moe_forward_mx")


# ------------------------------------------------------------------------------ the norm around a block
def _norm_row(t, dev: int, v, H: int) -> bool:
    return v is None or v.get_device() == dev and v.dtype is t.float32 and v.numel() == H and v.is_contiguous()


def _norm_args(t, dev: int, X, residual, d: NormDesc, w, residual_out, post_w, gate):
    """Checked arguments of the norm calls, up to and including the row stride of residual_out."""
    shape = X.shape
    M, H = shape
    if M | H > _INT_MAX:
        _check_int32(M, H)
    if dev != (t.device() if dev >= 0 else t.current()) or not _norm_row(t, dev, w, H) or not _norm_row(t, dev, post_w, H):
        _refuse((X, w, post_w), what="w and post_w must be contiguous float32 [H]")
    res, ldr, out, ldo, kind = None, H, None, H, X
    if residual is not None:
        if residual.get_device() != dev or residual.shape != shape:
            _refuse((X, residual), what="residual must have the shape of X")
        res, ldr, kind = residual.data_ptr(), _ld(residual, H, "residual"), residual
    if residual_out is residual:
        out, ldo = res, ldr
    elif residual_out is not None:
        if (residual_out.get_device() != dev or residual_out.shape != shape or
                residual is not None and residual_out.dtype is not residual.dtype):
            _refuse((X, residual_out), what="residual_out must have the shape of X and the type of residual")
        out, ldo, kind = residual_out.data_ptr(), _ld(residual_out, H, "residual_out"), residual_out
    ldg = 0
    if gate is not None:
        if (gate.get_device() != dev or gate.dtype is not X.dtype or gate.dim() != 2 or gate.shape[0] not in (1, M) or
                gate.shape[1] != H):
            _refuse((X, gate), what="gate must be [M, H] or [1, H] in the type of X")
        ldg = _row_stride(gate, "gate")
        if gate.shape[0] != M or M == 1:
            ldg = 0
    return (X.data_ptr(), _kind(t, X), _ld(X, H, "X"), res, _kind(t, kind), ldr, None if gate is None else gate.data_ptr(), ldg,
            None if post_w is None else post_w.data_ptr(), None if w is None else w.data_ptr(), d, M, H, out, ldo)


def w4a8_norm_residual(X, residual, d: NormDesc, w, residual_out, Y, post_w=None, gate=None, stream=None) -> None:
    """r' = residual + alpha gate u, u = X or its RMS norm times post_w; Y = RMS norm of r' times w.  residual, residual_out, Y,
    post_w and gate may be None."""
    t = _torch_of_calls or _torch()
    dev = X.get_device()
    args = _norm_args(t, dev, X, residual, d, w, residual_out, post_w, gate)
    y, ldy = None, args[12]
    if Y is not None:
        if Y.get_device() != dev or Y.shape != X.shape or Y.dtype is not X.dtype:
            _refuse((X, Y), what="Y must have the shape and type of X")
        y, ldy = Y.data_ptr(), _ld(Y, ldy, "Y")
    st = lib().w4a8_norm_residual(*args, y, ldy, t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_norm_residual")


def w4a8_norm_residual_quant(X, residual, d: NormDesc, w, residual_out, fmt: int, Xq, sx, post_w=None, gate=None,
                             stream=None) -> None:
    """The same with h quantized: MX codes and scales (mx_empty), or int8 [M, H] and float32 [M] for W4A8_QUANT_INT8."""
    t = _torch_of_calls or _torch()
    dev = X.get_device()
    args = _norm_args(t, dev, X, residual, d, w, residual_out, post_w, gate)
    M, H = args[11], args[12]
    if fmt == W4A8_QUANT_INT8:
        if not (Xq.get_device() == dev and sx.get_device() == dev and Xq.dtype is t.int8 and sx.dtype is t.float32 and
                Xq.shape == X.shape and sx.numel() == M and Xq.is_contiguous() and sx.is_contiguous()):
            _refuse((X, Xq, sx), what="Xq and sx must be contiguous int8 [M, H] and float32 [M]")
    elif not _mx_rows(t, dev, Xq, sx, fmt, M, H):
        _refuse((X, Xq, sx), ((Xq, sx, fmt, M, H),))
    st = lib().w4a8_norm_residual_quant(*args, fmt, Xq.data_ptr(), sx.data_ptr(),
                                        t.raw_stream(dev) if stream is None else int(stream))
    if st:
        _check(st, "w4a8_norm_residual_quant")


# ------------------------------------------------------------------------------ helpers
@dataclass
class DeviceWeights:
    """A packed blob (or E blobs back to back) resident on the device."""
    desc: WDesc
    blob: "object"          # torch uint8 cuda tensor
    stride: int             # bytes between experts (= packed size)
    experts: int = 1


def to_device(d: WDesc, blobs, device="cuda") -> DeviceWeights:
    """Copy one host blob or a list of host blobs (same desc) into one device buffer."""
    import torch
    if isinstance(blobs, np.ndarray):
        blobs = [blobs]
    n = w4a8_packed_size(d)
    for b in blobs:
        w4a8_blob_check(b, d)
    host = np.concatenate([np.ascontiguousarray(b[:n]) for b in blobs])
    dev = torch.from_numpy(host).to(device)
    return DeviceWeights(d, dev, n, len(blobs))


def experts_to_device(d: WDesc, E: int, blobs: dict, device="cuda") -> DeviceWeights:
    """E expert blobs of one desc in one zero-initialised device buffer; `blobs` maps expert
    id -> host blob and may omit experts that receive no rows (their bytes stay zero and
    are never read)."""
    import torch
    n = w4a8_packed_size(d)
    dev = torch.zeros(E * n, dtype=torch.uint8, device=device)
    for e, b in blobs.items():
        w4a8_blob_check(b, d)
        dev[e * n:(e + 1) * n].copy_(torch.from_numpy(np.ascontiguousarray(b[:n])))
    return DeviceWeights(d, dev, n, E)
