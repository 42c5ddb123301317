"""Python binding of the B200 NVFP4 + augmented-residual-channel library (libarc.so).

Argument marshalling only: every step of the path runs in the library's CUDA kernels. PyTorch
provides device memory and streams. There is no fallback: if libarc.so is missing or the GPU is
not an sm_100 device, calls raise.

The C ABI is documented in include/arc.h; the functions below carry the same names without the
``arc_`` prefix and allocate their outputs (and scratch) with torch when none are passed.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libarc.so")
_lib = None

ARC_STATUS = {0: "ARC_OK", 1: "ARC_ERR_INVALID_ARG", 2: "ARC_ERR_ALIGNMENT", 3: "ARC_ERR_UNSUPPORTED",
              4: "ARC_ERR_CUDA", 5: "ARC_ERR_TIMEOUT", 6: "ARC_ERR_WORKSPACE"}


class ArcError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {ARC_STATUS.get(code, code)}")
        self.code = code


class SwigluSublayer(ctypes.Structure):
    _fields_ = [
        ("rms_gain_bf16", ctypes.c_void_p), ("w_gateup_bf16", ctypes.c_void_p), ("w_down_bf16", ctypes.c_void_p),
        ("gateup_codes", ctypes.c_void_p), ("gateup_sf", ctypes.c_void_p), ("gateup_scale", ctypes.c_void_p),
        ("down_codes", ctypes.c_void_p), ("down_sf", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
        ("idx_gateup", ctypes.c_void_p), ("r_gateup", ctypes.c_int32),
        ("idx_down", ctypes.c_void_p), ("r_down", ctypes.c_int32),
        ("gateup_fp8", ctypes.c_void_p), ("gateup_fp8_scale", ctypes.c_void_p),
        ("down_fp8", ctypes.c_void_p), ("down_fp8_scale", ctypes.c_void_p),
    ]


class SwigluBlock(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int64), ("ffn", ctypes.c_int64), ("eps", ctypes.c_float),
                ("n_sublayers", ctypes.c_int32), ("sublayers", ctypes.POINTER(SwigluSublayer)),
                ("residual_scale", ctypes.c_float), ("inject_bf16", ctypes.c_void_p)]


STEP_BF16, STEP_NVFP4, STEP_FP8 = 0, 1, 2  # per-step formats of arc_recurrent_prefill_schedule


_SIGS = {
    "arc_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "arc_kpad": (ctypes.c_int64, [ctypes.c_int64]),
    "arc_nvfp4_codes_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "arc_nvfp4_sf_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "arc_quantize_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32]),
    "arc_calibrate_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64]),
    "arc_quantize_act_nvfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                              ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_pack_weight_nvfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_calibrate_outliers": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                              ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.c_void_p]),
    "arc_calibrate_order": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_quantize_act_nvfp4_reordered": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                                                        ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_pack_weight_nvfp4_reordered": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                       ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_gemm_nvfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
    "arc_mxfp4_sf_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "arc_quantize_act_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                              ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "arc_pack_weight_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p]),
    "arc_gemm_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "arc_gemm_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_void_p]),
    "arc_rmsnorm_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p]),
    "arc_silu_mul_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "arc_recurrent_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.POINTER(SwigluBlock)]),
    "arc_recurrent_prefill": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(SwigluBlock),
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                             ctypes.c_void_p]),
    "arc_recurrent_prefill_schedule": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                      ctypes.POINTER(SwigluBlock), ctypes.c_int32,
                                                      ctypes.POINTER(ctypes.c_uint8), ctypes.c_void_p,
                                                      ctypes.c_size_t, ctypes.c_void_p]),
    "arc_quantize_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "arc_gemm_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                    ctypes.c_int64, ctypes.c_void_p]),
    "arc_expert_plan_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    "arc_expert_sf_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64]),
    "arc_expert_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "arc_dispatch_experts_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                 ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                                 ctypes.c_int64, ctypes.c_void_p]),
    "arc_dispatch_experts_grad_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "arc_combine_experts_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                                ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                ctypes.c_int64, ctypes.c_void_p]),
    "arc_combine_experts_grad_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                     ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                                     ctypes.c_void_p]),
    "arc_quantize_act_experts_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_void_p]),
    "arc_quantize_swiglu_experts_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                         ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                         ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "arc_pack_weight_experts_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_void_p]),
    "arc_gemm_experts_mxfp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                              ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                              ctypes.c_void_p]),
    "arc_gemm_experts_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                             ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_void_p]),
    "arc_last_device_status": (ctypes.c_int, [ctypes.c_void_p]),
    "arc_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "arc_debug_inject": (ctypes.c_int, [ctypes.c_int32]),
    "arc_quantize_act_nvfp4_static_scratch": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                             ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                                                             ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                             ctypes.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """Load libarc.so (built in-tree by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def _check(fn: str, code: int):
    if code != 0:
        raise ArcError(fn, code)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("arc: tensors must be CUDA tensors")


def kpad(k_aug: int) -> int:
    return int(lib().arc_kpad(k_aug))


def codes_bytes(rows: int, k_aug: int) -> int:
    return int(lib().arc_nvfp4_codes_bytes(rows, k_aug))


def sf_bytes(rows: int, k_aug: int) -> int:
    return int(lib().arc_nvfp4_sf_bytes(rows, k_aug))


def quantize_workspace_bytes(rows: int, r: int) -> int:
    return int(lib().arc_quantize_workspace_bytes(rows, r))


def _u8(n: int, device):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _ws(n: int, device):
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


@dataclass
class NVFP4Tensor:
    """Packed NVFP4 operand: codes [rows, K_pad/2] u8, swizzled scale bytes, fp32 tensor scale."""
    codes: torch.Tensor
    sf: torch.Tensor
    scale: torch.Tensor
    rows: int
    k_aug: int


def quantize_act_nvfp4(x: torch.Tensor, idx: torch.Tensor | None = None, rms_gain: torch.Tensor | None = None,
                       eps: float = 1e-6, static_scale: torch.Tensor | None = None, out: NVFP4Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """arc_quantize_act_nvfp4: X [M, K] bf16 (row stride x.stride(0)) -> NVFP4 with r appended channels."""
    _need_cuda(x, idx, rms_gain, static_scale)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    r = 0 if idx is None else int(idx.numel())
    if out is None:
        out = NVFP4Tensor(_u8(codes_bytes(M, K + r), x.device), _u8(sf_bytes(M, K + r), x.device),
                          torch.empty(1, dtype=torch.float32, device=x.device), M, K + r)
    nws = quantize_workspace_bytes(M, r)
    if workspace is None:
        workspace = _ws(nws, x.device)
    _check("arc_quantize_act_nvfp4", lib().arc_quantize_act_nvfp4(
        _p(x), M, K, x.stride(0), _p(idx), r, _p(rms_gain), float(eps), _p(static_scale), _p(out.codes),
        _p(out.sf), _p(out.scale), _p(workspace), workspace.numel(), _stream(stream)))
    return out


def pack_weight_nvfp4(w: torch.Tensor, idx: torch.Tensor | None = None, out: NVFP4Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """arc_pack_weight_nvfp4: W [N, K] bf16 -> NVFP4 of [W | W[:, idx]] with its own tensor scale."""
    _need_cuda(w, idx)
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    N, K = w.shape
    r = 0 if idx is None else int(idx.numel())
    if out is None:
        out = NVFP4Tensor(_u8(codes_bytes(N, K + r), w.device), _u8(sf_bytes(N, K + r), w.device),
                          torch.empty(1, dtype=torch.float32, device=w.device), N, K + r)
    nws = quantize_workspace_bytes(N, r)
    if workspace is None:
        workspace = _ws(nws, w.device)
    _check("arc_pack_weight_nvfp4", lib().arc_pack_weight_nvfp4(
        _p(w), N, K, w.stride(0), _p(idx), r, _p(out.codes), _p(out.sf), _p(out.scale), _p(workspace),
        workspace.numel(), _stream(stream)))
    return out


def calibrate_outliers(x: torch.Tensor, r: int, stream=None) -> torch.Tensor:
    """arc_calibrate_outliers: top-r channels of X by abs-max (device int32[r])."""
    _need_cuda(x)
    M, K = x.shape
    idx = torch.empty(r, dtype=torch.int32, device=x.device)
    ws = _ws(int(lib().arc_calibrate_workspace_bytes(K)), x.device)
    _check("arc_calibrate_outliers", lib().arc_calibrate_outliers(_p(x), M, K, x.stride(0), r, _p(idx), _p(ws),
                                                                  ws.numel(), _stream(stream)))
    return idx


def calibrate_order(x: torch.Tensor, stream=None) -> torch.Tensor:
    """arc_calibrate_order: all K channels of X by descending abs-max (device int32[K])."""
    _need_cuda(x)
    M, K = x.shape
    perm = torch.empty(K, dtype=torch.int32, device=x.device)
    ws = _ws(int(lib().arc_calibrate_workspace_bytes(K)), x.device)
    _check("arc_calibrate_order", lib().arc_calibrate_order(_p(x), M, K, x.stride(0), _p(perm), _p(ws), ws.numel(),
                                                            _stream(stream)))
    return perm


def quantize_act_nvfp4_reordered(x: torch.Tensor, perm: torch.Tensor, r: int, rms_gain: torch.Tensor | None = None,
                                 eps: float = 1e-6, static_scale: torch.Tensor | None = None,
                                 out: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None,
                                 stream=None) -> NVFP4Tensor:
    """arc_quantize_act_nvfp4_reordered: X [M, K] bf16 -> NVFP4 of X[:, perm] with the residuals of
    the r channels perm[:r] appended."""
    _need_cuda(x, perm, rms_gain, static_scale)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert perm.dtype == torch.int32 and perm.numel() == x.shape[1]
    M, K = x.shape
    if out is None:
        out = NVFP4Tensor(_u8(codes_bytes(M, K + r), x.device), _u8(sf_bytes(M, K + r), x.device),
                          torch.empty(1, dtype=torch.float32, device=x.device), M, K + r)
    if workspace is None:
        workspace = _ws(quantize_workspace_bytes(M, r), x.device)
    _check("arc_quantize_act_nvfp4_reordered", lib().arc_quantize_act_nvfp4_reordered(
        _p(x), M, K, x.stride(0), _p(perm), int(r), _p(rms_gain), float(eps), _p(static_scale), _p(out.codes),
        _p(out.sf), _p(out.scale), _p(workspace), workspace.numel(), _stream(stream)))
    return out


def pack_weight_nvfp4_reordered(w: torch.Tensor, perm: torch.Tensor, r: int, out: NVFP4Tensor | None = None,
                                workspace: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """arc_pack_weight_nvfp4_reordered: W [N, K] bf16 -> NVFP4 of [W[:, perm] | W[:, perm[:r]]]."""
    _need_cuda(w, perm)
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    assert perm.dtype == torch.int32 and perm.numel() == w.shape[1]
    N, K = w.shape
    if out is None:
        out = NVFP4Tensor(_u8(codes_bytes(N, K + r), w.device), _u8(sf_bytes(N, K + r), w.device),
                          torch.empty(1, dtype=torch.float32, device=w.device), N, K + r)
    if workspace is None:
        workspace = _ws(quantize_workspace_bytes(N, r), w.device)
    _check("arc_pack_weight_nvfp4_reordered", lib().arc_pack_weight_nvfp4_reordered(
        _p(w), N, K, w.stride(0), _p(perm), int(r), _p(out.codes), _p(out.sf), _p(out.scale), _p(workspace),
        workspace.numel(), _stream(stream)))
    return out


def gemm_nvfp4(a: NVFP4Tensor, b: NVFP4Tensor, out: torch.Tensor | None = None, add: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """arc_gemm_nvfp4: Y [M, N] bf16 = s_A s_B * A_aug B_aug^T (+ add)."""
    assert a.k_aug == b.k_aug, "A and B must share the augmented depth K + r"
    M, N = a.rows, b.rows
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.codes.device)
    _check("arc_gemm_nvfp4", lib().arc_gemm_nvfp4(
        _p(a.codes), _p(a.sf), _p(a.scale), _p(b.codes), _p(b.sf), _p(b.scale), M, N, a.k_aug, _p(out),
        out.stride(0), _p(add), 0 if add is None else add.stride(0), _stream(stream)))
    return out


def gemm_bf16(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None, add: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """arc_gemm_bf16: Y [M, N] = bf16(X W^T (+ add))."""
    _need_cuda(x, w, out, add)
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    _check("arc_gemm_bf16", lib().arc_gemm_bf16(
        _p(x), x.stride(0), _p(w), w.stride(0), M, N, K, _p(out), out.stride(0), _p(add),
        0 if add is None else add.stride(0), _stream(stream)))
    return out


def rmsnorm_bf16(h: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    S, d = h.shape
    if out is None:
        out = torch.empty_like(h)
    _check("arc_rmsnorm_bf16", lib().arc_rmsnorm_bf16(_p(h), S, d, h.stride(0), _p(gain), float(eps), _p(out),
                                                      out.stride(0), _stream(stream)))
    return out


def silu_mul_bf16(gu: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    S, F2 = gu.shape
    F = F2 // 2
    if out is None:
        out = torch.empty(S, F, dtype=torch.bfloat16, device=gu.device)
    _check("arc_silu_mul_bf16", lib().arc_silu_mul_bf16(_p(gu), S, F, gu.stride(0), _p(out), out.stride(0),
                                                        _stream(stream)))
    return out


class RecurrentBlock:
    """Host description of the shared SwiGLU block (keeps the ctypes structs and tensors alive).
    Each sublayer dict holds gain, wgu, wd (bf16), gu_q, d_q (packed NVFP4 weights), idx_gu,
    idx_d, and optionally gu_f8, d_f8 (FP8Tensor weights, needed by FP8 steps).
    residual_scale is the damped residual's beta and inject an optional bf16 [S, d] term e added to
    it (h <- beta h + e + F(h); 1 and None: the plain residual block)."""

    def __init__(self, d: int, ffn: int, eps: float, sublayers: list[dict], residual_scale: float = 1.0,
                 inject: torch.Tensor | None = None):
        self.d, self.ffn, self.eps = d, ffn, eps
        self.sub = sublayers
        arr = (SwigluSublayer * len(sublayers))()
        for i, L in enumerate(sublayers):
            f8g, f8d = L.get("gu_f8"), L.get("d_f8")
            arr[i] = SwigluSublayer(
                L["gain"].data_ptr(), L["wgu"].data_ptr(), L["wd"].data_ptr(),
                L["gu_q"].codes.data_ptr(), L["gu_q"].sf.data_ptr(), L["gu_q"].scale.data_ptr(),
                L["d_q"].codes.data_ptr(), L["d_q"].sf.data_ptr(), L["d_q"].scale.data_ptr(),
                L["idx_gu"].data_ptr(), int(L["idx_gu"].numel()), L["idx_d"].data_ptr(), int(L["idx_d"].numel()),
                f8g.codes.data_ptr() if f8g is not None else None, f8g.scale.data_ptr() if f8g is not None else None,
                f8d.codes.data_ptr() if f8d is not None else None, f8d.scale.data_ptr() if f8d is not None else None)
        self._arr = arr
        self._inject = inject
        self.block = SwigluBlock(d, ffn, float(eps), len(sublayers), arr, float(residual_scale),
                                 inject.data_ptr() if inject is not None else None)

    def workspace_bytes(self, S: int) -> int:
        return int(lib().arc_recurrent_workspace_bytes(S, ctypes.byref(self.block)))


def recurrent_prefill(h: torch.Tensor, block: RecurrentBlock, T: int, k_low: int,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """arc_recurrent_prefill: apply the block T times in place (steps < k_low in NVFP4 + ARC)."""
    S = h.shape[0]
    n = block.workspace_bytes(S)
    if workspace is None:
        workspace = _ws(n, h.device)
    _check("arc_recurrent_prefill", lib().arc_recurrent_prefill(_p(h), S, ctypes.byref(block.block), T, k_low,
                                                                _p(workspace), workspace.numel(), _stream(stream)))
    return h


def recurrent_prefill_schedule(h: torch.Tensor, block: RecurrentBlock, schedule, workspace: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """arc_recurrent_prefill_schedule: apply the block len(schedule) times in place; step t in
    the format schedule[t]: STEP_BF16 (0 / False), STEP_NVFP4 (1 / True) or STEP_FP8 (2)."""
    S = h.shape[0]
    flags = (ctypes.c_uint8 * max(1, len(schedule)))(*[int(f) for f in schedule])
    n = block.workspace_bytes(S)
    if workspace is None:
        workspace = _ws(n, h.device)
    _check("arc_recurrent_prefill_schedule", lib().arc_recurrent_prefill_schedule(
        _p(h), S, ctypes.byref(block.block), len(schedule), flags, _p(workspace), workspace.numel(),
        _stream(stream)))
    return h


@dataclass
class MXFP4Tensor:
    """Packed MXFP4 operand: codes [rows, K_pad/2] u8 and swizzled E8M0 scale bytes (no tensor scale)."""
    codes: torch.Tensor
    sf: torch.Tensor
    rows: int
    k_aug: int


def mxfp4_sf_bytes(rows: int, k_aug: int) -> int:
    return int(lib().arc_mxfp4_sf_bytes(rows, k_aug))


def _mx_out(rows, k_aug, device):
    return MXFP4Tensor(_u8(codes_bytes(rows, k_aug), device), _u8(mxfp4_sf_bytes(rows, k_aug), device), rows, k_aug)


def quantize_act_mxfp4(x: torch.Tensor, idx: torch.Tensor | None = None, out: MXFP4Tensor | None = None,
                       stream=None) -> MXFP4Tensor:
    """arc_quantize_act_mxfp4: X [M, K] bf16 -> MXFP4 with r appended residual channels."""
    _need_cuda(x, idx)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    r = 0 if idx is None else int(idx.numel())
    if out is None:
        out = _mx_out(M, K + r, x.device)
    _check("arc_quantize_act_mxfp4", lib().arc_quantize_act_mxfp4(_p(x), M, K, x.stride(0), _p(idx), r, _p(out.codes),
                                                                  _p(out.sf), _stream(stream)))
    return out


def pack_weight_mxfp4(w: torch.Tensor, idx: torch.Tensor | None = None, out: MXFP4Tensor | None = None,
                      stream=None) -> MXFP4Tensor:
    """arc_pack_weight_mxfp4: W [N, K] bf16 -> W_aug = [W | W[:, idx]] in MXFP4."""
    _need_cuda(w, idx)
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    N, K = w.shape
    r = 0 if idx is None else int(idx.numel())
    if out is None:
        out = _mx_out(N, K + r, w.device)
    _check("arc_pack_weight_mxfp4", lib().arc_pack_weight_mxfp4(_p(w), N, K, w.stride(0), _p(idx), r, _p(out.codes),
                                                                _p(out.sf), _stream(stream)))
    return out


def gemm_mxfp4(a: MXFP4Tensor, b: MXFP4Tensor, out: torch.Tensor | None = None, add: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """arc_gemm_mxfp4: Y [M, N] bf16 = MXFP4(A) MXFP4(B)^T over depth K_aug (+ add)."""
    assert a.k_aug == b.k_aug
    M, N = a.rows, b.rows
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.codes.device)
    _check("arc_gemm_mxfp4", lib().arc_gemm_mxfp4(
        _p(a.codes), _p(a.sf), _p(b.codes), _p(b.sf), M, N, a.k_aug, _p(out), out.stride(0), _p(add),
        0 if add is None else add.stride(0), _stream(stream)))
    return out


class FP8Tensor:
    """E4M3 codes [rows, K] (row stride K bytes) and the device fp32 tensor scale."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        self.codes, self.scale = codes, scale
        self.rows, self.k = codes.shape


def quantize_fp8(x: torch.Tensor, static_scale: torch.Tensor | None = None, out: FP8Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> FP8Tensor:
    """arc_quantize_fp8: X [M, K] bf16 -> E4M3 codes with one per-tensor scale (amax/448)."""
    _need_cuda(x, static_scale)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        out = FP8Tensor(torch.empty(M, K, dtype=torch.uint8, device=x.device),
                        torch.empty(1, dtype=torch.float32, device=x.device))
    if workspace is None:
        workspace = _ws(quantize_workspace_bytes(M, 0), x.device)
    _check("arc_quantize_fp8", lib().arc_quantize_fp8(_p(x), M, K, x.stride(0), _p(static_scale), _p(out.codes),
                                                      out.codes.stride(0), _p(out.scale), _p(workspace),
                                                      workspace.numel(), _stream(stream)))
    return out


def gemm_fp8(a: FP8Tensor, b: FP8Tensor, out: torch.Tensor | None = None, add: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """arc_gemm_fp8: Y [M, N] bf16 = s_A s_B * E4M3(A) E4M3(B)^T (+ add)."""
    assert a.k == b.k
    M, N, K = a.rows, b.rows, a.k
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.codes.device)
    _check("arc_gemm_fp8", lib().arc_gemm_fp8(
        _p(a.codes), a.codes.stride(0), _p(a.scale), _p(b.codes), b.codes.stride(0), _p(b.scale), M, N, K,
        _p(out), out.stride(0), _p(add), 0 if add is None else add.stride(0), _stream(stream)))
    return out


# ---------------------------------------------------------------------------------------------
# Mixture-of-experts layers
# ---------------------------------------------------------------------------------------------


def _pad64(n: int) -> int:
    return (n + 63) // 64 * 64


class ExpertPlan:
    """The slots (token * k + choice) sorted stably by expert: one int32 device buffer with the
    sections that include/arc.h describes, seen through offsets, blocks, row_of_slot, slot_of_row and
    sf_row. Made by expert_plan, or put around a buffer of that layout."""

    __slots__ = ("buf", "tokens", "k", "experts", "slots")

    def __init__(self, buf: torch.Tensor, tokens: int, k: int, experts: int):
        slots = tokens * k
        if (buf.dtype is not torch.int32 or not buf.is_contiguous() or
                buf.numel() < 2 * _pad64(experts + 1) + 3 * _pad64(slots)):
            raise ValueError("ExpertPlan: the buffer does not hold a plan of these sizes")
        self.buf, self.tokens, self.k, self.experts, self.slots = buf, tokens, k, experts, slots

    @property
    def offsets(self) -> torch.Tensor:
        return self.buf[:self.experts + 1]

    @property
    def blocks(self) -> torch.Tensor:
        at = _pad64(self.experts + 1)
        return self.buf[at:at + self.experts + 1]

    @property
    def row_of_slot(self) -> torch.Tensor:
        at = 2 * _pad64(self.experts + 1)
        return self.buf[at:at + self.slots]

    @property
    def slot_of_row(self) -> torch.Tensor:
        at = 2 * _pad64(self.experts + 1) + _pad64(self.slots)
        return self.buf[at:at + self.slots]

    @property
    def sf_row(self) -> torch.Tensor:
        at = 2 * _pad64(self.experts + 1) + 2 * _pad64(self.slots)
        return self.buf[at:at + self.slots]


class ExpertMXFP4:
    """Sorted rows in MXFP4 in one u8 device buffer: codes [S, K_pad/2] and, from the next multiple of
    256 bytes on, the scale bytes, whose 128-row blocks begin anew with every expert. k_aug = K + r."""

    __slots__ = ("buf", "rows", "k_aug", "sf_at")

    def __init__(self, buf: torch.Tensor, rows: int, k_aug: int):
        self.buf, self.rows, self.k_aug = buf, rows, k_aug
        self.sf_at = (rows * (_pad64(k_aug) // 2) + 255) // 256 * 256

    @property
    def codes(self) -> torch.Tensor:
        half = _pad64(self.k_aug) // 2
        return self.buf[:self.rows * half].view(self.rows, half)

    @property
    def sf(self) -> torch.Tensor:
        return self.buf[self.sf_at:]


@dataclass
class ExpertWeightMXFP4:
    """Packed weights of all experts: codes [E * N, K_pad/2] u8 and their scale bytes."""
    codes: torch.Tensor
    sf: torch.Tensor
    experts: int
    n: int
    k_aug: int


# The handles alone: building Stream objects would cost a small call a tenth of its time.
_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _refuse(fn: str, name: str, t: torch.Tensor, dtype, dev: int, shape):
    if not t.is_cuda:
        raise ValueError(f"{fn}: tensors must be CUDA tensors ({name} is on {t.device})")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on cuda:{dev}")
    if t.dtype != dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{fn}: {name} must be {list(shape)}, not {list(t.shape)}")
    raise ValueError(f"{fn}: {name} must hold consecutive values")


def _rows_of(fn: str, name: str, t: torch.Tensor, dtype, dev: int, shape: tuple) -> int:
    """The leading dimension of a [rows, cols] argument; refuses one of another device, dtype, shape
    or with strided rows. A single row has the row's length, whatever its stride says."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(fn, name, t, dtype, dev, shape)
    ld, step = t.stride()
    if step != 1 and shape[1] != 1:
        _refuse(fn, name, t, dtype, dev, shape)
    return ld if shape[0] > 1 else shape[1]


def _flat(fn: str, name: str, t: torch.Tensor, dtype, dev: int, least: int):
    """Refuses a buffer of another device or dtype, with gaps, or with fewer than `least` values."""
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        _refuse(fn, name, t, dtype, dev, None)
    if t.numel() < least:
        raise ValueError(f"{fn}: {name} holds {t.numel()} values, {least} are needed")


def _plan_ptr(fn: str, plan: ExpertPlan, dev: int) -> int:
    if plan.buf.get_device() != dev:
        _refuse(fn, "plan", plan.buf, _I32, dev, None)
    return plan.buf.data_ptr()


def _on(fn: str, dev: int, stream):
    """Context in which a call on tensors of device `dev` runs when that is not the current device or
    a stream is given: both become the current ones, so that outputs are allocated for them."""
    if dev < 0:
        raise ValueError(f"{fn}: tensors must be CUDA tensors")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    return torch.cuda.stream(stream)


def _new_plan(ids: torch.Tensor, tokens: int, k: int, experts: int) -> ExpertPlan:
    """An ExpertPlan around a new buffer, without the checks of one that a caller brings."""
    p, slots = ExpertPlan.__new__(ExpertPlan), tokens * k
    p.buf = ids.new_empty(2 * ((experts + 64) // 64 * 64) + 3 * ((slots + 63) // 64 * 64), dtype=_I32)
    p.tokens, p.k, p.experts, p.slots = tokens, k, experts, slots
    return p


def expert_plan(ids: torch.Tensor, experts: int, out: ExpertPlan | None = None, stream=None) -> ExpertPlan:
    """arc_expert_plan: the slots of expert ids [T, k] (int32 or int64) sorted by expert; ids outside
    [0, experts) give their slots no row."""
    fn, dev, dtype = "expert_plan", ids.get_device(), ids.dtype
    if (dtype is not torch.int32 and dtype is not torch.int64) or ids.dim() != 2:
        raise ValueError("expert_plan: ids must be [tokens, k] of int32 or int64")
    shape = ids.shape
    T, k = shape
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return expert_plan(ids, experts, out)
    ld = _rows_of(fn, "ids", ids, dtype, dev, shape)
    if out is None:
        out = _new_plan(ids, T, k, experts)
    elif (out.tokens, out.k, out.experts) != (T, k, experts):
        raise ValueError("expert_plan: out was made for other sizes")
    _check("arc_expert_plan", lib().arc_expert_plan(
        ids.data_ptr(), 4 if dtype is _I32 else 8, ld, T, k, experts, _plan_ptr(fn, out, dev), out.buf.numel() * 4,
        _raw_stream(dev)))
    return out


def dispatch_experts(x: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """arc_dispatch_experts_bf16: tokens x [T, d] bf16 copied into sorted order [S, d]."""
    fn, dev, d, T, k = "dispatch_experts", x.get_device(), x.shape[-1], plan.tokens, plan.k
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return dispatch_experts(x, plan, out)
    ld = _rows_of(fn, "x", x, _BF16, dev, (T, d))
    if out is None:
        out, ld_out = x.new_empty(T * k, d), d
    else:
        ld_out = _rows_of(fn, "out", out, _BF16, dev, (T * k, d))
    _check("arc_dispatch_experts_bf16", lib().arc_dispatch_experts_bf16(
        x.data_ptr(), ld, d, _plan_ptr(fn, plan, dev), T, k, plan.experts, out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def dispatch_experts_grad(d_rows: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """arc_dispatch_experts_grad_bf16: the tokens' gradient [T, d] from the sorted rows' [S, d]."""
    fn, dev, d, T, k = "dispatch_experts_grad", d_rows.get_device(), d_rows.shape[-1], plan.tokens, plan.k
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return dispatch_experts_grad(d_rows, plan, out)
    ld = _rows_of(fn, "d_rows", d_rows, _BF16, dev, (T * k, d))
    if out is None:
        out, ld_out = d_rows.new_empty(T, d), d
    else:
        ld_out = _rows_of(fn, "out", out, _BF16, dev, (T, d))
    _check("arc_dispatch_experts_grad_bf16", lib().arc_dispatch_experts_grad_bf16(
        d_rows.data_ptr(), ld, d, _plan_ptr(fn, plan, dev), T, k, plan.experts, out.data_ptr(), ld_out,
        _raw_stream(dev)))
    return out


def combine_experts(rows: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan, add: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """arc_combine_experts_bf16: y [T, d] = sum over the token's choices of weights [T, k] (fp32) times
    the sorted rows [S, d] (+ add [T, d])."""
    fn, dev, d, T, k = "combine_experts", rows.get_device(), rows.shape[-1], plan.tokens, plan.k
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return combine_experts(rows, weights, plan, add, out)
    ld = _rows_of(fn, "rows", rows, _BF16, dev, (T * k, d))
    ld_w = _rows_of(fn, "weights", weights, _F32, dev, (T, k))
    if out is None:
        out, ld_out = rows.new_empty(T, d), d
    else:
        ld_out = _rows_of(fn, "out", out, _BF16, dev, (T, d))
    _check("arc_combine_experts_bf16", lib().arc_combine_experts_bf16(
        rows.data_ptr(), ld, d, weights.data_ptr(), ld_w, _plan_ptr(fn, plan, dev), T, k, plan.experts,
        None if add is None else add.data_ptr(), 0 if add is None else _rows_of(fn, "add", add, _BF16, dev, (T, d)),
        out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def combine_experts_grad(d_y: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan,
                         d_rows: torch.Tensor | None = None, d_weights: torch.Tensor | None = None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """arc_combine_experts_grad_bf16: (d_rows [S, d] bf16, d_weights [T, k] fp32) from d_y [T, d];
    d_rows may be rows."""
    fn, dev, d, T, k = "combine_experts_grad", rows.get_device(), rows.shape[-1], plan.tokens, plan.k
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return combine_experts_grad(d_y, rows, weights, plan, d_rows, d_weights)
    ld_dy = _rows_of(fn, "d_y", d_y, _BF16, dev, (T, d))
    ld = _rows_of(fn, "rows", rows, _BF16, dev, (T * k, d))
    ld_w = _rows_of(fn, "weights", weights, _F32, dev, (T, k))
    if d_rows is None:
        d_rows = rows.new_empty(T * k, d)
    if d_weights is None:
        d_weights = weights.new_empty(T, k)
    _check("arc_combine_experts_grad_bf16", lib().arc_combine_experts_grad_bf16(
        d_y.data_ptr(), ld_dy, rows.data_ptr(), ld, d, weights.data_ptr(), ld_w, _plan_ptr(fn, plan, dev), T, k,
        plan.experts, d_rows.data_ptr(), _rows_of(fn, "d_rows", d_rows, _BF16, dev, (T * k, d)),
        d_weights.data_ptr(), _rows_of(fn, "d_weights", d_weights, _F32, dev, (T, k)), _raw_stream(dev)))
    return d_rows, d_weights


def _expert_sf_bytes(plan: ExpertPlan, k_aug: int) -> int:
    S = plan.tokens * plan.k
    return (S + 127 * min(plan.experts, S)) // 128 * 1024 * ((_pad64(k_aug) + 255) // 256)


def _expert_quantize(fn: str, call, x: torch.Tensor, plan: ExpertPlan, K: int, idx, out: ExpertMXFP4 | None, stream,
                     rows: int):
    dev, S = x.get_device(), plan.slots
    r = 0 if idx is None else idx.numel()
    kp = _pad64(K + r)
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return _expert_quantize(fn, call, x, plan, K, idx, out, None, rows)
    ld = _rows_of(fn, "x" if rows == plan.tokens else "gu", x, _BF16, dev, (rows, x.shape[-1]))
    if idx is not None:
        _flat(fn, "idx", idx, _I32, dev, r)
    nsf = _expert_sf_bytes(plan, K + r)
    if out is None:
        out = ExpertMXFP4(x.new_empty((S * (kp // 2) + 255) // 256 * 256 + nsf, dtype=_U8), S, K + r)
    else:
        if out.rows != S or out.k_aug != K + r:
            raise ValueError(f"{fn}: out was made for other sizes")
        _flat(fn, "out", out.buf, _U8, dev, out.sf_at + nsf)
    codes = out.buf.data_ptr()
    _check("arc_" + fn, call(x.data_ptr(), ld, K, None if idx is None else idx.data_ptr(), r, _plan_ptr(fn, plan, dev),
                             plan.tokens, plan.k, plan.experts, codes, codes + out.sf_at, _raw_stream(dev)))
    return out


def quantize_act_experts_mxfp4(x: torch.Tensor, plan: ExpertPlan, idx: torch.Tensor | None = None,
                               out: ExpertMXFP4 | None = None, stream=None) -> ExpertMXFP4:
    """arc_quantize_act_experts_mxfp4: tokens x [T, K] bf16 in MXFP4 with r appended residual channels,
    written to their sorted rows."""
    return _expert_quantize("quantize_act_experts_mxfp4", lib().arc_quantize_act_experts_mxfp4, x, plan, x.shape[-1],
                            idx, out, stream, plan.tokens)


def quantize_swiglu_experts_mxfp4(gu: torch.Tensor, plan: ExpertPlan, idx: torch.Tensor | None = None,
                                  out: ExpertMXFP4 | None = None, stream=None) -> ExpertMXFP4:
    """arc_quantize_swiglu_experts_mxfp4: silu(gate) * up of the sorted rows gu [S, 2F], in MXFP4."""
    if gu.shape[-1] % 2:
        raise ValueError("quantize_swiglu_experts_mxfp4: gu must have as many gate as up columns")
    return _expert_quantize("quantize_swiglu_experts_mxfp4", lib().arc_quantize_swiglu_experts_mxfp4, gu, plan,
                            gu.shape[-1] // 2, idx, out, stream, plan.slots)


def _expert_weight_ld(fn: str, w: torch.Tensor, dev: int, E: int, N: int, K: int) -> int:
    if w.get_device() != dev or w.dtype is not _BF16 or w.shape != (E, N, K) or (w.stride(2) != 1 and K != 1):
        _refuse(fn, "w", w, _BF16, dev, (E, N, K))
    ld = w.stride(1) if N > 1 else (w.stride(0) if E > 1 else K)
    if E > 1 and w.stride(0) != N * ld:
        raise ValueError(f"{fn}: the experts' weights must lie one after another")
    return ld


def pack_weight_experts_mxfp4(w: torch.Tensor, idx: torch.Tensor | None = None, out: ExpertWeightMXFP4 | None = None,
                              stream=None) -> ExpertWeightMXFP4:
    """arc_pack_weight_experts_mxfp4: W [E, N, K] bf16 (experts one after another) -> MXFP4 of
    [W_e | W_e[:, idx]] for every expert."""
    fn, dev = "pack_weight_experts_mxfp4", w.get_device()
    if w.dim() != 3:
        raise ValueError("pack_weight_experts_mxfp4: w must be [experts, N, K]")
    E, N, K = w.shape
    r = 0 if idx is None else idx.numel()
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return pack_weight_experts_mxfp4(w, idx, out)
    ld = _expert_weight_ld(fn, w, dev, E, N, K)
    if idx is not None:
        _flat(fn, "idx", idx, _I32, dev, r)
    kp, nsf = _pad64(K + r), E * mxfp4_sf_bytes(N, K + r)
    if out is None:
        out = ExpertWeightMXFP4(torch.empty((E * N, kp // 2), dtype=_U8, device=w.device),
                                torch.empty(nsf, dtype=_U8, device=w.device), E, N, K + r)
    else:
        if (out.experts, out.n, out.k_aug) != (E, N, K + r):
            raise ValueError("pack_weight_experts_mxfp4: out was made for other sizes")
        _flat(fn, "out.codes", out.codes, _U8, dev, E * N * kp // 2)
        _flat(fn, "out.sf", out.sf, _U8, dev, nsf)
    _check("arc_pack_weight_experts_mxfp4", lib().arc_pack_weight_experts_mxfp4(
        w.data_ptr(), E, N, K, ld, None if idx is None else idx.data_ptr(), r, out.codes.data_ptr(),
        out.sf.data_ptr(), _raw_stream(dev)))
    return out


def gemm_experts_mxfp4(a: ExpertMXFP4, w: ExpertWeightMXFP4, plan: ExpertPlan, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """arc_gemm_experts_mxfp4: Y [S, N] bf16 = each sorted row times its expert's weights."""
    fn, dev, S, n, ka = "gemm_experts_mxfp4", a.buf.get_device(), plan.slots, w.n, a.k_aug
    if ka != w.k_aug or w.experts != plan.experts or a.rows != S:
        raise ValueError("gemm_experts_mxfp4: operands of other sizes than the plan's, or of two depths")
    kp = _pad64(ka)
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return gemm_experts_mxfp4(a, w, plan, out)
    _flat(fn, "a", a.buf, _U8, dev, a.sf_at + _expert_sf_bytes(plan, ka))
    _flat(fn, "w.codes", w.codes, _U8, dev, w.experts * n * kp // 2)
    _flat(fn, "w.sf", w.sf, _U8, dev, w.experts * ((n + 127) // 128) * ((kp + 127) // 128) * 512)
    if out is None:
        out, ld_out = a.buf.new_empty(S, n, dtype=_BF16), n
    else:
        ld_out = _rows_of(fn, "out", out, _BF16, dev, (S, n))
    codes = a.buf.data_ptr()
    _check("arc_gemm_experts_mxfp4", lib().arc_gemm_experts_mxfp4(
        codes, codes + a.sf_at, w.codes.data_ptr(), w.sf.data_ptr(), _plan_ptr(fn, plan, dev), plan.tokens,
        plan.k, plan.experts, n, ka, out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def gemm_experts_bf16(rows: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """arc_gemm_experts_bf16: Y [S, N] = bf16 of each sorted row [S, K] times its expert's W [E, N, K]."""
    fn, dev, S, K = "gemm_experts_bf16", rows.get_device(), plan.tokens * plan.k, rows.shape[-1]
    if w.dim() != 3:
        raise ValueError("gemm_experts_bf16: w must be [experts, N, K]")
    N = w.shape[1]
    if stream is not None or dev < 0 or dev != _device():
        with _on(fn, dev, stream):
            return gemm_experts_bf16(rows, w, plan, out)
    ld = _rows_of(fn, "rows", rows, _BF16, dev, (S, K))
    ld_w = _expert_weight_ld(fn, w, dev, plan.experts, N, K)
    if out is None:
        out, ld_out = rows.new_empty(S, N), N
    else:
        ld_out = _rows_of(fn, "out", out, _BF16, dev, (S, N))
    _check("arc_gemm_experts_bf16", lib().arc_gemm_experts_bf16(
        rows.data_ptr(), ld, w.data_ptr(), ld_w, _plan_ptr(fn, plan, dev), plan.tokens, plan.k, plan.experts, N, K,
        out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def last_device_status(stream=None) -> int:
    return int(lib().arc_last_device_status(_stream(stream)))


def set_wait_limit_ns(ns: int):
    _check("arc_set_wait_limit_ns", lib().arc_set_wait_limit_ns(int(ns)))


def debug_inject(kind: int):
    _check("arc_debug_inject", lib().arc_debug_inject(int(kind)))
