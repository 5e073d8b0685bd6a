"""Python binding of libqlora_nf4, the gfx950 QLoRA NF4 linear-layer library.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch supplies device memory (outputs and workspaces are allocated
here with torch.empty) and the current stream.  The functions carry the names
of the C entry points in include/qlora_nf4.h.

If the shared library has not been built, every entry point raises; there is
no fallback implementation.
"""
import ctypes
import functools
import os
from typing import NamedTuple, Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")

QLORA_OK = 0
QLORA_ERR_SCRATCH = 7
QLORA_ERR_FORMAT = 8
CODEBOOKS = {"nf4": 0, "int4": 1, "fp4": 2}   # qlora_codebook of the header
SCORES = {"softmax": 0, "sigmoid": 1}         # qlora_score of the header
NOALLOC_SCRATCH_BYTES = 32 << 20   # QLORA_NOALLOC_SCRATCH_BYTES of the header
_lib = None


class _Nf4Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("absmax_scale", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class _Q4Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("absmax_scale", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("codebook", ctypes.c_int32),
                ("double_quant", ctypes.c_int32)]


class _Dropout(ctypes.Structure):
    _fields_ = [("state", ctypes.c_void_p), ("p", ctypes.c_float)]


class _Act8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class _RouterConfig(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("topk", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class _AdamWConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


_SIGS = {
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_version": (ctypes.c_char_p, []),
    "qlora_nf4_levels": (ctypes.c_int, [ctypes.c_void_p]),
    "qlora_nf4_thresholds": (ctypes.c_int, [ctypes.c_void_p]),
    "qlora_nf4_codes_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "qlora_nf4_absmax_q_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "qlora_nf4_scale_count": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "qlora_nf4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "qlora_nf4_dequantize": (ctypes.c_int, [ctypes.POINTER(_Nf4Weight), ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "qlora_linear_fwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                           ctypes.c_int64, ctypes.c_int]),
    "qlora_linear_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_Nf4Weight), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                ctypes.POINTER(_Nf4Weight), ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                                ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_void_p]),
    "qlora_linear_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                           ctypes.c_int64, ctypes.c_int]),
    "qlora_linear_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_Nf4Weight), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "qlora_block_fwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int,
                                                          ctypes.c_int64, ctypes.c_int64,
                                                          ctypes.c_int]),
    "qlora_block_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Nf4Weight),
                                       ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "qlora_block_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int,
                                                          ctypes.c_int64, ctypes.c_int64,
                                                          ctypes.c_int]),
    "qlora_block_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.POINTER(_Nf4Weight), ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "qlora_lora16_fwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                           ctypes.c_int64, ctypes.c_int]),
    "qlora_lora16_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                           ctypes.c_int64, ctypes.c_int]),
    "qlora_lora16_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_lora16_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_q4_levels": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p]),
    "qlora_q4_thresholds": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p]),
    "qlora_q4_scale_count": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_q4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_q4_dequantize": (ctypes.c_int, [ctypes.POINTER(_Q4Weight), ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "qlora_q4_linear_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.POINTER(_Q4Weight), ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_q4_linear_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.POINTER(_Q4Weight), ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p]),
    "qlora_dropout_apply": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.POINTER(_Dropout), ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "qlora_linear_dropout_fwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_linear_dropout_bwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_linear_dropout_fwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Q4Weight), ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(_Dropout), ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear_dropout_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Q4Weight),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(_Dropout),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_grouped_fwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_grouped_bwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_grouped_fwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
        ctypes.POINTER(_Q4Weight), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
        ctypes.POINTER(_Dropout), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_grouped_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
        ctypes.POINTER(_Q4Weight), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
        ctypes.POINTER(_Dropout), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_expert_plan_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "qlora_expert_plan": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_expert_gather": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_expert_combine": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_expert_combine_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_act8_pack": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_Act8), ctypes.c_void_p]),
    "qlora_act8_unpack": (ctypes.c_int, [
        ctypes.POINTER(_Act8), ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_linear_act8_bwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_grouped_act8_bwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "qlora_linear_act8_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.POINTER(_Act8), ctypes.c_int64, ctypes.POINTER(_Q4Weight),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(_Dropout),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_grouped_act8_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.POINTER(_Act8), ctypes.c_int64, ctypes.c_void_p, ctypes.c_int,
        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(_Q4Weight),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(_Dropout),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_rms_norm_fwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.POINTER(_Act8), ctypes.c_void_p]),
    "qlora_rms_norm_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "qlora_rms_norm_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_router_fwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
        ctypes.POINTER(_RouterConfig), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_router_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
        ctypes.c_int, ctypes.POINTER(_RouterConfig), ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_adamw_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_AdamWConfig), ctypes.c_int64,
                                        ctypes.c_void_p]),
    "qlora_paged_state_create": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int,
                                                ctypes.POINTER(ctypes.c_void_p)]),
    "qlora_paged_state_destroy": (ctypes.c_int, [ctypes.c_void_p]),
    "qlora_paged_state_page_out": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_paged_state_page_in": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_paged_state_pointers": (ctypes.c_int, [ctypes.c_void_p,
                                                  ctypes.POINTER(ctypes.c_void_p),
                                                  ctypes.POINTER(ctypes.c_void_p)]),
    "qlora_paged_state_resident": (ctypes.c_int, [ctypes.c_void_p]),
    "qlora_paged_state_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "qlora_paged_state_write": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "qlora_probe_hbm_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                            ctypes.c_int, ctypes.c_void_p]),
    "qlora_probe_mfma_bf16": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_void_p]),
    "qlora_profile_enable": (ctypes.c_int, [ctypes.c_int]),
    "qlora_profile_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(ctypes.c_int64)]),
    "qlora_profile_reset": (ctypes.c_int, []),
}

EXPORTED = tuple(_SIGS)


def lib():
    """Load libqlora_nf4.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_fine_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().qlora_status_string(status).decode()


class QloraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")
        self.status = status


def _check(fn: str, status: int):
    if status != QLORA_OK:
        raise QloraError(fn, status)


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtype):
    """The C entry points trust their pointers to hold the documented
    [rows, cols] layout, so tensors are checked here before a call: first
    dtype, shape and contiguity of every argument, then (_on_gpu) that all
    of them sit on the same GPU."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(named):
    """named: (name, tensor or None) pairs; the first tensor's GPU is the one."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _check_weight(w):
    import torch
    n_codes, n_blocks = w.N * w.K // 2, w.N * w.K // 64
    _need(w.codes, "w.codes", (n_codes,), torch.uint8)
    _need(w.absmax_q, "w.absmax_q", (n_blocks,), torch.uint8)
    _need(w.absmax_scale, "w.absmax_scale", ((n_blocks + 255) // 256,), torch.float32)
    return [("w.codes", w.codes), ("w.absmax_q", w.absmax_q),
            ("w.absmax_scale", w.absmax_scale)]


def _check_adapters(A, B, w):
    import torch
    if A is None or B is None:
        if A is not None or B is not None:
            raise ValueError("A and B go together (both None selects r = 0)")
        return 0
    if A.dim() != 2:
        raise ValueError("A must be [K, r]")
    r = A.shape[1]
    _is(A, "A", (w.K, r), torch.bfloat16)
    _is(B, "B", (r, w.N), torch.bfloat16)
    return r


class NF4Weight(NamedTuple):
    codes: "torch.Tensor"          # uint8 [N*K/2]
    absmax_q: "torch.Tensor"       # uint8 [N*K/64]
    absmax_scale: "torch.Tensor"   # float32 [ceil(N*K/16384)]
    N: int
    K: int

    def _c(self) -> _Nf4Weight:
        return _Nf4Weight(self.codes.data_ptr(), self.absmax_q.data_ptr(),
                          self.absmax_scale.data_ptr(), self.N, self.K)

    def nbytes(self) -> int:
        return (self.codes.numel() + self.absmax_q.numel()
                + 4 * self.absmax_scale.numel())


def qlora_nf4_levels():
    """The 16 NF4 levels (list of float)."""
    buf = (ctypes.c_float * 16)()
    _check("qlora_nf4_levels", lib().qlora_nf4_levels(buf))
    return list(buf)


def qlora_nf4_thresholds():
    buf = (ctypes.c_float * 15)()
    _check("qlora_nf4_thresholds", lib().qlora_nf4_thresholds(buf))
    return list(buf)


def qlora_nf4_quantize(W, out: Optional[NF4Weight] = None) -> NF4Weight:
    """Quantize a float32 [N, K] CUDA tensor to NF4 + double-quantized constants."""
    import torch
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    _need(W, "W", (N, K), torch.float32)
    if out is not None and (out.N, out.K) != (N, K):
        raise ValueError(f"out is a {out.N} x {out.K} weight, W is {N} x {K}")
    _on_gpu([("W", W)] + (_check_weight(out) if out is not None else []))
    L = lib()
    if out is None:
        out = NF4Weight(
            torch.empty(L.qlora_nf4_codes_bytes(N, K), dtype=torch.uint8, device=W.device),
            torch.empty(L.qlora_nf4_absmax_q_bytes(N, K), dtype=torch.uint8, device=W.device),
            torch.empty(L.qlora_nf4_scale_count(N, K), dtype=torch.float32, device=W.device),
            N, K)
    _check("qlora_nf4_quantize",
           L.qlora_nf4_quantize(_ptr(W), N, K, _ptr(out.codes), _ptr(out.absmax_q),
                                _ptr(out.absmax_scale), _stream(W)))
    return out


def qlora_nf4_dequantize(w: NF4Weight):
    """bf16 [N, K] dequantized copy of an NF4 weight."""
    import torch
    _on_gpu(_check_weight(w))
    out = torch.empty((w.N, w.K), dtype=torch.bfloat16, device=w.codes.device)
    cw = w._c()
    _check("qlora_nf4_dequantize",
           lib().qlora_nf4_dequantize(ctypes.byref(cw), _ptr(out), _stream(out)))
    return out


def _ws(nbytes: int, device):
    import torch
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _fwd(fn, X, w, wt, cw, A, B, s, Y, T, workspace):
    """Marshal a forward call: fn is the C entry point's name, wt the weight's
    tensors (checked), cw its C struct."""
    import torch
    M = X.shape[0]
    r = _check_adapters(A, B, w)
    if Y is not None:
        _need(Y, "Y", (M, w.N), torch.bfloat16)
    if T is not None and r > 0:
        _need(T, "T", (M, r), torch.float32)
    if workspace is not None:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8)
    _on_gpu([("X", X)] + wt + [("A", A), ("B", B), ("Y", Y), ("T", T if r > 0 else None),
                               ("workspace", workspace)])
    dev = X.device
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    if T is None and r > 0:
        T = torch.empty((M, r), dtype=torch.float32, device=dev)
    need = lib().qlora_linear_fwd_workspace_bytes(M, w.N, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, X.device)
    _check(fn, getattr(lib(), fn)(_ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r, float(s),
                                  _ptr(Y), _ptr(T), _ptr(workspace), need, _stream(X)))
    return Y, T


def _x_rows(X, K):
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    _need(X, "X", (X.shape[0], K), torch.bfloat16)
    return X.shape[0]


def qlora_linear_fwd(X, w: NF4Weight, A=None, B=None, s: float = 1.0,
                     Y=None, T=None, workspace=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Y = X . deq(W)^T + s . (X . A) . B.  Returns (Y bf16 [M,N], T fp32 [M,r])."""
    _x_rows(X, w.K)
    return _fwd("qlora_linear_fwd", X, w, _check_weight(w), w._c(), A, B, s, Y, T, workspace)


def qlora_linear_fwd_noalloc(X, w: NF4Weight, A=None, B=None, s: float = 1.0,
                             Y=None, T=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """qlora_linear_fwd on the library's fixed per-GPU scratch instead of a
    workspace (for callers that cannot allocate device memory; pass Y and T
    to keep this call allocation-free on the Python side too).  Calls that
    overlap on one GPU race on that scratch."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    _need(X, "X", (M, w.K), torch.bfloat16)
    wt = _check_weight(w)
    r = _check_adapters(A, B, w)
    if Y is not None:
        _need(Y, "Y", (M, w.N), torch.bfloat16)
    if T is not None and r > 0:
        _need(T, "T", (M, r), torch.float32)
    _on_gpu([("X", X)] + wt + [("A", A), ("B", B), ("Y", Y), ("T", T if r > 0 else None)])
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    if T is None and r > 0:
        T = torch.empty((M, r), dtype=torch.float32, device=X.device)
    cw = w._c()
    _check("qlora_linear_fwd_noalloc",
           lib().qlora_linear_fwd_noalloc(_ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r,
                                          float(s), _ptr(Y), _ptr(T), _stream(X)))
    return Y, T


def _bwd(fn, dY, X, w, wt, cw, A, B, s, T, need_dx, dX, dA, dB, workspace):
    """Marshal a backward call (as _fwd)."""
    import torch
    M = X.shape[0]
    _need(dY, "dY", (M, w.N), torch.bfloat16)
    r = _check_adapters(A, B, w)
    if T is not None and r > 0:
        _need(T, "T", (M, r), torch.float32)
    if need_dx and dX is not None:
        _need(dX, "dX", (M, w.K), torch.bfloat16)
    if r > 0 and dA is not None:
        _need(dA, "dA", (w.K, r), torch.bfloat16)
    if r > 0 and dB is not None:
        _need(dB, "dB", (r, w.N), torch.bfloat16)
    if workspace is not None:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8)
    _on_gpu([("X", X), ("dY", dY)] + wt +
            [("A", A), ("B", B), ("T", T if r > 0 else None),
             ("dX", dX if need_dx else None), ("dA", dA if r > 0 else None),
             ("dB", dB if r > 0 else None), ("workspace", workspace)])
    dev = X.device
    if need_dx and dX is None:
        dX = torch.empty((M, w.K), dtype=torch.bfloat16, device=dev)
    if r > 0:
        if dA is None:
            dA = torch.empty((w.K, r), dtype=torch.bfloat16, device=dev)
        if dB is None:
            dB = torch.empty((r, w.N), dtype=torch.bfloat16, device=dev)
    need = lib().qlora_linear_bwd_workspace_bytes(M, w.N, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    _check(fn, getattr(lib(), fn)(_ptr(dY), _ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r,
                                  float(s), _ptr(T), _ptr(dX if need_dx else None), _ptr(dA),
                                  _ptr(dB), _ptr(workspace), need, _stream(X)))
    return (dX if need_dx else None), dA, dB


def qlora_linear_bwd(dY, X, w: NF4Weight, A=None, B=None, s: float = 1.0, T=None,
                     need_dx: bool = True, dX=None, dA=None, dB=None, workspace=None):
    """Returns (dX bf16 [M,K] or None, dA bf16 [K,r], dB bf16 [r,N]).

    T is the forward's T = X . A; None recomputes it (gradient checkpointing).
    """
    _x_rows(X, w.K)
    return _bwd("qlora_linear_bwd", dY, X, w, _check_weight(w), w._c(), A, B, s, T, need_dx,
                dX, dA, dB, workspace)


class Q4Weight(NamedTuple):
    """A 4-bit weight of any codebook: with double quantization the NF4
    format's constants, else absmax_q is None and absmax_scale holds one
    fp32 absmax per 64-block."""
    codes: "torch.Tensor"                    # uint8 [N*K/2]
    absmax_q: Optional["torch.Tensor"]       # uint8 [N*K/64], or None
    absmax_scale: "torch.Tensor"             # float32 [ceil(N*K/16384)] or [N*K/64]
    N: int
    K: int
    codebook: str                            # "nf4", "int4" or "fp4"
    double_quant: bool

    def _c(self) -> _Q4Weight:
        return _Q4Weight(self.codes.data_ptr(),
                         self.absmax_q.data_ptr() if self.absmax_q is not None else None,
                         self.absmax_scale.data_ptr(), self.N, self.K,
                         CODEBOOKS[self.codebook], int(self.double_quant))

    def nbytes(self) -> int:
        return (self.codes.numel() + (self.absmax_q.numel() if self.absmax_q is not None else 0)
                + 4 * self.absmax_scale.numel())


def _codebook_id(codebook: str) -> int:
    if codebook not in CODEBOOKS:
        raise ValueError(f"codebook must be one of {sorted(CODEBOOKS)}, got {codebook!r}")
    return CODEBOOKS[codebook]


def _check_q4_weight(w: Q4Weight):
    import torch
    _codebook_id(w.codebook)
    n_codes, n_blocks = w.N * w.K // 2, w.N * w.K // 64
    _need(w.codes, "w.codes", (n_codes,), torch.uint8)
    if w.double_quant:
        _need(w.absmax_q, "w.absmax_q", (n_blocks,), torch.uint8)
        _need(w.absmax_scale, "w.absmax_scale", ((n_blocks + 255) // 256,), torch.float32)
    else:
        _need(w.absmax_scale, "w.absmax_scale", (n_blocks,), torch.float32)
    return [("w.codes", w.codes), ("w.absmax_q", w.absmax_q),
            ("w.absmax_scale", w.absmax_scale)]


def qlora_q4_levels(codebook: str = "nf4"):
    """The 16 levels of a codebook (list of float)."""
    buf = (ctypes.c_float * 16)()
    _check("qlora_q4_levels", lib().qlora_q4_levels(_codebook_id(codebook), buf))
    return list(buf)


def qlora_q4_thresholds(codebook: str = "nf4"):
    """The 15 quantizer thresholds of a codebook (code = #{j : x > t_j})."""
    buf = (ctypes.c_float * 15)()
    _check("qlora_q4_thresholds", lib().qlora_q4_thresholds(_codebook_id(codebook), buf))
    return list(buf)


def qlora_q4_quantize(W, codebook: str = "nf4", double_quant: bool = True) -> Q4Weight:
    """Quantize a float32 [N, K] CUDA tensor with a codebook ("nf4", "int4",
    "fp4"), with double-quantized or fp32 block constants."""
    import torch
    cb = _codebook_id(codebook)
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    _need(W, "W", (N, K), torch.float32)
    _on_gpu([("W", W)])
    L = lib()
    dq = bool(double_quant)
    out = Q4Weight(
        torch.empty(L.qlora_nf4_codes_bytes(N, K), dtype=torch.uint8, device=W.device),
        torch.empty(L.qlora_nf4_absmax_q_bytes(N, K), dtype=torch.uint8, device=W.device)
        if dq else None,
        torch.empty(L.qlora_q4_scale_count(N, K, int(dq)), dtype=torch.float32, device=W.device),
        N, K, codebook, dq)
    _check("qlora_q4_quantize",
           L.qlora_q4_quantize(_ptr(W), N, K, cb, int(dq), _ptr(out.codes), _ptr(out.absmax_q),
                               _ptr(out.absmax_scale), _stream(W)))
    return out


def qlora_q4_dequantize(w: Q4Weight):
    """bf16 [N, K] dequantized copy of a 4-bit weight."""
    import torch
    _on_gpu(_check_q4_weight(w))
    out = torch.empty((w.N, w.K), dtype=torch.bfloat16, device=w.codes.device)
    cw = w._c()
    _check("qlora_q4_dequantize",
           lib().qlora_q4_dequantize(ctypes.byref(cw), _ptr(out), _stream(out)))
    return out


def qlora_q4_linear_fwd(X, w: Q4Weight, A=None, B=None, s: float = 1.0, Y=None, T=None,
                        workspace=None):
    """qlora_linear_fwd for a weight of any codebook and constant format."""
    _x_rows(X, w.K)
    return _fwd("qlora_q4_linear_fwd", X, w, _check_q4_weight(w), w._c(), A, B, s, Y, T,
                workspace)


def qlora_q4_linear_bwd(dY, X, w: Q4Weight, A=None, B=None, s: float = 1.0, T=None,
                        need_dx: bool = True, dX=None, dA=None, dB=None, workspace=None):
    """qlora_linear_bwd for a weight of any codebook and constant format."""
    _x_rows(X, w.K)
    return _bwd("qlora_q4_linear_bwd", dY, X, w, _check_q4_weight(w), w._c(), A, B, s, T,
                need_dx, dX, dA, dB, workspace)


# ---------------------------------------------------------------------------
# Dropout, layers grouped by expert and the exchange around them.  The same
# checks as above; as their smallest calls run for a few microseconds on the
# GPU, they are written to cost little on the host: one comparison a property,
# names and messages only where something is wrong.
# ---------------------------------------------------------------------------

def _is(t, name, shape, dtype):
    """_need for a torch.Size or tuple of ints."""
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _need(t, name, shape, dtype)


def _maybe(t, name, shape, dtype):
    if t is not None:
        _is(t, name, shape, dtype)


def _one_gpu(names, *tensors):
    """The GPU of all tensors given (None where an argument is absent); names
    holds theirs, separated by spaces."""
    dev = index = None
    for t in tensors:
        if t is not None:
            i = t.get_device()   # -1: not on a GPU
            if dev is None:
                dev, index = t.device, i
            if i != index or i < 0:
                _on_gpu(zip(names.split(), tensors))
    return dev


def _call(fn, dev, *args):
    """Call a C entry point on dev's current stream, with dev current."""
    import torch
    f = getattr(_lib or lib(), fn)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch._C._cuda_getDevice():
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != QLORA_OK:
        raise QloraError(fn, st)


def _at(t):
    """A tensor's address for a ctypes pointer argument."""
    return None if t is None else t.data_ptr()


def _q4(w):
    """The C view of an NF4Weight (or any object with its fields) or a Q4Weight,
    and its checked tensors."""
    import torch
    if isinstance(w, Q4Weight):   # (unpacked: half the time of reading the fields)
        codes, q, scale, N, K, book, dq = w
    else:
        book, dq = "nf4", True
        if isinstance(w, NF4Weight):
            codes, q, scale, N, K = w
        else:
            codes, q, scale, N, K = w.codes, w.absmax_q, w.absmax_scale, w.N, w.K
    n = N * K
    nb = n // 64
    cb = CODEBOOKS[book] if book in CODEBOOKS else _codebook_id(book)
    _is(codes, "w.codes", (n // 2,), torch.uint8)
    if dq:
        _is(q, "w.absmax_q", (nb,), torch.uint8)
        _is(scale, "w.absmax_scale", ((nb + 255) // 256,), torch.float32)
    else:
        _is(scale, "w.absmax_scale", (nb,), torch.float32)
        q = None
    return (_Q4Weight(codes.data_ptr(), _at(q), scale.data_ptr(), N, K, cb, 1 if dq else 0),
            codes, q, scale)


def _drop(p, state):
    """The C descriptor of dropout with probability p; state is an int64 [2]
    tensor {seed, offset} on the GPU (the 64-bit words as they are) and may be
    None when p is 0."""
    import torch
    if state is None:
        if p != 0:
            raise ValueError("state is required for p > 0")
        return _Dropout(None, p)
    _is(state, "state", (2,), torch.int64)
    return _Dropout(state.data_ptr(), p)


def _int32(names, *values):
    """Refuses numbers that ctypes would take modulo 2^32; names holds theirs,
    separated by spaces."""
    if max(values) >= 1 << 31 or min(values) < -1 << 31:
        for name, v in zip(names.split(), values):
            if not -1 << 31 <= v < 1 << 31:
                raise ValueError(f"{name} = {v} does not fit 32 bits")


def _scratch(workspace, need, dev):
    """The caller's workspace if it is large enough, else one of need bytes."""
    import torch
    if workspace is not None:
        _is(workspace, "workspace", (workspace.numel(),), torch.uint8)
        if workspace.numel() >= need:
            return workspace
    return _ws(need, dev)


def qlora_dropout(x, p: float, state, out=None):
    """x with its elements dropped with probability p and the rest scaled by
    1 / (1 - p) (to 16 bits of p): bf16, any shape, contiguous; the mask is a
    function of state (int64 [2] on the GPU: seed, offset) and the element's
    position.  The backward is the same call on the gradient; out may be x."""
    import torch
    _is(x, "x", x.shape, torch.bfloat16)
    _maybe(out, "out", x.shape, torch.bfloat16)
    d = _drop(p, state)
    dev = _one_gpu("x state out", x, state, out)
    if out is None:
        out = torch.empty_like(x)
    _call("qlora_dropout_apply", dev, x.data_ptr(), x.numel(), ctypes.byref(d), out.data_ptr())
    return out


def _rows(X, K):
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    _is(X, "X", (M, K), torch.bfloat16)
    return M


def qlora_linear_dropout_fwd(X, w, A=None, B=None, s: float = 1.0, p: float = 0.0, state=None,
                             Y=None, T=None, workspace=None):
    """The layer with dropout on its adapter's input: Y = X . deq(W)^T + s . T . B
    with T = drop(X) . A.  w is an NF4Weight or a Q4Weight.  Returns (Y bf16
    [M,N], T fp32 [M,r])."""
    import torch
    M = _rows(X, w.K)
    cw, *wt = _q4(w)
    r = _check_adapters(A, B, w)
    d = _drop(p, state)
    _maybe(Y, "Y", (M, w.N), torch.bfloat16)
    if r == 0:
        T = None
    _maybe(T, "T", (M, r), torch.float32)
    need = lib().qlora_linear_dropout_fwd_workspace_bytes(M, w.N, w.K, r)
    dev = _one_gpu("X w.codes w.absmax_q w.absmax_scale A B state Y T workspace", X, *wt, A, B,
                   state, Y, T, workspace)
    workspace = _scratch(workspace, need, dev)
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    if T is None and r > 0:
        T = torch.empty((M, r), dtype=torch.float32, device=dev)
    _call("qlora_linear_dropout_fwd", dev, X.data_ptr(), M, ctypes.byref(cw), _at(A), _at(B), r, s,
          ctypes.byref(d), Y.data_ptr(), _at(T), _at(workspace), need)
    return Y, T


def qlora_linear_dropout_bwd(dY, X, w, A=None, B=None, s: float = 1.0, p: float = 0.0, state=None,
                             T=None, need_dx: bool = True, dX=None, dA=None, dB=None,
                             workspace=None):
    """Backward of qlora_linear_dropout_fwd with the same p and state:
    (dX bf16 [M,K] or None, dA bf16 [K,r], dB bf16 [r,N]); T None recomputes
    it."""
    import torch
    M = _rows(X, w.K)
    cw, *wt = _q4(w)
    _is(dY, "dY", (M, w.N), torch.bfloat16)
    r = _check_adapters(A, B, w)
    d = _drop(p, state)
    return _grads("qlora_linear_dropout_bwd", (), dY, X, M, w.N, w.K, cw, wt, A, B, r, s, d, state,
                  T, need_dx, dX, dA, dB, (w.K, r), (r, w.N), workspace,
                  lib().qlora_linear_dropout_bwd_workspace_bytes(M, w.N, w.K, r))


def _grads(fn, groups, dY, X, M, N, K, cw, wt, A, B, r, s, d, state, T, need_dx, dX, dA, dB,
           shape_a, shape_b, workspace, need, kept=None):
    """The rest of a backward call: outputs, workspace, marshalling.  groups is
    () or (offsets, E).  With an 8-bit checkpoint in X's place, kept is (its C
    view, constants, further arguments, order or None) and X its codes."""
    import torch
    if r == 0:
        T = dA = dB = None
    if not need_dx:
        dX = None
    if T is not None:
        _is(T, "T", (M, r), torch.float32)
    if dX is not None:
        _is(dX, "dX", (M, K), torch.bfloat16)
    if dA is not None:
        _is(dA, "dA", shape_a, torch.bfloat16)
    if dB is not None:
        _is(dB, "dB", shape_b, torch.bfloat16)
    names = "X dY w.codes w.absmax_q w.absmax_scale offsets A B state T dX dA dB workspace"
    tensors = (X, dY, *wt, groups[0] if groups else None, A, B, state, T, dX, dA, dB, workspace)
    if kept is None:
        dev, x = _one_gpu(names, *tensors), (X.data_ptr(),)
    else:
        x8, scales, more, order = kept
        dev = _one_gpu("x8.codes" + names[1:] + " x8.scales order", *tensors, scales, order)
        x = (ctypes.byref(x8), *more)
    workspace = _scratch(workspace, need, dev)
    if need_dx and dX is None:
        dX = torch.empty_like(X) if kept is None else dY.new_empty((M, K))
    if r > 0 and dA is None:
        dA = torch.empty_like(A)
    if r > 0 and dB is None:
        dB = torch.empty_like(B)
    where = (groups[0].data_ptr(), groups[1]) if groups else ()
    _call(fn, dev, dY.data_ptr(), *x, M, *where, ctypes.byref(cw), _at(A), _at(B), r, s,
          ctypes.byref(d), _at(T), _at(dX), _at(dA), _at(dB), _at(workspace), need)
    return dX, dA, dB


def _experts(X, offsets, w, E, A, B):
    """Checks shared by the grouped calls: (M, N, r, C view, weight tensors)."""
    M = _rows(X, w.K)
    return (M, *_expert_layers(offsets, w, E, A, B))


def _expert_layers(offsets, w, E, A, B):
    """The same without X: (N, r, C view, weight tensors)."""
    import torch
    cw, *wt = _q4(w)
    if E < 1 or w.N % E:
        raise ValueError(f"w.N = {w.N} is not a multiple of E = {E}")
    N = w.N // E
    _is(offsets, "offsets", (E + 1,), torch.int32)
    if A is None or B is None:
        if A is not None or B is not None:
            raise ValueError("A and B go together (both None selects r = 0)")
        r = 0
    else:
        if A.dim() != 3:
            raise ValueError("A must be [E, K, r]")
        r = A.shape[2]
        _is(A, "A", (E, w.K, r), torch.bfloat16)
        _is(B, "B", (E, r, N), torch.bfloat16)
    return N, r, cw, wt


def qlora_grouped_fwd(X, offsets, w, E: int, A=None, B=None, s: float = 1.0, p: float = 0.0,
                      state=None, Y=None, T=None, workspace=None):
    """The layer grouped by expert: rows offsets[e] .. offsets[e+1]-1 of X [M, K]
    through expert e's rows of w [E*N, K] (NF4Weight or Q4Weight) and its
    adapters A [E, K, r], B [E, r, N]; p and state as in
    qlora_linear_dropout_fwd.  offsets is int32 [E+1] on the GPU.  Returns (Y
    bf16 [M,N], T fp32 [M,r]); rows outside all groups are left as they were."""
    import torch
    M, N, r, cw, wt = _experts(X, offsets, w, E, A, B)
    d = _drop(p, state)
    _maybe(Y, "Y", (M, N), torch.bfloat16)
    if r == 0:
        T = None
    _maybe(T, "T", (M, r), torch.float32)
    need = lib().qlora_grouped_fwd_workspace_bytes(M, E, N, w.K, r)
    dev = _one_gpu("X w.codes w.absmax_q w.absmax_scale offsets A B state Y T workspace", X, *wt,
                   offsets, A, B, state, Y, T, workspace)
    workspace = _scratch(workspace, need, dev)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if T is None and r > 0:
        T = torch.empty((M, r), dtype=torch.float32, device=dev)
    _call("qlora_grouped_fwd", dev, X.data_ptr(), M, offsets.data_ptr(), E, ctypes.byref(cw),
          _at(A), _at(B), r, s, ctypes.byref(d), Y.data_ptr(), _at(T), _at(workspace), need)
    return Y, T


def qlora_grouped_bwd(dY, X, offsets, w, E: int, A=None, B=None, s: float = 1.0, p: float = 0.0,
                      state=None, T=None, need_dx: bool = True, dX=None, dA=None, dB=None,
                      workspace=None):
    """Backward of qlora_grouped_fwd: (dX bf16 [M,K] or None, dA bf16 [E,K,r],
    dB bf16 [E,r,N]); T None recomputes it.  dA and dB are zero for an expert
    without rows."""
    import torch
    M, N, r, cw, wt = _experts(X, offsets, w, E, A, B)
    _is(dY, "dY", (M, N), torch.bfloat16)
    d = _drop(p, state)
    return _grads("qlora_grouped_bwd", (offsets, E), dY, X, M, N, w.K, cw, wt, A, B, r, s, d,
                  state, T, need_dx, dX, dA, dB, (E, w.K, r), (E, r, N), workspace,
                  lib().qlora_grouped_bwd_workspace_bytes(M, E, N, w.K, r))


def qlora_expert_plan(ids, E: int, workspace=None):
    """Slots sorted by expert, stably, on the GPU.  ids int32 [tokens, topk] (or
    any shape of n slots); an id outside 0 .. E-1 gets no row.  Returns int32
    tensors (offsets [E+1], order [n]: row -> slot or -1, inverse, of ids'
    shape: slot -> row or -1)."""
    import torch
    _is(ids, "ids", ids.shape, torch.int32)
    dev, n = _one_gpu("ids workspace", ids, workspace), ids.numel()
    need = lib().qlora_expert_plan_workspace_bytes(n, E)
    workspace = _scratch(workspace, need, dev)
    offsets = torch.empty(max(E, 0) + 1, dtype=torch.int32, device=dev)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    inverse = torch.empty_like(ids)
    _call("qlora_expert_plan", dev, ids.data_ptr(), n, E, offsets.data_ptr(), order.data_ptr(),
          inverse.data_ptr(), _at(workspace), need)
    return offsets, order, inverse


def _slots(inverse):
    import torch
    if inverse.dim() != 2:
        raise ValueError("inverse must be [tokens, topk]")
    _is(inverse, "inverse", inverse.shape, torch.int32)
    return inverse.shape


def qlora_expert_gather(X, inverse, out=None):
    """Token rows in expert order: row inverse[t, j] of the result [tokens*topk, K]
    is X[t].  Rows no slot has are left as they were (undefined in a result
    allocated here)."""
    import torch
    tokens, topk = _slots(inverse)
    if X.dim() != 2:
        raise ValueError("X must be [tokens, K]")
    K = X.shape[1]
    _is(X, "X", (tokens, K), torch.bfloat16)
    _maybe(out, "out", (tokens * topk, K), torch.bfloat16)
    dev = _one_gpu("X inverse out", X, inverse, out)
    if out is None:
        out = torch.empty((tokens * topk, K), dtype=torch.bfloat16, device=dev)
    _call("qlora_expert_gather", dev, X.data_ptr(), tokens, topk, K, inverse.data_ptr(),
          out.data_ptr())
    return out


def qlora_expert_combine(Y, inverse, weights=None, out=None):
    """Expert rows in token order: out[t] = sum_j weights[t, j] Y[inverse[t, j]]
    (weights fp32 [tokens, topk], or None for 1, which is the backward of
    qlora_expert_gather).  A slot without a row adds nothing."""
    import torch
    tokens, topk = _slots(inverse)
    if Y.dim() != 2:
        raise ValueError("Y must be [tokens*topk, K]")
    K = Y.shape[1]
    _is(Y, "Y", (tokens * topk, K), torch.bfloat16)
    _maybe(weights, "weights", (tokens, topk), torch.float32)
    _maybe(out, "out", (tokens, K), torch.bfloat16)
    dev = _one_gpu("Y inverse weights out", Y, inverse, weights, out)
    if out is None:
        out = torch.empty((tokens, K), dtype=torch.bfloat16, device=dev)
    _call("qlora_expert_combine", dev, Y.data_ptr(), tokens, topk, K, inverse.data_ptr(),
          _at(weights), out.data_ptr())
    return out


def qlora_expert_combine_bwd(dOut, Y, inverse, weights, dY=None, dweights=None):
    """Backward of qlora_expert_combine: (dY bf16 [tokens*topk, K] with rows
    inverse[t, j] = weights[t, j] dOut[t], the others left as they were;
    dweights fp32 [tokens, topk] = dOut[t] . Y[inverse[t, j]], 0 without a
    row)."""
    import torch
    tokens, topk = _slots(inverse)
    if Y.dim() != 2:
        raise ValueError("Y must be [tokens*topk, K]")
    K = Y.shape[1]
    _is(Y, "Y", (tokens * topk, K), torch.bfloat16)
    _is(dOut, "dOut", (tokens, K), torch.bfloat16)
    _is(weights, "weights", (tokens, topk), torch.float32)
    _maybe(dY, "dY", (tokens * topk, K), torch.bfloat16)
    _maybe(dweights, "dweights", (tokens, topk), torch.float32)
    dev = _one_gpu("dOut Y inverse weights dY dweights", dOut, Y, inverse, weights, dY, dweights)
    if dY is None:
        dY = torch.empty_like(Y)
    if dweights is None:
        dweights = torch.empty_like(weights)
    _call("qlora_expert_combine_bwd", dev, dOut.data_ptr(), Y.data_ptr(), tokens, topk, K,
          inverse.data_ptr(), weights.data_ptr(), dY.data_ptr(), dweights.data_ptr())
    return dY, dweights


# ---------------------------------------------------------------------------
# Activations in 8 bits and the backward pass from them, the norm in front of a
# layer, and the routing to experts.
# ---------------------------------------------------------------------------

class Act8(NamedTuple):
    """Activations [M, K] as an 8-bit checkpoint: one signed byte a value and one
    fp32 constant for each 64 of a row."""
    codes: "torch.Tensor"    # int8 [M, K]
    scales: "torch.Tensor"   # float32 [M, K/64]

    def _c(self) -> _Act8:
        return _Act8(self.codes.data_ptr(), self.scales.data_ptr())

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


def _new_act8(X, shape):
    import torch
    return Act8(torch.empty_like(X, dtype=torch.int8),
                X.new_empty((shape[0], shape[1] // 64), dtype=torch.float32))


def _check_act8(x8, name, M=None, K=None):
    """(M, K) of a checkpoint (of the given sizes)."""
    import torch
    if x8 is None:
        raise ValueError(f"{name} is required")
    if x8.codes.dim() != 2:
        raise ValueError(f"{name}.codes must be [M, K]")
    M, K = x8.codes.shape[0] if M is None else M, x8.codes.shape[1] if K is None else K
    if K % 64:
        raise ValueError(f"{name}: K = {K} is not a multiple of 64")
    _is(x8.codes, name + ".codes", (M, K), torch.int8)
    _is(x8.scales, name + ".scales", (M, K // 64), torch.float32)
    return M, K


def _matrix(t, name):
    """The shape of a bf16 matrix."""
    import torch
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be two-dimensional")
    if t.dtype is not torch.bfloat16 or not t.is_contiguous():
        _need(t, name, shape, torch.bfloat16)
    return shape


def qlora_act8_pack(X, out: Optional[Act8] = None) -> Act8:
    """The 8-bit checkpoint of X (bf16 [M, K], K % 64 == 0): blocks of 64 values
    along a row, codes rint(x / c) with c = max |x| / 127."""
    M, K = shape = _matrix(X, "X")
    if K % 64:
        raise ValueError(f"K = {K} is not a multiple of 64")
    if out is None:
        dev = _one_gpu("X", X)
        out = _new_act8(X, shape)
    else:
        _check_act8(out, "out", M, K)
        dev = _one_gpu("X out.codes out.scales", X, out.codes, out.scales)
    _call("qlora_act8_pack", dev, X.data_ptr(), M, K, ctypes.byref(out._c()))
    return out


def qlora_act8_unpack(x8: Act8, out=None):
    """The values (bf16 [M, K]) of an 8-bit checkpoint."""
    import torch
    M, K = _check_act8(x8, "x8")
    if out is not None:
        _is(out, "out", (M, K), torch.bfloat16)
    dev = _one_gpu("x8.codes x8.scales out", x8.codes, x8.scales, out)
    if out is None:
        out = torch.empty_like(x8.codes, dtype=torch.bfloat16)
    _call("qlora_act8_unpack", dev, ctypes.byref(x8._c()), M, K, out.data_ptr())
    return out


@functools.lru_cache(maxsize=1024)
def _act8_bwd_need(M, E, N, K, r):
    """Workspace bytes (E = 0: the plain layer)."""
    if E == 0:
        return lib().qlora_linear_act8_bwd_workspace_bytes(M, N, K, r)
    return lib().qlora_grouped_act8_bwd_workspace_bytes(M, E, N, K, r)


def qlora_linear_act8_bwd(dY, x8: Act8, w, A=None, B=None, s: float = 1.0, p: float = 0.0,
                          state=None, T=None, need_dx: bool = True, dX=None, dA=None, dB=None,
                          workspace=None):
    """qlora_linear_dropout_bwd from an 8-bit checkpoint of the layer's input:
    (dX bf16 [M,K] or None, dA bf16 [K,r], dB bf16 [r,N])."""
    import torch
    M, K = _check_act8(x8, "x8", K=w.K)
    cw, *wt = _q4(w)
    _is(dY, "dY", (M, w.N), torch.bfloat16)
    r = _check_adapters(A, B, w)
    d = _drop(p, state)
    return _grads("qlora_linear_act8_bwd", (), dY, x8.codes, M, w.N, K, cw, wt, A, B, r, s, d,
                  state, T, need_dx, dX, dA, dB, (K, r), (r, w.N), workspace,
                  _act8_bwd_need(M, 0, w.N, K, r),
                  (x8._c(), x8.scales, (), None))


def qlora_grouped_act8_bwd(dY, x8: Act8, offsets, w, E: int, A=None, B=None, s: float = 1.0,
                           p: float = 0.0, state=None, order=None, topk: int = 1, T=None,
                           need_dx: bool = True, dX=None, dA=None, dB=None, workspace=None):
    """qlora_grouped_bwd from an 8-bit checkpoint.  Without an order, x8 holds the
    rows of the grouped input; with order (int32 [M], as qlora_expert_plan gives
    it) it holds the tokens' rows, each once, and row i of the grouped input is
    row order[i] // topk of it.  Returns (dX bf16 [M,K] or None, dA bf16
    [E,K,r], dB bf16 [E,r,N])."""
    import torch
    _int32("topk", topk)
    if dY.dim() != 2:
        raise ValueError("dY must be [M, N]")
    M = dY.shape[0]
    tokens, K = _check_act8(x8, "x8", None if order is not None else M, w.K)
    _maybe(order, "order", (M,), torch.int32)
    N, r, cw, wt = _expert_layers(offsets, w, E, A, B)
    _is(dY, "dY", (M, N), torch.bfloat16)
    d = _drop(p, state)
    return _grads("qlora_grouped_act8_bwd", (offsets, E), dY, x8.codes, M, N, K, cw, wt, A, B, r,
                  s, d, state, T, need_dx, dX, dA, dB, (E, K, r), (E, r, N), workspace,
                  _act8_bwd_need(M, E, N, K, r),
                  (x8._c(), x8.scales, (tokens, _at(order), topk), order))


def _norm_weight(g, K):
    """1 if g [K] is fp32, 0 if bf16."""
    import torch
    if g.dtype is torch.float32:
        _is(g, "g", (K,), torch.float32)
        return 1
    _is(g, "g", (K,), torch.bfloat16)
    return 0


def qlora_rms_norm_fwd(x, g, residual=None, eps: float = 1e-5, act8=False, h=None, y=None,
                       rstd=None):
    """h = x + residual (x itself without one), y = h / rms(h) * g: (h bf16 [M,K],
    y bf16 [M,K], rstd fp32 [M]), and with act8 (True, or an Act8 to write to)
    the 8-bit checkpoint of y too.  g is fp32 or bf16 [K]; h may be x or
    residual."""
    import torch
    M, K = shape = _matrix(x, "x")
    g32 = _norm_weight(g, K)
    if residual is not None:
        _is(residual, "residual", shape, torch.bfloat16)
    elif h is None or h is x:
        h = x
    else:
        raise ValueError("without a residual h is x")
    if h is not None:
        _is(h, "h", shape, torch.bfloat16)
    if y is not None:
        _is(y, "y", shape, torch.bfloat16)
    if rstd is not None:
        _is(rstd, "rstd", (M,), torch.float32)
    keep = act8 is not False and act8 is not None
    if keep:
        if K % 64:
            raise ValueError(f"K = {K} is not a multiple of 64")
        if act8 is not True:
            _check_act8(act8, "act8", M, K)
    out = act8 if keep and act8 is not True else (None, None)
    dev = _one_gpu("x g residual h y rstd act8.codes act8.scales", x, g, residual, h, y, rstd, *out)
    if h is None:
        h = torch.empty_like(x)
    if y is None:
        y = torch.empty_like(x)
    if rstd is None:
        rstd = x.new_empty(M, dtype=torch.float32)
    if keep and act8 is True:
        out = _new_act8(x, shape)
    _call("qlora_rms_norm_fwd", dev, x.data_ptr(), _at(residual), g.data_ptr(), g32, M, K, eps,
          h.data_ptr(), y.data_ptr(), rstd.data_ptr(), ctypes.byref(out._c()) if keep else None)
    return (h, y, rstd, out) if keep else (h, y, rstd)


@functools.lru_cache(maxsize=1024)
def _norm_bwd_need(M, K):
    return lib().qlora_rms_norm_bwd_workspace_bytes(M, K)


def qlora_rms_norm_bwd(dy, h, rstd, g, dres=None, need_dg: bool = True, dx=None, dg=None,
                       workspace=None):
    """Backward of qlora_rms_norm_fwd: (dx bf16 [M,K], the gradient of x and of the
    residual, with dres, the gradient that reaches h from elsewhere, added; dg of
    g's type [K], or None without need_dg).  dx may be dres."""
    import torch
    M, K = shape = _matrix(h, "h")
    g32 = _norm_weight(g, K)
    _is(dy, "dy", shape, torch.bfloat16)
    _is(rstd, "rstd", (M,), torch.float32)
    if dres is not None:
        _is(dres, "dres", shape, torch.bfloat16)
    if dx is not None:
        _is(dx, "dx", shape, torch.bfloat16)
    need = 0
    if need_dg:
        need = _norm_bwd_need(M, K)
        if dg is not None:
            _is(dg, "dg", (K,), g.dtype)
    else:
        dg = None
    dev = _one_gpu("h dy rstd g dres dx dg workspace", h, dy, rstd, g, dres, dx, dg, workspace)
    if need or workspace is not None:
        workspace = _scratch(workspace, need, dev)
    if dx is None:
        dx = torch.empty_like(h)
    if need_dg and dg is None:
        dg = torch.empty_like(g)
    _call("qlora_rms_norm_bwd", dev, dy.data_ptr(), _at(dres), h.data_ptr(), rstd.data_ptr(),
          g.data_ptr(), g32, M, K, dx.data_ptr(), _at(dg), _at(workspace), need)
    return dx, dg


def _logits(logits):
    """(tokens, E, 1 for fp32 or 0 for bf16)."""
    import torch
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [tokens, E]")
    fp32 = logits.dtype is torch.float32
    if not (fp32 or logits.dtype is torch.bfloat16) or not logits.is_contiguous():
        _need(logits, "logits", shape, torch.float32 if fp32 else torch.bfloat16)
    return shape[0], shape[1], 1 if fp32 else 0


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def qlora_router_fwd(logits, topk: int, score: str = "softmax", bias=None, groups: int = 1,
                     top_groups: int = 1, group_top: int = 1, renorm: bool = True,
                     scale: float = 1.0, ids=None, weights=None):
    """The topk experts of every token, best first, and their weights: (ids int32
    [tokens, topk], weights fp32 [tokens, topk]).  logits are fp32 or bf16
    [tokens, E]; score is "softmax" or "sigmoid"; bias (fp32 [E]) takes part in
    the choice alone; of `groups` equal groups of experts the top_groups with the
    best sum of their group_top (1 or 2) best experts stay; renorm divides the
    weights by their sum.  Experts with a logit of -inf are not chosen; a slot
    left over has id -1 and weight 0."""
    import torch
    tokens, E, fp32 = _logits(logits)
    _int32("topk groups top_groups group_top", topk, groups, top_groups, group_top)
    cfg = _RouterConfig(_score(score), topk, groups, top_groups, group_top, 1 if renorm else 0,
                        scale)
    if bias is not None:
        _is(bias, "bias", (E,), torch.float32)
    if ids is not None:
        _is(ids, "ids", (tokens, topk), torch.int32)
    if weights is not None:
        _is(weights, "weights", (tokens, topk), torch.float32)
    dev = _one_gpu("logits bias ids weights", logits, bias, ids, weights)
    if ids is None:
        # (outputs of a topk that the call refuses have no room)
        ids = logits.new_empty((tokens, topk if 0 < topk <= 64 else 0), dtype=torch.int32)
    if weights is None:
        weights = torch.empty_like(ids, dtype=torch.float32)
    _call("qlora_router_fwd", dev, logits.data_ptr(), fp32, tokens, E, _at(bias),
          ctypes.byref(cfg), ids.data_ptr(), weights.data_ptr())
    return ids, weights


def qlora_router_bwd(dweights, logits, ids, score: str = "softmax", renorm: bool = True,
                     scale: float = 1.0, dlogits=None):
    """The gradient of the logits (of their type, [tokens, E]) from that of the
    weights (fp32 [tokens, topk]), the choice held fixed: ids, score, renorm and
    scale are those of qlora_router_fwd."""
    import torch
    tokens, E, fp32 = _logits(logits)
    shape = ids.shape
    if len(shape) != 2:
        raise ValueError("ids must be [tokens, topk]")
    topk = shape[1]
    _is(ids, "ids", (tokens, topk), torch.int32)
    _is(dweights, "dweights", shape, torch.float32)
    if dlogits is not None:
        _is(dlogits, "dlogits", logits.shape, logits.dtype)
    cfg = _RouterConfig(_score(score), topk, 1, 1, 1, 1 if renorm else 0, scale)
    dev = _one_gpu("logits dweights ids dlogits", logits, dweights, ids, dlogits)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    _call("qlora_router_bwd", dev, dweights.data_ptr(), logits.data_ptr(), fp32, ids.data_ptr(),
          tokens, E, ctypes.byref(cfg), dlogits.data_ptr())
    return dlogits


def _addr(x):
    """A torch tensor's data pointer, or an int address as it is."""
    return ctypes.c_void_p(x if isinstance(x, int) else x.data_ptr())


def qlora_adamw_step(param, grad, exp_avg, exp_avg_sq, step: int, lr: float = 2e-4,
                     beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                     weight_decay: float = 0.0):
    """One AdamW step, in place: param (bf16, 1-D) and the fp32 moments.
    exp_avg / exp_avg_sq are fp32 tensors on param's GPU, or device-visible
    addresses (ints) such as PagedState.pointers() gives."""
    import torch
    if param.dim() != 1:
        raise ValueError("param must be a flat [n] tensor (adapters as slices of one buffer)")
    n = param.numel()
    _need(param, "param", (n,), torch.bfloat16)
    _need(grad, "grad", (n,), torch.bfloat16)
    named = [("param", param), ("grad", grad)]
    for name, t in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if not isinstance(t, int):
            _need(t, name, (n,), torch.float32)
            named.append((name, t))
    _on_gpu(named)
    cfg = _AdamWConfig(lr, beta1, beta2, eps, weight_decay)
    _check("qlora_adamw_step",
           lib().qlora_adamw_step(_ptr(param), _ptr(grad), _addr(exp_avg), _addr(exp_avg_sq), n,
                                  ctypes.byref(cfg), int(step), _stream(param)))


class PagedState:
    """The library's paged optimizer state for n parameters: fp32 moments in
    HBM while resident, in pinned host memory (read and written by the GPU
    directly) when paged out."""

    def __init__(self, n: int, on_host: bool = False):
        h = ctypes.c_void_p()
        _check("qlora_paged_state_create",
               lib().qlora_paged_state_create(int(n), int(bool(on_host)), ctypes.byref(h)))
        self._h, self.n = h, int(n)

    def close(self):
        if self._h:
            _check("qlora_paged_state_destroy", lib().qlora_paged_state_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self):
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def page_out(self):
        _check("qlora_paged_state_page_out",
               lib().qlora_paged_state_page_out(self._h, self._stream()))

    def page_in(self):
        _check("qlora_paged_state_page_in",
               lib().qlora_paged_state_page_in(self._h, self._stream()))

    @property
    def resident(self) -> bool:
        return bool(lib().qlora_paged_state_resident(self._h))

    def pointers(self):
        """(exp_avg, exp_avg_sq) device-visible addresses of the current copy."""
        m, v = ctypes.c_void_p(), ctypes.c_void_p()
        _check("qlora_paged_state_pointers",
               lib().qlora_paged_state_pointers(self._h, ctypes.byref(m), ctypes.byref(v)))
        return m.value, v.value

    def read(self, out=None):
        """The moments as a [2, n] fp32 tensor (m, v) on the current GPU."""
        import torch
        if out is None:
            out = torch.empty((2, self.n), dtype=torch.float32, device="cuda")
        _need(out, "out", (2, self.n), torch.float32)
        _check("qlora_paged_state_read",
               lib().qlora_paged_state_read(self._h, _ptr(out), self._stream()))
        return out

    def write(self, src):
        """Set the moments from a [2, n] fp32 tensor (m, v)."""
        import torch
        _need(src, "src", (2, self.n), torch.float32)
        _check("qlora_paged_state_write",
               lib().qlora_paged_state_write(self._h, _ptr(src), self._stream()))

    def step(self, param, grad, step: int, **hp):
        m, v = self.pointers()
        qlora_adamw_step(param, grad, m, v, step, **hp)


class _Shape(NamedTuple):
    N: int
    K: int


def _dense_weight(W):
    import torch
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    _need(W, "W", tuple(W.shape), torch.bfloat16)
    return _Shape(int(W.shape[0]), int(W.shape[1]))


def qlora_lora16_fwd(X, W, A=None, B=None, s: float = 1.0, Y=None, T=None, workspace=None):
    """16-bit LoRA forward on the same kernels: Y = X . W^T + s . (X . A) . B
    with a bf16 base weight W [N, K].  Returns (Y bf16 [M,N], T fp32 [M,r])."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    w = _dense_weight(W)
    M = X.shape[0]
    _need(X, "X", (M, w.K), torch.bfloat16)
    r = _check_adapters(A, B, w)
    if Y is not None:
        _need(Y, "Y", (M, w.N), torch.bfloat16)
    if T is not None and r > 0:
        _need(T, "T", (M, r), torch.float32)
    if workspace is not None:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8)
    _on_gpu([("X", X), ("W", W), ("A", A), ("B", B), ("Y", Y), ("T", T if r > 0 else None),
             ("workspace", workspace)])
    dev = X.device
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=dev)
    if T is None and r > 0:
        T = torch.empty((M, r), dtype=torch.float32, device=dev)
    need = lib().qlora_lora16_fwd_workspace_bytes(M, w.N, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    _check("qlora_lora16_fwd",
           lib().qlora_lora16_fwd(_ptr(X), M, _ptr(W), w.N, w.K, _ptr(A), _ptr(B), r, float(s),
                                  _ptr(Y), _ptr(T), _ptr(workspace), need, _stream(X)))
    return Y, T


def qlora_lora16_bwd(dY, X, W, A=None, B=None, s: float = 1.0, T=None, need_dx: bool = True,
                     dX=None, dA=None, dB=None, workspace=None):
    """16-bit LoRA backward: (dX bf16 [M,K] or None, dA bf16 [K,r], dB bf16
    [r,N]) with a bf16 base weight W [N, K]; T None recomputes X . A."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    w = _dense_weight(W)
    M = X.shape[0]
    _need(X, "X", (M, w.K), torch.bfloat16)
    _need(dY, "dY", (M, w.N), torch.bfloat16)
    r = _check_adapters(A, B, w)
    if T is not None and r > 0:
        _need(T, "T", (M, r), torch.float32)
    if need_dx and dX is not None:
        _need(dX, "dX", (M, w.K), torch.bfloat16)
    if r > 0 and dA is not None:
        _need(dA, "dA", (w.K, r), torch.bfloat16)
    if r > 0 and dB is not None:
        _need(dB, "dB", (r, w.N), torch.bfloat16)
    if workspace is not None:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8)
    _on_gpu([("X", X), ("dY", dY), ("W", W), ("A", A), ("B", B), ("T", T if r > 0 else None),
             ("dX", dX if need_dx else None), ("dA", dA if r > 0 else None),
             ("dB", dB if r > 0 else None), ("workspace", workspace)])
    dev = X.device
    if need_dx and dX is None:
        dX = torch.empty((M, w.K), dtype=torch.bfloat16, device=dev)
    if r > 0:
        if dA is None:
            dA = torch.empty((w.K, r), dtype=torch.bfloat16, device=dev)
        if dB is None:
            dB = torch.empty((r, w.N), dtype=torch.bfloat16, device=dev)
    need = lib().qlora_lora16_bwd_workspace_bytes(M, w.N, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    _check("qlora_lora16_bwd",
           lib().qlora_lora16_bwd(_ptr(dY), _ptr(X), M, _ptr(W), w.N, w.K, _ptr(A), _ptr(B), r,
                                  float(s), _ptr(T), _ptr(dX if need_dx else None), _ptr(dA),
                                  _ptr(dB), _ptr(workspace), need, _stream(X)))
    return (dX if need_dx else None), dA, dB


def qlora_profile_enable(enable: bool = True):
    _check("qlora_profile_enable", lib().qlora_profile_enable(int(enable)))


def qlora_profile_reset():
    _check("qlora_profile_reset", lib().qlora_profile_reset())


def qlora_profile_read(family: int):
    """(total milliseconds, launches) of a timed kernel family."""
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check("qlora_profile_read", lib().qlora_profile_read(family, ctypes.byref(ms),
                                                           ctypes.byref(n)))
    return ms.value, n.value


def _check_block_adapters(A, B, w, S):
    import torch
    if A is None or B is None or A.dim() != 2:
        raise ValueError("A [K, S*r] and B [r, S*nseg] are required")
    if A.shape[1] % S:
        raise ValueError(f"A has {A.shape[1]} columns, not a multiple of S = {S}")
    r = A.shape[1] // S
    _need(A, "A", (w.K, S * r), torch.bfloat16)
    _need(B, "B", (r, w.N), torch.bfloat16)
    return r


def qlora_block_fwd(X, w: NF4Weight, S: int, A, B, s: float = 1.0, Y=None, T=None,
                    workspace=None):
    """S projections sharing X, stacked along N in w: returns Y [M, S*nseg]
    (projection j in columns j*nseg ..) and T [M, S*r]."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    _need(X, "X", (M, w.K), torch.bfloat16)
    wt = _check_weight(w)
    if S < 1 or w.N % S:
        raise ValueError(f"w.N = {w.N} is not a multiple of S = {S}")
    r = _check_block_adapters(A, B, w, S)
    nseg = w.N // S
    if Y is not None:
        _need(Y, "Y", (M, w.N), torch.bfloat16)
    if T is not None:
        _need(T, "T", (M, S * r), torch.float32)
    _on_gpu([("X", X)] + wt + [("A", A), ("B", B), ("Y", Y), ("T", T), ("workspace", workspace)])
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    if T is None:
        T = torch.empty((M, S * r), dtype=torch.float32, device=X.device)
    need = lib().qlora_block_fwd_workspace_bytes(M, S, nseg, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, X.device)
    cw = w._c()
    _check("qlora_block_fwd",
           lib().qlora_block_fwd(_ptr(X), M, ctypes.byref(cw), S, _ptr(A), _ptr(B), r, float(s),
                                 _ptr(Y), _ptr(T), _ptr(workspace), need, _stream(X)))
    return Y, T


def qlora_block_bwd(dY, X, w: NF4Weight, S: int, A, B, s: float = 1.0, T=None,
                    need_dx: bool = True, dX=None, dA=None, dB=None, workspace=None):
    """Backward of the fused block: (dX [M, K] summed over the projections or
    None, dA [K, S*r], dB [r, S*nseg])."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    _need(X, "X", (M, w.K), torch.bfloat16)
    _need(dY, "dY", (M, w.N), torch.bfloat16)
    wt = _check_weight(w)
    if S < 1 or w.N % S:
        raise ValueError(f"w.N = {w.N} is not a multiple of S = {S}")
    r = _check_block_adapters(A, B, w, S)
    nseg = w.N // S
    if T is not None:
        _need(T, "T", (M, S * r), torch.float32)
    _on_gpu([("X", X), ("dY", dY)] + wt + [("A", A), ("B", B), ("T", T)])
    dev = X.device
    if need_dx and dX is None:
        dX = torch.empty((M, w.K), dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((w.K, S * r), dtype=torch.bfloat16, device=dev)
    if dB is None:
        dB = torch.empty((r, w.N), dtype=torch.bfloat16, device=dev)
    need = lib().qlora_block_bwd_workspace_bytes(M, S, nseg, w.K, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    cw = w._c()
    _check("qlora_block_bwd",
           lib().qlora_block_bwd(_ptr(dY), _ptr(X), M, ctypes.byref(cw), S, _ptr(A), _ptr(B), r,
                                 float(s), _ptr(T), _ptr(dX if need_dx else None), _ptr(dA),
                                 _ptr(dB), _ptr(workspace), need, _stream(X)))
    return (dX if need_dx else None), dA, dB


def qlora_probe_hbm_read(buf, workgroups: int, sink):
    """Enqueue one streaming read of the uint8 device tensor buf."""
    _check("qlora_probe_hbm_read",
           lib().qlora_probe_hbm_read(_ptr(buf), buf.numel(), _ptr(sink), workgroups,
                                      _stream(buf)))


def qlora_probe_mfma_bf16(iters: int, workgroups: int, sink):
    """Enqueue the bf16 MFMA loop; returns its flop count."""
    _check("qlora_probe_mfma_bf16",
           lib().qlora_probe_mfma_bf16(iters, workgroups, _ptr(sink), _stream(sink)))
    return workgroups * 4 * iters * 8 * 32768


PROFILE_FAMILIES = {0: "fwd_gemm", 1: "dx_gemm", 2: "fwd_decode", 3: "quantize", 4: "rank"}
