"""Exact minimax FP16 group scales for W4/G128 quantization on MI355X (gfx950).

A thin ctypes binding over ``libcq.so`` (C ABI in ``include/cq.h``).  The
functions named ``cq_*`` mirror the C entry points one to one and only
marshal arguments: torch tensors already on the GPU are passed by pointer on
the current stream, and a non-OK status raises ``CQError``.  The helpers
without the prefix allocate outputs and a workspace with torch and call the
``cq_*`` functions.  Every step of the computation runs in the HIP kernels;
there is no CPU path, and importing this package on a machine without the
built library raises.

The method (CliffQuant repository README, "What CliffQuant changes"): per
group of 128 weights, the positive finite binary16 scale minimising the worst
environment's diagonal-weighted squared error, codes round-half-even then
clipped to [-8, 7], exact ties to the lower bit pattern; the result is stored
in the GPTQ-v1 layout (Qwen3.5-0.8B-Base-CliffQuant-W4A16-G128 model card,
"Quantization configuration").
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "CQError", "GROUP", "MAX_GROUP", "EXHAUSTIVE", "CANDIDATE", "BOUNDED", "ABSMAX", "POOLED_WMSE",
    "FLAG_BAD_INPUT", "FLAG_NEAR_TIE", "FLAG_EXACT_TIE", "FLAG_FALLBACK", "FLAG_FP64_SWEEP",
    "library_path", "load", "cq_abi_version", "cq_status_string", "cq_workspace_size",
    "cq_quantize_groups", "cq_quantize_groups_spec", "cq_quantize_groups_noalloc", "cq_baseline_scales",
    "cq_baseline_scales_spec", "cq_proxy_worst_env_wmse_multi_spec",
    "cq_pack_gptq_v1", "cq_pack_gptq_v1_spec",
    "cq_pack_gptq_v1_multi", "pack_gptq_v1_multi", "cq_proxy_workspace_size",
    "cq_proxy_worst_env_wmse", "cq_proxy_worst_env_wmse_multi", "quantize_groups", "baseline_scales",
    "pack_gptq_v1", "proxy_worst_env_wmse", "proxy_worst_env_wmse_multi", "solve_breakpoint_exact",
    "cq_heldout_workspace_size", "cq_heldout_compare", "heldout_compare", "cq_diagonals_workspace_size",
    "cq_environment_diagonals", "environment_diagonals", "cq_w4a16_matmul", "w4a16_matmul", "EXPORTED_SYMBOLS",
    "cq_probe_valu_fma", "probe_valu_fma",
    "BF16", "F16", "F32", "ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "MAX_REQUESTS",
    "MAX_HEAD_DIM", "PagedAttentionArgs", "cq_w4a16_linear", "w4a16_linear", "cq_kv_block_map", "kv_block_map",
    "cq_kv_cache_write", "kv_cache_write", "cq_paged_attention_workspace_size", "cq_paged_attention",
    "paged_attention",
    "MXFP4", "MXFP8", "MX_BLOCK", "MxCache", "cq_mx_quantize", "mx_quantize", "cq_mx_dequantize", "mx_dequantize",
    "cq_kv_cache_write_mx", "kv_cache_write_mx", "Mxfp4LinearArgs", "cq_mxfp4_linear_workspace_size", "cq_mxfp4_linear",
    "mxfp4_linear", "cq_paged_attention_mx_workspace_size", "cq_paged_attention_mx", "paged_attention_mx",
]

GROUP = 128
MAX_GROUP = 256
EXHAUSTIVE, CANDIDATE, BOUNDED = 0, 1, 2
ABSMAX, POOLED_WMSE = 0, 1
FLAG_BAD_INPUT, FLAG_NEAR_TIE, FLAG_EXACT_TIE, FLAG_FALLBACK, FLAG_FP64_SWEEP = 1, 2, 4, 8, 16
BF16, F16, F32 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)
MXFP4, MXFP8 = 3, 4
MX_BLOCK = 32
MAX_REQUESTS = 4096
MAX_HEAD_DIM = 256
_TYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
_BINARY16 = (torch.int16, torch.float16, torch.uint16)
_MX_FORMATS = {"mxfp4": MXFP4, "mxfp8": MXFP8}
_MX_CODES = (torch.uint8, torch.float8_e4m3fn)
_MX_SCALES = (torch.uint8, torch.float8_e8m0fnu)
_ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}
_METHODS = {"exhaustive": EXHAUSTIVE, "candidate": CANDIDATE, "bounded": BOUNDED}
EXPORTED_SYMBOLS = ("cq_abi_version", "cq_status_string", "cq_workspace_size", "cq_quantize_groups",
                    "cq_quantize_groups_spec", "cq_quantize_groups_noalloc",
                    "cq_baseline_scales", "cq_baseline_scales_spec", "cq_pack_gptq_v1", "cq_pack_gptq_v1_spec",
                    "cq_pack_gptq_v1_multi", "cq_proxy_worst_env_wmse_multi_spec",
                    "cq_proxy_workspace_size",
                    "cq_proxy_worst_env_wmse", "cq_proxy_worst_env_wmse_multi", "cq_heldout_workspace_size",
                    "cq_heldout_compare", "cq_diagonals_workspace_size", "cq_environment_diagonals",
                    "cq_w4a16_matmul", "cq_probe_valu_fma", "cq_w4a16_linear", "cq_kv_block_map",
                    "cq_kv_cache_write", "cq_paged_attention_workspace_size", "cq_paged_attention",
                    "cq_mx_quantize", "cq_mx_dequantize", "cq_kv_cache_write_mx", "cq_mxfp4_linear_workspace_size",
                    "cq_mxfp4_linear", "cq_paged_attention_mx_workspace_size", "cq_paged_attention_mx")

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


class CQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {cq_status_string(status)} (status {status})")
        self.status = status


class PagedAttentionArgs(ctypes.Structure):
    """cq_paged_attention_args of cq.h: device pointers as integers, strides in elements."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k_cache", "v_cache", "block_table", "cu_q", "kv_len", "out",
                                               "lse")] + \
               [(n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "out_token_stride",
                                              "out_head_stride", "page_stride", "head_stride", "row_stride",
                                              "table_stride")] + \
               [(n, ctypes.c_int32) for n in ("type", "n_tokens", "n_requests", "max_q", "max_kv", "heads",
                                              "kv_heads", "head_dim", "page_size", "n_pages", "max_pages",
                                              "causal", "window")] + [("scale", ctypes.c_float)]


class MxCache(ctypes.Structure):
    """cq_mx_cache of cq.h: device pointers as integers, strides in bytes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + \
               [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "row_stride", "scale_page_stride",
                                              "scale_head_stride", "scale_row_stride")] + \
               [(n, ctypes.c_int32) for n in ("format", "n_pages", "page_size", "kv_heads", "head_dim")]


class Mxfp4LinearArgs(ctypes.Structure):
    """cq_mxfp4_linear_args of cq.h: device pointers as integers, leading dimensions in elements (of codes: bytes)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "x_scales", "qweight", "scales", "bias", "residual", "y")] + \
               [(n, ctypes.c_int64) for n in ("ldx", "ldxs", "ldr", "ldy", "M", "out", "inp")] + \
               [(n, ctypes.c_int32) for n in ("type", "x_format", "y_type", "activation", "gated")]


def library_path() -> str:
    return os.environ.get("CQ_LIBRARY", os.path.join(_HERE, "libcq.so"))


def load():
    """Load libcq.so (raises when it has not been built: there is no fallback)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m post_weight_quantization_group_amd.build`")
        lib = ctypes.CDLL(path)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.cq_abi_version.restype = I32
        lib.cq_abi_version.argtypes = []
        lib.cq_status_string.restype = ctypes.c_char_p
        lib.cq_status_string.argtypes = [I32]
        lib.cq_workspace_size.restype = SZ
        lib.cq_workspace_size.argtypes = [I32, I32, I64]
        lib.cq_quantize_groups.restype = I32
        lib.cq_quantize_groups.argtypes = [P, P, I64, I32, I64, I32, P, P, P, P, P, P, P, SZ, P]
        lib.cq_quantize_groups_noalloc.restype = I32
        lib.cq_quantize_groups_noalloc.argtypes = [P, P, I64, I32, I64, I32, P, P, P, P, P, P, P]
        lib.cq_quantize_groups_spec.restype = I32
        lib.cq_quantize_groups_spec.argtypes = [P, P, I32, I32, I32, I64, I32, I64, I32, P, P, P, P, P, P, P, SZ, P]
        lib.cq_baseline_scales.restype = I32
        lib.cq_baseline_scales.argtypes = [P, P, I64, I32, I64, I32, P, P, P, P, SZ, P]
        lib.cq_pack_gptq_v1.restype = I32
        lib.cq_pack_gptq_v1.argtypes = [P, P, I64, I64, P, P, P]
        lib.cq_pack_gptq_v1_spec.restype = I32
        lib.cq_baseline_scales_spec.restype = I32
        lib.cq_baseline_scales_spec.argtypes = [P, P, I32, I32, I32, I64, I32, I64, I32, P, P, P, P, SZ, P]
        lib.cq_proxy_worst_env_wmse_multi_spec.restype = I32
        lib.cq_proxy_worst_env_wmse_multi_spec.argtypes = [P, P, I32, I32, I32, I64, I32, I64, I32, P, P, I32, P, P,
                                                           P, P, SZ, P]
        lib.cq_pack_gptq_v1_spec.argtypes = [P, P, I64, I64, I32, I32, P, P, P]
        lib.cq_pack_gptq_v1_multi.restype = I32
        lib.cq_pack_gptq_v1_multi.argtypes = [P, P, I32, P, P, P, P, P]
        lib.cq_proxy_workspace_size.restype = SZ
        lib.cq_proxy_workspace_size.argtypes = [I64]
        lib.cq_proxy_worst_env_wmse.restype = I32
        lib.cq_proxy_worst_env_wmse.argtypes = [P, P, I64, I32, I64, P, P, I32, P, P, P, P, SZ, P]
        lib.cq_proxy_worst_env_wmse_multi.restype = I32
        lib.cq_proxy_worst_env_wmse_multi.argtypes = [P, P, I64, I32, I64, I32, P, P, I32, P, P, P, P, SZ, P]
        lib.cq_w4a16_matmul.restype = I32
        lib.cq_w4a16_matmul.argtypes = [P, P, P, I64, I64, I64, P, P]
        lib.cq_diagonals_workspace_size.restype = SZ
        lib.cq_diagonals_workspace_size.argtypes = [I32, I64, I64]
        lib.cq_environment_diagonals.restype = I32
        lib.cq_environment_diagonals.argtypes = [P, I32, I64, I64, P, P, SZ, P]
        lib.cq_heldout_workspace_size.restype = SZ
        lib.cq_heldout_workspace_size.argtypes = [I32, I32]
        lib.cq_heldout_compare.restype = I32
        lib.cq_heldout_compare.argtypes = [P, P, I64, P, I32, P, I32, ctypes.c_double, P, P, P, P, P, SZ, P]
        lib.cq_probe_valu_fma.restype = I32
        lib.cq_probe_valu_fma.argtypes = [I32, I32, I32, P, P, ctypes.POINTER(ctypes.c_double), P]
        lib.cq_w4a16_linear.restype = I32
        lib.cq_w4a16_linear.argtypes = [P, I64, I32, P, P, P, P, I64, I32, I32, I64, I64, I64, P, I64, I32, P]
        lib.cq_kv_block_map.restype = I32
        lib.cq_kv_block_map.argtypes = [P, P, I32, I32, P, P, I32, P, I64, I32, I32, P, P, P, P, P, P, P]
        lib.cq_kv_cache_write.restype = I32
        lib.cq_kv_cache_write.argtypes = [P, I64, I64, P, I64, I64, P, P, I64, I64, I64, I32, I32, I32, I32, P, I32, P]
        lib.cq_paged_attention_workspace_size.restype = SZ
        lib.cq_paged_attention_workspace_size.argtypes = [I32] * 7
        lib.cq_paged_attention.restype = I32
        lib.cq_paged_attention.argtypes = [ctypes.POINTER(PagedAttentionArgs), P, SZ, P]
        lib.cq_mx_quantize.restype = I32
        lib.cq_mx_quantize.argtypes = [P, I64, I32, I64, I64, I32, P, I64, P, I64, P]
        lib.cq_mx_dequantize.restype = I32
        lib.cq_mx_dequantize.argtypes = [P, I64, P, I64, I32, I64, I64, P, I64, I32, P]
        lib.cq_kv_cache_write_mx.restype = I32
        lib.cq_kv_cache_write_mx.argtypes = [P, I64, I64, P, I64, I64, I32, ctypes.POINTER(MxCache), P, I32, P]
        lib.cq_mxfp4_linear_workspace_size.restype = SZ
        lib.cq_mxfp4_linear_workspace_size.argtypes = [I64, I64, I64, I32, I32, I32]
        lib.cq_mxfp4_linear.restype = I32
        lib.cq_mxfp4_linear.argtypes = [ctypes.POINTER(Mxfp4LinearArgs), P, SZ, P]
        lib.cq_paged_attention_mx_workspace_size.restype = SZ
        lib.cq_paged_attention_mx_workspace_size.argtypes = [I32] * 7
        lib.cq_paged_attention_mx.restype = I32
        lib.cq_paged_attention_mx.argtypes = [ctypes.POINTER(PagedAttentionArgs), ctypes.POINTER(MxCache), P, SZ, P]
        _lib = lib
    return _lib


# ---------------------------------------------------------------- marshalling
def _p(t):
    """Device pointer of a CUDA/HIP tensor (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("arrays passed to the library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("arrays passed to the library must be contiguous")
    return t.data_ptr()


def _rows(t):
    """Device pointer of a strided CUDA/HIP tensor (None -> NULL); its strides are passed beside it."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("arrays passed to the library must live on the GPU")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The helpers on a hot path call themselves with their arrays' GPU current where another one is: the default stream is
# that of the current GPU, whose kernels would work on another one's memory.
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_on(stream, device: int):
    """_stream for the helpers on a hot path: the current stream of `device` without building an object."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise CQError(status, where)


# ---------------------------------------------------------------- C entry points
def cq_abi_version() -> int:
    return load().cq_abi_version()


def cq_status_string(status: int) -> str:
    return load().cq_status_string(status).decode()


def cq_workspace_size(method: int, E: int, n_groups: int) -> int:
    return load().cq_workspace_size(method, E, n_groups)


def cq_proxy_workspace_size(n_groups: int) -> int:
    return load().cq_proxy_workspace_size(n_groups)


def cq_quantize_groups(w, d, d_period, E, n_groups, method, scales, codes=None, objective=None, flags=None,
                       pooled_scales=None, pooled_objective=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_quantize_groups(_p(w), _p(d), d_period, E, n_groups, method, _p(scales), _p(codes),
                                     _p(objective), _p(flags), _p(pooled_scales), _p(pooled_objective),
                                     _p(workspace), ws_bytes, _stream(stream)), "cq_quantize_groups")


def cq_quantize_groups_noalloc(w, d, d_period, E, n_groups, method, scales, codes=None, objective=None, flags=None,
                               pooled_scales=None, pooled_objective=None, stream=None):
    _check(load().cq_quantize_groups_noalloc(_p(w), _p(d), d_period, E, n_groups, method, _p(scales), _p(codes),
                                             _p(objective), _p(flags), _p(pooled_scales), _p(pooled_objective),
                                             _stream(stream)), "cq_quantize_groups_noalloc")


def cq_quantize_groups_spec(w, d, group_len, qmin, qmax, d_period, E, n_groups, method, scales, codes=None,
                            objective=None, flags=None, pooled_scales=None, pooled_objective=None, workspace=None,
                            stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_quantize_groups_spec(_p(w), _p(d), group_len, qmin, qmax, d_period, E, n_groups, method,
                                          _p(scales), _p(codes), _p(objective), _p(flags), _p(pooled_scales),
                                          _p(pooled_objective), _p(workspace), ws_bytes, _stream(stream)),
           "cq_quantize_groups_spec")


def cq_baseline_scales(w, d, d_period, E, n_groups, which, scales, codes=None, objective=None, workspace=None,
                       stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_baseline_scales(_p(w), _p(d), d_period, E, n_groups, which, _p(scales), _p(codes),
                                     _p(objective), _p(workspace), ws_bytes, _stream(stream)),
           "cq_baseline_scales")


def cq_pack_gptq_v1(codes, grp_scales, out, inp, qweight, scales, stream=None):
    _check(load().cq_pack_gptq_v1(_p(codes), _p(grp_scales), out, inp, _p(qweight), _p(scales),
                                  _stream(stream)), "cq_pack_gptq_v1")


def cq_baseline_scales_spec(w, d, group_len, qmin, qmax, d_period, E, n_groups, which, scales, codes=None,
                            objective=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_baseline_scales_spec(_p(w), _p(d), group_len, qmin, qmax, d_period, E, n_groups, which,
                                          _p(scales), _p(codes), _p(objective), _p(workspace), ws_bytes,
                                          _stream(stream)), "cq_baseline_scales_spec")


def cq_proxy_worst_env_wmse_multi_spec(w, d_eval, group_len, qmin, qmax, d_period, E, n_groups, n_policies, scales,
                                       module_offsets, n_modules, module_mean, macro, per_group=None,
                                       workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_proxy_worst_env_wmse_multi_spec(_p(w), _p(d_eval), group_len, qmin, qmax, d_period, E,
                                                     n_groups, n_policies, _p(scales), _p(module_offsets),
                                                     n_modules, _p(module_mean), _p(macro), _p(per_group),
                                                     _p(workspace), ws_bytes, _stream(stream)),
           "cq_proxy_worst_env_wmse_multi_spec")


def cq_pack_gptq_v1_spec(codes, grp_scales, out, inp, bits, group_len, qweight, scales, stream=None):
    _check(load().cq_pack_gptq_v1_spec(_p(codes), _p(grp_scales), out, inp, bits, group_len, _p(qweight),
                                       _p(scales), _stream(stream)), "cq_pack_gptq_v1_spec")


def cq_pack_gptq_v1_multi(codes, grp_scales, n_mats, outs, ins, qweight, scales, stream=None):
    """outs, ins: host sequences of n_mats shapes (marshalled to int64 host arrays)."""
    o = (ctypes.c_int64 * max(1, n_mats))(*[int(x) for x in outs])
    i = (ctypes.c_int64 * max(1, n_mats))(*[int(x) for x in ins])
    _check(load().cq_pack_gptq_v1_multi(_p(codes), _p(grp_scales), n_mats, ctypes.cast(o, ctypes.c_void_p),
                                        ctypes.cast(i, ctypes.c_void_p), _p(qweight), _p(scales), _stream(stream)),
           "cq_pack_gptq_v1_multi")


def cq_proxy_worst_env_wmse(w, d_eval, d_period, E, n_groups, scales, module_offsets, n_modules, module_mean,
                            macro, per_group=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_proxy_worst_env_wmse(_p(w), _p(d_eval), d_period, E, n_groups, _p(scales),
                                          _p(module_offsets), n_modules, _p(module_mean), _p(macro),
                                          _p(per_group), _p(workspace), ws_bytes, _stream(stream)),
           "cq_proxy_worst_env_wmse")


def cq_proxy_worst_env_wmse_multi(w, d_eval, d_period, E, n_groups, n_policies, scales, module_offsets, n_modules,
                                  module_mean, macro, per_group=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_proxy_worst_env_wmse_multi(_p(w), _p(d_eval), d_period, E, n_groups, n_policies, _p(scales),
                                                _p(module_offsets), n_modules, _p(module_mean), _p(macro),
                                                _p(per_group), _p(workspace), ws_bytes, _stream(stream)),
           "cq_proxy_worst_env_wmse_multi")


def cq_w4a16_matmul(x, qweight, scales, M, out, inp, y, stream=None):
    _check(load().cq_w4a16_matmul(_p(x), _p(qweight), _p(scales), M, out, inp, _p(y), _stream(stream)),
           "cq_w4a16_matmul")


def w4a16_matmul(x, qweight, scales, stream=None):
    """y [M, out] float32 = x [M, in] (bfloat16, or int16 bit patterns) times the dequantized
    GPTQ-v1 tensors (qweight int32 [in/8, out], scales int16 binary16 bits [in/128, out])."""
    M, inp = x.shape
    out = qweight.shape[1]
    xb = x.view(torch.int16) if x.dtype == torch.bfloat16 else x
    y = torch.empty((M, out), dtype=torch.float32, device=x.device)
    cq_w4a16_matmul(xb, qweight, scales, M, out, inp, y, stream)
    return y


def cq_probe_valu_fma(iters, blocks, mode, out, clocks, stream=None) -> float:
    """Runs the fp32 fma issue probe; returns the wall clock's rate in Hz."""
    hz = ctypes.c_double(0.0)
    _check(load().cq_probe_valu_fma(iters, blocks, mode, _p(out), _p(clocks), ctypes.byref(hz), _stream(stream)),
           "cq_probe_valu_fma")
    return hz.value


def probe_valu_fma(iters: int, blocks: int, mode: int = 1, device="cuda", stream=None) -> dict:
    """The issue probe on `blocks` workgroups (mode 0: v_fma_f32, 1: v_fmac_f32, 2: v_fma_f32
    with a scalar operand): the sums,
    per-workgroup (shader cycles, wall ticks) and the wall clock's rate.  The caller times the
    launch."""
    out = torch.empty(blocks * 256, dtype=torch.float32, device=device)
    clocks = torch.empty((blocks, 2), dtype=torch.int64, device=device)
    hz = cq_probe_valu_fma(iters, blocks, mode, out, clocks, stream)
    return {"out": out, "clocks": clocks, "wall_clock_hz": hz}


def cq_diagonals_workspace_size(E: int, T: int, inp: int) -> int:
    return load().cq_diagonals_workspace_size(E, T, inp)


def cq_environment_diagonals(x, E, T, inp, d, workspace, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_environment_diagonals(_p(x), E, T, inp, _p(d), _p(workspace), ws_bytes, _stream(stream)),
           "cq_environment_diagonals")


def cq_heldout_workspace_size(n_boot: int, n_modules: int) -> int:
    return load().cq_heldout_workspace_size(n_boot, n_modules)


def cq_heldout_compare(pa, pb, n_groups, module_offsets, n_modules, boot_idx, n_boot, alpha, counts, effect, boot,
                       ci, workspace, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_heldout_compare(_p(pa), _p(pb), n_groups, _p(module_offsets), n_modules, _p(boot_idx), n_boot,
                                     float(alpha), _p(counts), _p(effect), _p(boot), _p(ci), _p(workspace), ws_bytes,
                                     _stream(stream)), "cq_heldout_compare")


def cq_w4a16_linear(x, ldx, x_type, qweight, scales, bias, residual, ldr, activation, gated, M, out, inp, y, ldy,
                    y_type, stream=None):
    """x, residual and y may be strided rows (their leading dimensions are arguments)."""
    _check(load().cq_w4a16_linear(_rows(x), ldx, x_type, _p(qweight), _p(scales), _p(bias), _rows(residual), ldr,
                                  activation, gated, M, out, inp, _rows(y), ldy, y_type, _stream(stream)),
           "cq_w4a16_linear")


def cq_kv_block_map(ctx_len, new_len, n_requests, page_size, free_pages, n_free, free_capacity, block_table,
                    table_stride, max_pages, max_tokens, cu_q, kv_len, slots, positions, status, n_left, stream=None):
    _check(load().cq_kv_block_map(_p(ctx_len), _p(new_len), n_requests, page_size, _p(free_pages), _p(n_free),
                                  free_capacity, _rows(block_table), table_stride, max_pages, max_tokens, _p(cu_q),
                                  _p(kv_len), _p(slots), _p(positions), _p(status), _p(n_left), _stream(stream)),
           "cq_kv_block_map")


def cq_kv_cache_write(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, k_cache, v_cache,
                      page_stride, head_stride, row_stride, n_pages, page_size, kv_heads, head_dim, slots, n_tokens,
                      stream=None):
    _check(load().cq_kv_cache_write(_rows(k), k_token_stride, k_head_stride, _rows(v), v_token_stride, v_head_stride,
                                    _rows(k_cache), _rows(v_cache), page_stride, head_stride, row_stride, n_pages,
                                    page_size, kv_heads, head_dim, _p(slots), n_tokens, _stream(stream)),
           "cq_kv_cache_write")


def cq_paged_attention_workspace_size(n_tokens: int, n_requests: int, max_q: int, max_kv: int, heads: int,
                                      kv_heads: int, head_dim: int) -> int:
    return load().cq_paged_attention_workspace_size(n_tokens, n_requests, max_q, max_kv, heads, kv_heads, head_dim)


def cq_paged_attention(args: PagedAttentionArgs, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_paged_attention(args, _p(workspace), ws_bytes, _stream(stream)), "cq_paged_attention")


def cq_mx_quantize(x, ldx, x_type, rows, length, format, codes, ldc, scales, lds, stream=None):
    _check(load().cq_mx_quantize(_rows(x), ldx, x_type, rows, length, format, _rows(codes), ldc, _rows(scales), lds,
                                 _stream(stream)), "cq_mx_quantize")


def cq_mx_dequantize(codes, ldc, scales, lds, format, rows, length, y, ldy, y_type, stream=None):
    _check(load().cq_mx_dequantize(_rows(codes), ldc, _rows(scales), lds, format, rows, length, _rows(y), ldy, y_type,
                                   _stream(stream)), "cq_mx_dequantize")


def cq_kv_cache_write_mx(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, type, cache: MxCache,
                         slots, n_tokens, stream=None):
    _check(load().cq_kv_cache_write_mx(_rows(k), k_token_stride, k_head_stride, _rows(v), v_token_stride,
                                       v_head_stride, type, cache, _p(slots), n_tokens, _stream(stream)),
           "cq_kv_cache_write_mx")


def cq_mxfp4_linear_workspace_size(M: int, out: int, inp: int, gated: int, x_format: int, codes: int) -> int:
    return load().cq_mxfp4_linear_workspace_size(M, out, inp, gated, x_format, codes)


def cq_mxfp4_linear(args: Mxfp4LinearArgs, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_mxfp4_linear(args, _p(workspace), ws_bytes, _stream(stream)), "cq_mxfp4_linear")


def cq_paged_attention_mx_workspace_size(n_tokens: int, n_requests: int, max_q: int, max_kv: int, heads: int,
                                         kv_heads: int, head_dim: int) -> int:
    return load().cq_paged_attention_mx_workspace_size(n_tokens, n_requests, max_q, max_kv, heads, kv_heads, head_dim)


def cq_paged_attention_mx(args: PagedAttentionArgs, cache: MxCache, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().cq_paged_attention_mx(args, cache, _p(workspace), ws_bytes, _stream(stream)), "cq_paged_attention_mx")


# ---------------------------------------------------------------- helpers
def _workspace(nbytes: int, device):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _shape_check(w, d):
    if w.dim() != 2 or w.shape[1] != GROUP or w.dtype != torch.float32:
        raise ValueError("w must be float32 [n_groups, 128]")
    if d.dim() != 3 or d.shape[2] != GROUP or d.dtype != torch.float32:
        raise ValueError("d must be float32 [n_d, E, 128]")


def _spec_shape(w, d, qmin, qmax):
    """(G, spec): G from w; spec is True unless the quantizer is the pages' (G = 128, [-8, 7])."""
    G = w.shape[1] if w.dim() == 2 else -1
    spec = (G, int(qmin), int(qmax)) != (GROUP, -8, 7)
    if spec:
        if w.dim() != 2 or not 1 <= G <= MAX_GROUP or w.dtype != torch.float32:
            raise ValueError("w must be float32 [n_groups, G] with 1 <= G <= 256")
        if d.dim() != 3 or d.shape[2] != G or d.dtype != torch.float32:
            raise ValueError("d must be float32 [n_d, E, G]")
    else:
        _shape_check(w, d)
    return G, spec


def quantize_groups(w, d, d_period=None, method="exhaustive", codes=True, pooled=False, workspace=None,
                    stream=None, qmin=-8, qmax=7):
    """Minimax scales (and codes, objective, flags; optionally the pooled policy) for every group.

    w is float32 [n_groups, G] and d float32 [n_d, E, G]; G = 128 with codes in [qmin, qmax] =
    [-8, 7] is the pages' quantizer, any other G <= 256 or range goes through
    cq_quantize_groups_spec (method "exhaustive", or "candidate" for G <= 128 and
    -8 <= qmin, qmax <= 8).  method: "exhaustive" (every scale), "bounded" (branch and bound) or
    "candidate"; all give the same result.
    Returns a dict of device tensors: scales (uint16 bit patterns held in int16
    storage -> use ``.view(torch.uint16)`` or ``& 0xFFFF``), codes, objective,
    flags and, with ``pooled=True``, pooled_scales and pooled_objective.
    """
    G, spec = _spec_shape(w, d, qmin, qmax)
    n, E = w.shape[0], d.shape[1]
    d_period = d.shape[0] if d_period is None else int(d_period)
    m = _METHODS[method] if isinstance(method, str) else int(method)
    dev = w.device
    out = {
        "scales": torch.empty(n, dtype=torch.int16, device=dev),
        "codes": torch.empty((n, G), dtype=torch.int8, device=dev) if codes else None,
        "objective": torch.empty(n, dtype=torch.float64, device=dev),
        "flags": torch.empty(n, dtype=torch.uint8, device=dev),
    }
    if pooled:
        out["pooled_scales"] = torch.empty(n, dtype=torch.int16, device=dev)
        out["pooled_objective"] = torch.empty(n, dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = _workspace(cq_workspace_size(m, E, n), dev)
    if spec:
        cq_quantize_groups_spec(w, d, G, qmin, qmax, d_period, E, n, m, out["scales"], out["codes"], out["objective"],
                                out["flags"], out.get("pooled_scales"), out.get("pooled_objective"), workspace, stream)
    else:
        cq_quantize_groups(w, d, d_period, E, n, m, out["scales"], out["codes"], out["objective"], out["flags"],
                           out.get("pooled_scales"), out.get("pooled_objective"), workspace, stream)
    return out


def baseline_scales(w, d, d_period=None, which="absmax", codes=True, objective=True, workspace=None,
                    stream=None, qmin=-8, qmax=7):
    """AbsMax or pooled-WMSE scales: dict with scales, codes, objective.  Another group length
    (w [n_groups, G], d [n_d, E, G]) or code range goes through cq_baseline_scales_spec."""
    G, spec = _spec_shape(w, d, qmin, qmax)
    n, E = w.shape[0], d.shape[1]
    d_period = d.shape[0] if d_period is None else int(d_period)
    k = {"absmax": ABSMAX, "pooled": POOLED_WMSE}[which] if isinstance(which, str) else int(which)
    dev = w.device
    out = {
        "scales": torch.empty(n, dtype=torch.int16, device=dev),
        "codes": torch.empty((n, G), dtype=torch.int8, device=dev) if codes else None,
        "objective": torch.empty(n, dtype=torch.float64, device=dev) if objective else None,
    }
    if k == POOLED_WMSE and workspace is None:
        workspace = _workspace(cq_workspace_size(EXHAUSTIVE, E, n), dev)
    if spec:
        cq_baseline_scales_spec(w, d, G, qmin, qmax, d_period, E, n, k, out["scales"], out["codes"],
                                out["objective"], workspace, stream)
    else:
        cq_baseline_scales(w, d, d_period, E, n, k, out["scales"], out["codes"], out["objective"], workspace,
                           stream)
    return out


def pack_gptq_v1(codes, grp_scales, out: int, inp: int, stream=None, bits: int = 4, group: int = GROUP):
    """GPTQ-v1 (qweight int32 [in*bits/32, out], scales int16-stored fp16 bits [in/group, out]);
    4-bit fields and groups of 128 by default, else bits in {2, 4, 8} and any group length."""
    qweight = torch.empty((inp * bits // 32, out), dtype=torch.int32, device=codes.device)
    scales = torch.empty((inp // group, out), dtype=torch.int16, device=codes.device)
    if bits == 4 and group == GROUP:
        cq_pack_gptq_v1(codes, grp_scales, out, inp, qweight, scales, stream)
    else:
        cq_pack_gptq_v1_spec(codes, grp_scales, out, inp, bits, group, qweight, scales, stream)
    return qweight, scales


def pack_gptq_v1_multi(codes, grp_scales, shapes, stream=None):
    """GPTQ-v1 packing of several matrices in one launch.  codes int8 and grp_scales int16 (binary16
    bits) hold the matrices back to back (flat, or any contiguous tensor); shapes is a list of
    (out, in).  Returns (qweight, scales) as flat int32 and int16 tensors holding each matrix's
    [in/8, out] and [in/128, out] blocks back to back."""
    n_el = sum(int(o) * int(i) for o, i in shapes)
    qweight = torch.empty(n_el // 8, dtype=torch.int32, device=codes.device)
    scales = torch.empty(n_el // GROUP, dtype=torch.int16, device=codes.device)
    cq_pack_gptq_v1_multi(codes, grp_scales, len(shapes), [o for o, _ in shapes], [i for _, i in shapes], qweight,
                          scales, stream)
    return qweight, scales


def proxy_worst_env_wmse(w, d_eval, scales, module_offsets, d_period=None, per_group=True, stream=None):
    """(per_group or None, module_mean [n_modules], macro [1]) as float64 device tensors."""
    _shape_check(w, d_eval)
    n, E = w.shape[0], d_eval.shape[1]
    d_period = d_eval.shape[0] if d_period is None else int(d_period)
    n_modules = module_offsets.numel() - 1
    dev = w.device
    mm = torch.empty(n_modules, dtype=torch.float64, device=dev)
    macro = torch.empty(1, dtype=torch.float64, device=dev)
    pg = torch.empty(n, dtype=torch.float64, device=dev) if per_group else None
    ws = None if per_group else _workspace(cq_proxy_workspace_size(n), dev)
    cq_proxy_worst_env_wmse(w, d_eval, d_period, E, n, scales, module_offsets, n_modules, mm, macro, pg, ws,
                            stream)
    return pg, mm, macro


def proxy_worst_env_wmse_multi(w, d_eval, scales, module_offsets, d_period=None, per_group=True, stream=None,
                               qmin=-8, qmax=7):
    """The proxy for several policies at once: scales [P, n_groups] int16 on the device.
    Returns (per_group [P, n] or None, module_mean [P, n_modules], macro [P]) as float64 device tensors.
    Another group length or code range goes through cq_proxy_worst_env_wmse_multi_spec."""
    G, spec = _spec_shape(w, d_eval, qmin, qmax)
    n, E = w.shape[0], d_eval.shape[1]
    if scales.dim() != 2 or scales.shape[1] != n:
        raise ValueError("scales must be [n_policies, n_groups]")
    n_pol = scales.shape[0]
    d_period = d_eval.shape[0] if d_period is None else int(d_period)
    n_modules = module_offsets.numel() - 1
    dev = w.device
    mm = torch.empty((n_pol, n_modules), dtype=torch.float64, device=dev)
    macro = torch.empty(n_pol, dtype=torch.float64, device=dev)
    pg = torch.empty((n_pol, n), dtype=torch.float64, device=dev) if per_group else None
    ws = None if per_group else _workspace(cq_proxy_workspace_size(n * n_pol), dev)
    if spec:
        cq_proxy_worst_env_wmse_multi_spec(w, d_eval, G, qmin, qmax, d_period, E, n, n_pol, scales, module_offsets,
                                           n_modules, mm, macro, pg, ws, stream)
    else:
        cq_proxy_worst_env_wmse_multi(w, d_eval, d_period, E, n, n_pol, scales, module_offsets, n_modules, mm,
                                      macro, pg, ws, stream)
    return pg, mm, macro


def _empty(shape, dtype, like, stream):
    """An output (or workspace) in the memory pool of the stream that the kernels run on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _on(device: int, *named):
    """Device pointers of (name, tensor or None) pairs, all of which must be on `device`."""
    ptrs = []
    for name, t in named:
        if t is None:
            ptrs.append(None)
        elif t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}; all arrays must live on one GPU")
        else:
            ptrs.append(t.data_ptr())
    return ptrs


def _same_gpu(device: int, **arrays):
    """_on for the helpers on a hot path that take the pointers themselves."""
    for name, t in arrays.items():
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}; all arrays must live on one GPU")


def _gpu(t) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError("arrays passed to the library must live on the GPU")
    return d


def _contiguous(**arrays):
    for name, t in arrays.items():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _int32(**arrays):
    for name, t in arrays.items():
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")


def _ld(t):
    """Leading dimension of a row-major matrix; that of a single row is its length."""
    if t.is_contiguous():
        return t.shape[1]
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("the rows of x, residual, out and block_table must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _step(t, dim):
    """Stride of a dimension; that of a single entry is never used, and 0."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def w4a16_linear(x, qweight, scales, bias=None, residual=None, activation="none", gated=False, out_dtype=None,
                 out=None, stream=None):
    """y [M, out] = act(x W + bias) + residual over GPTQ-v1 tensors; gated: qweight holds the gate's
    columns, then as many others, and y = act(x Wg + bg) * (x Wu + bu) + residual.

    x is bfloat16 or float16 [M, in] (rows may be strided: 16-byte aligned, stride a multiple of
    8), qweight int32 [in/8, cols], scales int16, uint16 or float16 [in/128, cols]; bias [cols] and residual
    [M, out] have x's type.  activation: "none", "relu", "silu", "gelu" or "gelu_tanh".  The result
    has x's type, or float32 with out_dtype=torch.float32, or goes into ``out`` (which may be the
    residual itself)."""
    dt = x.dtype
    if x.dim() != 2 or (dt != torch.bfloat16 and dt != torch.float16):
        raise ValueError("x must be bfloat16 or float16 [M, in]")
    M, inp = x.shape
    if qweight.dim() != 2 or qweight.dtype != torch.int32 or qweight.shape[0] * 8 != inp or inp % GROUP:
        raise ValueError("qweight must be int32 [in/8, cols], in a multiple of 128")
    cols = qweight.shape[1]
    if scales.shape != (inp // GROUP, cols) or scales.dtype not in _BINARY16:
        raise ValueError("scales must be float16, or its bits as int16 or uint16, [in/128, cols]")
    if gated and cols % 2:
        raise ValueError("gated needs an even number of columns")
    n = cols // 2 if gated else cols
    if bias is not None and (bias.shape != (cols,) or bias.dtype != dt):
        raise ValueError("bias must be [cols], of x's type")
    if residual is not None and (residual.shape != (M, n) or residual.dtype != dt):
        raise ValueError("residual must be [M, out], of x's type")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    _contiguous(qweight=qweight, scales=scales)
    if bias is not None:
        _contiguous(bias=bias)
    device = _gpu(x)
    if device != _device_now():
        with torch.cuda.device(device):
            return w4a16_linear(x, qweight, scales, bias, residual, activation, gated, out_dtype, out, stream)
    if out is None:
        out = _empty((M, n), out_dtype or dt, x, stream)
    elif out.shape != (M, n) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [M, out], of the type asked for")
    if out.dtype != dt and out.dtype != torch.float32:
        raise ValueError("the result has x's type or float32")
    px, pq, ps, pb, pr, py = _on(device, ("x", x), ("qweight", qweight), ("scales", scales), ("bias", bias),
                                 ("residual", residual), ("out", out))
    _check((_lib or load()).cq_w4a16_linear(px, _ld(x), _TYPES[dt], pq, ps, pb, pr,
                                            0 if residual is None else _ld(residual), act, int(gated), M, n, inp, py,
                                            _ld(out), _TYPES[out.dtype], _stream_on(stream, device)),
           "cq_w4a16_linear")
    return out


def kv_block_map(ctx_len, new_len, free_pages, n_free, block_table, page_size, max_tokens, stream=None):
    """Block tables and slot maps of a paged cache from the requests' lengths.

    ctx_len, new_len int32 [R]: tokens held and to come; free_pages int32 [capacity] of which the
    first n_free (int32 [1]) are free, taken from the end; block_table int32 [R, max_pages], updated in
    place.  Returns a dict of int32 tensors: cu_q [R + 1], kv_len [R], slots and positions
    [max_tokens] (slot -1 past the last token), status [R] (0 served, 1 refused for want of pages
    or tokens, 2 invalid) and n_left [1]."""
    R = ctx_len.numel()
    _int32(ctx_len=ctx_len, new_len=new_len, free_pages=free_pages, n_free=n_free, block_table=block_table)
    if new_len.numel() != R or n_free.numel() != 1 or block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("ctx_len and new_len must be [R], n_free [1], block_table [R, max_pages]")
    _contiguous(ctx_len=ctx_len, new_len=new_len, free_pages=free_pages)
    device, most = _gpu(ctx_len), block_table.shape[1]
    if device != _device_now():
        with torch.cuda.device(device):
            return kv_block_map(ctx_len, new_len, free_pages, n_free, block_table, page_size, max_tokens, stream)
    sizes = (R + 1, R, max_tokens, max_tokens, R, 1)
    buf = _empty(2 * R + R + 2 + 2 * max_tokens, torch.int32, ctx_len, stream)
    cu, kv, slots, pos, status, left = buf.split_with_sizes(sizes)
    pc, pn, pf, pfree, pt, at = _on(device, ("ctx_len", ctx_len), ("new_len", new_len), ("free_pages", free_pages),
                                    ("n_free", n_free), ("block_table", block_table), ("the result", buf))
    kv_at = at + 4 * (R + 1)
    slots_at = kv_at + 4 * R
    pos_at = slots_at + 4 * max_tokens
    status_at = pos_at + 4 * max_tokens
    _check((_lib or load()).cq_kv_block_map(pc, pn, R, page_size, pf, pfree, free_pages.numel(), pt, _ld(block_table),
                                            most, max_tokens, at, kv_at, slots_at, pos_at, status_at,
                                            status_at + 4 * R, _stream_on(stream, device)), "cq_kv_block_map")
    return {"cu_q": cu, "kv_len": kv, "slots": slots, "positions": pos, "status": status, "n_left": left}


def _cache_shape(k_cache, v_cache):
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or \
            (v_cache.stride() != strides and any(shape[i] > 1 and v_cache.stride(i) != strides[i] for i in range(4))):
        raise ValueError("k_cache and v_cache must be [pages, kv_heads, page_size, head_dim], strided alike")
    dt = k_cache.dtype
    if (dt != torch.bfloat16 and dt != torch.float16) or v_cache.dtype != dt:
        raise ValueError("k_cache and v_cache must be bfloat16 or float16")
    if strides[3] != 1:
        raise ValueError("head_dim must be contiguous")
    return shape, [st if n > 1 else 0 for st, n in zip(strides, shape)]


def kv_cache_write(k, v, k_cache, v_cache, slots, stream=None):
    """Writes k, v [T, kv_heads, head_dim] (strided views allowed) into the caches
    [pages, kv_heads, page_size, head_dim] at slots int32 [T] (page * page_size + offset; a
    negative slot is skipped)."""
    (pages, heads, page, D), (c_page, c_head, c_row, _) = _cache_shape(k_cache, v_cache)
    T = slots.numel()
    _int32(slots=slots)
    want, dt = (T, heads, D), k_cache.dtype
    if k.shape != want or v.shape != want or k.dtype != dt or v.dtype != dt:
        raise ValueError("k and v must be [T, kv_heads, head_dim] of the caches' type, slots int32 [T]")
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("head_dim must be contiguous")
    _contiguous(slots=slots)
    device = _gpu(k_cache)
    if device != _device_now():
        with torch.cuda.device(device):
            return kv_cache_write(k, v, k_cache, v_cache, slots, stream)
    pk, pv, pkc, pvc, ps = _on(device, ("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache), ("slots", slots))
    _check((_lib or load()).cq_kv_cache_write(pk, _step(k, 0), _step(k, 1), pv, _step(v, 0), _step(v, 1), pkc, pvc,
                                              c_page, c_head, c_row, pages, page, heads, D, ps, T,
                                              _stream_on(stream, device)), "cq_kv_cache_write")


_ATTENTION_ARGS = struct.Struct("@8P8q13if")  # PagedAttentionArgs, field by field
assert _ATTENTION_ARGS.size == ctypes.sizeof(PagedAttentionArgs)


def paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale=None, causal=True, window=0,
                    out=None, lse=None, workspace=None, stream=None):
    """Attention of packed new tokens over a paged cache, the new tokens' keys in it already.

    q [T, heads, head_dim] (a strided view allowed), caches [pages, kv_heads, page_size, head_dim],
    block_table int32 [R, max_pages], cu_q int32 [R + 1], kv_len int32 [R] (the new tokens
    included); max_q and max_kv are the host's bounds of the requests' new and cached tokens.
    scale defaults to 1/sqrt(head_dim).  Returns out [T, heads, head_dim] of q's type; ``lse``, if
    given, is a contiguous float32 [T, heads] to fill."""
    (pages, Hkv, page, D), (c_page, c_head, c_row, _) = _cache_shape(k_cache, v_cache)
    dt = q.dtype
    if q.dim() != 3 or dt != k_cache.dtype or q.shape[2] != D or q.stride(2) != 1:
        raise ValueError("q must be [T, heads, head_dim] of the caches' type, head_dim contiguous")
    _int32(block_table=block_table, cu_q=cu_q, kv_len=kv_len)
    T, H, _ = q.shape
    R = kv_len.numel()
    if cu_q.numel() != R + 1 or block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("cu_q must be [R + 1], kv_len [R], block_table [R, max_pages]")
    _contiguous(cu_q=cu_q, kv_len=kv_len)
    if lse is not None:
        if lse.shape != (T, H) or lse.dtype != torch.float32:
            raise ValueError("lse must be float32 [T, heads]")
        _contiguous(lse=lse)
    device = _gpu(q)
    if device != _device_now():
        with torch.cuda.device(device):
            return paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale, causal, window,
                                   out, lse, workspace, stream)
    if out is None:
        out = _empty((T, H, D), dt, q, stream)
    elif out.shape != q.shape or out.dtype != dt or out.stride(2) != 1:
        raise ValueError("out must be [T, heads, head_dim] of q's type, head_dim contiguous")
    lib = _lib or load()
    need = lib.cq_paged_attention_workspace_size(T, R, max_q, max_kv, H, Hkv, D)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q, stream)
    pq, pk, pv, pt, pcu, pkv, po, pl, pw = _on(
        device, ("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table), ("cu_q", cu_q),
        ("kv_len", kv_len), ("out", out), ("lse", lse), ("workspace", workspace))
    args = PagedAttentionArgs.from_buffer_copy(_ATTENTION_ARGS.pack(
        pq, pk, pv, pt, pcu, pkv, po, pl or 0, _step(q, 0), _step(q, 1), _step(out, 0), _step(out, 1), c_page, c_head,
        c_row, _ld(block_table), _TYPES[dt], T, R, max_q, max_kv, H, Hkv, D, page, pages, block_table.shape[1],
        int(causal), window, D ** -0.5 if scale is None else scale))
    _check(lib.cq_paged_attention(args, pw, 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                  _stream_on(stream, device)), "cq_paged_attention")
    return out


def _mx_format(format):
    form = _MX_FORMATS.get(format)
    if form is None:
        raise ValueError(f"format must be one of {', '.join(_MX_FORMATS)}")
    return form


def _mx_rows(t, name):
    """(rows, leading dimension) of an array of rows: contiguous, or a matrix whose rows are."""
    n = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // n, n
    if t.dim() != 2 or (n > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be contiguous, or a matrix with contiguous rows")
    return t.shape[0], _ld(t)


def mx_quantize(x, format="mxfp4", stream=None):
    """Values as microscaled blocks of 32 along the last axis: (codes, scales), both uint8.

    x is bfloat16, float16 or float32 [..., n], n a multiple of 32 (contiguous, or a matrix with strided rows: 16-byte
    aligned, stride a multiple of 8).  format "mxfp4": e2m1 elements, codes [..., n/2] with the first of two in the low
    four bits; "mxfp8": e4m3, [..., n] (view it as torch.float8_e4m3fn).  scales [..., n/32] hold powers of two with a
    bias of 127: 2^(floor(log2 of the block's largest magnitude) - 2) (mxfp8: - 8); 255 (NaN) for a block with an
    infinity or a NaN.  Elements are rounded to nearest even and saturate at 6 (448)."""
    form, kind, shape = _mx_format(format), _TYPES.get(x.dtype), x.shape
    n = shape[-1] if len(shape) else 0
    if kind is None or n % MX_BLOCK or not n:
        raise ValueError("x must be bfloat16, float16 or float32 [..., n], n a multiple of 32")
    rows, ldx = _mx_rows(x, "x")
    device = _gpu(x)
    if device != _device_now():
        with torch.cuda.device(device):
            return mx_quantize(x, format, stream)
    width = n // 2 if form == MXFP4 else n
    codes = _empty((*shape[:-1], width), torch.uint8, x, stream)
    scales = _empty((*shape[:-1], n // MX_BLOCK), torch.uint8, x, stream)
    status = (_lib or load()).cq_mx_quantize(x.data_ptr(), ldx, kind, rows, n, form, codes.data_ptr(), width,
                                             scales.data_ptr(), n // MX_BLOCK, _stream_on(stream, device))
    if status:
        raise CQError(status, "cq_mx_quantize")
    return codes, scales


def _mx_pair(codes, scales, form, what="codes"):
    """Values a row of codes stands for, with the types and shapes of codes and scales checked."""
    if codes.dim() < 1 or codes.dtype not in _MX_CODES or (form == MXFP4 and codes.dtype != torch.uint8):
        raise ValueError(f"{what} must be uint8 (mxfp8: or float8_e4m3fn)")
    n = codes.shape[-1] * (2 if form == MXFP4 else 1)
    if n % MX_BLOCK or scales.dtype not in _MX_SCALES or scales.shape != codes.shape[:-1] + (n // MX_BLOCK,):
        raise ValueError(f"the scales of {what} must be uint8 or float8_e8m0fnu, one for each 32 values of a row")
    return n


def mx_dequantize(codes, scales, format="mxfp4", out_dtype=torch.bfloat16, stream=None):
    """The values [..., n] that the blocks of mx_quantize stand for, as bfloat16, float16 or float32 (rounded once)."""
    form = _mx_format(format)
    n = _mx_pair(codes, scales, form)
    if out_dtype not in _TYPES:
        raise ValueError("out_dtype must be bfloat16, float16 or float32")
    if not n:
        raise ValueError("rows without values")
    rows, ldc = _mx_rows(codes, "codes")
    _, lds = _mx_rows(scales, "scales")
    device = _gpu(codes)
    if device != _device_now():
        with torch.cuda.device(device):
            return mx_dequantize(codes, scales, format, out_dtype, stream)
    y = _empty((*codes.shape[:-1], n), out_dtype, codes, stream)
    _same_gpu(device, scales=scales)
    status = (_lib or load()).cq_mx_dequantize(codes.data_ptr(), ldc, scales.data_ptr(), lds, form, rows, n,
                                               y.data_ptr(), n, _TYPES[out_dtype], _stream_on(stream, device))
    if status:
        raise CQError(status, "cq_mx_dequantize")
    return y


_MXFP4_LINEAR = struct.Struct("@7P7q5i4x")  # Mxfp4LinearArgs, field by field
assert _MXFP4_LINEAR.size == ctypes.sizeof(Mxfp4LinearArgs)


def mxfp4_linear(x, qweight, scales, x_scales=None, x_format="mxfp8", bias=None, residual=None, activation="none",
                 gated=False, out_dtype=None, out=None, workspace=None, stream=None):
    """y [M, out] = act(X W^T + bias) + residual over MXFP4 weights; gated: W holds the gate's rows, then as many others,
    and y = act(X Wg^T + bg) * (X Wu^T + bu) + residual.

    qweight uint8 [cols, in/2] and scales uint8 [cols, in/32] are mx_quantize's of a [cols, in] matrix, in a multiple of
    128.  x is bfloat16 or float16 [M, in] (rows may be strided: 16-byte aligned, stride a multiple of 8), and X its rows
    quantized to x_format ("mxfp8" or "mxfp4") as mx_quantize does; or x holds codes of x_format with their x_scales.
    bias [cols] and residual [M, out] have x's type; beside codes they have one 16-bit type, which is the result's too
    (bfloat16 where there is neither).  activation: "none", "relu", "silu", "gelu" or "gelu_tanh".  The result has that
    type, or float32 with out_dtype=torch.float32, or goes into ``out`` (which may be the residual itself)."""
    form = _mx_format(x_format)
    if x.dim() != 2:
        raise ValueError("x must be a matrix [M, in], of values or of codes")
    M = x.shape[0]
    if x_scales is None:
        dt, inp = x.dtype, x.shape[1]
        if dt != torch.bfloat16 and dt != torch.float16:
            raise ValueError("x must be bfloat16 or float16 [M, in], or codes with x_scales")
    else:
        inp = _mx_pair(x, x_scales, form, "x")
        dt = next((t.dtype for t in (bias, residual) if t is not None), None)
        if dt is None:
            dt = next((d for d in (out_dtype, None if out is None else out.dtype) if d not in (None, torch.float32)),
                      torch.bfloat16)
        if dt != torch.bfloat16 and dt != torch.float16:
            raise ValueError("bias, residual and result must be bfloat16 or float16 (the result also float32)")
    if qweight.dim() != 2 or qweight.dtype != torch.uint8 or qweight.shape[1] * 2 != inp or inp % GROUP or not inp:
        raise ValueError("qweight must be uint8 [cols, in/2], in a multiple of 128")
    cols = qweight.shape[0]
    if scales.shape != (cols, inp // MX_BLOCK) or scales.dtype not in _MX_SCALES:
        raise ValueError("scales must be uint8 or float8_e8m0fnu [cols, in/32]")
    if gated and cols % 2:
        raise ValueError("gated needs an even number of columns")
    n = cols // 2 if gated else cols
    if bias is not None and (bias.shape != (cols,) or bias.dtype != dt):
        raise ValueError("bias must be [cols], of x's type (beside codes: of the residual's)")
    if residual is not None and (residual.shape != (M, n) or residual.dtype != dt):
        raise ValueError("residual must be [M, out], of x's type (beside codes: of the bias's)")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    if not (qweight.is_contiguous() and scales.is_contiguous() and (bias is None or bias.is_contiguous())):
        raise ValueError("qweight, scales and bias must be contiguous")
    device = _gpu(x)
    if device != _device_now():
        with torch.cuda.device(device):
            return mxfp4_linear(x, qweight, scales, x_scales, x_format, bias, residual, activation, gated, out_dtype,
                                out, workspace, stream)
    if out is None:
        out = _empty((M, n), out_dtype or dt, x, stream)
    elif out.shape != (M, n) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [M, out], of the type asked for")
    if out.dtype != dt and out.dtype != torch.float32:
        raise ValueError("the result has the 16-bit type of the other arrays, or float32")
    lib = _lib or load()
    need = lib.cq_mxfp4_linear_workspace_size(M, n, inp, int(gated), form, int(x_scales is not None))
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, x, stream)
    _same_gpu(device, x_scales=x_scales, qweight=qweight, scales=scales, bias=bias, residual=residual, out=out,
              workspace=workspace)
    args = Mxfp4LinearArgs.from_buffer_copy(_MXFP4_LINEAR.pack(
        x.data_ptr(), 0 if x_scales is None else x_scales.data_ptr(), qweight.data_ptr(), scales.data_ptr(),
        0 if bias is None else bias.data_ptr(), 0 if residual is None else residual.data_ptr(), out.data_ptr(), _ld(x),
        0 if x_scales is None else _ld(x_scales), 0 if residual is None else _ld(residual), _ld(out), M, n, inp,
        _TYPES[dt], form, _TYPES[out.dtype], act, int(gated)))
    status = lib.cq_mxfp4_linear(args, None if workspace is None else workspace.data_ptr(),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _stream_on(stream, device))
    if status:
        raise CQError(status, "cq_mxfp4_linear")
    return out


_MX_CACHE = struct.Struct("@4P6q5i4x")  # MxCache, field by field
assert _MX_CACHE.size == ctypes.sizeof(MxCache)


def _strides_like(a, b, shape):
    """a's strides, which b must share where they matter."""
    st, other = a.stride(), b.stride()
    if st != other and any(n > 1 and i != j for n, i, j in zip(shape, st, other)):
        raise ValueError("the caches of keys and of values must be strided alike, and so their scales")
    return st


def _mx_cache(k_cache, k_scales, v_cache, v_scales, heads, D, device):
    """The cache that a call reads or writes: its format follows from the width of its rows."""
    shape, sshape = k_cache.shape, k_scales.shape
    if len(shape) != 4 or v_cache.shape != shape or shape[1] != heads or (shape[3] != D and shape[3] * 2 != D):
        raise ValueError("k_cache and v_cache must be [pages, kv_heads, page_size, head_dim (mxfp8) or head_dim / 2 "
                         "(mxfp4)]")
    form = MXFP8 if shape[3] == D else MXFP4
    if D % MX_BLOCK or not 0 < D <= MAX_HEAD_DIM:
        raise ValueError("head_dim must be a multiple of 32 up to 256")
    pages, _, page, _ = shape
    if sshape != (pages, heads, page, D // MX_BLOCK) or v_scales.shape != sshape:
        raise ValueError("k_scales and v_scales must be [pages, kv_heads, page_size, head_dim / 32]")
    u8 = torch.uint8
    if k_cache.dtype != u8 or v_cache.dtype != u8 or k_scales.dtype != u8 or v_scales.dtype != u8:
        for c, e in ((k_cache, k_scales), (v_cache, v_scales)):
            if c.dtype not in _MX_CODES or (form == MXFP4 and c.dtype != u8) or e.dtype not in _MX_SCALES:
                raise ValueError("caches must be uint8 (mxfp8: or float8_e4m3fn), their scales uint8 or float8_e8m0fnu")
    a, b, c, d = _strides_like(k_cache, v_cache, shape)
    sa, sb, sc, sd = _strides_like(k_scales, v_scales, sshape)
    if d != 1 or (sd != 1 and sshape[3] > 1):
        raise ValueError("the rows of caches and scales must be contiguous")
    _same_gpu(device, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales, v_scales=v_scales)
    if pages < 2:  # (a dimension of one entry has no stride)
        a = sa = 0
    if heads < 2:
        b = sb = 0
    if page < 2:
        c = sc = 0
    return MxCache.from_buffer_copy(_MX_CACHE.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), a, b, c, sa, sb, sc, form,
        pages, page, heads, D))


def kv_cache_write_mx(k, v, k_cache, k_scales, v_cache, v_scales, slots, stream=None):
    """Quantizes k, v [T, kv_heads, head_dim] (bfloat16 or float16, strided views allowed) in blocks of 32 into caches of
    codes uint8 [pages, kv_heads, page_size, head_dim] (mxfp8) or [.., head_dim / 2] (mxfp4) and of scales uint8 [..,
    head_dim / 32], each block as by mx_quantize, at slots int32 [T] (page * page_size + offset; a negative slot is
    skipped, and none may occur twice)."""
    shape, dt = k.shape, k.dtype
    if len(shape) != 3 or v.shape != shape or v.dtype != dt or (dt != torch.bfloat16 and dt != torch.float16):
        raise ValueError("k and v must be bfloat16 or float16 [T, kv_heads, head_dim]")
    T, heads, D = shape
    if slots.dtype != torch.int32 or slots.numel() != T or not slots.is_contiguous():
        raise ValueError("slots must be int32 [T], contiguous")
    kt, kh, kd = k.stride()
    vt, vh, vd = v.stride()
    if kd != 1 or vd != 1:
        raise ValueError("head_dim must be contiguous")
    if T < 2:  # (a dimension of one entry has no stride)
        kt = vt = 0
    if heads < 2:
        kh = vh = 0
    device = _gpu(k_cache)
    if device != _device_now():
        with torch.cuda.device(device):
            return kv_cache_write_mx(k, v, k_cache, k_scales, v_cache, v_scales, slots, stream)
    cache = _mx_cache(k_cache, k_scales, v_cache, v_scales, heads, D, device)
    _same_gpu(device, k=k, v=v, slots=slots)
    status = (_lib or load()).cq_kv_cache_write_mx(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _TYPES[dt], cache,
                                                   slots.data_ptr(), T, _stream_on(stream, device))
    if status:
        raise CQError(status, "cq_kv_cache_write_mx")


def paged_attention_mx(q, k_cache, k_scales, v_cache, v_scales, block_table, cu_q, kv_len, max_q, max_kv, scale=None,
                       causal=True, window=0, out=None, lse=None, workspace=None, stream=None):
    """paged_attention over a cache of microscaled blocks, as kv_cache_write_mx fills it: codes uint8 [pages, kv_heads,
    page_size, head_dim] (mxfp8) or [.., head_dim / 2] (mxfp4), scales uint8 [.., head_dim / 32]; head_dim a multiple of
    32.  Everything else as there."""
    dt, shape, i32 = q.dtype, q.shape, torch.int32
    if len(shape) != 3 or (dt != torch.bfloat16 and dt != torch.float16) or q.stride(2) != 1:
        raise ValueError("q must be bfloat16 or float16 [T, heads, head_dim], head_dim contiguous")
    if block_table.dtype != i32 or cu_q.dtype != i32 or kv_len.dtype != i32:
        raise ValueError("block_table, cu_q and kv_len must be int32")
    T, H, D = shape
    R = kv_len.numel()
    if cu_q.numel() != R + 1 or block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("cu_q must be [R + 1], kv_len [R], block_table [R, max_pages]")
    if not (cu_q.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError("cu_q and kv_len must be contiguous")
    if lse is not None and (lse.shape != (T, H) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be float32 [T, heads], contiguous")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, head_dim (mxfp8) or head_dim / 2 (mxfp4)]")
    device = _gpu(q)
    if device != _device_now():
        with torch.cuda.device(device):
            return paged_attention_mx(q, k_cache, k_scales, v_cache, v_scales, block_table, cu_q, kv_len, max_q, max_kv,
                                      scale, causal, window, out, lse, workspace, stream)
    pages, Hkv, page, _ = k_cache.shape
    cache = _mx_cache(k_cache, k_scales, v_cache, v_scales, Hkv, D, device)
    if out is None:
        out = _empty((T, H, D), dt, q, stream)
    elif out.shape != q.shape or out.dtype != dt or out.stride(2) != 1:
        raise ValueError("out must be [T, heads, head_dim] of q's type, head_dim contiguous")
    lib = _lib or load()
    need = lib.cq_paged_attention_mx_workspace_size(T, R, max_q, max_kv, H, Hkv, D)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q, stream)
    _same_gpu(device, block_table=block_table, cu_q=cu_q, kv_len=kv_len, out=out, lse=lse, workspace=workspace)
    args = PagedAttentionArgs.from_buffer_copy(_ATTENTION_ARGS.pack(
        q.data_ptr(), 0, 0, block_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), out.data_ptr(),
        0 if lse is None else lse.data_ptr(), _step(q, 0), _step(q, 1), _step(out, 0), _step(out, 1), 0, 0, 0,
        _ld(block_table), _TYPES[dt], T, R, max_q, max_kv, H, Hkv, D, page, pages, block_table.shape[1], int(causal),
        window, D ** -0.5 if scale is None else scale))
    status = lib.cq_paged_attention_mx(args, cache, None if workspace is None else workspace.data_ptr(),
                                       0 if workspace is None else workspace.numel() * workspace.element_size(),
                                       _stream_on(stream, device))
    if status:
        raise CQError(status, "cq_paged_attention_mx")
    return out


def environment_diagonals(x, stream=None):
    """Diagonals [in/128, E, 128] float32 from bfloat16 activations x [E, T, in] (a torch.bfloat16
    or int16 device tensor holding the bit patterns)."""
    if x.dim() != 3:
        raise ValueError("x must be [E, T, in]")
    E, T, inp = x.shape
    xb = x.view(torch.int16) if x.dtype == torch.bfloat16 else x
    d = torch.empty((inp // GROUP, E, GROUP), dtype=torch.float32, device=x.device)
    ws = _workspace(cq_diagonals_workspace_size(E, T, inp), x.device)
    cq_environment_diagonals(xb, E, T, inp, d, ws, stream)
    return d


def heldout_compare(pa, pb, module_offsets, boot_idx, alpha=0.05, stream=None):
    """Policy A against policy B on per-group proxy values (float64 [n] device tensors), with the
    bootstrap draws boot_idx (int32 [n_boot, n] device tensor).  Returns (counts int64 [3] =
    wins/ties/losses of A, effect [1], replicates [n_boot] sorted, ci [2]) as device tensors."""
    n = pa.numel()
    n_modules = module_offsets.numel() - 1
    n_boot = boot_idx.shape[0] if boot_idx is not None else 0
    dev = pa.device
    counts = torch.empty(3, dtype=torch.int64, device=dev)
    effect = torch.empty(1, dtype=torch.float64, device=dev)
    boot = torch.empty(max(n_boot, 1), dtype=torch.float64, device=dev)
    ci = torch.empty(2, dtype=torch.float64, device=dev)
    ws = _workspace(cq_heldout_workspace_size(n_boot, n_modules), dev)
    cq_heldout_compare(pa, pb, n, module_offsets, n_modules, boot_idx if n_boot > 0 else None, n_boot, alpha, counts,
                       effect, boot, ci, ws, stream)
    return counts, effect, boot[:n_boot], ci


def solve_breakpoint_exact(weights, environment_diagonals, qmin: int = -8, qmax: int = 7, method=None,
                           device="cuda"):
    """One group, in the shape of the pages' solver call (CliffQuant README, "Use the solver": the
    weights, the environment diagonals and a quantizer specification with qmin and qmax).

    ``weights`` has at most 256 entries, ``environment_diagonals`` is [E][len(weights)].  For
    the pages' range [-8, 7] a group shorter than 128 is zero-padded to 128 (a zero weight adds
    nothing at any scale) and any method serves it (default "candidate"); other ranges run the
    group at its own length, by default through the candidate solver where it takes the
    quantizer (at most 128 weights, -8 <= qmin, qmax <= 8) and the exhaustive method elsewhere.
    Returns (scale as float, objective, codes list).
    """
    n = len(weights)
    if not 1 <= n <= MAX_GROUP:
        raise ValueError("1..256 weights")
    E = len(environment_diagonals)
    L = GROUP if (qmin, qmax) == (-8, 7) and n <= GROUP else n
    if method is None:
        method = "candidate" if L <= GROUP and qmin >= -8 and qmax <= 8 else "exhaustive"
    w = torch.zeros((1, L), dtype=torch.float32)
    w[0, :n] = torch.tensor(weights, dtype=torch.float32)
    d = torch.zeros((1, E, L), dtype=torch.float32)
    d[0, :, :n] = torch.tensor(environment_diagonals, dtype=torch.float32)
    r = quantize_groups(w.to(device), d.to(device), method=method, qmin=qmin, qmax=qmax)
    torch.cuda.current_stream().synchronize()
    bits = int(r["scales"].cpu().view(torch.uint16)[0]) if hasattr(torch, "uint16") else \
        int(r["scales"].cpu()[0]) & 0xFFFF
    scale = float(torch.tensor([bits], dtype=torch.int16).view(torch.float16)[0])
    return scale, float(r["objective"].cpu()[0]), r["codes"].cpu()[0, :n].tolist()
