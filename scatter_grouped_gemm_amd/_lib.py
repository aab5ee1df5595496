"""ctypes binding of libmoe (include/moe.h), one Python function per C entry point.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, then their data pointers and torch's current HIP stream are handed
to the C call.  Every step of the computation runs in the library's HIP
kernels; there is no fallback.  If libmoe.so has not been built, loading fails
with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")
_lib = None

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ECAPACITY, MOE_EDEVICE = 0, 1, 2, 3, 4
MOE_DTYPE_BF16, MOE_DTYPE_FP8_E4M3_UE8M0, MOE_DTYPE_FP8_E4M3_MXFP8, MOE_DTYPE_FP8_MXFP4 = 0, 1, 2, 3
MOE_DTYPE_FP32 = 16
MOE_MX_E4M3, MOE_MX_E2M1 = 0, 1
# activations of the products with an epilogue; the gated ones take two halves of a row
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu2": 4,
               "silu_mul": 9, "gelu_mul": 10, "gelu_tanh_mul": 11, "swiglu_clamp": 12}
GATED_ACTIVATIONS = ("silu_mul", "gelu_mul", "gelu_tanh_mul", "swiglu_clamp")
MOE_DEVERR_MASKED_OVERFLOW = 1
MOE_SCATTER_NOALLOC_MAX_BYTES = 4 << 20

# name -> (restype, argtypes); the exported symbols of include/moe.h
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_F = ctypes.c_float
SIGNATURES = {
    "moe_compact_rows_bound": (_I64, [_I64, _I32, _I32]),
    "moe_use_masked_layout": (_I32, [_I32, _I32]),
    "moe_choose_layout": (_I32, [_I64, _I32, _I32, _I32, _I32]),
    "moe_scatter_ws_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "moe_status_str": (ctypes.c_char_p, [_I32]),
    "moe_get_device_error": (_I32, [_P, _P, _P]),
    "moe_route_topk": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_scatter_compact": (_I32, [_P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I64, _I32,
                                   _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_scatter_compact_noalloc": (_I32, [_P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I64, _I32,
                                           _P, _P, _P, _P, _P, _P, _P]),
    "moe_scatter_masked": (_I32, [_P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32,
                                  _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_quant_fp8_ue8m0": (_I32, [_P, _I64, _I32, _I64, _P, _P, _P, _P]),
    "moe_quant_weight_fp8_ue8m0": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_requant_weight_fp8_ue8m0": (_I32, [_P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_quant_weight_mx": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_mx_scales_tile": (_I32, [_P, _I32, _I32, _I32, _P, _P]),
    "grouped_gemm_rows_executed": (_I64, [_I32, _I32, _P, _I32, _I32, _I64, _I32, _I32]),
    "grouped_gemm_contig": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P]),
    "grouped_gemm_masked": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P]),
    "grouped_gemm_contig_silu": (_I32, [_I32, _P, _P, _P, _P, _I32, _P, _P, _P, _I64, _I32, _I32,
                                        _I32, _P]),
    "grouped_gemm_masked_silu": (_I32, [_I32, _P, _P, _P, _P, _I32, _P, _P, _P, _I32, _I32, _I32,
                                        _I32, _I32, _P]),
    "silu_and_mul": (_I32, [_P, _I64, _I32, _P, _P, _I32, _I32, _P, _P, _P]),
    "moe_combine": (_I32, [_P, _I64, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_combine_bwd": (_I32, [_P, _P, _I64, _P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_route_topk_bwd": (_I32, [_P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_scatter_bwd": (_I32, [_P, _I64, _P, _I32, _I32, _I32, _P, _P]),
    "silu_and_mul_bwd": (_I32, [_P, _P, _I64, _I32, _P, _P, _I32, _P, _P, _P]),
    "grouped_gemm_contig_dgrad": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _P]),
    "grouped_gemm_contig_wgrad": (_I32, [_P, _P, _P, _P, _I32, _I32, _P, _I64, _I32, _I32, _I32, _P]),
    "moe_linear": (_I32, [_P, _I64, _P, _P, _I32, _I32, _F, _F, _P, _I64, _I32, _P, _I64, _P, _I64, _I32, _I32, _P]),
    "grouped_gemm_contig_act": (_I32, [_I32, _P, _P, _P, _P, _P, _I32, _I32, _F, _F, _I32, _P, _P, _P, _P, _I64,
                                       _I32, _I32, _I32, _P]),
    "grouped_gemm_masked_act": (_I32, [_I32, _P, _P, _P, _P, _P, _I32, _I32, _F, _F, _I32, _P, _P, _P, _P, _I32,
                                       _I32, _I32, _I32, _I32, _P]),
    "moe_act_bwd_ws_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_act_bwd": (_I32, [_P, _I32, _P, _I64, _I32, _I32, _F, _F, _P, _P, _I32, _P, _P, _I32, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "moe_adamw_plan_bytes": (_SZ, [_P, _I32]),
    "moe_adamw_plan": (_I32, [_P, _I32, _P, _SZ]),
    "moe_adamw_step": (_I32, [_P, _SZ, _P, _P, _P, ctypes.c_double, ctypes.c_double, ctypes.c_float,
                              ctypes.c_uint32, _P]),
}


class AdamwTensor(ctypes.Structure):
    """moe_adamw_tensor of include/moe.h."""
    _fields_ = [("param", _P), ("master", _P), ("grad", _P), ("m", _P), ("v", _P), ("m_scale", _P),
                ("v_scale", _P), ("numel", _I64), ("weight_decay", ctypes.c_float),
                ("param_dtype", _I32), ("grad_dtype", _I32), ("state_bits", _I32)]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_str(status)})")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is not built; run `python -m scatter_grouped_gemm_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def lib_path() -> str:
    return _LIB_PATH


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status)


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "device tensors must be contiguous"
    return t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(fp8: bool) -> int:
    return MOE_DTYPE_FP8_E4M3_UE8M0 if fp8 else MOE_DTYPE_BF16


def _gemm_dtype(fp8) -> int:
    """GEMM operand dtype: False -> BF16, True -> FP8 with 128x128 weight
    blocks, "mxfp8" -> FP8 activations with MX e4m3 weights."""
    if fp8 == "mxfp8":
        return MOE_DTYPE_FP8_E4M3_MXFP8
    if fp8 == "mxfp4":
        return MOE_DTYPE_FP8_MXFP4
    if isinstance(fp8, str):
        raise ValueError(f"unknown GEMM weight format {fp8!r}")
    return _dtype_code(bool(fp8))


# --- host helpers ---------------------------------------------------------------

def moe_compact_rows_bound(num_assignments: int, num_local_experts: int, block_e: int = 128) -> int:
    return int(lib().moe_compact_rows_bound(num_assignments, num_local_experts, block_e))


def moe_use_masked_layout(num_experts: int, num_local_experts: int) -> bool:
    return bool(lib().moe_use_masked_layout(num_experts, num_local_experts))


def moe_choose_layout(max_tokens: int, top_k: int, num_experts: int, num_local_experts: int,
                      block_e: int = 128) -> bool:
    r = lib().moe_choose_layout(max_tokens, top_k, num_experts, num_local_experts, block_e)
    if r < 0:
        raise ValueError("moe_choose_layout: sizes must be positive, num_local_experts <= num_experts "
                         "and top_k <= num_experts")
    return bool(r)


def moe_scatter_ws_bytes(T: int, k: int, num_local_experts: int, H: int) -> int:
    return int(lib().moe_scatter_ws_bytes(T, k, num_local_experts, H))


def moe_get_device_error(ws: torch.Tensor) -> int:
    out = ctypes.c_int32(0)
    _check("moe_get_device_error", lib().moe_get_device_error(_ptr(ws), ctypes.byref(out), _stream()))
    return int(out.value)



def grouped_gemm_rows_executed(fp8, masked: bool, counts, expected_m: int, M: int, N: int, K: int) -> int:
    """Rows the grouped GEMM with these arguments runs its MFMAs on (whole
    16-row blocks of its tiles) for per-expert valid counts."""
    import numpy as np
    c = np.ascontiguousarray(np.asarray(counts, np.int32))
    r = lib().grouped_gemm_rows_executed(_gemm_dtype(fp8), int(bool(masked)),
                                         c.ctypes.data_as(ctypes.c_void_p), len(c), expected_m, M, N, K)
    if r < 0:
        raise ValueError("grouped_gemm_rows_executed: bad arguments")
    return int(r)


# --- device calls ----------------------------------------------------------------

def moe_route_topk(logits: torch.Tensor, k: int, topk_ids: torch.Tensor, topk_weights: torch.Tensor):
    assert logits.dtype == torch.float32 and logits.dim() == 2
    T, E = logits.shape
    assert topk_ids.dtype == torch.int32 and topk_ids.shape == (T, k)
    assert topk_weights.dtype == torch.float32 and topk_weights.shape == (T, k)
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_ids),
                                                  _ptr(topk_weights), _stream()))


def moe_scatter_compact(x, topk_ids, expert_start, num_local_experts, block_e, rows_capacity,
                        fp8, x_out, scale_out, m_indices, expert_start_loc, num_valid, src2dst, ws):
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    T, H = x.shape
    k = topk_ids.shape[1]
    _check("moe_scatter_compact", lib().moe_scatter_compact(
        _ptr(x), T, H, _ptr(topk_ids), k, expert_start, num_local_experts, block_e, rows_capacity,
        _dtype_code(fp8), _ptr(x_out), _ptr(scale_out), _ptr(m_indices), _ptr(expert_start_loc),
        _ptr(num_valid), _ptr(src2dst), _ptr(ws), ws.numel() * ws.element_size(), _stream()))


def moe_scatter_compact_noalloc(x, topk_ids, expert_start, num_local_experts, block_e, rows_capacity,
                                fp8, x_out, scale_out, m_indices, expert_start_loc, num_valid, src2dst):
    """moe_scatter_compact on the library's static per-device scratch (no ws)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    T, H = x.shape
    k = topk_ids.shape[1]
    _check("moe_scatter_compact_noalloc", lib().moe_scatter_compact_noalloc(
        _ptr(x), T, H, _ptr(topk_ids), k, expert_start, num_local_experts, block_e, rows_capacity,
        _dtype_code(fp8), _ptr(x_out), _ptr(scale_out), _ptr(m_indices), _ptr(expert_start_loc),
        _ptr(num_valid), _ptr(src2dst), _stream()))


def moe_scatter_masked(x, topk_ids, expert_start, num_local_experts, max_m, fp8, x_out, scale_out,
                       masked_m, src2dst, ws):
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    T, H = x.shape
    k = topk_ids.shape[1]
    _check("moe_scatter_masked", lib().moe_scatter_masked(
        _ptr(x), T, H, _ptr(topk_ids), k, expert_start, num_local_experts, max_m, _dtype_code(fp8),
        _ptr(x_out), _ptr(scale_out), _ptr(masked_m), _ptr(src2dst), _ptr(ws),
        ws.numel() * ws.element_size(), _stream()))


def moe_quant_fp8_ue8m0(x, q, scale, m_indices=None):
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    _check("moe_quant_fp8_ue8m0", lib().moe_quant_fp8_ue8m0(
        x.data_ptr(), M, K, x.stride(0), _ptr(m_indices), _ptr(q), _ptr(scale), _stream()))


def moe_quant_weight_fp8_ue8m0(w, q, scale):
    assert w.dtype == torch.bfloat16 and w.dim() == 3
    G, N, K = w.shape
    _check("moe_quant_weight_fp8_ue8m0", lib().moe_quant_weight_fp8_ue8m0(
        _ptr(w), G, N, K, _ptr(q), _ptr(scale), _stream()))


def moe_requant_weight_fp8_ue8m0(q_in, s_in, q_out, s_out):
    """Block-FP8 weights (e4m3 [G,N,K] + fp32 [G,N/128,K/128]) -> e4m3 + UE8M0."""
    G, N, K = q_in.shape
    assert q_in.dtype == torch.uint8 and s_in.dtype == torch.float32 and q_out.shape == (G, N, K)
    assert s_in.shape == (G, N // 128, K // 128) and s_out.shape == s_in.shape and s_out.dtype == torch.uint8
    _check("moe_requant_weight_fp8_ue8m0", lib().moe_requant_weight_fp8_ue8m0(
        _ptr(q_in), _ptr(s_in), G, N, K, _ptr(q_out), _ptr(s_out), _stream()))


def moe_quant_weight_mx(w, fmt, q, scale_tiled):
    """bf16 w [G,N,K] -> MX codes q (e4m3 [G,N,K] or e2m1 pairs [G,N,K/2]) and
    tiled scales scale_tiled [G, N/64, K/128, 256]."""
    G, N, K = w.shape
    f = {"e4m3": MOE_MX_E4M3, "e2m1": MOE_MX_E2M1}[fmt]
    assert w.dtype == torch.bfloat16 and q.dtype == torch.uint8 and scale_tiled.dtype == torch.uint8
    assert q.shape == (G, N, K if f == MOE_MX_E4M3 else K // 2)
    assert scale_tiled.numel() == G * N * (K // 32)
    _check("moe_quant_weight_mx", lib().moe_quant_weight_mx(
        _ptr(w), G, N, K, f, _ptr(q), _ptr(scale_tiled), _stream()))


def moe_mx_scales_tile(scale_plain, scale_tiled):
    """Plain MX scales [G,N,K/32] -> the GEMM's tiled layout."""
    G, N, KB = scale_plain.shape
    assert scale_plain.dtype == torch.uint8 and scale_tiled.dtype == torch.uint8
    assert scale_tiled.numel() == scale_plain.numel()
    _check("moe_mx_scales_tile", lib().moe_mx_scales_tile(
        _ptr(scale_plain), G, N, KB * 32, _ptr(scale_tiled), _stream()))


def _bk(fp8, B):
    """(G, N, K) of a weight tensor: e2m1 weights hold two k per byte."""
    G, N, Kb = B.shape
    return G, N, Kb * 2 if fp8 == "mxfp4" else Kb


def grouped_gemm_contig(fp8, A, A_scale, B, B_scale, C, m_indices):
    M, K = A.shape
    G, N, K2 = _bk(fp8, B)
    assert K == K2 and C.shape == (M, N) and C.dtype == torch.bfloat16
    _check("grouped_gemm_contig", lib().grouped_gemm_contig(
        _gemm_dtype(fp8), _ptr(A), _ptr(A_scale), _ptr(B), _ptr(B_scale), _ptr(C), _ptr(m_indices),
        M, N, K, G, _stream()))


def grouped_gemm_masked(fp8, A, A_scale, B, B_scale, C, masked_m, expected_m):
    G, max_m, K = A.shape
    G2, N, K2 = _bk(fp8, B)
    assert G == G2 and K == K2 and C.shape == (G, max_m, N) and C.dtype == torch.bfloat16
    _check("grouped_gemm_masked", lib().grouped_gemm_masked(
        _gemm_dtype(fp8), _ptr(A), _ptr(A_scale), _ptr(B), _ptr(B_scale), _ptr(C), _ptr(masked_m),
        expected_m, max_m, N, K, G, _stream()))


def grouped_gemm_contig_silu(fp8, A, A_scale, B, B_scale, out, m_indices, out_scale=None):
    """w13 GEMM with SiLU-and-mul fused: out [M][I] is bf16, or e4m3 (uint8)
    with out_scale [I/128][M]."""
    M, K = A.shape
    G, N, K2 = _bk(fp8, B)
    I = N // 2
    q8 = out.dtype == torch.uint8
    assert K == K2 and out.shape == (M, I) and (q8 or out.dtype == torch.bfloat16)
    _check("grouped_gemm_contig_silu", lib().grouped_gemm_contig_silu(
        _gemm_dtype(fp8), _ptr(A), _ptr(A_scale), _ptr(B), _ptr(B_scale), _dtype_code(q8),
        _ptr(out), _ptr(out_scale), _ptr(m_indices), M, I, K, G, _stream()))


def grouped_gemm_masked_silu(fp8, A, A_scale, B, B_scale, out, masked_m, expected_m,
                             out_scale=None):
    """Masked-layout w13 GEMM with SiLU-and-mul fused: out [G][max_m][I];
    FP8 out_scale [G][I/128][max_m]."""
    G, max_m, K = A.shape
    G2, N, K2 = _bk(fp8, B)
    I = N // 2
    q8 = out.dtype == torch.uint8
    assert G == G2 and K == K2 and out.shape == (G, max_m, I) and (q8 or out.dtype == torch.bfloat16)
    _check("grouped_gemm_masked_silu", lib().grouped_gemm_masked_silu(
        _gemm_dtype(fp8), _ptr(A), _ptr(A_scale), _ptr(B), _ptr(B_scale), _dtype_code(q8),
        _ptr(out), _ptr(out_scale), _ptr(masked_m), expected_m, max_m, I, K, G, _stream()))


def silu_and_mul(gateup, out, fp8=False, out_scale=None, m_indices=None, masked_m=None, max_m=0):
    M, N = gateup.shape
    _check("silu_and_mul", lib().silu_and_mul(
        _ptr(gateup), M, N // 2, _ptr(m_indices), _ptr(masked_m), max_m, _dtype_code(fp8),
        _ptr(out), _ptr(out_scale), _stream()))


def moe_combine(Y, src2dst, topk_weights, out):
    T, k = src2dst.shape
    H = Y.shape[-1]
    rows = Y.numel() // H
    _check("moe_combine", lib().moe_combine(_ptr(Y), rows, _ptr(src2dst), _ptr(topk_weights), T, k,
                                            H, _ptr(out), _stream()))


# --- training: gradients and the optimizer step -------------------------------------

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# The current stream of a device without building a Stream object (a third of a
# small call's time); the public way where torch does not have it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _dev(name: str, dtype, shape, t, dev: int) -> int:
    """Data pointer of an operand of the training calls: a contiguous tensor of
    this dtype and shape on the current device (the stream's)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: is on {t.device}, not on the current device")
    raise ValueError(f"{name}: must be contiguous")


def _current() -> int:
    """The current device; -2, which no operand is on, where there is none."""
    if torch.cuda.is_initialized() or torch.cuda.is_available():
        return torch.cuda.current_device()
    return -2


_BF16, _F32, _INT32 = torch.bfloat16, torch.float32, torch.int32


def moe_combine_bwd(dout, Y, src2dst, topk_weights, dY, dtopk_weights):
    """Gradient of moe_combine: dY [rows, H] (rows that no slot names keep what
    they hold) and dtopk_weights [T, k]."""
    _need(dout.dim() == 2 and src2dst.dim() == 2, "moe_combine_bwd: dout and src2dst are matrices")
    T, H = dout.shape
    k = src2dst.shape[1]
    _need(Y.shape[-1] == H, "moe_combine_bwd: Y and dout differ in width")
    rows = Y.numel() // H if H else 0
    dev = _current()
    _check("moe_combine_bwd", lib().moe_combine_bwd(
        _dev("dout", _BF16, (T, H), dout, dev), _dev("Y", _BF16, Y.shape, Y, dev), rows,
        _dev("src2dst", _INT32, (T, k), src2dst, dev), _dev("topk_weights", _F32, (T, k), topk_weights, dev), T, k, H,
        _dev("dY", _BF16, Y.shape, dY, dev), _dev("dtopk_weights", _F32, (T, k), dtopk_weights, dev), _raw_stream(dev)))


def moe_route_topk_bwd(topk_ids, topk_weights, dtopk_weights, dlogits):
    """Gradient of moe_route_topk: dlogits [T, E], zero outside the kept experts."""
    _need(topk_ids.dim() == 2 and dlogits.dim() == 2, "moe_route_topk_bwd: topk_ids and dlogits are matrices")
    T, k = topk_ids.shape
    E = dlogits.shape[1]
    dev = _current()
    _check("moe_route_topk_bwd", lib().moe_route_topk_bwd(
        _dev("topk_ids", _INT32, (T, k), topk_ids, dev), _dev("topk_weights", _F32, (T, k), topk_weights, dev),
        _dev("dtopk_weights", _F32, (T, k), dtopk_weights, dev), T, E, k,
        _dev("dlogits", _F32, (T, E), dlogits, dev), _raw_stream(dev)))


def moe_scatter_bwd(dX, src2dst, dx):
    """Gradient of the scatter: dx [T, H], the sum of a token's gradient rows."""
    _need(src2dst.dim() == 2 and dx.dim() == 2, "moe_scatter_bwd: src2dst and dx are matrices")
    T, k = src2dst.shape
    H = dx.shape[1]
    _need(dX.shape[-1] == H, "moe_scatter_bwd: dX and dx differ in width")
    rows = dX.numel() // H if H else 0
    dev = _current()
    _check("moe_scatter_bwd", lib().moe_scatter_bwd(
        _dev("dX", _BF16, dX.shape, dX, dev), rows, _dev("src2dst", _INT32, (T, k), src2dst, dev), T, k, H,
        _dev("dx", _BF16, (T, H), dx, dev), _raw_stream(dev)))


def silu_and_mul_bwd(gateup, dact, dgateup, act=None, m_indices=None, masked_m=None, max_m=0):
    """Gradient of silu_and_mul: dgateup [M, 2I] (may be gateup itself) and, if
    given, the activation act [M, I] again."""
    _need(gateup.dim() == 2 and gateup.shape[1] % 2 == 0, "silu_and_mul_bwd: gateup is [M, 2I]")
    M, N = gateup.shape
    I = N // 2
    _need(masked_m is None or (max_m > 0 and masked_m.numel() * max_m == M),
          "silu_and_mul_bwd: masked_m and max_m do not make up M rows")
    dev = _current()
    _check("silu_and_mul_bwd", lib().silu_and_mul_bwd(
        _dev("gateup", _BF16, (M, N), gateup, dev), _dev("dact", _BF16, (M, I), dact, dev), M, I,
        None if m_indices is None else _dev("m_indices", _INT32, (M,), m_indices, dev),
        None if masked_m is None else _dev("masked_m", _INT32, masked_m.shape, masked_m, dev), max_m,
        _dev("dgateup", _BF16, (M, N), dgateup, dev),
        None if act is None else _dev("act", _BF16, (M, I), act, dev), _raw_stream(dev)))


def _act(act: str) -> int:
    try:
        return ACTIVATIONS[act]
    except KeyError:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}") from None


def _rows(name: str, dtype, shape, t, dev: int):
    """Data pointer and row stride of a matrix on the current device whose rows are contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous() or shape[0] <= 1 and (shape[1] <= 1 or t.stride(1) == 1):
            return t.data_ptr(), shape[1]
        if shape[1] <= 1 or t.stride(1) == 1:
            return t.data_ptr(), t.stride(0)
        raise ValueError(f"{name}: rows must be contiguous")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name}: is on {t.device}, not on the current device")


def _bias(bias, shape, dev: int):
    """Pointer and type of a bias, or (None, 0)."""
    if bias is None:
        return None, MOE_DTYPE_BF16
    if bias.dtype is _F32:
        return _dev("bias", _F32, shape, bias, dev), MOE_DTYPE_FP32
    return _dev("bias", _BF16, shape, bias, dev), MOE_DTYPE_BF16


def moe_linear(x, w, out, bias=None, act="none", residual=None, pre=None, alpha=1.702, limit=7.0):
    """out = act(x w^T + bias) + residual: x bf16 [T, K], w bf16 [N, K], out bf16 or
    fp32 [T, N] ([T, N/2] with a gated activation).  Rows of x, out and residual
    (out's type; may be out) may be a stride apart.  pre bf16 [T, N] receives the
    product with its bias, which moe_act_bwd needs."""
    _need(x.dim() == 2 and w.dim() == 2, "moe_linear: x is [T, K] and w [N, K]")
    code = _act(act)
    T, K = x.shape
    N = w.shape[0]
    odt = out.dtype
    _need(code < 8 or N % 2 == 0, "moe_linear: a gated activation takes an even number of columns")
    _need(odt is _BF16 or odt is _F32, "moe_linear: out is bf16 or fp32")
    dev = _current()
    shape = (T, N // 2 if code >= 8 else N)
    px, ldx = _rows("x", _BF16, (T, K), x, dev)
    po, ldo = _rows("out", odt, shape, out, dev)
    pr, ldr = (None, 0) if residual is None else _rows("residual", odt, shape, residual, dev)
    pb, bdt = _bias(bias, (N,), dev)
    _check("moe_linear", lib().moe_linear(
        px, ldx, _dev("w", _BF16, (N, K), w, dev), pb, bdt, code, alpha, limit, pr, ldr,
        MOE_DTYPE_FP32 if odt is _F32 else MOE_DTYPE_BF16, po, ldo,
        None if pre is None else _dev("pre", _BF16, (T, N), pre, dev), T, N, K, _raw_stream(dev)))


def _product_operands(name, fp8, A, A_scale, B, B_scale, out, out_scale, rows, K, G, N, K2, per_row, dev):
    """Pointers of a grouped product's tensors: (A, A_scale, B, B_scale, out dtype, out, out_scale)."""
    if K != K2:
        raise ValueError(f"{name}: A and B differ in their reduction")
    if not fp8 and out.dtype is _BF16:
        return (_dev("A", _BF16, A.shape, A, dev), None, _dev("B", _BF16, B.shape, B, dev), None, MOE_DTYPE_BF16,
                _dev("out", _BF16, per_row, out, dev), None)
    q8 = out.dtype is torch.uint8
    _need(q8 or out.dtype is _BF16, f"{name}: out is bf16 or uint8 (e4m3)")
    adt = torch.uint8 if fp8 else _BF16
    w_scale = G * N * (K // 32) if fp8 in ("mxfp8", "mxfp4") else G * (N // 128) * (K // 128)
    return (_dev("A", adt, A.shape, A, dev), _scale("A_scale", A_scale, rows * (K // 128), dev) if fp8 else None,
            _dev("B", adt, B.shape, B, dev), _scale("B_scale", B_scale, w_scale, dev) if fp8 else None,
            MOE_DTYPE_FP8_E4M3_UE8M0 if q8 else MOE_DTYPE_BF16, _dev("out", out.dtype, per_row, out, dev),
            _scale("out_scale", out_scale, rows * (per_row[-1] // 128), dev) if q8 else None)


def _scale(name: str, t, n: int, dev: int):
    _need(t is not None, f"{name}: needed with FP8")
    _need(t.numel() == n, f"{name}: want {n} bytes, got {t.numel()}")
    return _dev(name, torch.uint8, t.shape, t, dev)


def grouped_gemm_contig_act(fp8, A, A_scale, B, B_scale, out, m_indices, bias=None, act="none", out_scale=None,
                            pre=None, alpha=1.702, limit=7.0):
    """Compact-layout product with each expert's bias [G, N] and an activation: out
    [M, N], [M, N/2] with a gated one (then also e4m3 with out_scale [N/256, M]).
    pre [M, N] (bf16 weights) receives the product with its bias for moe_act_bwd.
    Rows with m_indices < 0 keep what they hold."""
    _need(A.dim() == 2 and B.dim() == 3, "grouped_gemm_contig_act: A is [M, K] and B [G, N, K]")
    code = _act(act)
    M, K = A.shape
    G, N, K2 = _bk(fp8, B)
    dev = _current()
    ops = _product_operands("grouped_gemm_contig_act", fp8, A, A_scale, B, B_scale, out, out_scale, M, K, G, N, K2,
                            (M, N // 2 if code >= 8 else N), dev)
    pb, bdt = _bias(bias, (G, N), dev)
    _check("grouped_gemm_contig_act", lib().grouped_gemm_contig_act(
        _gemm_dtype(fp8), *ops[:4], pb, bdt, code, alpha, limit, *ops[4:],
        None if pre is None else _dev("pre", _BF16, (M, N), pre, dev), _dev("m_indices", _INT32, (M,), m_indices, dev),
        M, N, K, G, _raw_stream(dev)))


def grouped_gemm_masked_act(fp8, A, A_scale, B, B_scale, out, masked_m, expected_m, bias=None, act="none",
                            out_scale=None, pre=None, alpha=1.702, limit=7.0):
    """grouped_gemm_contig_act for the masked layout: out [G, max_m, N or N/2], FP8
    out_scale [G, N/256, max_m], pre [G, max_m, N].  Rows at or past masked_m keep
    what they hold."""
    _need(A.dim() == 3 and B.dim() == 3, "grouped_gemm_masked_act: A is [G, max_m, K] and B [G, N, K]")
    code = _act(act)
    G2, max_m, K = A.shape
    G, N, K2 = _bk(fp8, B)
    _need(G == G2, "grouped_gemm_masked_act: A and B differ in their experts")
    dev = _current()
    ops = _product_operands("grouped_gemm_masked_act", fp8, A, A_scale, B, B_scale, out, out_scale, G * max_m, K, G, N,
                            K2, (G, max_m, N // 2 if code >= 8 else N), dev)
    pb, bdt = _bias(bias, (G, N), dev)
    _check("grouped_gemm_masked_act", lib().grouped_gemm_masked_act(
        _gemm_dtype(fp8), *ops[:4], pb, bdt, code, alpha, limit, *ops[4:],
        None if pre is None else _dev("pre", _BF16, (G, max_m, N), pre, dev), _dev("masked_m", _INT32, (G,), masked_m, dev),
        expected_m, max_m, N, K, G, _raw_stream(dev)))


def moe_act_bwd_ws_bytes(M: int, N: int, G: int) -> int:
    return int(lib().moe_act_bwd_ws_bytes(M, N, G))


def moe_act_bwd(pre, dout, dpre, act, dbias=None, m_indices=None, expert_start_loc=None, num_valid=None, masked_m=None,
                max_m=0, alpha=1.702, limit=7.0, accumulate=False, ws=None):
    """Gradient of the epilogue of moe_linear and the grouped products: dpre [M, N]
    (may be pre) from pre [M, N] and dout [M, N or N/2] (bf16 or fp32), and the bias gradients
    dbias [G, N] ([N] or [1, N] without a layout) in bf16 or fp32, replaced or
    (accumulate) added to.  Rows: m_indices (with expert_start_loc and num_valid for
    dbias), masked_m with max_m, or all.  act "none": pre and dpre may be None.  ws:
    scratch of moe_act_bwd_ws_bytes, allocated here if not given."""
    code = _act(act)
    _need(dout.dim() == 2 and dout.dtype in (_BF16, _F32), "moe_act_bwd: dout is a matrix of bf16 or fp32")
    M, cols = dout.shape
    N = 2 * cols if code >= 8 else cols
    _need(code == 0 or (pre is not None and dpre is not None), "moe_act_bwd: pre and dpre are needed")
    _need(masked_m is None or (max_m > 0 and masked_m.numel() * max_m == M),
          "moe_act_bwd: masked_m and max_m do not make up M rows")
    dev = _current()
    G, pd, pw, nw, ddt, pst, pnv = 1, None, None, 0, MOE_DTYPE_FP32, None, None
    if dbias is not None:
        if masked_m is not None:
            G = masked_m.numel()
        elif m_indices is not None:
            _need(expert_start_loc is not None and num_valid is not None,
                  "moe_act_bwd: dbias in the compact layout needs expert_start_loc and num_valid")
            G = num_valid.numel()
            pst = _dev("expert_start_loc", _INT32, (G,), expert_start_loc, dev)
            pnv = _dev("num_valid", _INT32, (G,), num_valid, dev)
        _need(dbias.dtype in (_BF16, _F32), "moe_act_bwd: dbias is bf16 or fp32")
        ddt = MOE_DTYPE_FP32 if dbias.dtype is _F32 else MOE_DTYPE_BF16
        pd = _dev("dbias", dbias.dtype, (N,) if dbias.dim() == 1 and G == 1 else (G, N), dbias, dev)
        if ws is None:
            nw = moe_act_bwd_ws_bytes(M, N, G)
            if nw:
                ws = torch.empty(nw, dtype=torch.uint8, device=dout.device)
                pw = ws.data_ptr()
        else:
            pw, nw = _dev("ws", ws.dtype, ws.shape, ws, dev), ws.numel() * ws.element_size()
    _check("moe_act_bwd", lib().moe_act_bwd(
        None if pre is None else _dev("pre", _BF16, (M, N), pre, dev), MOE_DTYPE_FP32 if dout.dtype is _F32 else MOE_DTYPE_BF16,
        _dev("dout", dout.dtype, (M, cols), dout, dev), M, N, code, alpha, limit, None if m_indices is None else _dev("m_indices", _INT32, (M,), m_indices, dev),
        None if masked_m is None else _dev("masked_m", _INT32, masked_m.shape, masked_m, dev), max_m, pst, pnv, G,
        None if dpre is None else _dev("dpre", _BF16, (M, N), dpre, dev), ddt, int(bool(accumulate)), pd, pw, nw,
        _raw_stream(dev)))


def grouped_gemm_contig_dgrad(dC, B, dA, m_indices):
    """Gradient of grouped_gemm_contig (bf16) with respect to A: dA [M, K] from
    dC [M, N] and B [G, N, K]; rows with m_indices < 0 keep what they hold."""
    _need(dC.dim() == 2 and B.dim() == 3, "grouped_gemm_contig_dgrad: dC is [M, N] and B [G, N, K]")
    M = dC.shape[0]
    G, N, K = B.shape
    dev = _current()
    _check("grouped_gemm_contig_dgrad", lib().grouped_gemm_contig_dgrad(
        _dev("dC", _BF16, (M, N), dC, dev), _dev("B", _BF16, (G, N, K), B, dev), _dev("dA", _BF16, (M, K), dA, dev),
        _dev("m_indices", _INT32, (M,), m_indices, dev), M, N, K, G, _raw_stream(dev)))


def grouped_gemm_contig_wgrad(dC, A, expert_start_loc, num_valid, dB, accumulate=False):
    """Gradient of grouped_gemm_contig (bf16) with respect to B: dB [G, N, K] in
    bf16 or fp32, replaced or (accumulate) added to."""
    _need(dC.dim() == 2 and dB.dim() == 3, "grouped_gemm_contig_wgrad: dC is [M, N] and dB [G, N, K]")
    M = dC.shape[0]
    G, N, K = dB.shape
    _need(dB.dtype in (_BF16, _F32), "grouped_gemm_contig_wgrad: dB is bf16 or fp32")
    dev = _current()
    _check("grouped_gemm_contig_wgrad", lib().grouped_gemm_contig_wgrad(
        _dev("dC", _BF16, (M, N), dC, dev), _dev("A", _BF16, (M, K), A, dev),
        _dev("expert_start_loc", _INT32, (G,), expert_start_loc, dev), _dev("num_valid", _INT32, (G,), num_valid, dev),
        MOE_DTYPE_FP32 if dB.dtype is _F32 else MOE_DTYPE_BF16, int(bool(accumulate)),
        _dev("dB", dB.dtype, (G, N, K), dB, dev), M, N, K, G, _raw_stream(dev)))


def grouped_gemm_grads_supported(M: int, N: int, K: int, G: int) -> bool:
    """Whether the two gradient products cover these sizes (their limits are the
    same).  Host only: the call checks sizes before pointers, and without pointers
    it ends there."""
    if not all(0 <= x < 1 << 31 for x in (M, N, K, G)):
        return False
    st = lib().grouped_gemm_contig_wgrad(None, None, None, None, MOE_DTYPE_BF16, 0, None, M, N, K, G, None)
    return st == MOE_EINVAL and N > 0 and K > 0 and G > 0


def moe_adamw_plan(tensors) -> torch.Tensor:
    """Host plan (uint8 tensor) of a list of AdamwTensor; copy it to the device."""
    arr = (AdamwTensor * len(tensors))(*tensors)
    n = lib().moe_adamw_plan_bytes(arr, len(tensors))
    plan = torch.zeros(max(n, 16), dtype=torch.uint8)
    _check("moe_adamw_plan", lib().moe_adamw_plan(arr, len(tensors), plan.data_ptr(), n))
    return plan


def moe_adamw_step(plan, lr, counter, beta1, beta2, eps, seed=0, grad_scale=None):
    """One AdamW step over the tensors of a device plan."""
    dev = _current()
    _check("moe_adamw_step", lib().moe_adamw_step(
        _dev("plan", torch.uint8, plan.shape, plan, dev), plan.numel(), _dev("lr", _F32, (1,), lr, dev),
        None if grad_scale is None else _dev("grad_scale", _F32, (1,), grad_scale, dev),
        _dev("counter", torch.int64, (2,), counter, dev), beta1, beta2, eps, seed & 0xffffffff, _raw_stream(dev)))
