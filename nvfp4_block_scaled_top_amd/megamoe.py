"""Thin ctypes binding of libmegamoe.so: the C entry points under the same names.

Argument marshalling only: each function takes torch tensors that already live on the GPU,
passes their device pointers, sizes and the current HIP stream to the C ABI, and raises
``MegaMoEError`` on a non-zero return code.  Every step of the layer runs in the library's HIP
kernels; there is no fallback.  If the library has not been built, loading it raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmegamoe.so")
_lib = None

#: Slots of per-workgroup h amax written by moe_grouped_gemm_l1_silu (MEGAMOE_L1_AMAX_PARTS).
L1_AMAX_PARTS = 1280

#: Index of the error word in the sync buffer of moe_grouped_ffn_fused (MEGAMOE_FFN_SYNC_ERROR_WORD).
FFN_SYNC_ERROR_WORD = 352

#: Bytes of the static per-GPU scratch of moe_route_permute_noalloc (MEGAMOE_ROUTE_NOALLOC_SCRATCH_BYTES).
ROUTE_NOALLOC_SCRATCH_BYTES = 1 << 20

ERRORS = {
    -1: "MEGAMOE_ERR_NULL",
    -2: "MEGAMOE_ERR_SHAPE",
    -3: "MEGAMOE_ERR_WORKSPACE",
    -4: "MEGAMOE_ERR_LAUNCH",
    -5: "MEGAMOE_ERR_DEVICE",
    -6: "MEGAMOE_ERR_ALIGN",
}

#: Scores of moe_router_scores (MEGAMOE_SCORE_*).
SCORES = {"softmax": 0, "sigmoid": 1}

#: Element types of the calls that take two (MEGAMOE_DTYPE_*); bf16 may be viewed as int16.
DTYPES = {torch.bfloat16: 0, torch.int16: 0, torch.float32: 1}

#: Those of the int8 calls (a quantizer takes all of them, a product writes the two of 16 bits) and of the
#: 16-bit experts' products.
ANY_DTYPES = {**DTYPES, torch.float16: 2}
HALF_DTYPES = {torch.bfloat16: 0, torch.int16: 0, torch.float16: 2}

#: Exported symbols and their C signatures (restype, argtypes), as declared in include/megamoe.h.
_P = ctypes.c_void_p
_I32, _I64, _SZ, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "megamoe_row_capacity": (_I64, [_I32, _I32, _I32, _I32]),
    "megamoe_sched_len": (_I64, [_I32]),
    "megamoe_route_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "megamoe_quant_workspace_bytes": (_SZ, [_I64, _I64]),
    "moe_router_topk": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_route_logits": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                _SZ, _P]),
    "moe_router_scores": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32, _F, _P, _P, _P]),
    "moe_route_scores": (_I32, [_P, _I32, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32, _F, _I32, _I32, _I32,
                                _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_router_scores_bwd": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _F, _P, _P, _P, _P]),
    "mxfp4_quantize_act": (_I32, [_P, _I32, _I64, _I64, _P, _P, _P, _P]),
    "mxfp4_dequantize": (_I32, [_P, _P, _I64, _I64, _P, _P]),
    "mxfp4_linear": (_I32, [_P, _P, _I64, _I32, _P, _P, _I32, _P, _P]),
    "mxfp4_linear_gate_up_silu": (_I32, [_P, _P, _I64, _I32, _P, _P, _I32, _P, _P]),
    "moe_grouped_gemm_l1_silu_mxfp4": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _P, _P]),
    "moe_grouped_gemm_l2_mxfp4": (_I32, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _P, _P]),
    "int8_quantize_act": (_I32, [_P, _I32, _I64, _I64, _P, _P, _P, _P]),
    "int8_dequantize": (_I32, [_P, _P, _I64, _I64, _I32, _P, _P]),
    "int8_linear": (_I32, [_P, _P, _I64, _I32, _P, _P, _I32, _I32, _P, _P]),
    "int8_linear_gate_up_silu": (_I32, [_P, _P, _I64, _I32, _P, _P, _I32, _I32, _P, _P]),
    "moe_grouped_gemm_l1_silu_int8": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _P, _P]),
    "moe_grouped_gemm_l2_int8": (_I32, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _P, _P]),
    "moe_grouped_gemm": (_I32, [_P, _I32, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _P, _P]),
    "moe_grouped_gemm_dgrad": (_I32, [_P, _I32, _P, _P, _P, _I32, _I32, _I32, _I64, _P, _P]),
    "moe_grouped_gemm_wgrad": (_I32, [_P, _P, _I32, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32, _P, _P]),
    "moe_route_quantize": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _I64,
                                  _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_gemm_l1_silu_nvfp4": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32,
                                              _I32, _P, _P, _P, _P, _P]),
    "moe_route_permute": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_permute_noalloc": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "nvfp4_quantize_act": (_I32, [_P, _I64, _I64, _P, _P, _I32, _P, _P, _P, _P, _SZ, _P]),
    "nvfp4_quantize_act_gs": (_I32, [_P, _I64, _I64, _P, _P, _P, _P, _P]),
    "moe_grouped_gemm_l1_silu": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32,
                                        _P, _P, _P]),
    "moe_grouped_gemm_l2": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32, _P, _P]),
    "nvfp4_pack_weight_codes": (_I32, [_P, _I64, _I64, _P, _P]),
    "moe_grouped_ffn_fused_packed": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32,
                                            _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_gemm_l1_silu_packed": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64,
                                               _I32, _I32, _P, _P, _P]),
    "moe_grouped_gemm_l1_silu_nvfp4_packed": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32,
                                                     _I64, _I32, _I32, _P, _P, _P, _P, _P]),
    "moe_grouped_gemm_l2_packed": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _I32, _I32,
                                          _P, _P]),
    "moe_combine": (_I32, [_P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_combine_shared": (_I32, [_P, _P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "megamoe_dense_workspace_bytes": (_SZ, [_I64]),
    "megamoe_ffn_sync_bytes": (_SZ, [_I32]),
    "moe_grouped_ffn_fused": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I64, _P,
                                     _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "nvfp4_linear": (_I32, [_P, _P, _P, _I64, _I32, _P, _P, _P, _I32, _P, _P, _SZ, _P]),
    "nvfp4_linear_gate_up_silu": (_I32, [_P, _P, _P, _I64, _I32, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "nvfp4_linear_gate_up_silu_nvfp4": (_I32, [_P, _P, _P, _I64, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _SZ,
                                               _P]),
}


class MegaMoEError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libmegamoe.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise MegaMoEError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m nvfp4_block_scaled_top_amd.build_lib")
        h = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def _check(name: str, rc: int) -> None:
    if rc != 0:
        raise MegaMoEError(f"{name} returned {rc} ({ERRORS.get(rc, 'unknown')})")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise MegaMoEError("tensors passed to libmegamoe must be on the GPU")
    if not t.is_contiguous():
        raise MegaMoEError("tensors passed to libmegamoe must be contiguous")
    return t.data_ptr()


#: bf16 tensors; their 16 bits may be viewed as integers.
_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)


def _bf16(name: str, t: Optional[torch.Tensor]):
    """_ptr of a bf16 tensor: a tensor of another type (float16 among them) would be taken for bf16 bits."""
    if t is not None and t.dtype not in _BF16_BITS:
        raise MegaMoEError(f"{name} is {t.dtype}, expected one of {list(_BF16_BITS)}")
    return _ptr(t)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ---- size helpers ------------------------------------------------------------------------------

def megamoe_row_capacity(T: int, k: int, num_experts: int, pad_multiple: int) -> int:
    return int(lib().megamoe_row_capacity(T, k, num_experts, pad_multiple))


def megamoe_sched_len(num_experts: int) -> int:
    return int(lib().megamoe_sched_len(num_experts))


def megamoe_route_workspace_bytes(T: int, k: int, num_experts: int) -> int:
    return int(lib().megamoe_route_workspace_bytes(T, k, num_experts))


def megamoe_quant_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().megamoe_quant_workspace_bytes(rows, cols))


# ---- entry points --------------------------------------------------------------------------------

def moe_router_topk(logits, k, topk_ids, topk_weights, stream=None):
    T, Eg = logits.shape
    _check("moe_router_topk", lib().moe_router_topk(_ptr(logits), T, Eg, k, _ptr(topk_ids), _ptr(topk_weights),
                                                    _stream(stream)))


def moe_route_logits(logits, k, expert_begin, num_experts, pad_multiple, topk_ids, topk_weights, counts,
                     expert_offsets, padded_offsets, row_token, token_rows, sched, workspace, block_m_override=0,
                     stream=None):
    T, Eg = logits.shape
    _check("moe_route_logits", lib().moe_route_logits(
        _ptr(logits), T, Eg, k, expert_begin, num_experts, pad_multiple, block_m_override, _ptr(topk_ids),
        _ptr(topk_weights), _ptr(counts), _ptr(expert_offsets), _ptr(padded_offsets), _ptr(row_token),
        _ptr(token_rows), _ptr(sched), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_route_permute(topk_ids, expert_begin, num_experts, pad_multiple, counts, expert_offsets, padded_offsets,
                      row_token, token_rows, sched, workspace, block_m_override=0, stream=None):
    T, k = topk_ids.shape
    _check("moe_route_permute", lib().moe_route_permute(
        _ptr(topk_ids), T, k, expert_begin, num_experts, pad_multiple, block_m_override, _ptr(counts),
        _ptr(expert_offsets), _ptr(padded_offsets), _ptr(row_token), _ptr(token_rows), _ptr(sched),
        _ptr(workspace), _nbytes(workspace), _stream(stream)))


def moe_route_permute_noalloc(topk_ids, expert_begin, num_experts, pad_multiple, counts, expert_offsets,
                              padded_offsets, row_token, token_rows, sched, block_m_override=0, stream=None):
    """moe_route_permute with the library's static per-GPU scratch instead of a workspace."""
    T, k = topk_ids.shape
    _check("moe_route_permute_noalloc", lib().moe_route_permute_noalloc(
        _ptr(topk_ids), T, k, expert_begin, num_experts, pad_multiple, block_m_override, _ptr(counts),
        _ptr(expert_offsets), _ptr(padded_offsets), _ptr(row_token), _ptr(token_rows), _ptr(sched),
        _stream(stream)))


def moe_route_quantize(topk_ids, expert_begin, num_experts, pad_multiple, counts, expert_offsets, padded_offsets,
                       row_token, token_rows, sched, route_workspace, x_bf16, x_codes, x_scales, x_global_scale,
                       quant_workspace, block_m_override=0, stream=None, x_gs_in=None):
    """x_gs_in (float32 [1] on the device): calibrated global scale; x_global_scale and
    quant_workspace are then not used (may be None)."""
    T, k = topk_ids.shape
    H = x_bf16.shape[1]
    _check("moe_route_quantize", lib().moe_route_quantize(
        _ptr(topk_ids), T, k, expert_begin, num_experts, pad_multiple, block_m_override, _ptr(counts),
        _ptr(expert_offsets), _ptr(padded_offsets), _ptr(row_token), _ptr(token_rows), _ptr(sched),
        _ptr(route_workspace), _nbytes(route_workspace), _bf16("x_bf16", x_bf16), H, _ptr(x_gs_in), _ptr(x_codes),
        _ptr(x_scales), _ptr(x_global_scale), _ptr(quant_workspace), _nbytes(quant_workspace), _stream(stream)))


def nvfp4_quantize_act(x_bf16, codes, scales, global_scale, workspace=None, row_valid=None, amax_in=None,
                       stream=None):
    rows, cols = x_bf16.shape
    n_amax = 0 if amax_in is None else amax_in.numel()
    _check("nvfp4_quantize_act", lib().nvfp4_quantize_act(
        _bf16("x_bf16", x_bf16), rows, cols, _ptr(row_valid), _ptr(amax_in), n_amax, _ptr(codes), _ptr(scales),
        _ptr(global_scale), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def nvfp4_quantize_act_gs(x_bf16, global_scale_in, codes, scales, row_valid=None, stream=None):
    rows, cols = x_bf16.shape
    _check("nvfp4_quantize_act_gs", lib().nvfp4_quantize_act_gs(
        _bf16("x_bf16", x_bf16), rows, cols, _ptr(row_valid), _ptr(global_scale_in), _ptr(codes), _ptr(scales),
        _stream(stream)))


def nvfp4_pack_weight_codes(codes, packed, stream=None):
    """codes: uint8 [..., rows, K/2] (leading dimensions folded into rows); packed: as many bytes."""
    K = 2 * codes.shape[-1]
    rows = codes.numel() // codes.shape[-1]
    if packed.numel() != codes.numel():
        raise MegaMoEError("packed must hold as many bytes as codes")
    _check("nvfp4_pack_weight_codes", lib().nvfp4_pack_weight_codes(_ptr(codes), rows, K, _ptr(packed), _stream(stream)))


def moe_grouped_gemm_l1_silu(x_codes, x_scales, x_gs, row_token, padded_offsets, counts, sched, w13_codes,
                             w13_scales, w13_gs, h_bf16, h_amax_parts, block_m_override=0, max_rows_per_expert=0,
                             stream=None, w13_packed=None):
    """w13_packed: optional, the codes packed by nvfp4_pack_weight_codes (moe_grouped_gemm_l1_silu_packed)."""
    E, I2, Hh = w13_codes.shape
    M_cap = h_bf16.shape[0]
    if h_amax_parts.numel() < L1_AMAX_PARTS:
        raise MegaMoEError(f"h_amax_parts needs {L1_AMAX_PARTS} floats")
    head = (_ptr(x_codes), _ptr(x_scales), _ptr(x_gs), _ptr(row_token), _ptr(padded_offsets), _ptr(counts),
            _ptr(sched), _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_gs))
    tail = (E, 2 * Hh, I2 // 2, M_cap, block_m_override, max_rows_per_expert, _bf16("h_bf16", h_bf16),
            _ptr(h_amax_parts), _stream(stream))
    if w13_packed is None:
        _check("moe_grouped_gemm_l1_silu", lib().moe_grouped_gemm_l1_silu(*head, *tail))
    else:
        _check("moe_grouped_gemm_l1_silu_packed", lib().moe_grouped_gemm_l1_silu_packed(*head, _ptr(w13_packed), *tail))


def moe_grouped_gemm_l1_silu_nvfp4(x_codes, x_scales, x_gs, row_token, padded_offsets, counts, sched, w13_codes,
                                   w13_scales, w13_gs, h_gs, h_codes, h_scales, h_amax_parts, block_m_override=0,
                                   max_rows_per_expert=0, stream=None, w13_packed=None):
    E, I2, Hh = w13_codes.shape
    M_cap = h_codes.shape[0]
    if h_amax_parts.numel() < L1_AMAX_PARTS:
        raise MegaMoEError(f"h_amax_parts needs {L1_AMAX_PARTS} floats")
    head = (_ptr(x_codes), _ptr(x_scales), _ptr(x_gs), _ptr(row_token), _ptr(padded_offsets), _ptr(counts),
            _ptr(sched), _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_gs))
    tail = (E, 2 * Hh, I2 // 2, M_cap, block_m_override, max_rows_per_expert, _ptr(h_gs), _ptr(h_codes),
            _ptr(h_scales), _ptr(h_amax_parts), _stream(stream))
    if w13_packed is None:
        _check("moe_grouped_gemm_l1_silu_nvfp4", lib().moe_grouped_gemm_l1_silu_nvfp4(*head, *tail))
    else:
        _check("moe_grouped_gemm_l1_silu_nvfp4_packed",
               lib().moe_grouped_gemm_l1_silu_nvfp4_packed(*head, _ptr(w13_packed), *tail))


def moe_grouped_gemm_l2(h_codes, h_scales, h_gs, padded_offsets, counts, sched, w2_codes, w2_scales, w2_gs, y_bf16,
                        block_m_override=0, max_rows_per_expert=0, stream=None, w2_packed=None):
    E, H, Ih = w2_codes.shape
    M_cap = y_bf16.shape[0]
    head = (_ptr(h_codes), _ptr(h_scales), _ptr(h_gs), _ptr(padded_offsets), _ptr(counts), _ptr(sched),
            _ptr(w2_codes), _ptr(w2_scales), _ptr(w2_gs))
    tail = (E, H, 2 * Ih, M_cap, block_m_override, max_rows_per_expert, _bf16("y_bf16", y_bf16), _stream(stream))
    if w2_packed is None:
        _check("moe_grouped_gemm_l2", lib().moe_grouped_gemm_l2(*head, *tail))
    else:
        _check("moe_grouped_gemm_l2_packed", lib().moe_grouped_gemm_l2_packed(*head, _ptr(w2_packed), *tail))


def megamoe_ffn_sync_bytes(num_experts: int) -> int:
    return int(lib().megamoe_ffn_sync_bytes(num_experts))


def moe_grouped_ffn_fused(x_codes, x_scales, x_gs, row_token, padded_offsets, counts, sched, w13_codes, w13_scales,
                          w13_gs, w2_codes, w2_scales, w2_gs, h_amax_parts, h_codes, h_scales, y_bf16, sync,
                          h_gs_in=None, h_bf16=None, h_gs_out=None, stream=None, w13_packed=None, w2_packed=None):
    """w13_packed, w2_packed: optional, both weights' packed codes (moe_grouped_ffn_fused_packed)."""
    E, I2, Hh = w13_codes.shape
    M_cap = y_bf16.shape[0]
    if h_amax_parts.numel() < L1_AMAX_PARTS:
        raise MegaMoEError(f"h_amax_parts needs {L1_AMAX_PARTS} floats")
    head = (_ptr(x_codes), _ptr(x_scales), _ptr(x_gs), _ptr(row_token), _ptr(padded_offsets), _ptr(counts),
            _ptr(sched), _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_gs), _ptr(w2_codes), _ptr(w2_scales),
            _ptr(w2_gs))
    tail = (E, 2 * Hh, I2 // 2, M_cap, _ptr(h_gs_in), _bf16("h_bf16", h_bf16), _ptr(h_amax_parts), _ptr(h_codes),
            _ptr(h_scales), _ptr(h_gs_out), _bf16("y_bf16", y_bf16), _ptr(sync), _nbytes(sync), _stream(stream))
    if w13_packed is None or w2_packed is None:
        _check("moe_grouped_ffn_fused", lib().moe_grouped_ffn_fused(*head, *tail))
    else:
        _check("moe_grouped_ffn_fused_packed",
               lib().moe_grouped_ffn_fused_packed(*head, _ptr(w13_packed), _ptr(w2_packed), *tail))


def _combine_extents(y_bf16, token_rows, topk_weights, out_bf16):
    """T, k and H of a combine, whose tensors must hold as much as the kernel reads and writes (buffers made for
    more tokens may be longer)."""
    T, k = topk_weights.shape
    H = out_bf16.shape[1]
    if topk_weights.dtype != torch.float32 or token_rows.dtype != torch.int32:
        raise MegaMoEError(f"topk_weights is {topk_weights.dtype} and token_rows {token_rows.dtype}, "
                           "expected torch.float32 and torch.int32")
    if y_bf16.dim() != 2 or y_bf16.shape[1] != H:
        raise MegaMoEError(f"y_bf16 has shape {tuple(y_bf16.shape)}, expected (rows, {H})")
    if out_bf16.shape[0] < T or token_rows.numel() < T * k:
        raise MegaMoEError(f"out_bf16 has {out_bf16.shape[0]} rows and token_rows {token_rows.numel()} entries, "
                           f"expected {T} and {T * k}")
    return T, k, H


def moe_combine(y_bf16, token_rows, topk_weights, out_bf16, stream=None):
    """y_bf16 [rows, H] and out_bf16 [T, H] bf16 (also viewed as 16-bit integers; float16 is refused), token_rows
    int32 [T * k], topk_weights float32 [T, k]."""
    T, k, H = _combine_extents(y_bf16, token_rows, topk_weights, out_bf16)
    _check("moe_combine", lib().moe_combine(
        _bf16("y_bf16", y_bf16), _ptr(token_rows), _ptr(topk_weights), T, k, H, _bf16("out_bf16", out_bf16),
        _stream(stream)))


def moe_combine_shared(y_bf16, token_rows, topk_weights, y_shared_bf16, out_bf16, stream=None):
    """moe_combine with y_shared_bf16 [T, H] added to each token's sum."""
    T, k, H = _combine_extents(y_bf16, token_rows, topk_weights, out_bf16)
    if y_shared_bf16.dim() != 2 or y_shared_bf16.shape[0] < T or y_shared_bf16.shape[1] != H:
        raise MegaMoEError(f"y_shared_bf16 has shape {tuple(y_shared_bf16.shape)}, expected {(T, H)}")
    _check("moe_combine_shared", lib().moe_combine_shared(
        _bf16("y_bf16", y_bf16), _ptr(token_rows), _ptr(topk_weights), T, k, H,
        _bf16("y_shared_bf16", y_shared_bf16), _bf16("out_bf16", out_bf16), _stream(stream)))


# ---- dense layers ------------------------------------------------------------------------------

def megamoe_dense_workspace_bytes(M: int) -> int:
    return int(lib().megamoe_dense_workspace_bytes(M))


def nvfp4_linear(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, out_bf16, workspace, stream=None):
    M, Kh = a_codes.shape
    N = w_codes.shape[0]
    _check("nvfp4_linear", lib().nvfp4_linear(
        _ptr(a_codes), _ptr(a_scales), _ptr(a_gs), M, 2 * Kh, _ptr(w_codes), _ptr(w_scales), _ptr(w_gs), N,
        _bf16("out_bf16", out_bf16), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def nvfp4_linear_gate_up_silu(a_codes, a_scales, a_gs, w13_codes, w13_scales, w13_gs, h_bf16, h_amax_parts,
                              workspace, stream=None):
    M, Kh = a_codes.shape
    I = w13_codes.shape[0] // 2
    if h_amax_parts.numel() < L1_AMAX_PARTS:
        raise MegaMoEError(f"h_amax_parts needs {L1_AMAX_PARTS} floats")
    _check("nvfp4_linear_gate_up_silu", lib().nvfp4_linear_gate_up_silu(
        _ptr(a_codes), _ptr(a_scales), _ptr(a_gs), M, 2 * Kh, _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_gs), I,
        _bf16("h_bf16", h_bf16), _ptr(h_amax_parts), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def nvfp4_linear_gate_up_silu_nvfp4(a_codes, a_scales, a_gs, w13_codes, w13_scales, w13_gs, h_gs, h_codes, h_scales,
                                    h_amax_parts, workspace, stream=None):
    M, Kh = a_codes.shape
    I = w13_codes.shape[0] // 2
    if h_amax_parts.numel() < L1_AMAX_PARTS:
        raise MegaMoEError(f"h_amax_parts needs {L1_AMAX_PARTS} floats")
    _check("nvfp4_linear_gate_up_silu_nvfp4", lib().nvfp4_linear_gate_up_silu_nvfp4(
        _ptr(a_codes), _ptr(a_scales), _ptr(a_gs), M, 2 * Kh, _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_gs), I,
        _ptr(h_gs), _ptr(h_codes), _ptr(h_scales), _ptr(h_amax_parts), _ptr(workspace), _nbytes(workspace),
        _stream(stream)))


# ---- scored router -----------------------------------------------------------------------------

# The checks below run on every call, beside kernels of a few microseconds: one device query and one raw
# stream query a call, and five cheap tests a tensor (a router call takes 6.5 us of the host, 10.5 with torch's
# public queries).

def _arg(name: str, t: torch.Tensor, dtypes, shape, dev: int) -> int:
    """Device pointer of a tensor that must have one of these types and this shape, be contiguous and
    lie on device `dev`, the current one (the one the kernels are launched on)."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == dev and dev >= 0 and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise MegaMoEError(f"{name} is {t.dtype}, expected one of {list(dtypes)}")
    if t.shape != shape:
        raise MegaMoEError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise MegaMoEError("tensors passed to libmegamoe must be on the GPU")
    if t.get_device() != dev:
        raise MegaMoEError(f"{name} is on another device than the current one")
    raise MegaMoEError("tensors passed to libmegamoe must be contiguous")


def _on(t: torch.Tensor, stream):
    """Current device and raw stream for a call on t's device (-1 and no stream if t is not on a GPU:
    _arg then refuses it)."""
    if not t.is_cuda:
        return -1, None
    dev = torch._C._cuda_getDevice()  # torch.cuda.current_device() of an initialized runtime
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_U8 = (torch.uint8,)
_INT = (torch.int32,)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16, torch.int16)


def _score_args(logits, k, bias, score, n_group, topk_group, group_top, renormalize, scale, dev):
    T, Eg = logits.shape
    if score not in SCORES:
        raise MegaMoEError(f"score is {score!r}, expected one of {list(SCORES)}")
    return (_arg("logits", logits, DTYPES, (T, Eg), dev), DTYPES[logits.dtype], T, Eg, k,
            None if bias is None else _arg("bias", bias, _F32, (Eg,), dev), SCORES[score], n_group, topk_group, group_top,
            int(renormalize), scale)


def moe_router_scores(logits, k, topk_ids, topk_weights, bias=None, score="sigmoid", n_group=1, topk_group=1,
                      group_top=2, renormalize=True, scale=1.0, stream=None):
    """Top-k ids and weights by sigmoid or softmax scores, with a balance bias, expert groups and
    renormalised weights.  logits [T, E] float32 or bf16."""
    T = logits.shape[0]
    dev, st = _on(logits, stream)
    _check("moe_router_scores", lib().moe_router_scores(
        *_score_args(logits, k, bias, score, n_group, topk_group, group_top, renormalize, scale, dev),
        _arg("topk_ids", topk_ids, _INT, (T, k), dev), _arg("topk_weights", topk_weights, _F32, (T, k), dev), st))


def moe_route_scores(logits, k, expert_begin, num_experts, pad_multiple, topk_ids, topk_weights, counts,
                     expert_offsets, padded_offsets, row_token, token_rows, sched, workspace, bias=None,
                     score="sigmoid", n_group=1, topk_group=1, group_top=2, renormalize=True, scale=1.0,
                     block_m_override=0, stream=None):
    """moe_router_scores, then moe_route_permute on its ids."""
    T = logits.shape[0]
    dev, st = _on(logits, stream)
    _check("moe_route_scores", lib().moe_route_scores(
        *_score_args(logits, k, bias, score, n_group, topk_group, group_top, renormalize, scale, dev), expert_begin,
        num_experts, pad_multiple, block_m_override, _arg("topk_ids", topk_ids, _INT, (T, k), dev),
        _arg("topk_weights", topk_weights, _F32, (T, k), dev), _ptr(counts), _ptr(expert_offsets), _ptr(padded_offsets),
        _ptr(row_token), _ptr(token_rows), _ptr(sched), _ptr(workspace), _nbytes(workspace), st))


def moe_router_scores_bwd(logits, topk_ids, grad_weights, grad_logits, score="sigmoid", renormalize=True, scale=1.0,
                          stream=None):
    """Gradient of moe_router_scores' weights with respect to the logits (dtype of the logits)."""
    T, Eg = logits.shape
    k = topk_ids.shape[1]
    if score not in SCORES:
        raise MegaMoEError(f"score is {score!r}, expected one of {list(SCORES)}")
    dev, st = _on(logits, stream)
    _check("moe_router_scores_bwd", lib().moe_router_scores_bwd(
        _arg("logits", logits, DTYPES, (T, Eg), dev), DTYPES[logits.dtype], T, Eg, k, SCORES[score], int(renormalize),
        scale, _arg("topk_ids", topk_ids, _INT, (T, k), dev), _arg("grad_weights", grad_weights, _F32, (T, k), dev),
        _arg("grad_logits", grad_logits, (logits.dtype,), (T, Eg), dev), st))


# ---- MXFP4 -------------------------------------------------------------------------------------

def _rows_of(tokens: int, M_cap: int) -> int:
    """Rows of a call that gathers from `tokens` rows: without a token none, although the padding leaves room for some
    (an empty tensor has no address, which the library would refuse beside M_cap > 0)."""
    return M_cap if tokens else 0


def mxfp4_quantize_act(x, codes, scales, row_valid=None, stream=None):
    """x [rows, cols] bf16 (also viewed as int16) or float32 -> codes [rows, cols/2], scales [rows, cols/32]."""
    rows, cols = x.shape
    dev, st = _on(x, stream)
    _check("mxfp4_quantize_act", lib().mxfp4_quantize_act(
        _arg("x", x, DTYPES, (rows, cols), dev), DTYPES[x.dtype], rows, cols,
        None if row_valid is None else _arg("row_valid", row_valid, _INT, (rows,), dev),
        _arg("codes", codes, _U8, (rows, cols // 2), dev), _arg("scales", scales, _U8, (rows, cols // 32), dev),
        st))


def mxfp4_dequantize(codes, scales, out_bf16, stream=None):
    rows, cols = out_bf16.shape
    dev, st = _on(codes, stream)
    _check("mxfp4_dequantize", lib().mxfp4_dequantize(
        _arg("codes", codes, _U8, (rows, cols // 2), dev), _arg("scales", scales, _U8, (rows, cols // 32), dev), rows, cols,
        _arg("out_bf16", out_bf16, _BF16, (rows, cols), dev), st))


def mxfp4_linear(a_codes, a_scales, w_codes, w_scales, out_bf16, stream=None):
    M, Kh = a_codes.shape
    N = w_codes.shape[0]
    dev, st = _on(a_codes, stream)
    _check("mxfp4_linear", lib().mxfp4_linear(
        _arg("a_codes", a_codes, _U8, (M, Kh), dev), _arg("a_scales", a_scales, _U8, (M, Kh // 16), dev), M, 2 * Kh,
        _arg("w_codes", w_codes, _U8, (N, Kh), dev), _arg("w_scales", w_scales, _U8, (N, Kh // 16), dev), N,
        _arg("out_bf16", out_bf16, _BF16, (M, N), dev), st))


def mxfp4_linear_gate_up_silu(a_codes, a_scales, w13_codes, w13_scales, h_bf16, stream=None):
    M, Kh = a_codes.shape
    I = h_bf16.shape[1]
    dev, st = _on(a_codes, stream)
    _check("mxfp4_linear_gate_up_silu", lib().mxfp4_linear_gate_up_silu(
        _arg("a_codes", a_codes, _U8, (M, Kh), dev), _arg("a_scales", a_scales, _U8, (M, Kh // 16), dev), M, 2 * Kh,
        _arg("w13_codes", w13_codes, _U8, (2 * I, Kh), dev), _arg("w13_scales", w13_scales, _U8, (2 * I, Kh // 16), dev), I,
        _arg("h_bf16", h_bf16, _BF16, (M, I), dev), st))


def moe_grouped_gemm_l1_silu_mxfp4(x_codes, x_scales, row_token, padded_offsets, counts, w13_codes, w13_scales,
                                   h_bf16, max_rows_per_expert=0, stream=None):
    """row_token, padded_offsets and counts as moe_route_permute wrote them (row_token holds token ids
    of x_codes' rows); h_bf16 [M_cap, I]."""
    T, Hh = x_codes.shape
    E, I2, _ = w13_codes.shape
    M_cap, I = h_bf16.shape
    if T * Hh >= 1 << 36:  # row offsets are 32-bit counts of 16 bytes; the library is not told T
        raise MegaMoEError(f"x_codes has {T * Hh} bytes, expected less than 2^36")
    dev, st = _on(x_codes, stream)
    _check("moe_grouped_gemm_l1_silu_mxfp4", lib().moe_grouped_gemm_l1_silu_mxfp4(
        _arg("x_codes", x_codes, _U8, (T, Hh), dev), _arg("x_scales", x_scales, _U8, (T, Hh // 16), dev),
        _arg("row_token", row_token, _INT, (M_cap,), dev), _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev),
        _arg("counts", counts, _INT, (E,), dev), _arg("w13_codes", w13_codes, _U8, (E, 2 * I, Hh), dev),
        _arg("w13_scales", w13_scales, _U8, (E, 2 * I, Hh // 16), dev), E, 2 * Hh, I, _rows_of(T, M_cap),
        max_rows_per_expert,
        _arg("h_bf16", h_bf16, _BF16, (M_cap, I), dev), st))


def moe_grouped_gemm_l2_mxfp4(h_codes, h_scales, padded_offsets, counts, w2_codes, w2_scales, y_bf16,
                              max_rows_per_expert=0, stream=None):
    M_cap, Ih = h_codes.shape
    E, H, _ = w2_codes.shape
    dev, st = _on(h_codes, stream)
    _check("moe_grouped_gemm_l2_mxfp4", lib().moe_grouped_gemm_l2_mxfp4(
        _arg("h_codes", h_codes, _U8, (M_cap, Ih), dev), _arg("h_scales", h_scales, _U8, (M_cap, Ih // 16), dev),
        _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev), _arg("counts", counts, _INT, (E,), dev),
        _arg("w2_codes", w2_codes, _U8, (E, H, Ih), dev), _arg("w2_scales", w2_scales, _U8, (E, H, Ih // 16), dev), E, H,
        2 * Ih, M_cap, max_rows_per_expert, _arg("y_bf16", y_bf16, _BF16, (M_cap, H), dev), st))


# ---- 8-bit integers ------------------------------------------------------------------------------

_I8 = (torch.int8,)


def int8_quantize_act(x, codes, scales, row_valid=None, stream=None):
    """x [rows, cols] bf16 (also viewed as int16), float16 or float32 -> codes int8 [rows, cols], scales
    float32 [rows]."""
    rows, cols = x.shape
    dev, st = _on(x, stream)
    _check("int8_quantize_act", lib().int8_quantize_act(
        _arg("x", x, ANY_DTYPES, (rows, cols), dev), ANY_DTYPES[x.dtype], rows, cols,
        None if row_valid is None else _arg("row_valid", row_valid, _INT, (rows,), dev),
        _arg("codes", codes, _I8, (rows, cols), dev), _arg("scales", scales, _F32, (rows,), dev), st))


def int8_dequantize(codes, scales, out, stream=None):
    """out [rows, cols] bf16, float16 or float32."""
    rows, cols = codes.shape
    dev, st = _on(codes, stream)
    _check("int8_dequantize", lib().int8_dequantize(
        _arg("codes", codes, _I8, (rows, cols), dev), _arg("scales", scales, _F32, (rows,), dev), rows, cols,
        ANY_DTYPES.get(out.dtype, -1), _arg("out", out, ANY_DTYPES, (rows, cols), dev), st))


def int8_linear(a_codes, a_scales, w_codes, w_scales, out, stream=None):
    """out [M, N] bf16 or float16."""
    M, K = a_codes.shape
    N = w_codes.shape[0]
    dev, st = _on(a_codes, stream)
    _check("int8_linear", lib().int8_linear(
        _arg("a_codes", a_codes, _I8, (M, K), dev), _arg("a_scales", a_scales, _F32, (M,), dev), M, K,
        _arg("w_codes", w_codes, _I8, (N, K), dev), _arg("w_scales", w_scales, _F32, (N,), dev), N,
        HALF_DTYPES.get(out.dtype, -1), _arg("out", out, HALF_DTYPES, (M, N), dev), st))


def int8_linear_gate_up_silu(a_codes, a_scales, w13_codes, w13_scales, h, stream=None):
    """h [M, I] bf16 or float16."""
    M, K = a_codes.shape
    I = h.shape[1]
    dev, st = _on(a_codes, stream)
    _check("int8_linear_gate_up_silu", lib().int8_linear_gate_up_silu(
        _arg("a_codes", a_codes, _I8, (M, K), dev), _arg("a_scales", a_scales, _F32, (M,), dev), M, K,
        _arg("w13_codes", w13_codes, _I8, (2 * I, K), dev), _arg("w13_scales", w13_scales, _F32, (2 * I,), dev), I,
        HALF_DTYPES.get(h.dtype, -1), _arg("h", h, HALF_DTYPES, (M, I), dev), st))


def _gathered_bytes(name, t):
    """The products' limit on their rows; the library is not told how many a gathered tensor has."""
    if _nbytes(t) >= 1 << 36:
        raise MegaMoEError(f"{name} has {_nbytes(t)} bytes, expected less than 2^36")


def moe_grouped_gemm_l1_silu_int8(x_codes, x_scales, row_token, padded_offsets, counts, w13_codes, w13_scales, h_bf16,
                                  max_rows_per_expert=0, stream=None):
    """row_token, padded_offsets and counts as moe_route_permute wrote them (row_token holds token ids
    of x_codes' rows); h_bf16 [M_cap, I]."""
    T, H = x_codes.shape
    E, I2, _ = w13_codes.shape
    M_cap, I = h_bf16.shape
    _gathered_bytes("x_codes", x_codes)
    dev, st = _on(x_codes, stream)
    _check("moe_grouped_gemm_l1_silu_int8", lib().moe_grouped_gemm_l1_silu_int8(
        _arg("x_codes", x_codes, _I8, (T, H), dev), _arg("x_scales", x_scales, _F32, (T,), dev),
        _arg("row_token", row_token, _INT, (M_cap,), dev), _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev),
        _arg("counts", counts, _INT, (E,), dev), _arg("w13_codes", w13_codes, _I8, (E, 2 * I, H), dev),
        _arg("w13_scales", w13_scales, _F32, (E, 2 * I), dev), E, H, I, _rows_of(T, M_cap), max_rows_per_expert,
        _arg("h_bf16", h_bf16, _BF16, (M_cap, I), dev), st))


def moe_grouped_gemm_l2_int8(h_codes, h_scales, padded_offsets, counts, w2_codes, w2_scales, y_bf16,
                             max_rows_per_expert=0, stream=None):
    M_cap, I = h_codes.shape
    E, H, _ = w2_codes.shape
    dev, st = _on(h_codes, stream)
    _check("moe_grouped_gemm_l2_int8", lib().moe_grouped_gemm_l2_int8(
        _arg("h_codes", h_codes, _I8, (M_cap, I), dev), _arg("h_scales", h_scales, _F32, (M_cap,), dev),
        _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev), _arg("counts", counts, _INT, (E,), dev),
        _arg("w2_codes", w2_codes, _I8, (E, H, I), dev), _arg("w2_scales", w2_scales, _F32, (E, H), dev), E, H, I, M_cap,
        max_rows_per_expert, _arg("y_bf16", y_bf16, _BF16, (M_cap, H), dev), st))


# ---- experts in 16 bits --------------------------------------------------------------------------

def moe_grouped_gemm(x, w, padded_offsets, counts, y, row_token=None, max_rows_per_expert=0, stream=None):
    """y[r] = x[row_token[r] or r] @ w[e].T for the rows r of each expert e.  x [T or M_cap, K], w [E, N, K] and
    y [M_cap, N], all bf16 (also viewed as int16) or all float16."""
    rows, K = x.shape
    E, N, _ = w.shape
    M_cap = y.shape[0]
    _gathered_bytes("x", x)
    dev, st = _on(x, stream)
    dt = (x.dtype,)
    _check("moe_grouped_gemm", lib().moe_grouped_gemm(
        _arg("x", x, HALF_DTYPES, (rows if row_token is not None else M_cap, K), dev), HALF_DTYPES[x.dtype],
        None if row_token is None else _arg("row_token", row_token, _INT, (M_cap,), dev),
        _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev), _arg("counts", counts, _INT, (E,), dev),
        _arg("w", w, dt, (E, N, K), dev), E, K, N, _rows_of(rows, M_cap), max_rows_per_expert,
        _arg("y", y, dt, (M_cap, N), dev), st))


def moe_grouped_gemm_dgrad(dy, w, padded_offsets, counts, dx, stream=None):
    """Gradient of moe_grouped_gemm with respect to its rows: dx[r] = dy[r] @ w[e].  dy [M_cap, N], w [E, N, K],
    dx [M_cap, K]; a gathered x's gradient is the sum of the rows that read it."""
    M_cap, N = dy.shape
    E, _, K = w.shape
    dev, st = _on(dy, stream)
    dt = (dy.dtype,)
    _check("moe_grouped_gemm_dgrad", lib().moe_grouped_gemm_dgrad(
        _arg("dy", dy, HALF_DTYPES, (M_cap, N), dev), HALF_DTYPES[dy.dtype],
        _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev), _arg("counts", counts, _INT, (E,), dev),
        _arg("w", w, dt, (E, N, K), dev), E, K, N, M_cap, _arg("dx", dx, dt, (M_cap, K), dev), st))


def moe_grouped_gemm_wgrad(dy, x, padded_offsets, counts, dw, row_token=None, accumulate=False, stream=None):
    """Gradient of moe_grouped_gemm with respect to the weights: dw[e] (+)= dy[rows of e].T @ x[their sources].
    dw [E, N, K] in the type of dy and x, or float32."""
    M_cap, N = dy.shape
    rows, K = x.shape
    E = dw.shape[0]
    _gathered_bytes("x", x)
    dev, st = _on(dy, stream)
    dt = (dy.dtype,)
    _check("moe_grouped_gemm_wgrad", lib().moe_grouped_gemm_wgrad(
        _arg("dy", dy, HALF_DTYPES, (M_cap, N), dev),
        _arg("x", x, dt, (rows if row_token is not None else M_cap, K), dev), HALF_DTYPES[dy.dtype],
        None if row_token is None else _arg("row_token", row_token, _INT, (M_cap,), dev),
        _arg("padded_offsets", padded_offsets, _INT, (E + 1,), dev), _arg("counts", counts, _INT, (E,), dev), E, K, N,
        _rows_of(rows, M_cap), ANY_DTYPES.get(dw.dtype, -1), int(accumulate), _arg("dw", dw, (dy.dtype, torch.float32), (E, N, K), dev),
        st))
