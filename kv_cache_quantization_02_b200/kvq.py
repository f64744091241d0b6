"""Thin Python binding of libkvq.so (include/kvq.h), argument marshalling only.

The raw entry points keep the C names and take integer device addresses:

    kvq_quantize(x, lam, signs, n_vec, D, group, packed, scales, stream) -> status
    kvq_dequantize(packed, scales, lam, signs, n_vec, D, group, x_out, stream) -> status
    kvq_attention_decode(q, k_packed, k_scales, v_packed, v_scales, seq_len,
                         lam_k, s_k, lam_v, s_v, B, Hq, Hkv, T, D, group,
                         sm_scale, out, workspace, workspace_bytes, stream) -> status

``quantize`` / ``dequantize`` accept torch CUDA tensors, allocate outputs
with torch when none are given, call the C entry point on the current (or
given) stream and raise ``KvqError`` on a non-zero status.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.  If the
library is missing, importing this module raises ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # loads libcudart first, so the library shares torch's runtime

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libkvq.so")

if not os.path.exists(LIBRARY):
    raise ImportError(
        f"{LIBRARY} is not built; run `python -m kv_cache_quantization_02_b200.build`")

_lib = ctypes.CDLL(LIBRARY)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int

_lib.kvq_quantize.restype = _I
_lib.kvq_quantize.argtypes = [_P, _P, _P, _I64, _I, _I, _P, _P, _P]
_lib.kvq_quantize_rows.restype = _I
_lib.kvq_quantize_rows.argtypes = [_P, _P, _P, _I64, _I, _I, _P, _I64, _P, _P, _P]
_lib.kvq_roundtrip.restype = _I
_lib.kvq_roundtrip.argtypes = [_P, _P, _P, _I64, _I, _I, _P, _P, _P, _P]
_lib.kvq_dequantize.restype = _I
_lib.kvq_dequantize.argtypes = [_P, _P, _P, _P, _I64, _I, _I, _P, _P]
_lib.kvq_dequantize_tc.restype = _I
_lib.kvq_dequantize_tc.argtypes = [_P, _P, _P, _P, _I64, _I, _I, _P, _P]
_lib.kvq_quantize_ex.restype = _I
_lib.kvq_quantize_ex.argtypes = [_P, _P, _P, _I64, _I, _I, _I, _I, _I64, _I, _P, _P, _P]
_lib.kvq_dequantize_ex.restype = _I
_lib.kvq_dequantize_ex.argtypes = [_P, _P, _P, _P, _I64, _I, _I, _I, _I, _I64, _I, _P, _P]
_lib.kvq_attention_decode.restype = _I
_lib.kvq_attention_decode.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _I64, _P]
_lib.kvq_attention_decode_ex.restype = _I
_lib.kvq_attention_decode_ex.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                         _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _I64, _P]
_lib.kvq_attention_decode_static.restype = _I
_lib.kvq_attention_decode_static.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                             _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P]
_lib.kvq_attention_workspace_bytes.restype = _I64
_lib.kvq_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.kvq_paged_write.restype = _I
_lib.kvq_paged_write.argtypes = [_P, _P, _I, _I64, _I64, _P, _P, _P, _I, _I, _I64, _I, _I, _I, _I, _I64,
                                 _P, _P, _P, _P, _P]
_lib.kvq_paged_read.restype = _I
_lib.kvq_paged_read.argtypes = [_P, _P, _P, _I, _I, _I64, _I, _I, _I, _I, _I64, _P, _P, _P, _P, _I, _P, _P, _P]
_lib.kvq_paged_attention_decode.restype = _I
_lib.kvq_paged_attention_decode.argtypes = [_P, _I, _I64, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I64, _P, _P, _P, _P,
                                            ctypes.c_float, _I, _P, _P, _I64, _P]
_lib.kvq_paged_attention_prefill.restype = _I
_lib.kvq_paged_attention_prefill.argtypes = [_P, _I, _I64, _P, _P, _P, _I, _I, _I64, _I, _I, _I, _I, _I, _I64,
                                             _P, _P, _P, _P, ctypes.c_float, _I, _P, _P, _I64, _P]
_lib.kvq_paged_decode_workspace_bytes.restype = _I64
_lib.kvq_paged_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I, _I]
_lib.kvq_paged_prefill_workspace_bytes.restype = _I64
_lib.kvq_paged_prefill_workspace_bytes.argtypes = [_I, _I, _I64, _I, _I, _I, _I, _I]
_lib.kvq_status_string.restype = ctypes.c_char_p
_lib.kvq_status_string.argtypes = [_I]
_lib.kvq_last_cuda_error.restype = _I
_lib.kvq_last_cuda_error.argtypes = []
_lib.kvq_version.restype = _I
_lib.kvq_version.argtypes = []
_lib.kvq_fault_status.restype = _I
_lib.kvq_fault_status.argtypes = [_I]
_lib.kvq_selftest_wait_timeout.restype = _I
_lib.kvq_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _P]
_lib.kvq_selftest_rcp_f16.restype = _I
_lib.kvq_selftest_rcp_f16.argtypes = [_P, _P]

KVQ_OK = 0
KVQ_ERR_NULL = -1
KVQ_ERR_ALIGN = -2
KVQ_ERR_DIM = -3
KVQ_ERR_GROUP = -4
KVQ_ERR_COUNT = -5
KVQ_ERR_LAUNCH = -6
KVQ_ERR_FORMAT = -7


class KvqError(RuntimeError):
    def __init__(self, status: int):
        msg = kvq_status_string(status)
        if status == KVQ_ERR_LAUNCH:
            msg += f" (cudaError {kvq_last_cuda_error()})"
        super().__init__(msg)
        self.status = status


# ---- raw C entry points -------------------------------------------------

def kvq_quantize(x: int, lam: int, signs: int, n_vec: int, D: int, group: int,
                 packed: int, scales: int, stream: int = 0) -> int:
    return _lib.kvq_quantize(x, lam, signs, n_vec, D, group, packed, scales, stream)


def kvq_quantize_rows(x: int, lam: int, signs: int, n_vec: int, D: int, group: int,
                      row_idx: int, cache_rows: int, packed: int, scales: int,
                      stream: int = 0) -> int:
    return _lib.kvq_quantize_rows(x, lam, signs, n_vec, D, group, row_idx, cache_rows,
                                  packed, scales, stream)


def kvq_roundtrip(x: int, lam: int, signs: int, n_vec: int, D: int, group: int,
                  x_hat: int, packed: int = 0, scales: int = 0, stream: int = 0) -> int:
    return _lib.kvq_roundtrip(x, lam, signs, n_vec, D, group, x_hat, packed, scales, stream)


def kvq_dequantize(packed: int, scales: int, lam: int, signs: int, n_vec: int,
                   D: int, group: int, x_out: int, stream: int = 0) -> int:
    return _lib.kvq_dequantize(packed, scales, lam, signs, n_vec, D, group, x_out, stream)


KVQ_LAMBDA_AFTER = 1
KVQ_SRFT = 2


def kvq_dequantize_tc(packed: int, scales: int, lam: int, signs: int, n_vec: int,
                      D: int, group: int, x_out: int, stream: int = 0) -> int:
    return _lib.kvq_dequantize_tc(packed, scales, lam, signs, n_vec, D, group, x_out, stream)


def kvq_quantize_ex(x: int, lam: int, signs: int, n_vec: int, D: int, group: int, bits: int,
                    flags: int, lambda_rows: int, n_lambda: int, codes: int, scales: int,
                    stream: int = 0) -> int:
    return _lib.kvq_quantize_ex(x, lam, signs, n_vec, D, group, bits, flags, lambda_rows,
                                n_lambda, codes, scales, stream)


def kvq_dequantize_ex(codes: int, scales: int, lam: int, signs: int, n_vec: int, D: int,
                      group: int, bits: int, flags: int, lambda_rows: int, n_lambda: int,
                      x_out: int, stream: int = 0) -> int:
    return _lib.kvq_dequantize_ex(codes, scales, lam, signs, n_vec, D, group, bits, flags,
                                  lambda_rows, n_lambda, x_out, stream)


def _ex_flags(lambda_after: bool, srft: bool) -> int:
    return (KVQ_LAMBDA_AFTER if lambda_after else 0) | (KVQ_SRFT if srft else 0)


def kvq_attention_decode(q: int, k_packed: int, k_scales: int, v_packed: int, v_scales: int,
                         seq_len: int, lam_k: int, s_k: int, lam_v: int, s_v: int,
                         B: int, Hq: int, Hkv: int, T: int, D: int, group: int,
                         sm_scale: float, out: int, workspace: int = 0,
                         workspace_bytes: int = 0, stream: int = 0) -> int:
    return _lib.kvq_attention_decode(q, k_packed, k_scales, v_packed, v_scales, seq_len,
                                     lam_k, s_k, lam_v, s_v, B, Hq, Hkv, T, D, group,
                                     sm_scale, out, workspace, workspace_bytes, stream)


def kvq_attention_decode_ex(q: int, k_packed: int, k_scales: int, v_packed: int, v_scales: int,
                            seq_len: int, lam_k: int, s_k: int, lam_v: int, s_v: int,
                            B: int, Hq: int, Hkv: int, T: int, D: int, group: int, flags: int,
                            sm_scale: float, out: int, workspace: int = 0,
                            workspace_bytes: int = 0, stream: int = 0) -> int:
    return _lib.kvq_attention_decode_ex(q, k_packed, k_scales, v_packed, v_scales, seq_len,
                                        lam_k, s_k, lam_v, s_v, B, Hq, Hkv, T, D, group, flags,
                                        sm_scale, out, workspace, workspace_bytes, stream)


def kvq_attention_decode_static(q: int, k_packed: int, k_scales: int, v_packed: int,
                                v_scales: int, seq_len: int, lam_k: int, s_k: int, lam_v: int,
                                s_v: int, B: int, Hq: int, Hkv: int, T: int, D: int, group: int,
                                sm_scale: float, out: int, stream: int = 0) -> int:
    return _lib.kvq_attention_decode_static(q, k_packed, k_scales, v_packed, v_scales, seq_len,
                                            lam_k, s_k, lam_v, s_v, B, Hq, Hkv, T, D, group,
                                            sm_scale, out, stream)


def kvq_attention_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, D: int, group: int) -> int:
    return _lib.kvq_attention_workspace_bytes(B, Hq, Hkv, T, D, group)


KVQ_FP16 = 0
KVQ_BF16 = 1
KVQ_INT8 = 0
KVQ_E4M3 = 1


def kvq_paged_write(k: int, v: int, dtype: int, k_stride: int, v_stride: int, cu_tokens: int, start: int,
                    block_table: int, B: int, max_blocks: int, n_tokens: int, Hkv: int, D: int, block: int,
                    format: int, num_blocks: int, k_codes: int, v_codes: int, k_scales: int, v_scales: int,
                    stream: int = 0) -> int:
    return _lib.kvq_paged_write(k, v, dtype, k_stride, v_stride, cu_tokens, start, block_table, B, max_blocks,
                                n_tokens, Hkv, D, block, format, num_blocks, k_codes, v_codes, k_scales, v_scales,
                                stream)


def kvq_paged_read(cu_tokens: int, start: int, block_table: int, B: int, max_blocks: int, n_tokens: int, Hkv: int,
                   D: int, block: int, format: int, num_blocks: int, k_codes: int, v_codes: int, k_scales: int,
                   v_scales: int, dtype: int, k_out: int, v_out: int, stream: int = 0) -> int:
    return _lib.kvq_paged_read(cu_tokens, start, block_table, B, max_blocks, n_tokens, Hkv, D, block, format,
                               num_blocks, k_codes, v_codes, k_scales, v_scales, dtype, k_out, v_out, stream)


def kvq_paged_attention_decode(q: int, dtype: int, q_stride: int, seq_len: int, block_table: int, B: int,
                               max_blocks: int, Hq: int, Hkv: int, D: int, block: int, format: int, num_blocks: int,
                               k_codes: int, v_codes: int, k_scales: int, v_scales: int, sm_scale: float, window: int,
                               out: int, workspace: int = 0, workspace_bytes: int = 0, stream: int = 0) -> int:
    return _lib.kvq_paged_attention_decode(q, dtype, q_stride, seq_len, block_table, B, max_blocks, Hq, Hkv, D, block,
                                           format, num_blocks, k_codes, v_codes, k_scales, v_scales, sm_scale, window,
                                           out, workspace, workspace_bytes, stream)


def kvq_paged_attention_prefill(q: int, dtype: int, q_stride: int, cu_q: int, seq_len: int, block_table: int, B: int,
                                max_blocks: int, total_q: int, Hq: int, Hkv: int, D: int, block: int, format: int,
                                num_blocks: int, k_codes: int, v_codes: int, k_scales: int, v_scales: int,
                                sm_scale: float, window: int, out: int, workspace: int = 0, workspace_bytes: int = 0,
                                stream: int = 0) -> int:
    return _lib.kvq_paged_attention_prefill(q, dtype, q_stride, cu_q, seq_len, block_table, B, max_blocks, total_q,
                                            Hq, Hkv, D, block, format, num_blocks, k_codes, v_codes, k_scales,
                                            v_scales, sm_scale, window, out, workspace, workspace_bytes, stream)


def kvq_paged_decode_workspace_bytes(B: int, max_blocks: int, Hq: int, Hkv: int, D: int, block: int,
                                     window: int = 0) -> int:
    return _lib.kvq_paged_decode_workspace_bytes(B, max_blocks, Hq, Hkv, D, block, window)


def kvq_paged_prefill_workspace_bytes(B: int, max_blocks: int, total_q: int, Hq: int, Hkv: int, D: int, block: int,
                                      window: int = 0) -> int:
    return _lib.kvq_paged_prefill_workspace_bytes(B, max_blocks, total_q, Hq, Hkv, D, block, window)


def kvq_status_string(status: int) -> str:
    return _lib.kvq_status_string(status).decode()


def kvq_last_cuda_error() -> int:
    return _lib.kvq_last_cuda_error()


def kvq_version() -> int:
    return _lib.kvq_version()


def kvq_fault_status(clear: bool = False) -> int:
    return _lib.kvq_fault_status(1 if clear else 0)


def kvq_selftest_wait_timeout(limit: int, stream: int = 0) -> int:
    return _lib.kvq_selftest_wait_timeout(limit, stream)


def kvq_selftest_rcp_f16(out: int, stream: int = 0) -> int:
    return _lib.kvq_selftest_rcp_f16(out, stream)


# ---- torch-tensor convenience --------------------------------------------

def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _need(t: torch.Tensor, dtype, shape, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def quantize(x: torch.Tensor, lam: torch.Tensor, signs: torch.Tensor, group: int,
             packed: torch.Tensor | None = None, scales: torch.Tensor | None = None,
             stream=None):
    """x: fp16 [n, D] -> (packed uint8 [n, D/2], scales fp16 [n, D/group])."""
    if x.dim() != 2:
        raise ValueError("x must be [n_vec, D]")
    n, D = x.shape
    _need(x, torch.float16, (n, D), "x")
    _need(lam, torch.float32, (D,), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    if packed is None:
        packed = torch.empty((n, D // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, max(D // group, 1)), dtype=torch.float16, device=x.device)
    _need(packed, torch.uint8, (n, D // 2), "packed")
    _need(scales, torch.float16, (n, max(D // group, 1)), "scales")
    rc = kvq_quantize(x.data_ptr(), lam.data_ptr(), signs.data_ptr(), n, D, group,
                      packed.data_ptr(), scales.data_ptr(), _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return packed, scales


def quantize_rows(x: torch.Tensor, lam: torch.Tensor, signs: torch.Tensor, group: int,
                  row_idx: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                  stream=None):
    """Encode x: fp16 [n, D] into rows row_idx (int64 [n]) of the cache
    (packed uint8 [N, D/2], scales fp16 [N, D/group]); other rows untouched."""
    if x.dim() != 2:
        raise ValueError("x must be [n_vec, D]")
    n, D = x.shape
    _need(x, torch.float16, (n, D), "x")
    _need(lam, torch.float32, (D,), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    _need(row_idx, torch.int64, (n,), "row_idx")
    N = packed.shape[0]
    _need(packed, torch.uint8, (N, D // 2), "packed")
    _need(scales, torch.float16, (N, max(D // group, 1)), "scales")
    rc = kvq_quantize_rows(x.data_ptr(), lam.data_ptr(), signs.data_ptr(), n, D, group,
                           row_idx.data_ptr(), N, packed.data_ptr(), scales.data_ptr(),
                           _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return packed, scales


def roundtrip(x: torch.Tensor, lam: torch.Tensor, signs: torch.Tensor, group: int,
              out: torch.Tensor | None = None, packed: torch.Tensor | None = None,
              scales: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x_hat = dequantize(quantize(x)) in one kernel; codes/scales optional."""
    if x.dim() != 2:
        raise ValueError("x must be [n_vec, D]")
    n, D = x.shape
    _need(x, torch.float16, (n, D), "x")
    _need(lam, torch.float32, (D,), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    if out is None:
        out = torch.empty((n, D), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, (n, D), "out")
    if (packed is None) != (scales is None):
        raise ValueError("pass both packed and scales, or neither")
    pk = sc = 0
    if packed is not None:
        _need(packed, torch.uint8, (n, D // 2), "packed")
        _need(scales, torch.float16, (n, max(D // group, 1)), "scales")
        pk, sc = packed.data_ptr(), scales.data_ptr()
    rc = kvq_roundtrip(x.data_ptr(), lam.data_ptr(), signs.data_ptr(), n, D, group,
                       out.data_ptr(), pk, sc, _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return out


def quantize_ex(x: torch.Tensor, lam: torch.Tensor, signs: torch.Tensor, group: int,
                bits: int = 4, lambda_after: bool = False, lambda_rows: int | None = None,
                codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                stream=None, srft: bool = False):
    """Format variants.  x fp16 [n, D]; lam fp32 [n_lambda, D] (or [D]); row r
    uses table (r // lambda_rows) % n_lambda.  -> (codes uint8 [n, D/2 or D],
    scales fp16 [n, D/group]).  D = 128, or 64, 96, 128, 256 with srft=True."""
    if x.dim() != 2:
        raise ValueError("x must be [n_vec, D]")
    n, D = x.shape
    _need(x, torch.float16, (n, D), "x")
    lam2 = lam.reshape(-1, D)
    _need(lam2, torch.float32, (lam2.shape[0], D), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    cb = D // 2 if bits == 4 else D
    if codes is None:
        codes = torch.empty((n, cb), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, D // group), dtype=torch.float16, device=x.device)
    _need(codes, torch.uint8, (n, cb), "codes")
    _need(scales, torch.float16, (n, D // group), "scales")
    rows = lambda_rows if lambda_rows is not None else max(n, 1)
    rc = kvq_quantize_ex(x.data_ptr(), lam2.data_ptr(), signs.data_ptr(), n, D, group, bits,
                         _ex_flags(lambda_after, srft), rows, lam2.shape[0], codes.data_ptr(),
                         scales.data_ptr(), _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return codes, scales


def dequantize_ex(codes: torch.Tensor, scales: torch.Tensor, lam: torch.Tensor,
                  signs: torch.Tensor, group: int, bits: int = 4, lambda_after: bool = False,
                  lambda_rows: int | None = None, out: torch.Tensor | None = None,
                  stream=None, srft: bool = False) -> torch.Tensor:
    """Inverse of quantize_ex -> fp16 [n, D]."""
    if codes.dim() != 2:
        raise ValueError("codes must be [n_vec, bytes]")
    n = codes.shape[0]
    D = codes.shape[1] * (2 if bits == 4 else 1)
    _need(codes, torch.uint8, (n, codes.shape[1]), "codes")
    _need(scales, torch.float16, (n, D // group), "scales")
    lam2 = lam.reshape(-1, D)
    _need(lam2, torch.float32, (lam2.shape[0], D), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    if out is None:
        out = torch.empty((n, D), dtype=torch.float16, device=codes.device)
    _need(out, torch.float16, (n, D), "out")
    rows = lambda_rows if lambda_rows is not None else max(n, 1)
    rc = kvq_dequantize_ex(codes.data_ptr(), scales.data_ptr(), lam2.data_ptr(), signs.data_ptr(),
                           n, D, group, bits, _ex_flags(lambda_after, srft), rows, lam2.shape[0],
                           out.data_ptr(), _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return out


def attention_decode(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor,
                     v_packed: torch.Tensor, v_scales: torch.Tensor, seq_len: torch.Tensor,
                     lam_k: torch.Tensor, s_k: torch.Tensor, lam_v: torch.Tensor,
                     s_v: torch.Tensor, group: int, sm_scale: float,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | bool = True,
                     stream=None, lambda_after: bool = False, srft: bool = False) -> torch.Tensor:
    """Decode attention over the int4 cache.  q fp16 [B, Hq, D]; packed uint8
    [B, Hkv, T, D/2]; scales fp16 [B, Hkv, T, D/group]; seq_len int32 [B]
    -> fp16 [B, Hq, D].  ``workspace``: a uint8 CUDA tensor, True to allocate
    the size the library asks for, or False to run without splitting.
    ``lambda_after`` / ``srft``: the cache's rows are quantize_ex rows of that
    format (int4)."""
    if q.dim() != 3 or k_packed.dim() != 4:
        raise ValueError("q must be [B, Hq, D] and the caches [B, Hkv, T, D/2]")
    B, Hq, D = q.shape
    Hkv, T = k_packed.shape[1], k_packed.shape[2]
    _need(q, torch.float16, (B, Hq, D), "q")
    for name, t in (("k_packed", k_packed), ("v_packed", v_packed)):
        _need(t, torch.uint8, (B, Hkv, T, D // 2), name)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _need(t, torch.float16, (B, Hkv, T, max(D // group, 1)), name)
    _need(seq_len, torch.int32, (B,), "seq_len")
    for name, t in (("lambda_k", lam_k), ("lambda_v", lam_v)):
        _need(t, torch.float32, (D,), name)
    for name, t in (("signs_k", s_k), ("signs_v", s_v)):
        _need(t, torch.int8, (D,), name)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, (B, Hq, D), "out")
    ws, wsb = 0, 0
    if workspace is True:
        need = kvq_attention_workspace_bytes(B, Hq, Hkv, T, D, group)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            workspace = None
    if isinstance(workspace, torch.Tensor):
        if not workspace.is_cuda or workspace.dtype != torch.uint8:
            raise ValueError("workspace must be a uint8 CUDA tensor")
        ws, wsb = workspace.data_ptr(), workspace.numel()
    rc = kvq_attention_decode_ex(q.data_ptr(), k_packed.data_ptr(), k_scales.data_ptr(),
                                 v_packed.data_ptr(), v_scales.data_ptr(), seq_len.data_ptr(),
                                 lam_k.data_ptr(), s_k.data_ptr(), lam_v.data_ptr(), s_v.data_ptr(),
                                 B, Hq, Hkv, T, D, group, _ex_flags(lambda_after, srft),
                                 float(sm_scale), out.data_ptr(), ws, wsb, _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return out


def dequantize(packed: torch.Tensor, scales: torch.Tensor, lam: torch.Tensor,
               signs: torch.Tensor, group: int, out: torch.Tensor | None = None,
               stream=None, tensor_cores: bool = False) -> torch.Tensor:
    """(packed uint8 [n, D/2], scales fp16 [n, D/group]) -> fp16 [n, D].
    ``tensor_cores``: run kvq_dequantize_tc (the in-group Hadamard on the
    tensor cores; D = 128, group 16/32/64), bit-identical."""
    if packed.dim() != 2:
        raise ValueError("packed must be [n_vec, D/2]")
    n, D = packed.shape[0], packed.shape[1] * 2
    _need(packed, torch.uint8, (n, D // 2), "packed")
    _need(scales, torch.float16, (n, max(D // group, 1)), "scales")
    _need(lam, torch.float32, (D,), "lambda")
    _need(signs, torch.int8, (D,), "signs")
    if out is None:
        out = torch.empty((n, D), dtype=torch.float16, device=packed.device)
    _need(out, torch.float16, (n, D), "out")
    fn = kvq_dequantize_tc if tensor_cores else kvq_dequantize
    rc = fn(packed.data_ptr(), scales.data_ptr(), lam.data_ptr(),
            signs.data_ptr(), n, D, group, out.data_ptr(),
            _stream_handle(stream))
    if rc != KVQ_OK:
        raise KvqError(rc)
    return out


# ---- the paged 8-bit cache ------------------------------------------------
#
# A decode step's calls are short, so these wrappers check each tensor once and
# call the library directly.

_PAGED_FORMAT = {torch.int8: KVQ_INT8, torch.float8_e4m3fn: KVQ_E4M3}
_PAGED_DTYPE = {torch.float16: KVQ_FP16, torch.bfloat16: KVQ_BF16}
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8

# torch.cuda.current_device() and the handle of current_stream(index) without
# the objects around them (a microsecond a call)
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _paged_need(t, dtype, shape, index, name):
    """`t` is a contiguous tensor of this type and shape on CUDA device `index`."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return
    _need(t, dtype, shape, name)
    raise ValueError(f"{name} must be on cuda:{index} as the other tensors, got {t.device}")


def _paged_cache(block_table, k_cache, v_cache, k_scales, v_scales):
    """Checks the cache and its table; (device, format, B, max_blocks, num_blocks, Hkv, block, D)."""
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache must be [num_blocks, Hkv, block, D] and block_table [B, max_blocks]")
    dtype, shape, index = k_cache.dtype, k_cache.shape, k_cache.get_device()
    fmt = _PAGED_FORMAT.get(dtype)
    if fmt is None:
        raise ValueError(f"k_cache must be torch.int8 or torch.float8_e4m3fn, got {dtype}")
    if index < 0:
        raise ValueError("k_cache must be a CUDA tensor")
    num_blocks, Hkv, block, D = shape
    B, max_blocks = block_table.shape
    one = (num_blocks, Hkv)
    if not (v_cache.dtype is dtype and v_cache.shape == shape and k_scales.dtype is _F32 and k_scales.shape == one
            and v_scales.dtype is _F32 and v_scales.shape == one and block_table.dtype is _I32
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scales.is_contiguous()
            and v_scales.is_contiguous() and block_table.is_contiguous()
            and v_cache.get_device() == k_scales.get_device() == v_scales.get_device()
            == block_table.get_device() == index):
        _paged_need(k_cache, dtype, shape, index, "k_cache")
        _paged_need(v_cache, dtype, shape, index, "v_cache")
        _paged_need(k_scales, _F32, one, index, "k_scales")
        _paged_need(v_scales, _F32, one, index, "v_scales")
        _paged_need(block_table, _I32, (B, max_blocks), index, "block_table")
    return index, fmt, B, max_blocks, num_blocks, Hkv, block, D


def _paged_lists(cu, cu_name, each, each_name, B, index):
    """Checks offsets [B + 1] and a list [B], int32."""
    if not (cu.dtype is _I32 and each.dtype is _I32 and cu.shape == (B + 1,) and each.shape == (B,)
            and cu.is_contiguous() and each.is_contiguous() and cu.get_device() == each.get_device() == index):
        _paged_need(cu, _I32, (B + 1,), index, cu_name)
        _paged_need(each, _I32, (B,), index, each_name)


def _paged_rows(x, name, D, index):
    """Checks token rows [n, heads, D] that may lie apart; (element type, n, heads, stride)."""
    dtype = _PAGED_DTYPE.get(x.dtype)
    if dtype is None:
        raise ValueError(f"{name} must be torch.float16 or torch.bfloat16, got {x.dtype}")
    shape = x.shape
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"{name} must be [tokens, heads, {D}], got {tuple(shape)}")
    if x.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index} as the cache, got {x.device}")
    n, heads, _ = shape
    s0, s1, s2 = x.stride()
    if s2 != 1 or (s1 != D and heads > 1):
        raise ValueError(f"{name}: the channels and heads of a token must be contiguous")
    return dtype, n, heads, s0 if n > 1 else heads * D


def _paged_call(index, fn, *args):
    """fn(*args) with device `index` current; raises KvqError."""
    if index == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != KVQ_OK:
        raise KvqError(rc)


def _on_stream(fn, stream, index, *args, **kwargs):
    """A call under `stream`: what it allocates belongs to that stream, and is
    not handed out again before its work."""
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the cache on cuda:{index}")
    with torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def paged_write(k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor,
                block_table: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                v_scales: torch.Tensor, stream=None) -> None:
    """Quantise new tokens into a paged 8-bit cache, in place.

    k, v: fp16 or bf16 [n, Hkv, D]; tokens may lie apart (slices of a fused
    projection).  Sequence b's tokens are rows cu_tokens[b] .. cu_tokens[b + 1]
    (int32 [B + 1]) and take the positions from start[b] (int32 [B]) on;
    position p is slot p % block of block block_table[b, p // block] (int32
    [B, max_blocks]).  k_cache, v_cache: int8 or float8_e4m3fn [num_blocks,
    Hkv, block, D] with fp32 scales [num_blocks, Hkv].  This call and the three
    below run on the current stream of the tensors' device, or on ``stream``."""
    if stream is not None:
        return _on_stream(paged_write, stream, k_cache.get_device(), k, v, cu_tokens, start, block_table, k_cache,
                          v_cache, k_scales, v_scales)
    index, fmt, B, max_blocks, num_blocks, Hkv, block, D = _paged_cache(block_table, k_cache, v_cache, k_scales,
                                                                        v_scales)
    dtype, n, heads, k_stride = _paged_rows(k, "k", D, index)
    v_dtype, v_n, v_heads, v_stride = _paged_rows(v, "v", D, index)
    if heads != Hkv or v_heads != Hkv or v_n != n or v_dtype != dtype:
        raise ValueError(f"k and v must both be [n, {Hkv}, {D}] of one type, "
                         f"got {tuple(k.shape)} {k.dtype} and {tuple(v.shape)} {v.dtype}")
    _paged_lists(cu_tokens, "cu_tokens", start, "start", B, index)
    _paged_call(index, _lib.kvq_paged_write, k.data_ptr(), v.data_ptr(), dtype, k_stride, v_stride,
                cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), B, max_blocks, n, Hkv, D, block, fmt,
                num_blocks, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                _current_stream(index))


def paged_read(cu_tokens: torch.Tensor, start: torch.Tensor, block_table: torch.Tensor, k_cache: torch.Tensor,
               v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, n_tokens: int,
               dtype: torch.dtype = torch.float16, k_out: torch.Tensor | None = None,
               v_out: torch.Tensor | None = None, stream=None):
    """The tokens of paged_write back out of the cache -> (k, v), each
    [n_tokens, Hkv, D] of `dtype`.  Rows from cu_tokens[B] on are not written."""
    if stream is not None:
        return _on_stream(paged_read, stream, k_cache.get_device(), cu_tokens, start, block_table, k_cache, v_cache,
                          k_scales, v_scales, n_tokens, dtype, k_out, v_out)
    index, fmt, B, max_blocks, num_blocks, Hkv, block, D = _paged_cache(block_table, k_cache, v_cache, k_scales,
                                                                        v_scales)
    code = _PAGED_DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
    _paged_lists(cu_tokens, "cu_tokens", start, "start", B, index)
    shape = (n_tokens, Hkv, D)
    if k_out is None:
        k_out = k_cache.new_empty(shape, dtype=dtype)
    else:
        _paged_need(k_out, dtype, shape, index, "k_out")
    if v_out is None:
        v_out = k_cache.new_empty(shape, dtype=dtype)
    else:
        _paged_need(v_out, dtype, shape, index, "v_out")
    _paged_call(index, _lib.kvq_paged_read, cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), B,
                max_blocks, n_tokens, Hkv, D, block, fmt, num_blocks, k_cache.data_ptr(), v_cache.data_ptr(),
                k_scales.data_ptr(), v_scales.data_ptr(), code, k_out.data_ptr(), v_out.data_ptr(),
                _current_stream(index))
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _paged_workspace_bytes(size, index, *shape):
    with torch.cuda.device(index):
        return size(*shape)


def _paged_workspace(workspace, like, size, index, *shape):
    """(tensor or None, address, bytes): `workspace` True allocates what the library asks for."""
    if workspace is True:
        need = _paged_workspace_bytes(size, index, *shape)
        if need <= 0:
            return None, 0, 0
        workspace = like.new_empty(need, dtype=_U8)
        return workspace, workspace.data_ptr(), need
    if not isinstance(workspace, torch.Tensor):
        return None, 0, 0
    _paged_need(workspace, _U8, (workspace.numel(),), index, "workspace")
    return workspace, workspace.data_ptr(), workspace.numel()


def paged_attention_decode(q: torch.Tensor, seq_len: torch.Tensor, block_table: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, sm_scale: float,
                           window: int = 0, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | bool = True, stream=None) -> torch.Tensor:
    """Attention of one token per sequence over a paged 8-bit cache.  q fp16 or
    bf16 [B, Hq, D] (sequences may lie apart); seq_len int32 [B], the positions
    in the cache, the query's own among them; window > 0 keeps the last
    `window` of them -> [B, Hq, D].  ``workspace``: a uint8 CUDA tensor, True
    to allocate the size the library asks for, or False to run unsplit."""
    if stream is not None:
        return _on_stream(paged_attention_decode, stream, k_cache.get_device(), q, seq_len, block_table, k_cache,
                          v_cache, k_scales, v_scales, sm_scale, window, out, workspace)
    index, fmt, B, max_blocks, num_blocks, Hkv, block, D = _paged_cache(block_table, k_cache, v_cache, k_scales,
                                                                        v_scales)
    dtype, n, Hq, q_stride = _paged_rows(q, "q", D, index)
    if n != B:
        raise ValueError(f"q must have one row for each of the {B} sequences, got {n}")
    _paged_need(seq_len, _I32, (B,), index, "seq_len")
    window = int(window)
    if out is None:
        out = q.new_empty((B, Hq, D))
    else:
        _paged_need(out, q.dtype, (B, Hq, D), index, "out")
    ws, ws_ptr, ws_bytes = _paged_workspace(workspace, q, kvq_paged_decode_workspace_bytes, index, B, max_blocks, Hq, Hkv,
                                            D, block, window)
    _paged_call(index, _lib.kvq_paged_attention_decode, q.data_ptr(), dtype, q_stride, seq_len.data_ptr(),
                block_table.data_ptr(), B, max_blocks, Hq, Hkv, D, block, fmt, num_blocks, k_cache.data_ptr(),
                v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), float(sm_scale), window, out.data_ptr(),
                ws_ptr, ws_bytes, _current_stream(index))
    return out


def paged_attention_prefill(q: torch.Tensor, cu_q: torch.Tensor, seq_len: torch.Tensor, block_table: torch.Tensor,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                            v_scales: torch.Tensor, sm_scale: float, window: int = 0,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | bool = True,
                            stream=None) -> torch.Tensor:
    """Causal attention of any number of new tokens per sequence.  q fp16 or
    bf16 [n, Hq, D], sequence b's in rows cu_q[b] .. cu_q[b + 1] (int32
    [B + 1]), the last of them at position seq_len[b] - 1; the rest as for
    paged_attention_decode -> [n, Hq, D].  Rows from cu_q[B] on are not
    written."""
    if stream is not None:
        return _on_stream(paged_attention_prefill, stream, k_cache.get_device(), q, cu_q, seq_len, block_table,
                          k_cache, v_cache, k_scales, v_scales, sm_scale, window, out, workspace)
    index, fmt, B, max_blocks, num_blocks, Hkv, block, D = _paged_cache(block_table, k_cache, v_cache, k_scales,
                                                                        v_scales)
    dtype, n, Hq, q_stride = _paged_rows(q, "q", D, index)
    _paged_lists(cu_q, "cu_q", seq_len, "seq_len", B, index)
    window = int(window)
    if out is None:
        out = q.new_empty((n, Hq, D))
    else:
        _paged_need(out, q.dtype, (n, Hq, D), index, "out")
    ws, ws_ptr, ws_bytes = _paged_workspace(workspace, q, kvq_paged_prefill_workspace_bytes, index, B, max_blocks, n, Hq,
                                            Hkv, D, block, window)
    _paged_call(index, _lib.kvq_paged_attention_prefill, q.data_ptr(), dtype, q_stride, cu_q.data_ptr(),
                seq_len.data_ptr(), block_table.data_ptr(), B, max_blocks, n, Hq, Hkv, D, block, fmt, num_blocks,
                k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), float(sm_scale), window,
                out.data_ptr(), ws_ptr, ws_bytes, _current_stream(index))
    return out
