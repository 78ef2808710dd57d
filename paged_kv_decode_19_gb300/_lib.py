"""ctypes binding of libpageddecode (include/pageddecode.h).

Argument marshalling only: tensors are turned into device pointers, shapes and
dtype codes, and every call goes to the C ABI.  The library must be built
(``__graft_entry__.build()`` or ``python -m paged_kv_decode_19_gb300.build``);
if it is missing, loading raises — there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

_LIB_PATH = _build.LIB
_lock = threading.Lock()
_lib = None

STATUS = {
    0: "PD_OK",
    1: "PD_ERR_INVALID_ARG",
    2: "PD_ERR_UNSUPPORTED",
    3: "PD_ERR_CUDA",
    4: "PD_ERR_BAD_PAGE",
    5: "PD_ERR_BAD_LENGTH",
    6: "PD_ERR_BAD_SLOT",
    7: "PD_ERR_TIMEOUT",
    8: "PD_ERR_WORKSPACE",
    9: "PD_ERR_NO_PAGES",
}
DTYPE_CODES = {
    torch.float32: 0,
    torch.float16: 1,
    torch.bfloat16: 2,
    torch.float8_e4m3fn: 3,
}
# codes of a block-scaled cache (the _bs entry points)
BS_DTYPE_CODES = {torch.float8_e4m3fn: 3, torch.int8: 4}
# a 4-bit cache, by the type of its scales, and the dims that share one (the _mx entry points); power-of-two
# scales want a torch that has their type
MX_DTYPE_CODES = {torch.float8_e4m3fn: (5, 16)}
if hasattr(torch, "float8_e8m0fnu"):
    MX_DTYPE_CODES[torch.float8_e8m0fnu] = (6, 32)
DTYPE_NAMES = {"f32": 0, "f16": 1, "bf16": 2, "e4m3": 3}

# Every entry point declared in include/pageddecode.h.
EXPORTS = (
    "pd_batch_decode_paged_kv",
    "pd_batch_decode_paged_kv_noalloc",
    "pd_batch_decode_paged_kv_mq",
    "pd_workspace_size_mq",
    "pd_append_paged_kv_rope",
    "pd_merge_state_inplace",
    "pd_merge_states",
    "pd_cp_shard_plan",
    "pd_append_paged_kv",
    "pd_workspace_size",
    "pd_workspace_init",
    "pd_release_stream_workspace",
    "pd_plan",
    "pd_append_paged_kv_bs",
    "pd_batch_decode_paged_kv_bs",
    "pd_workspace_size_bs",
    "pd_append_paged_kv_mx",
    "pd_batch_decode_paged_kv_mx",
    "pd_workspace_size_mx",
    "pd_build_page_tables",
    "pd_qk_norm_rope",
    "pd_rope_frequencies",
    "pd_check_device_errors",
    "pd_last_decode_variant",
    "pd_get_last_error_string",
    "pd_version",
)


class PDError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{self.status_name}: {message}")


class DecodeDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32),
        ("H_qo", ctypes.c_int32),
        ("H_kv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("sliding_window", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("max_pages", ctypes.c_int64),
        ("nnz_pages", ctypes.c_int64),
        ("max_kv_len_hint", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("flags", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("sink", ctypes.c_void_p),
        ("host_indptr", ctypes.c_void_p),
        ("host_length_info", ctypes.c_void_p),
    ]


class QkDesc(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32),
        ("H_q", ctypes.c_int32),
        ("H_k", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("rotary_mode", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("attention_factor", ctypes.c_float),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("q_out_stride", ctypes.c_int64),
        ("k_out_stride", ctypes.c_int64),
        ("q_out_head_stride", ctypes.c_int64),
        ("k_out_head_stride", ctypes.c_int64),
    ]


class AppendBsDesc(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("H_kv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("scale_rows", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("max_pages", ctypes.c_int64),
        ("nnz_pages", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("flags", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class AppendMxDesc(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32),
        ("H_kv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("max_pages", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("flags", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class TablesDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("T", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("table_stride", ctypes.c_int64),
        ("values_capacity", ctypes.c_int64),
        ("free_capacity", ctypes.c_int64),
    ]


def lib():
    """Load libpageddecode.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"libpageddecode is not built ({_LIB_PATH} missing); run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(_LIB_PATH)
            P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
            L.pd_batch_decode_paged_kv.argtypes = [P, P, P, P, P, P, P, P, P, i32, f32, f32, f32,
                                                   ctypes.POINTER(DecodeDesc), P]
            L.pd_batch_decode_paged_kv.restype = i32
            L.pd_batch_decode_paged_kv_noalloc.argtypes = L.pd_batch_decode_paged_kv.argtypes
            L.pd_batch_decode_paged_kv_noalloc.restype = i32
            a = list(L.pd_batch_decode_paged_kv.argtypes)
            L.pd_batch_decode_paged_kv_mq.argtypes = a[:9] + [i32] + a[9:]
            L.pd_batch_decode_paged_kv_mq.restype = i32
            L.pd_workspace_size_mq.argtypes = [ctypes.POINTER(DecodeDesc), i32]
            L.pd_workspace_size_mq.restype = ctypes.c_size_t
            L.pd_merge_state_inplace.argtypes = [P, P, P, P, i32, i32, i32, i32, P]
            L.pd_merge_state_inplace.restype = i32
            L.pd_merge_states.argtypes = [P, P, P, P, i64, i64, i32, i32, i32, i32, i32, P]
            L.pd_merge_states.restype = i32
            L.pd_cp_shard_plan.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, i64, P, P]
            L.pd_cp_shard_plan.restype = i32
            L.pd_append_paged_kv.argtypes = [P, P, P, P, i32, i32, i32, i32, i64, i32, i32, f32,
                                             f32, P]
            L.pd_append_paged_kv.restype = i32
            L.pd_append_paged_kv_rope.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i64, i32,
                                                  i32, f32, f32, i32, f32, f32, P]
            L.pd_append_paged_kv_rope.restype = i32
            L.pd_append_paged_kv_bs.argtypes = [P] * 10
            L.pd_append_paged_kv_bs.restype = i32
            L.pd_batch_decode_paged_kv_bs.argtypes = [P] * 8 + [i32, i32, f32, P, P]
            L.pd_batch_decode_paged_kv_bs.restype = i32
            L.pd_workspace_size_bs.argtypes = [ctypes.POINTER(DecodeDesc), i32, i32]
            L.pd_workspace_size_bs.restype = ctypes.c_size_t
            L.pd_append_paged_kv_mx.argtypes = [P] * 7
            L.pd_append_paged_kv_mx.restype = i32
            L.pd_batch_decode_paged_kv_mx.argtypes = [P] * 8 + [i32, f32, P, P]
            L.pd_batch_decode_paged_kv_mx.restype = i32
            L.pd_workspace_size_mx.argtypes = [ctypes.POINTER(DecodeDesc), i32]
            L.pd_workspace_size_mx.restype = ctypes.c_size_t
            L.pd_build_page_tables.argtypes = [P] * 13
            L.pd_build_page_tables.restype = i32
            L.pd_qk_norm_rope.argtypes = [P] * 8 + [P, P]
            L.pd_qk_norm_rope.restype = i32
            f64 = ctypes.c_double
            L.pd_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, P]
            L.pd_rope_frequencies.restype = i32
            L.pd_workspace_size.argtypes = [ctypes.POINTER(DecodeDesc)]
            L.pd_workspace_size.restype = ctypes.c_size_t
            L.pd_workspace_init.argtypes = [P, ctypes.c_size_t, P]
            L.pd_workspace_init.restype = i32
            L.pd_release_stream_workspace.argtypes = [P]
            L.pd_release_stream_workspace.restype = i32
            L.pd_plan.argtypes = [ctypes.POINTER(DecodeDesc), i32, i32, ctypes.POINTER(i32),
                                  ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_size_t)]
            L.pd_plan.restype = i32
            L.pd_check_device_errors.argtypes = [P]
            L.pd_check_device_errors.restype = i32
            L.pd_last_decode_variant.restype = ctypes.c_char_p
            L.pd_get_last_error_string.restype = ctypes.c_char_p
            L.pd_version.restype = i32
            _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise PDError(status, lib().pd_get_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    """Device address of a contiguous tensor (the C functions take it as void*)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    """cudaStream_t of `stream` (a torch stream or a raw handle); None: the current stream."""
    if stream is None:
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


DECODE_EARLY_INPUTS = 1
DECODE_K_ROTATED = 2


def make_desc(Q, pages, indptr, values, length_info, out, *, num_splits=0, max_kv_len_hint=0,
              k_scale=1.0, v_scale=1.0, workspace=None, early_inputs=False,
              sink=None, k_rotated=False, host_meta=None) -> DecodeDesc:
    """host_meta: optional (indptr, length_info) numpy int32 host copies (the caller keeps
    them alive for the call)."""
    B, H_qo, D = Q.shape
    max_pages, two, H_kv, P, D2 = pages.shape
    if two != 2 or D2 != D:
        raise ValueError(f"pages must be [max_pages, 2, H_kv, P, {D}], got {tuple(pages.shape)}")
    # windowed: [3, B]; else the first B entries of a list (a flat window is no list of lengths)
    n_li = length_info.numel()
    if length_info.shape != (3, B) and (length_info.dim() != 1 or n_li < B or n_li == 3 * B > 0):
        raise ValueError(f"length_info must be [{B}] or [3, {B}], got {tuple(length_info.shape)}")
    return DecodeDesc(
        B=B, H_qo=H_qo, H_kv=H_kv, D=D, page_size=P, q_dtype=DTYPE_CODES[Q.dtype],
        kv_dtype=DTYPE_CODES[pages.dtype], out_dtype=DTYPE_CODES[out.dtype],
        sliding_window=int(length_info.dim() == 2), num_splits=int(num_splits),
        max_pages=max_pages, nnz_pages=int(values.numel()) if values is not None else 0,
        max_kv_len_hint=int(max_kv_len_hint), k_scale=float(k_scale), v_scale=float(v_scale),
        flags=(DECODE_EARLY_INPUTS if early_inputs else 0) | (DECODE_K_ROTATED if k_rotated else 0),
        workspace=None if workspace is None else workspace.data_ptr(),
        workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
        sink=_sink_ptr(sink, H_qo),
        host_indptr=None if host_meta is None else _host_i32(host_meta[0], B + 1),
        host_length_info=None if host_meta is None else _host_i32(host_meta[1], length_info.numel()))


def _host_i32(a, n):
    try:
        if a.size != n or a.dtype.char != "i" or not a.dtype.isnative:
            raise ValueError
        return ctypes.addressof(ctypes.c_char.from_buffer(a))  # (a writable C-contiguous buffer)
    except (AttributeError, TypeError, ValueError):
        ai = getattr(a, "__array_interface__", None)
        if ai is None or ai["typestr"] != "<i4" or ai["strides"] is not None or a.size != n:
            raise ValueError(f"host copies must be contiguous numpy int32 arrays of {n} entries") from None
        return ai["data"][0]


def host_meta_of(indptr, length_info):
    """Host copies (numpy int32) of a page table's indptr and length_info, for host_meta."""
    import numpy as np
    return (np.ascontiguousarray(indptr.cpu().numpy(), dtype=np.int32),
            np.ascontiguousarray(length_info.cpu().numpy(), dtype=np.int32).reshape(-1))


def _sink_ptr(sink, H_qo):
    if sink is None:
        return None
    if sink.dtype != torch.float32 or sink.numel() != H_qo or not sink.is_contiguous():
        raise ValueError("sink must be a contiguous float32 tensor of H_qo values")
    return sink.data_ptr()


def batch_decode_paged_kv(Q, pages, page_table_indptr, page_table_values, length_info,
                          k_rope_pos_offset, q_rope_position, output, lse, rotary_mode=0,
                          rope_scale=1.0, rope_theta=1e4, sm_scale=None, *, k_scale=1.0,
                          v_scale=1.0, num_splits=0, max_kv_len_hint=0, workspace=None,
                          early_inputs=False, sink=None, k_rotated=False, host_meta=None,
                          stream=None):
    """pd_batch_decode_paged_kv on device tensors; writes `output` and `lse`.
    host_meta=(indptr, length_info) numpy int32 host copies: the split is planned on the
    host (desc->host_indptr / host_length_info).
    early_inputs=True sets PD_DECODE_EARLY_INPUTS: only right after append_paged_kv (or
    another kernel that writes none of Q, the page table, lengths and positions)."""
    if sm_scale is None:
        sm_scale = Q.shape[-1] ** -0.5
    desc = make_desc(Q, pages, page_table_indptr, page_table_values, length_info, output,
                     num_splits=num_splits, max_kv_len_hint=max_kv_len_hint, k_scale=k_scale,
                     v_scale=v_scale, workspace=workspace, early_inputs=early_inputs,
                     sink=sink, k_rotated=k_rotated, host_meta=host_meta)
    _check(lib().pd_batch_decode_paged_kv(
        _ptr(Q), _ptr(pages), _ptr(page_table_indptr), _ptr(page_table_values),
        _ptr(length_info), _ptr(k_rope_pos_offset), _ptr(q_rope_position), _ptr(output),
        _ptr(lse), int(rotary_mode), float(rope_scale), float(rope_theta), float(sm_scale),
        ctypes.byref(desc), _stream(stream)))
    return output, lse


def batch_decode_paged_kv_noalloc(Q, pages, page_table_indptr, page_table_values,
                                  length_info, k_rope_pos_offset, q_rope_position, output, lse,
                                  rotary_mode=0, rope_scale=1.0, rope_theta=1e4, sm_scale=None,
                                  *, k_scale=1.0, v_scale=1.0, num_splits=0, max_kv_len_hint=0,
                                  early_inputs=False, sink=None, k_rotated=False, stream=None):
    """pd_batch_decode_paged_kv_noalloc: same result, split scratch in the library's
    static device array (no device allocation)."""
    if sm_scale is None:
        sm_scale = Q.shape[-1] ** -0.5
    desc = make_desc(Q, pages, page_table_indptr, page_table_values, length_info, output,
                     num_splits=num_splits, max_kv_len_hint=max_kv_len_hint, k_scale=k_scale,
                     v_scale=v_scale, early_inputs=early_inputs, sink=sink, k_rotated=k_rotated)
    _check(lib().pd_batch_decode_paged_kv_noalloc(
        _ptr(Q), _ptr(pages), _ptr(page_table_indptr), _ptr(page_table_values),
        _ptr(length_info), _ptr(k_rope_pos_offset), _ptr(q_rope_position), _ptr(output),
        _ptr(lse), int(rotary_mode), float(rope_scale), float(rope_theta), float(sm_scale),
        ctypes.byref(desc), _stream(stream)))
    return output, lse


def batch_decode_paged_kv_mq(Q, pages, page_table_indptr, page_table_values, length_info,
                             k_rope_pos_offset, q_rope_position, output, lse, rotary_mode=0,
                             rope_scale=1.0, rope_theta=1e4, sm_scale=None, *, k_scale=1.0,
                             v_scale=1.0, num_splits=0, max_kv_len_hint=0, workspace=None,
                             early_inputs=False, sink=None, k_rotated=False, host_meta=None,
                             stream=None):
    """pd_batch_decode_paged_kv_mq: Q [B, q_len, H_qo, D], output [B, q_len, H_qo, D],
    lse [B, q_len, H_qo]; token t of a sequence sees its rows up to itself."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, q_len, H_qo, D]")
    B, q_len, H_qo, D = Q.shape
    if sm_scale is None:
        sm_scale = D ** -0.5
    desc = make_desc(Q[:, 0], pages, page_table_indptr,
                     page_table_values, length_info, output, num_splits=num_splits,
                     max_kv_len_hint=max_kv_len_hint, k_scale=k_scale, v_scale=v_scale,
                     workspace=workspace, early_inputs=early_inputs, sink=sink,
                     k_rotated=k_rotated, host_meta=host_meta)
    _check(lib().pd_batch_decode_paged_kv_mq(
        _ptr(Q), _ptr(pages), _ptr(page_table_indptr), _ptr(page_table_values),
        _ptr(length_info), _ptr(k_rope_pos_offset), _ptr(q_rope_position), _ptr(output),
        _ptr(lse), int(q_len), int(rotary_mode), float(rope_scale), float(rope_theta),
        float(sm_scale), ctypes.byref(desc), _stream(stream)))
    return output, lse


def _refuse(dev, *tensors):
    """The error of a call whose tensors are not all on device `dev`, or not contiguous."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on the same GPU")
    raise ValueError("tensors must be contiguous")


def _device(t):
    """The index of the tensor's device, which must be the current one: the kernels run there."""
    dev = t.get_device()  # (-1: not on a GPU)
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current GPU")
    return dev


def _bs_refuse(pages, scales, page_table_indptr, page_table_values, length_info, B):
    """What is wrong with a block-scaled cache or its table."""
    if pages.dim() != 5 or pages.shape[1] != 2 or pages.dtype not in BS_DTYPE_CODES:
        raise ValueError("pages must be [max_pages, 2, H_kv, P, D] of float8_e4m3fn or int8")
    if scales.dtype != torch.float32 or scales.dim() != 4 or scales.shape[:3] != pages.shape[:3]:
        raise ValueError("scales must be float32 [max_pages, 2, H_kv, P / scale_rows]")
    if scales.shape[3] < 1 or pages.shape[3] % scales.shape[3]:
        raise ValueError("the blocks of a page must divide it")
    for t in (page_table_indptr, page_table_values, length_info):
        if t is not None and t.dtype != torch.int32:
            raise ValueError("the page table and length_info must be int32")
    if page_table_values is None and page_table_indptr.numel() == B + 1 and length_info.shape in ((B,), (3, B)):
        raise ValueError("page_table_values must be int32")
    raise ValueError(f"page_table_indptr [{B} + 1] and length_info [{B}] or [3, {B}]")


# The calls below are made once per layer and step, mostly on small batches: their checks stand in
# one expression each, and the descs are packed rather than filled field by field (a
# ctypes.Structure of twenty fields costs more to fill than the call it is passed to).
_PACK_DECODE = struct.Struct("@10i2qi2fi5Q").pack
_PACK_APPEND = struct.Struct("@8i4q2i").pack
_PACK_QK = struct.Struct("@8i3f8q").pack
_I32, _F32 = torch.int32, torch.float32


def batch_decode_paged_kv_bs(Q, pages, scales, page_table_indptr, page_table_values, length_info,
                             output, lse, sm_scale=None, *, num_splits=0, workspace=None,
                             early_inputs=False, sink=None, host_meta=None, stream=None):
    """pd_batch_decode_paged_kv_bs: decode over 8-bit pages (float8_e4m3fn or int8) with
    scales [max_pages, 2, H_kv, blocks per page] float32.  Q [B, H_qo, D], or
    [B, q_len, H_qo, D] for several query tokens per sequence (causal among them); output
    like Q, lse [B, H_qo] or [B, q_len, H_qo].  K is used as stored and Q as given: rotate
    both with qk_norm_rope."""
    shape, pshape, sshape, kv = Q.shape, pages.shape, scales.shape, BS_DTYPE_CODES.get(pages.dtype)
    rank = len(shape)
    if rank == 3:
        (B, H_qo, D), q_len = shape, 1
    elif rank == 4:
        B, q_len, H_qo, D = shape
    else:
        raise ValueError("Q must be [B, H_qo, D] or [B, q_len, H_qo, D]")
    vals, li_shape = page_table_values, length_info.shape
    if (kv is None or len(pshape) != 5 or len(sshape) != 4 or pshape[1] != 2 or sshape[1] != 2
            or sshape[0] != pshape[0] or sshape[2] != pshape[2] or scales.dtype != _F32
            or sshape[3] < 1 or pshape[3] % sshape[3] or page_table_indptr.dtype != _I32
            or length_info.dtype != _I32 or page_table_indptr.numel() != B + 1
            or (li_shape != (B,) and li_shape != (3, B)) or (vals is not None and vals.dtype != _I32)):
        _bs_refuse(pages, scales, page_table_indptr, vals, length_info, B)
    max_pages, _, H_kv, P, D_kv = pshape
    if D_kv != D:
        raise ValueError("Q must be [B, H_qo, D] or [B, q_len, H_qo, D]")
    if output.shape != shape or lse.shape != shape[:-1] or lse.dtype != _F32:
        raise ValueError("output must be shaped like Q and lse float32 like its heads")
    q_code, out_code = DTYPE_CODES.get(Q.dtype), DTYPE_CODES.get(output.dtype)
    if q_code is None or out_code is None:
        raise ValueError("Q and output must be float32, float16 or bfloat16")
    dev = _device(Q)
    if not (pages.get_device() == scales.get_device()
            == page_table_indptr.get_device() == length_info.get_device() == output.get_device()
            == lse.get_device() == dev and Q.is_contiguous() and pages.is_contiguous()
            and scales.is_contiguous() and page_table_indptr.is_contiguous()
            and length_info.is_contiguous() and output.is_contiguous() and lse.is_contiguous()):
        _refuse(dev, Q, pages, scales, page_table_indptr, length_info, output, lse)
    vals_at = n_vals = ws_at = ws_bytes = sink_at = host_ip = host_li = 0
    if vals is not None:
        if vals.get_device() != dev or not vals.is_contiguous():
            _refuse(dev, vals)
        vals_at, n_vals = vals.data_ptr(), vals.numel()
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(dev, workspace)
        ws_at, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if sink is not None:
        sink_at = _sink_ptr(sink, H_qo)
        if sink.get_device() != dev:
            _refuse(dev, sink)
    if host_meta is not None:
        host_ip, host_li = _host_i32(host_meta[0], B + 1), _host_i32(host_meta[1], length_info.numel())
    desc = _PACK_DECODE(B, H_qo, H_kv, D, P, q_code, kv, out_code,
                        len(li_shape) == 2, num_splits, max_pages, n_vals, 0, 1.0, 1.0,
                        DECODE_EARLY_INPUTS if early_inputs else 0, ws_at, ws_bytes, sink_at,
                        host_ip, host_li)
    st = (_lib or lib()).pd_batch_decode_paged_kv_bs(
        Q.data_ptr(), pages.data_ptr(), scales.data_ptr(), page_table_indptr.data_ptr(),
        vals_at or None, length_info.data_ptr(), output.data_ptr(), lse.data_ptr(), q_len,
        P // sshape[3], D ** -0.5 if sm_scale is None else sm_scale, desc,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return output, lse


def workspace_size_bs(desc: DecodeDesc, q_len: int, scale_rows: int) -> int:
    return int(lib().pd_workspace_size_bs(ctypes.byref(desc), q_len, scale_rows))


def append_paged_kv_bs(pages, scales, k_new, v_new, append_indptr, page_table_indptr,
                       page_table_values, length_info, stream=None):
    """pd_append_paged_kv_bs: quantises new tokens' K/V [T, H_kv, D] into 8-bit pages with
    block scales (both updated in place).  append_indptr [B+1] int32: sequence b brings
    tokens append_indptr[b] .. append_indptr[b+1] - 1, its last rows in the page table and
    length_info as they stand after the append.  k_new and v_new may be slices of a larger
    tensor along the heads (any token stride)."""
    pshape, sshape, kv = pages.shape, scales.shape, BS_DTYPE_CODES.get(pages.dtype)
    B, li_shape, vals = append_indptr.numel() - 1, length_info.shape, page_table_values
    if B < 0 or append_indptr.dtype != _I32:
        raise ValueError("append_indptr must be int32 [B+1]")
    if (kv is None or len(pshape) != 5 or len(sshape) != 4 or pshape[1] != 2 or sshape[1] != 2
            or sshape[0] != pshape[0] or sshape[2] != pshape[2] or scales.dtype != _F32
            or sshape[3] < 1 or pshape[3] % sshape[3] or page_table_indptr.dtype != _I32
            or length_info.dtype != _I32 or page_table_indptr.numel() != B + 1
            or (li_shape != (B,) and li_shape != (3, B)) or vals is None or vals.dtype != _I32):
        _bs_refuse(pages, scales, page_table_indptr, vals, length_info, B)
    max_pages, _, H_kv, P, D = pshape
    shape, dtype = k_new.shape, k_new.dtype
    if len(shape) != 3 or shape[1] != H_kv or shape[2] != D or v_new.shape != shape or v_new.dtype != dtype:
        raise ValueError("k_new and v_new must be [T, H_kv, D] of one dtype")
    T, in_code = shape[0], DTYPE_CODES.get(dtype)
    if in_code is None:
        raise ValueError("k_new and v_new must be float32, float16 or bfloat16")
    (ks, kh, kd), (vs, vh, vd) = k_new.stride(), v_new.stride()
    if T and (kd != 1 or vd != 1 or (H_kv > 1 and (kh != D or vh != D))):
        raise ValueError("the heads of k_new and v_new must be contiguous")
    if T < 2:
        ks = vs = H_kv * D
    dev = _device(pages)
    if not (scales.get_device() == k_new.get_device() == v_new.get_device()
            == append_indptr.get_device() == page_table_indptr.get_device() == vals.get_device()
            == length_info.get_device() == dev and pages.is_contiguous() and scales.is_contiguous()
            and append_indptr.is_contiguous() and page_table_indptr.is_contiguous()
            and vals.is_contiguous() and length_info.is_contiguous()):
        _refuse(dev, pages, scales, k_new, v_new, append_indptr, page_table_indptr, vals, length_info)
    desc = _PACK_APPEND(T, B, H_kv, D, P, P // sshape[3], in_code, kv, max_pages,
                        vals.numel(), ks, vs, 0, 0)
    st = (_lib or lib()).pd_append_paged_kv_bs(
        pages.data_ptr(), scales.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        append_indptr.data_ptr(), page_table_indptr.data_ptr(), vals.data_ptr(),
        length_info.data_ptr(), desc,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return pages, scales


# ----------------------------------------------------------------------------- 4-bit cache
_PACK_APPEND_MX = struct.Struct("@6i3q2f2i").pack
_PACK_TABLES = struct.Struct("@8i3q").pack
_U8, _I64 = torch.uint8, torch.int64
# bytes of two codes: uint8, or torch's own type of two e2m1 values where it has one
_MX_PAGES = (_U8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())


def _mx_refuse(pages, scales):
    """What is wrong with a 4-bit cache."""
    if pages.dim() != 5 or pages.shape[1] != 2 or pages.dtype not in _MX_PAGES:
        raise ValueError("pages must be [max_pages, 2, H_kv, P, D / 2] of uint8 (two codes a byte)")
    if scales.dtype not in MX_DTYPE_CODES:
        raise ValueError("scales must be float8_e4m3fn (of 16 dims) or float8_e8m0fnu (of 32)")
    n = MX_DTYPE_CODES[scales.dtype][1]
    raise ValueError(f"scales must be [max_pages, 2, H_kv, P, D / {n}] for these pages")


def batch_decode_paged_kv_mx(Q, pages, scales, page_table_indptr, page_table_values, length_info,
                             output, lse, sm_scale=None, *, k_scale=1.0, v_scale=1.0, num_splits=0,
                             workspace=None, early_inputs=False, sink=None, host_meta=None, stream=None):
    """pd_batch_decode_paged_kv_mx: decode over 4-bit pages [max_pages, 2, H_kv, P, D / 2] (uint8,
    two e2m1 codes a byte) with scales [max_pages, 2, H_kv, P, D / 16] float8_e4m3fn or
    [..., D / 32] float8_e8m0fnu, times k_scale and v_scale.  Power-of-two scales must lie in
    [2^-14, 2^13], as append_paged_kv_mx writes them (a smaller one counts as 0, a larger one as NaN; the
    cache's k_scale and v_scale move the range).  Q [B, H_qo, D], or [B, q_len, H_qo, D]
    for several query tokens per sequence (causal among them); output like Q, lse [B, H_qo] or
    [B, q_len, H_qo].  K is used as stored and Q as given: rotate both with qk_norm_rope."""
    shape, pshape, sshape = Q.shape, pages.shape, scales.shape
    kv, block = MX_DTYPE_CODES.get(scales.dtype, (None, 1))
    rank = len(shape)
    if rank == 3:
        (B, H_qo, D), q_len = shape, 1
    elif rank == 4:
        B, q_len, H_qo, D = shape
    else:
        raise ValueError("Q must be [B, H_qo, D] or [B, q_len, H_qo, D]")
    vals, li_shape = page_table_values, length_info.shape
    if (kv is None or len(pshape) != 5 or pshape[1] != 2 or pages.dtype not in _MX_PAGES
            or len(sshape) != 5 or sshape[:4] != pshape[:4] or sshape[4] * block != 2 * pshape[4]):
        _mx_refuse(pages, scales)
    if (page_table_indptr.dtype != _I32 or length_info.dtype != _I32 or page_table_indptr.numel() != B + 1
            or (li_shape != (B,) and li_shape != (3, B)) or (vals is not None and vals.dtype != _I32)):
        _table_refuse(page_table_indptr, vals, length_info, B)
    max_pages, _, H_kv, P, half = pshape
    if 2 * half != D:
        raise ValueError("Q must be [B, H_qo, D] or [B, q_len, H_qo, D]")
    if output.shape != shape or lse.shape != shape[:-1] or lse.dtype != _F32:
        raise ValueError("output must be shaped like Q and lse float32 like its heads")
    q_code, out_code = DTYPE_CODES.get(Q.dtype), DTYPE_CODES.get(output.dtype)
    if q_code is None or out_code is None:
        raise ValueError("Q and output must be float32, float16 or bfloat16")
    dev = _device(Q)
    if not (pages.get_device() == scales.get_device()
            == page_table_indptr.get_device() == length_info.get_device() == output.get_device()
            == lse.get_device() == dev and Q.is_contiguous() and pages.is_contiguous()
            and scales.is_contiguous() and page_table_indptr.is_contiguous()
            and length_info.is_contiguous() and output.is_contiguous() and lse.is_contiguous()):
        _refuse(dev, Q, pages, scales, page_table_indptr, length_info, output, lse)
    vals_at = n_vals = ws_at = ws_bytes = sink_at = host_ip = host_li = 0
    if vals is not None:
        if vals.get_device() != dev or not vals.is_contiguous():
            _refuse(dev, vals)
        vals_at, n_vals = vals.data_ptr(), vals.numel()
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(dev, workspace)
        ws_at, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if sink is not None:
        sink_at = _sink_ptr(sink, H_qo)
        if sink.get_device() != dev:
            _refuse(dev, sink)
    if host_meta is not None:
        host_ip, host_li = _host_i32(host_meta[0], B + 1), _host_i32(host_meta[1], length_info.numel())
    desc = _PACK_DECODE(B, H_qo, H_kv, D, P, q_code, kv, out_code,
                        len(li_shape) == 2, num_splits, max_pages, n_vals, 0, k_scale, v_scale,
                        DECODE_EARLY_INPUTS if early_inputs else 0, ws_at, ws_bytes, sink_at,
                        host_ip, host_li)
    st = (_lib or lib()).pd_batch_decode_paged_kv_mx(
        Q.data_ptr(), pages.data_ptr(), scales.data_ptr(), page_table_indptr.data_ptr(),
        vals_at or None, length_info.data_ptr(), output.data_ptr(), lse.data_ptr(), q_len,
        D ** -0.5 if sm_scale is None else sm_scale, desc,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return output, lse


def _table_refuse(page_table_indptr, page_table_values, length_info, B):
    """What is wrong with a page table."""
    for t in (page_table_indptr, page_table_values, length_info):
        if t is not None and t.dtype != torch.int32:
            raise ValueError("page_table_indptr, page_table_values and length_info must be int32")
    raise ValueError(f"page_table_indptr must be [{B} + 1] and length_info [{B}] or [3, {B}]")


def workspace_size_mx(desc: DecodeDesc, q_len: int) -> int:
    return int(lib().pd_workspace_size_mx(ctypes.byref(desc), q_len))


def append_paged_kv_mx(pages, scales, k_new, v_new, slot_mapping, k_scale=1.0, v_scale=1.0, stream=None):
    """pd_append_paged_kv_mx: quantises new tokens' K/V [T, H_kv, D] into the slots (int64 [T],
    negative: skipped) of 4-bit pages with scales (both updated in place).  k_new and v_new may be
    slices of a larger tensor along the heads (any token stride)."""
    pshape, sshape = pages.shape, scales.shape
    kv, block = MX_DTYPE_CODES.get(scales.dtype, (None, 1))
    if (kv is None or len(pshape) != 5 or pshape[1] != 2 or pages.dtype not in _MX_PAGES
            or len(sshape) != 5 or sshape[:4] != pshape[:4] or sshape[4] * block != 2 * pshape[4]):
        _mx_refuse(pages, scales)
    max_pages, _, H_kv, P, half = pshape
    D, shape, dtype = 2 * half, k_new.shape, k_new.dtype
    if len(shape) != 3 or shape[1] != H_kv or shape[2] != D or v_new.shape != shape or v_new.dtype != dtype:
        raise ValueError("k_new and v_new must be [T, H_kv, D] of one dtype")
    T, in_code = shape[0], DTYPE_CODES.get(dtype)
    if in_code is None:
        raise ValueError("k_new and v_new must be float32, float16 or bfloat16")
    if slot_mapping.dtype != _I64 or slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be int64 [T]")
    (ks, kh, kd), (vs, vh, vd) = k_new.stride(), v_new.stride()
    if T and (kd != 1 or vd != 1 or (H_kv > 1 and (kh != D or vh != D))):
        raise ValueError("the heads of k_new and v_new must be contiguous")
    if T < 2:
        ks = vs = H_kv * D
    dev = _device(pages)
    if not (scales.get_device() == k_new.get_device() == v_new.get_device() == slot_mapping.get_device() == dev
            and pages.is_contiguous() and scales.is_contiguous() and slot_mapping.is_contiguous()):
        _refuse(dev, pages, scales, k_new, v_new, slot_mapping)
    desc = _PACK_APPEND_MX(T, H_kv, D, P, in_code, kv, max_pages, ks, vs, k_scale, v_scale, 0, 0)
    st = (_lib or lib()).pd_append_paged_kv_mx(
        pages.data_ptr(), scales.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr(), desc,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return pages, scales


def page_pool(num_pages, device="cuda"):
    """(free_pages, state) of a pool of pages 0 .. num_pages - 1, all free, for build_page_tables."""
    return (torch.arange(num_pages, dtype=_I32, device=device),
            torch.tensor([0, num_pages, 0, 0], dtype=_I64, device=device))


def _tables_refuse(page_table, lengths, new_tokens, state, page_table_indptr, page_table_values, length_info, window):
    """What is wrong with the arguments of build_page_tables that every call has."""
    if page_table.dim() != 2 or page_table.dtype != _I32:
        raise ValueError("page_table must be int32 [B, pages]")
    B = page_table.shape[0]
    if lengths.dtype != _I32 or new_tokens.dtype != _I32 or lengths.shape != (B,) or new_tokens.shape != (B,):
        raise ValueError("lengths and new_tokens must be int32 [B]")
    if state.dtype != _I64 or state.shape != (4,):
        raise ValueError("state must be int64 [4]")
    if page_table_values.dtype != _I32 or page_table_values.dim() != 1:
        raise ValueError("page_table_values must be int32 [capacity]")
    if page_table_indptr.dtype != _I32 or page_table_indptr.shape != (B + 1,):
        raise ValueError("page_table_indptr must be int32 [B+1]")
    raise ValueError("length_info must be int32 [B], with a window [3, B]")


def build_page_tables(page_table, lengths, new_tokens, state, page_size, page_table_indptr, page_table_values,
                      length_info, append_indptr=None, slot_mapping=None, positions=None, *, free_pages=None,
                      window=0, sinks=0, stream=None):
    """pd_build_page_tables: the tables of a step, on the device, from the requests' lengths.
    page_table int32 [B, pages] (each request's pages; rows may be strided), lengths int32 [B] and
    state int64 [4] are moved on in place; new_tokens int32 [B] (negative: rows dropped).  Written:
    page_table_indptr [B+1], page_table_values, length_info ([B], with a window [3, B]), append_indptr
    [B+1] (all int32), slot_mapping int64 [T] and positions int32 [T], as the appends and decodes take
    them.  free_pages int32: the ring of free pages (page_pool); None: page_table holds its pages."""
    tshape, i32, i64 = page_table.shape, _I32, _I64
    B = tshape[0] if len(tshape) == 2 else -1
    of_b, of_b1 = (B,), (B + 1,)
    slots_at = pos_at = append_at = free_at = None
    T = n_free = 0
    if (B < 0 or page_table.dtype != i32 or lengths.dtype != i32 or new_tokens.dtype != i32 or lengths.shape != of_b
            or new_tokens.shape != of_b or state.dtype != i64 or state.shape != (4,)
            or page_table_values.dtype != i32 or page_table_values.dim() != 1 or page_table_indptr.dtype != i32
            or page_table_indptr.shape != of_b1 or length_info.dtype != i32
            or length_info.shape != ((3, B) if window else of_b)):
        _tables_refuse(page_table, lengths, new_tokens, state, page_table_indptr, page_table_values, length_info, window)
    dev, width = state.get_device(), tshape[1]
    stride, last = page_table.stride()
    if (width > 1 and last != 1) or (B > 1 and stride < width):
        raise ValueError("the rows of page_table must be contiguous, and apart")
    if append_indptr is not None:
        if append_indptr.dtype != i32 or append_indptr.shape != of_b1:
            raise ValueError("append_indptr must be int32 [B+1]")
        if append_indptr.get_device() != dev or not append_indptr.is_contiguous():
            _refuse(dev, append_indptr)
        append_at = append_indptr.data_ptr()
    if slot_mapping is not None:
        if slot_mapping.dtype != i64 or slot_mapping.dim() != 1:
            raise ValueError("slot_mapping must be int64 [T]")
        if slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
            _refuse(dev, slot_mapping)
        # (one of no entries has no address: any other stands for it, so that it still holds no token)
        T, slots_at = slot_mapping.numel(), slot_mapping.data_ptr() or state.data_ptr()
    if positions is not None:
        n = positions.numel()
        if positions.dtype != i32 or positions.dim() != 1 or (slot_mapping is not None and n != T):
            raise ValueError("positions must be int32 [T]")
        if positions.get_device() != dev or not positions.is_contiguous():
            _refuse(dev, positions)
        T, pos_at = n, positions.data_ptr() or state.data_ptr()
    if free_pages is not None:
        n_free = free_pages.numel()
        if free_pages.dtype != i32 or free_pages.dim() != 1 or not n_free:
            raise ValueError("free_pages must be int32 [pages]")
        if free_pages.get_device() != dev or not free_pages.is_contiguous():
            _refuse(dev, free_pages)
        free_at = free_pages.data_ptr()
    if not (page_table.get_device() == lengths.get_device() == new_tokens.get_device()
            == page_table_indptr.get_device() == page_table_values.get_device() == length_info.get_device() == dev
            and lengths.is_contiguous() and new_tokens.is_contiguous() and state.is_contiguous()
            and page_table_indptr.is_contiguous() and page_table_values.is_contiguous()
            and length_info.is_contiguous()):
        _refuse(dev, page_table, lengths, new_tokens, state, page_table_indptr, page_table_values, length_info)
    _device(state)
    desc = _PACK_TABLES(B, page_size, width, T, window, sinks, 0, 0, stride, page_table_values.numel(), n_free)
    st = (_lib or lib()).pd_build_page_tables(
        page_table.data_ptr(), lengths.data_ptr(), new_tokens.data_ptr(), state.data_ptr(), free_at,
        page_table_indptr.data_ptr(), page_table_values.data_ptr(), length_info.data_ptr(), append_at, slots_at,
        pos_at, desc, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return page_table_indptr, page_table_values, length_info


ROPE_SCALINGS = {None: 0, "linear": 1, "theta": 2, "parts": 3}


def rope_frequencies(rotary_dim, rope_theta=1e4, scaling=None, factor=1.0, original_context=0.0,
                     low_turns=1.0, high_turns=4.0, device="cuda"):
    """pd_rope_frequencies: float64 [rotary_dim / 2] radians per position on `device`, plain or
    extended to longer contexts ("linear", "theta" or "parts" scaling by `factor`)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(1, int(rotary_dim) // 2))()
    _check(lib().pd_rope_frequencies(int(rotary_dim), float(rope_theta), ROPE_SCALINGS[scaling],
                                     float(factor), float(original_context), float(low_turns),
                                     float(high_turns), out))
    return torch.tensor(list(out), dtype=torch.float64, device=device)


def _heads(t, T, H, D, dtype, dev, what, written=False):
    """(token stride, head stride) of rows [T, H, D], checked."""
    if t.shape != (T, H, D) or t.dtype != dtype:
        raise ValueError(f"{what} must be [T, heads, D] like the other rows")
    a, b, c = t.stride()
    if c != 1 and D > 1:
        raise ValueError(f"the last dim of {what} must be contiguous")
    if written and ((a == 0 and T > 1) or (b == 0 and H > 1)):
        raise ValueError(f"{what} must not be an expanded tensor")
    if t.get_device() != dev:
        _refuse(dev, t)
    return a, b


def _new(shape, dtype, device, stream):
    """A tensor for work on `stream`: memory of the current stream's, freed but still in use there,
    is not taken for another."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)  # (up to 2: the default streams)
        stream = torch.cuda.ExternalStream(handle, device) if handle > 2 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, q_out=None, k_out=None, *,
                 rotary_mode=1, eps=1e-6, weight_offset=0.0, attention_factor=1.0, stream=None):
    """pd_qk_norm_rope: RMS norm of each head of q [T, H_q, D] and k [T, H_k, D] (weights [D],
    or None: no norm), then the rotation of the first 2 * len(inv_freq) dims at positions
    (int32 [T]; rotary_mode 1 rotate-half, 2 interleaved; inv_freq None: no rotation).
    k may be None.  q and k may be slices along the heads of a projection's output; q_out and
    k_out default to new tensors (of `stream`'s memory) and may be q and k.  Returns (q_out, k_out)."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [T, heads, D]")
    T, H_q, D = q.shape
    dtype, dev = q.dtype, q.get_device()
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError("q must be float32, float16 or bfloat16")
    if q_out is None:
        q_out = _new((T, H_q, D), dtype, q.device, stream)
    qs, qh = _heads(q, T, H_q, D, dtype, dev, "q")
    qos, qoh = _heads(q_out, T, H_q, D, dtype, dev, "q_out", True)
    H_k = ks = kh = kos = koh = 0
    k_at = ko_at = qw_at = kw_at = pos_at = freq_at = None
    if k is not None:
        H_k = k.shape[1]
        if k_out is None:
            k_out = _new((T, H_k, D), dtype, k.device, stream)
        ks, kh = _heads(k, T, H_k, D, dtype, dev, "k")
        kos, koh = _heads(k_out, T, H_k, D, dtype, dev, "k_out", True)
        k_at, ko_at = k.data_ptr(), k_out.data_ptr()
    wdt = 0
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (D,) or w.get_device() != dev or not w.is_contiguous()):
            if w.shape != (D,):
                raise ValueError("the weights must be [D], of one dtype")
            _refuse(dev, w)
    if q_weight is not None:
        qw_at, wdt = q_weight.data_ptr(), DTYPE_CODES.get(q_weight.dtype)
    if k_weight is not None:
        if q_weight is not None and k_weight.dtype != q_weight.dtype:
            raise ValueError("the weights must be [D], of one dtype")
        kw_at, wdt = k_weight.data_ptr(), DTYPE_CODES.get(k_weight.dtype)
    if wdt is None:
        raise ValueError("the weights must be float32, float16 or bfloat16")
    rd = 0
    if inv_freq is not None and rotary_mode:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be float64 [rotary_dim / 2]")
        if positions is None or positions.dtype != _I32 or positions.shape != (T,):
            raise ValueError("positions must be int32 [T]")
        if not (positions.get_device() == inv_freq.get_device() == dev
                and positions.is_contiguous() and inv_freq.is_contiguous()):
            _refuse(dev, positions, inv_freq)
        rd = 2 * inv_freq.numel()
        pos_at, freq_at = positions.data_ptr(), inv_freq.data_ptr()
    _device(q)
    desc = _PACK_QK(T, H_q, H_k, D, code, wdt, rotary_mode, rd, eps, weight_offset,
                    attention_factor, qs, ks, qh, kh, qos, kos, qoh, koh)
    st = (_lib or lib()).pd_qk_norm_rope(
        q.data_ptr(), k_at, qw_at, kw_at, pos_at, freq_at, q_out.data_ptr(), ko_at, desc,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if st:
        _check(st)
    return q_out, k_out


def merge_state_inplace(V, S, V_other, S_other, stream=None):
    """pd_merge_state_inplace: V [N,H,D], S [N,H] float32 updated in place."""
    N, H, D = V.shape
    if V_other.shape != V.shape or V_other.dtype != V.dtype or S.shape != (N, H) or S_other.shape != (N, H):
        raise ValueError("merge_state_inplace: shape/dtype mismatch")
    _check(lib().pd_merge_state_inplace(_ptr(V), _ptr(S), _ptr(V_other), _ptr(S_other), N, H, D,
                                        DTYPE_CODES[V.dtype], _stream(stream)))
    return V, S


def merge_states(V_out, S_out, V_parts, S_parts, stream=None):
    """pd_merge_states: V_parts [R,N,H,D] float32, S_parts [R,N,H] float32 -> V_out [N,H,D]
    (F32/F16/BF16), S_out [N,H] float32."""
    R, N, H, D = V_parts.shape
    if V_parts.dtype != torch.float32 or S_parts.dtype != torch.float32 or S_parts.shape != (R, N, H):
        raise ValueError("merge_states: V_parts [R,N,H,D] and S_parts [R,N,H] must be float32")
    if V_out.shape != (N, H, D) or S_out.shape != (N, H) or S_out.dtype != torch.float32:
        raise ValueError("merge_states: V_out [N,H,D], S_out [N,H] float32")
    _check(lib().pd_merge_states(_ptr(V_out), _ptr(S_out), _ptr(V_parts), _ptr(S_parts),
                                 N * H * D, N * H, R, N, H, D, DTYPE_CODES[V_out.dtype],
                                 _stream(stream)))
    return V_out, S_out


def merge_states_packed(V_out, S_out, packed, stream=None):
    """pd_merge_states on R packed partials: packed [R, N*H*D + N*H] float32, each row a
    partner's outputs followed by its lse (the layout an all-gather of packed partials
    gives)."""
    N, H, D = V_out.shape
    R, width = packed.shape
    if packed.dtype != torch.float32 or width != N * H * (D + 1) or not packed.is_contiguous():
        raise ValueError("merge_states_packed: packed must be float32 [R, N*H*(D+1)]")
    base = packed.data_ptr()
    _check(lib().pd_merge_states(_ptr(V_out), _ptr(S_out), ctypes.c_void_p(base),
                                 ctypes.c_void_p(base + 4 * N * H * D), width, width, R, N, H, D,
                                 DTYPE_CODES[V_out.dtype], _stream(stream)))
    return V_out, S_out


def cp_shard_plan(indptr, values, length_info, k_rope_pos_offset, page_size, world, rank):
    """pd_cp_shard_plan on host int32 arrays: returns (indptr, values, length_info,
    k_rope_pos_offset) of rank `rank`'s page-aligned slice, as numpy int32 arrays."""
    import numpy as np
    ip = np.ascontiguousarray(indptr, np.int32)
    vals = np.ascontiguousarray(values, np.int32)
    li = np.ascontiguousarray(length_info, np.int32)
    B = len(li)
    ko = None if k_rope_pos_offset is None else np.ascontiguousarray(k_rope_pos_offset, np.int32)
    npg = ip[1:] - ip[:-1]
    cap = int(np.sum(-(-npg // world))) if B and world >= 1 else 0
    o_ip = np.zeros(B + 1, np.int32)
    o_vals = np.zeros(max(cap, 1), np.int32)
    o_li = np.zeros(B, np.int32)
    o_ko = np.zeros(B, np.int32)
    p = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    _check(lib().pd_cp_shard_plan(p(ip), p(vals), p(li), p(ko), B, int(page_size), int(world),
                                  int(rank), p(o_ip), p(o_vals), cap, p(o_li), p(o_ko)))
    return o_ip, o_vals[:o_ip[-1]], o_li, o_ko


def append_paged_kv(pages, k_new, v_new, slot_mapping, k_scale=1.0, v_scale=1.0, stream=None):
    """pd_append_paged_kv: writes new tokens' K/V into their slots (in place)."""
    T, H_kv, D = k_new.shape
    max_pages, _, H2, P, D2 = pages.shape
    if v_new.shape != k_new.shape or H2 != H_kv or D2 != D or slot_mapping.dtype != torch.int64:
        raise ValueError("append_paged_kv: shape/dtype mismatch")
    _check(lib().pd_append_paged_kv(_ptr(pages), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                    T, H_kv, D, P, max_pages, DTYPE_CODES[k_new.dtype],
                                    DTYPE_CODES[pages.dtype], float(k_scale), float(v_scale),
                                    _stream(stream)))
    return pages


def check_device_errors(stream=None) -> str:
    """Synchronises and returns the device error status name ("PD_OK" if clean)."""
    st = lib().pd_check_device_errors(_stream(stream))
    return STATUS.get(st, str(st))


def workspace_size(desc: DecodeDesc) -> int:
    return int(lib().pd_workspace_size(ctypes.byref(desc)))


def append_paged_kv_rope(pages, k_new, v_new, slot_mapping, positions, rotary_mode=1,
                         rope_scale=1.0, rope_theta=1e4, k_scale=1.0, v_scale=1.0, stream=None):
    """pd_append_paged_kv_rope: appends with each K row rotated at positions[t] (int32)."""
    T, H_kv, D = k_new.shape
    max_pages, _, H2, P, D2 = pages.shape
    if v_new.shape != k_new.shape or H2 != H_kv or D2 != D or slot_mapping.dtype != torch.int64:
        raise ValueError("k_new/v_new [T,H_kv,D] must match pages; slot_mapping int64")
    if positions.dtype != torch.int32 or positions.numel() != T:
        raise ValueError("positions must be int32 [T]")
    _check(lib().pd_append_paged_kv_rope(
        _ptr(pages), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(positions), T, H_kv, D, P,
        max_pages, DTYPE_CODES[k_new.dtype], DTYPE_CODES[pages.dtype], float(k_scale),
        float(v_scale), int(rotary_mode), float(rope_scale), float(rope_theta), _stream(stream)))
    return pages


def release_stream_workspace(stream=None):
    """pd_release_stream_workspace: frees the library-managed workspace of `stream`
    (stream-ordered)."""
    _check(lib().pd_release_stream_workspace(_stream(stream)))


def workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().pd_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def plan(desc: DecodeDesc, num_sms: int, ctas_per_sm: int):
    """Host-only split plan: (schedule, grid_blocks, workspace_bytes); schedule 0 =
    balanced shares of all pages, 1 = one block per (sequence, head slice)."""
    c, g, w = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t()
    _check(lib().pd_plan(ctypes.byref(desc), num_sms, ctas_per_sm, ctypes.byref(c),
                         ctypes.byref(g), ctypes.byref(w)))
    return c.value, g.value, w.value


def last_decode_variant() -> str:
    return lib().pd_last_decode_variant().decode()


def version() -> int:
    return int(lib().pd_version())
