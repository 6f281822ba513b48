"""fp8_paged_kv_gb300 -- Python binding of libfp8kv (the C ABI in include/fp8kv.h).

Argument marshalling only: every function takes torch CUDA tensors, checks
dtype / device / contiguity, and passes raw pointers, sizes and the current
CUDA stream to the C entry point of the same name.  All computation happens in
the library's CUDA kernels; there is no CPU or PyTorch fallback.  If the
library is missing or cannot be loaded the first call raises.

The decode-pool path (Cloudflare Kimi/GLM serving write-up): quantise-on-append
of each new token's K/V into e4m3 pages, page-tag bump on reallocation, the
separate batched tag check that aborts stale requests, and split-KV decode
attention over the FP8 (or BF16) cache with a cross-split combine.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8kv.so")

FPK_OK, FPK_EINVAL, FPK_EUNSUPPORTED, FPK_ENOSPC, FPK_ECUDA = 0, 1, 2, 3, 4

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

# name -> (restype, argtypes); mirrors include/fp8kv.h
SIGNATURES = {
    "fpk_version": (ctypes.c_int, []),
    "fpk_selftest_bounded_wait": (ctypes.c_int, [_P, _P, _P]),
    "fpk_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "fpk_kv_append_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                         _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_append_bf16": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                          _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_prefill_fp8": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P, _P, _I32, _P, _P, _P,
                                          _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_prefill_bf16": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I32, _P, _P, _P,
                                           _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_quantize_e4m3": (ctypes.c_int, [_P, _P, _P, _I64, _P]),
    "fpk_amax_scale_bf16": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
    "fpk_page_tags_bump": (ctypes.c_int, [_P, _P, _I32, _I32, _P]),
    "fpk_page_tags_validate": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _P]),
    "fpk_decode_append_check_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                                   _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_decode_append_check_bf16": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                                    _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_decode_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "fpk_paged_decode_attn_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P,
                                                 _SZ, _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32,
                                                 _P]),
    "fpk_paged_decode_attn_fp8_tc": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P,
                                                    _SZ, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                                    _I32, _P]),
    "fpk_paged_decode_attn_bf16": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P, _P, _P, _SZ,
                                                  _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_paged_decode_attn_fp8_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P,
                                                         _P, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                                         _I32, _P]),
    "fpk_decode_step_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P,
                                           _P, _P, _SZ, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                           _I32, _P]),
    "fpk_decode_step_bf16": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                            _SZ, _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_prefix_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "fpk_paged_decode_attn_fp8_prefix": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _I32,
                                                        _P, _P, _P, _SZ, _F, _I32, _I32, _I32, _I32,
                                                        _I32, _I32, _P]),
    "fpk_paged_decode_attn_bf16_prefix": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P, _P, _I32,
                                                         _P, _P, _P, _SZ, _F, _I32, _I32, _I32, _I32,
                                                         _I32, _I32, _P]),
    "fpk_rope_append_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                           _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_rope_append_bf16": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                            _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_rope_prefill_fp8": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _I32,
                                            _P, _P, _P, _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                            _I32, _P]),
    "fpk_rope_prefill_bf16": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _I32,
                                             _P, _P, _P, _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                             _I32, _P]),
    "fpk_rope_append_fp8_block": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                                 _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_rope_prefill_fp8_block": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _I32,
                                                  _P, _P, _P, _I32, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                                  _I32, _P]),
    "fpk_kv_append_fp8_block": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                               _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_prefill_fp8_block": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P, _P, _I32, _P, _P, _P,
                                                _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_paged_decode_attn_fp8_block": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P,
                                                       _SZ, _I32, _F, _I32, _I32, _I32, _I32, _I32,
                                                       _I32, _P]),
    "fpk_prefill_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "fpk_paged_prefill_attn_fp8_block": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _I32, _P, _P, _I32,
                                                        _P, _P, _P, _SZ, _F, _I32, _I32, _I32, _I32,
                                                        _I32, _I32, _P]),
    "fpk_kv_fork_block": (ctypes.c_int, [_P, _I32, _I64, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _P, _P,
                                         _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_compact_block": (ctypes.c_int, [_P, _I32, _I64, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _I32,
                                            _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_fork": (ctypes.c_int, [_P, _I32, _I32, _I64, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _I32,
                                   _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_kv_compact": (ctypes.c_int, [_P, _I32, _I32, _I64, _P, _I32, _P, _P, _P, _P, _P, _I32,
                                      _I32, _I32, _I32, _I32, _I32, _P]),
    "fpk_decode_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
    "fpk_w4_quantize": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _P]),
    "fpk_w4_gemv": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _P]),
    "fpk_w8_quantize": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _P]),
    "fpk_w8_gemv": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _P]),
}

_lock = threading.Lock()
_lib = None


class FpkError(RuntimeError):
    pass


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp8kv.so (built by fp8_paged_kv_gb300.build); raises if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise FpkError(f"{path} not found: build it first "
                               "(python -m fp8_paged_kv_gb300.build); there is no fallback")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(status: int, what: str) -> None:
    if status != FPK_OK:
        msg = load_library().fpk_status_str(status).decode()
        raise FpkError(f"{what}: status {status} ({msg})")


def _ptr(t, dtype=None, name="tensor", allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise FpkError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise FpkError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise FpkError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise FpkError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise FpkError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _launch_stream(stream, device):
    """The handle alone: the current stream's object costs as much as a launch."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _expect(t, name, shape):
    """The tensor's shape (an int: its number of elements), where the call's other arguments settle it."""
    if t is None or shape is None:
        return
    if isinstance(shape, int):
        if t.numel() != shape:
            raise FpkError(f"{name} has {t.numel()} elements, expected {shape}")
    elif tuple(t.shape) != shape:
        raise FpkError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _same_device(*tensors):
    """Every tensor is on the current device: the launch goes to that device's stream."""
    dev = None
    for t in tensors:
        if t is None or not t.is_cuda:
            continue  # host tensors are refused by name when their pointer is taken
        if dev is None:
            dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise FpkError(f"tensor on device {t.get_device()}, the current device is {dev}")


def _pointers(*specs):
    """Addresses of a call's tensors, each (tensor, dtypes, name, shape or None, optional).  One pass
    over what nearly every call has; if anything is not as it should be, the checks by name say what."""
    try:
        dev, out = specs[0][0].get_device(), []
        if dev >= 0 and dev == torch.cuda.current_device():
            for t, dtypes, _, shape, optional in specs:
                if t is None:
                    if not optional:
                        break
                    out.append(None)
                elif (t.dtype in dtypes and t.get_device() == dev and t.is_contiguous()
                      and (shape is None or t.shape == shape
                           or (shape.__class__ is int and t.numel() == shape))):
                    out.append(t.data_ptr())
                else:
                    break
            else:
                return out
    except AttributeError:
        pass  # no tensor
    for t, _, name, shape, _ in specs:
        if t is None or isinstance(t, torch.Tensor):
            _expect(t, name, shape)
    _same_device(*(t for t, *_ in specs if isinstance(t, torch.Tensor)))
    return [_ptr(t, dtypes, name, optional) for t, dtypes, name, _, optional in specs]


_U8 = torch.uint8
_I32T = torch.int32
_U8S, _I32S, _F32S, _BF16S = (torch.uint8,), (torch.int32,), (torch.float32,), (torch.bfloat16,)
_F32 = torch.float32
_BF16 = torch.bfloat16
_TAGS = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)


def version() -> int:
    return load_library().fpk_version()


def fpk_kv_append_fp8(k_new, v_new, kv_pool, k_scale, v_scale, page_table, seq_lens,
                      live_tags=None, expected_tags=None, abort_mask=None, *, Hkv, D, page_size,
                      num_pages, stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_kv_append_fp8(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"),
        _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), max_pages, _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), B, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_kv_append_fp8")


def fpk_kv_append_bf16(k_new, v_new, kv_pool, page_table, seq_lens, live_tags=None,
                       expected_tags=None, abort_mask=None, *, Hkv, D, page_size, num_pages,
                       stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_kv_append_bf16(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"),
        _ptr(kv_pool, _BF16_LIKE, "kv_pool"),
        _ptr(page_table, _I32T, "page_table"), max_pages, _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), B, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_kv_append_bf16")


def fpk_kv_prefill_fp8(k, v, cu_seqlens, kv_pool, k_scale, v_scale, page_table,
                       live_tags=None, expected_tags=None, abort_mask=None, *, Hkv, D, page_size,
                       num_pages, stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_kv_prefill_fp8(
        _ptr(k, _BF16_LIKE, "k"), _ptr(v, _BF16_LIKE, "v"), _ptr(cu_seqlens, _I32T, "cu_seqlens"),
        k.shape[0], _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), max_pages,
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), B, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_kv_prefill_fp8")


def fpk_kv_prefill_bf16(k, v, cu_seqlens, kv_pool, page_table, live_tags=None,
                        expected_tags=None, abort_mask=None, *, Hkv, D, page_size, num_pages,
                        stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_kv_prefill_bf16(
        _ptr(k, _BF16_LIKE, "k"), _ptr(v, _BF16_LIKE, "v"), _ptr(cu_seqlens, _I32T, "cu_seqlens"),
        k.shape[0], _ptr(kv_pool, _BF16_LIKE, "kv_pool"),
        _ptr(page_table, _I32T, "page_table"), max_pages,
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), B, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_kv_prefill_bf16")


def fpk_decode_append_check_fp8(k_new, v_new, kv_pool, k_scale, v_scale, page_table, seq_lens,
                                live_tags, expected_tags, abort_mask, *, Hkv, D, page_size,
                                num_pages, stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_decode_append_check_fp8(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"),
        _ptr(kv_pool, _U8, "kv_pool"), _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), max_pages, _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags"), _ptr(expected_tags, _TAGS, "expected_tags"),
        _ptr(abort_mask, _U8, "abort_mask"), B, Hkv, D, page_size, num_pages, _stream(stream)),
        "fpk_decode_append_check_fp8")


def fpk_decode_append_check_bf16(k_new, v_new, kv_pool, page_table, seq_lens, live_tags,
                                 expected_tags, abort_mask, *, Hkv, D, page_size, num_pages,
                                 stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_decode_append_check_bf16(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"),
        _ptr(kv_pool, _BF16_LIKE, "kv_pool"),
        _ptr(page_table, _I32T, "page_table"), max_pages, _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags"), _ptr(expected_tags, _TAGS, "expected_tags"),
        _ptr(abort_mask, _U8, "abort_mask"), B, Hkv, D, page_size, num_pages, _stream(stream)),
        "fpk_decode_append_check_bf16")


def fpk_quantize_e4m3(x, scale, out, stream=None):
    _check(load_library().fpk_quantize_e4m3(_ptr(x, _F32, "x"), _ptr(scale, _F32, "scale"),
                                            _ptr(out, _U8, "out"), x.numel(), _stream(stream)),
           "fpk_quantize_e4m3")


def fpk_amax_scale_bf16(x, scale, scratch, stream=None):
    _check(load_library().fpk_amax_scale_bf16(_ptr(x, _BF16_LIKE, "x"), x.numel(),
                                              _ptr(scale, _F32, "scale"), _ptr(scratch, _TAGS, "scratch"),
                                              _stream(stream)), "fpk_amax_scale_bf16")


def fpk_page_tags_bump(live_tags, pages, *, num_pages, stream=None):
    _check(load_library().fpk_page_tags_bump(_ptr(live_tags, _TAGS, "live_tags"),
                                             _ptr(pages, _I32T, "pages"), pages.numel(), num_pages,
                                             _stream(stream)), "fpk_page_tags_bump")


def fpk_page_tags_validate(page_table, expected_tags, seq_lens, live_tags, abort_mask,
                           abort_count=None, *, num_pages, page_size, stream=None):
    B, max_pages = page_table.shape
    _check(load_library().fpk_page_tags_validate(
        _ptr(page_table, _I32T, "page_table"), _ptr(expected_tags, _TAGS, "expected_tags"),
        _ptr(seq_lens, _I32T, "seq_lens"), max_pages, _ptr(live_tags, _TAGS, "live_tags"),
        num_pages, B, page_size, _ptr(abort_mask, _U8, "abort_mask"),
        _ptr(abort_count, _I32T, "abort_count", True), _stream(stream)), "fpk_page_tags_validate")


def fpk_decode_workspace_bytes(B, Hq, Hkv, D=128, num_splits=0) -> int:
    n = load_library().fpk_decode_workspace_bytes(B, Hq, Hkv, D, num_splits)
    if n == 0 and B > 0:
        raise FpkError("fpk_decode_workspace_bytes: invalid shape or no CUDA device")
    return int(n)


def fpk_paged_decode_attn_fp8(q, kv_pool, k_scale, v_scale, page_table, seq_lens,
                              abort_mask, out, lse, workspace, *, Hkv, page_size, num_pages,
                              sm_scale, num_splits=0, stream=None):
    B, Hq, D = q.shape
    _check(load_library().fpk_paged_decode_attn_fp8(
        _ptr(q, _BF16_LIKE, "q"), _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True), _ptr(workspace, _U8, "workspace"),
        workspace.numel(), num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_paged_decode_attn_fp8")


def fpk_paged_decode_attn_fp8_tc(q, kv_pool, k_scale, v_scale, page_table, seq_lens,
                                 abort_mask, out, lse, workspace, *, Hkv, page_size, num_pages,
                                 sm_scale, num_splits=0, stream=None):
    """fpk_paged_decode_attn_fp8 on the tcgen05 tensor cores (same arguments)."""
    B, Hq, D = q.shape
    _check(load_library().fpk_paged_decode_attn_fp8_tc(
        _ptr(q, _BF16_LIKE, "q"), _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True), _ptr(workspace, _U8, "workspace"),
        workspace.numel(), num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_paged_decode_attn_fp8_tc")


def fpk_decode_step_fp8(k_new, v_new, kv_pool, k_scale, v_scale, page_table, seq_lens, live_tags,
                        expected_tags, abort_mask, q, out, lse, workspace, *, Hkv, page_size,
                        num_pages, sm_scale, num_splits=0, stream=None):
    B, Hq, D = q.shape
    _check(load_library().fpk_decode_step_fp8(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"), _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(q, _BF16_LIKE, "q"), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True), _ptr(workspace, _U8, "workspace"), workspace.numel(),
        num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages, _stream(stream)),
        "fpk_decode_step_fp8")


def fpk_decode_step_bf16(k_new, v_new, kv_pool, page_table, seq_lens, live_tags, expected_tags,
                         abort_mask, q, out, lse, workspace, *, Hkv, page_size, num_pages, sm_scale,
                         num_splits=0, stream=None):
    B, Hq, D = q.shape
    _check(load_library().fpk_decode_step_bf16(
        _ptr(k_new, _BF16_LIKE, "k_new"), _ptr(v_new, _BF16_LIKE, "v_new"),
        _ptr(kv_pool, _BF16_LIKE, "kv_pool"), _ptr(page_table, _I32T, "page_table"),
        page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(live_tags, _TAGS, "live_tags", True), _ptr(expected_tags, _TAGS, "expected_tags", True),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(q, _BF16_LIKE, "q"), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True),
        _ptr(workspace, _U8, "workspace"), workspace.numel(), num_splits, sm_scale, B, Hq, Hkv, D,
        page_size, num_pages, _stream(stream)), "fpk_decode_step_bf16")


def fpk_paged_decode_attn_bf16(q, kv_pool, page_table, seq_lens, abort_mask, out, lse,
                               workspace, *, Hkv, page_size, num_pages, sm_scale, num_splits=0,
                               stream=None):
    B, Hq, D = q.shape
    _check(load_library().fpk_paged_decode_attn_bf16(
        _ptr(q, _BF16_LIKE, "q"), _ptr(kv_pool, _BF16_LIKE, "kv_pool"),
        _ptr(page_table, _I32T, "page_table"),
        page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True), _ptr(workspace, _U8, "workspace"),
        workspace.numel(), num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_paged_decode_attn_bf16")


def fpk_paged_decode_attn_fp8_noalloc(q, kv_pool, k_scale, v_scale, page_table, seq_lens,
                                      abort_mask, out, lse, *, Hkv, page_size, num_pages, sm_scale,
                                      num_splits=0, stream=None):
    """FP8 decode attention without a caller workspace, for callers that cannot
    allocate device memory; the scratch is a fixed array inside the library
    (batches needing more than 16 MiB of it are rejected).  Calls that overlap
    on the GPU share that scratch and race."""
    B, Hq, D = q.shape
    _check(load_library().fpk_paged_decode_attn_fp8_noalloc(
        _ptr(q, _BF16_LIKE, "q"), _ptr(kv_pool, _U8, "kv_pool"),
        _ptr(k_scale, _F32, "k_scale"), _ptr(v_scale, _F32, "v_scale"),
        _ptr(page_table, _I32T, "page_table"), page_table.shape[1], _ptr(seq_lens, _I32T, "seq_lens"),
        _ptr(abort_mask, _U8, "abort_mask", True), _ptr(out, _F32, "out"),
        _ptr(lse, _F32, "lse", True), num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages,
        _stream(stream)), "fpk_paged_decode_attn_fp8_noalloc")


# ---------------------------------------------------------- shared prefixes
def fpk_prefix_workspace_bytes(B, Hq, Hkv, D=128) -> int:
    n = load_library().fpk_prefix_workspace_bytes(B, Hq, Hkv, D)
    if n == 0 and B > 0:
        raise FpkError("fpk_prefix_workspace_bytes: invalid shape or no CUDA device")
    return int(n)


def _groups(group_starts, prefix_lens):
    n = prefix_lens.numel()
    if group_starts.numel() != n + 1:
        raise FpkError(f"group_starts has {group_starts.numel()} entries, expected {n + 1} "
                       "(one more than prefix_lens)")
    return n


def _prefix(name, fp8, q, kv_pool, scales, page_table, seq_lens, abort_mask, group_starts, prefix_lens,
            out, lse, workspace, Hkv, page_size, num_pages, sm_scale, stream):
    B, Hq, D = q.shape
    max_pages, n_groups = page_table.shape[-1], _groups(group_starts, prefix_lens)
    (q_p, pool_p, table_p, lens_p, abort_p, starts_p, prefix_p, out_p, lse_p, ws_p, *scales_p) = _pointers(
        (q, _BF16S, "q", None, False),
        (kv_pool, _U8S if fp8 else _BF16_LIKE, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        (page_table, _I32S, "page_table", (B, max_pages), False), (seq_lens, _I32S, "seq_lens", (B,), False),
        (abort_mask, _U8S, "abort_mask", (B,), True), (group_starts, _I32S, "group_starts", None, False),
        (prefix_lens, _I32S, "prefix_lens", None, False), (out, _BF16S, "out", (B, Hq, D), False),
        (lse, _F32S, "lse", (B, Hq), True), (workspace, _U8S, "workspace", None, False), *scales)
    _check(getattr(_lib or load_library(), name)(
        q_p, pool_p, *scales_p, table_p, max_pages, lens_p, abort_p, starts_p, prefix_p, n_groups, out_p, lse_p,
        ws_p, workspace.numel(), sm_scale, B, Hq, Hkv, D, page_size, num_pages, _launch_stream(stream, kv_pool.get_device())), name)


def _scales(k_scale, v_scale):
    return (k_scale, _F32S, "k_scale", None, False), (v_scale, _F32S, "v_scale", None, False)


def fpk_paged_decode_attn_fp8_prefix(q, kv_pool, k_scale, v_scale, page_table, seq_lens, abort_mask,
                                     group_starts, prefix_lens, out, lse, workspace, *, Hkv, page_size,
                                     num_pages, sm_scale, stream=None):
    """Decode attention that reads each group's shared prefix once (out: bf16)."""
    _prefix("fpk_paged_decode_attn_fp8_prefix", True, q, kv_pool, _scales(k_scale, v_scale), page_table, seq_lens,
            abort_mask, group_starts, prefix_lens, out, lse, workspace, Hkv, page_size, num_pages, sm_scale, stream)


def fpk_paged_decode_attn_bf16_prefix(q, kv_pool, page_table, seq_lens, abort_mask, group_starts,
                                      prefix_lens, out, lse, workspace, *, Hkv, page_size, num_pages,
                                      sm_scale, stream=None):
    """BF16-cache variant of fpk_paged_decode_attn_fp8_prefix."""
    _prefix("fpk_paged_decode_attn_bf16_prefix", False, q, kv_pool, (), page_table, seq_lens, abort_mask,
            group_starts, prefix_lens, out, lse, workspace, Hkv, page_size, num_pages, sm_scale, stream)


# ------------------------------------------------- caches with block scales
def _block_scales(kv_scales, num_pages, Hkv, page_size):
    return (kv_scales, _U8S, "kv_scales", 2 * num_pages * Hkv * (page_size // 16), False)


def block_scales(num_pages, Hkv, page_size, layers=1, device="cuda"):
    """Block scales of fresh pools: uint8 [layers][num_pages][Hkv][page_size/16][2]."""
    return torch.zeros((layers, num_pages, Hkv, page_size // 16, 2), dtype=torch.uint8, device=device)


def fpk_rope_append_fp8_block(q, k_new, v_new, inv_freq, q_out, kv_pool, kv_scales, page_table,
                              seq_lens, live_tags=None, expected_tags=None, abort_mask=None, *, Hkv,
                              page_size, num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    """fpk_rope_append_fp8 into blocks whose scales follow their largest value (rot_dim 0: no rotation)."""
    _rope("fpk_rope_append_fp8_block", True, q, k_new, v_new, (seq_lens,), inv_freq, q_out, kv_pool,
          (kv_scales,), page_table, live_tags, expected_tags, abort_mask, Hkv, page_size,
          num_pages, rot_dim, interleaved, rot_scale, stream)


def fpk_rope_prefill_fp8_block(q, k, v, cu_seqlens, start_pos, inv_freq, q_out, kv_pool, kv_scales,
                               page_table, live_tags=None, expected_tags=None, abort_mask=None, *, Hkv,
                               page_size, num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    """fpk_rope_prefill_fp8 into blocks whose scales follow their largest value (rot_dim 0: no rotation)."""
    _rope("fpk_rope_prefill_fp8_block", True, q, k, v, (cu_seqlens, start_pos), inv_freq, q_out, kv_pool,
          (kv_scales,), page_table, live_tags, expected_tags, abort_mask, Hkv, page_size,
          num_pages, rot_dim, interleaved, rot_scale, stream)


def fpk_kv_append_fp8_block(k_new, v_new, kv_pool, kv_scales, page_table, seq_lens, live_tags=None,
                            expected_tags=None, abort_mask=None, *, Hkv, D, page_size, num_pages, stream=None):
    """One token per request, without rotation (k_new, v_new: [B][Hkv][D])."""
    B, max_pages = page_table.shape
    (k_p, v_p, pool_p, scales_p, table_p, lens_p, live_p, expected_p, abort_p) = _pointers(
        (k_new, _BF16_LIKE, "k_new", (B, Hkv, D), False), (v_new, _BF16_LIKE, "v_new", (B, Hkv, D), False),
        (kv_pool, _U8S, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        _block_scales(kv_scales, num_pages, Hkv, page_size), (page_table, _I32S, "page_table", None, False),
        (seq_lens, _I32S, "seq_lens", (B,), False), (live_tags, _TAGS, "live_tags", (num_pages,), True),
        (expected_tags, _TAGS, "expected_tags", (B, max_pages), True), (abort_mask, _U8S, "abort_mask", (B,), True))
    _check((_lib or load_library()).fpk_kv_append_fp8_block(
        k_p, v_p, pool_p, scales_p, table_p, max_pages, lens_p, live_p, expected_p, abort_p, B, Hkv, D, page_size,
        num_pages, _launch_stream(stream, kv_pool.get_device())), "fpk_kv_append_fp8_block")


def fpk_kv_prefill_fp8_block(k, v, cu_seqlens, start_pos, kv_pool, kv_scales, page_table, live_tags=None,
                             expected_tags=None, abort_mask=None, *, Hkv, D, page_size, num_pages, stream=None):
    """Prompts or their chunks (from start_pos, None: 0), without rotation."""
    T = k.shape[0]
    B, max_pages = page_table.shape
    (k_p, v_p, cu_p, start_p, pool_p, scales_p, table_p, live_p, expected_p, abort_p) = _pointers(
        (k, _BF16_LIKE, "k", (T, Hkv, D), False), (v, _BF16_LIKE, "v", (T, Hkv, D), False),
        (cu_seqlens, _I32S, "cu_seqlens", (B + 1,), False), (start_pos, _I32S, "start_pos", (B,), True),
        (kv_pool, _U8S, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        _block_scales(kv_scales, num_pages, Hkv, page_size), (page_table, _I32S, "page_table", None, False),
        (live_tags, _TAGS, "live_tags", (num_pages,), True),
        (expected_tags, _TAGS, "expected_tags", (B, max_pages), True), (abort_mask, _U8S, "abort_mask", (B,), True))
    _check((_lib or load_library()).fpk_kv_prefill_fp8_block(
        k_p, v_p, cu_p, T, start_p, pool_p, scales_p, table_p, max_pages, live_p, expected_p, abort_p, B, Hkv, D,
        page_size, num_pages, _launch_stream(stream, kv_pool.get_device())), "fpk_kv_prefill_fp8_block")


def fpk_paged_decode_attn_fp8_block(q, kv_pool, kv_scales, page_table, seq_lens, abort_mask, out, lse,
                                    workspace, *, Hkv, page_size, num_pages, sm_scale, num_splits=0, stream=None):
    """fpk_paged_decode_attn_fp8 over a cache with block scales."""
    B, Hq, D = q.shape
    max_pages = page_table.shape[-1]
    (q_p, pool_p, scales_p, table_p, lens_p, abort_p, out_p, lse_p, ws_p) = _pointers(
        (q, _BF16_LIKE, "q", None, False),
        (kv_pool, _U8S, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        _block_scales(kv_scales, num_pages, Hkv, page_size),
        (page_table, _I32S, "page_table", (B, max_pages), False), (seq_lens, _I32S, "seq_lens", (B,), False),
        (abort_mask, _U8S, "abort_mask", (B,), True), (out, _F32S, "out", (B, Hq, D), False),
        (lse, _F32S, "lse", (B, Hq), True), (workspace, _U8S, "workspace", None, False))
    _check((_lib or load_library()).fpk_paged_decode_attn_fp8_block(
        q_p, pool_p, scales_p, table_p, max_pages, lens_p, abort_p, out_p, lse_p, ws_p, workspace.numel(),
        num_splits, sm_scale, B, Hq, Hkv, D, page_size, num_pages, _launch_stream(stream, kv_pool.get_device())),
        "fpk_paged_decode_attn_fp8_block")


def fpk_prefill_workspace_bytes(B, n_tokens, Hq, Hkv, D=128) -> int:
    n = load_library().fpk_prefill_workspace_bytes(B, n_tokens, Hq, Hkv, D)
    if n == 0 and B > 0 and n_tokens > 0:
        raise FpkError("fpk_prefill_workspace_bytes: invalid shape or no CUDA device")
    return int(n)


def fpk_paged_prefill_attn_fp8_block(q, cu_seqlens, kv_pool, kv_scales, page_table, seq_lens, abort_mask,
                                     out, lse, workspace, *, causal=True, Hkv, page_size, num_pages,
                                     sm_scale, stream=None):
    """Attention of several query tokens per request (out: bf16): causal at the end of each
    context, or over all of it (cross attention to an encoder's states)."""
    T, Hq, D = q.shape
    B, max_pages = page_table.shape
    (q_p, cu_p, pool_p, scales_p, table_p, lens_p, abort_p, out_p, lse_p, ws_p) = _pointers(
        (q, _BF16S, "q", None, False), (cu_seqlens, _I32S, "cu_seqlens", (B + 1,), False),
        (kv_pool, _U8S, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        _block_scales(kv_scales, num_pages, Hkv, page_size), (page_table, _I32S, "page_table", None, False),
        (seq_lens, _I32S, "seq_lens", (B,), False), (abort_mask, _U8S, "abort_mask", (B,), True),
        (out, _BF16S, "out", (T, Hq, D), False), (lse, _F32S, "lse", (T, Hq), True),
        (workspace, _U8S, "workspace", None, False))
    _check((_lib or load_library()).fpk_paged_prefill_attn_fp8_block(
        q_p, cu_p, T, pool_p, scales_p, table_p, max_pages, lens_p, abort_p, int(bool(causal)), out_p, lse_p, ws_p,
        workspace.numel(), sm_scale, B, Hq, Hkv, D, page_size, num_pages,
        _launch_stream(stream, kv_pool.get_device())), "fpk_paged_prefill_attn_fp8_block")


# --------------------------------------------------------- rotary positions
def _rope(name, fp8, q, k, v, pos, inv_freq, q_out, kv_pool, scales, page_table, live_tags,
          expected_tags, abort_mask, Hkv, page_size, num_pages, rot_dim, interleaved, rot_scale,
          stream):
    """pos: (seq_lens,) of an append or (cu_seqlens, start_pos) of a prefill."""
    T, _, D = k.shape
    Hq = 0 if q is None else q.shape[1]
    B, max_pages = page_table.shape
    append = len(pos) == 1
    if append and T != B:
        raise FpkError(f"k has {T} rows for {B} requests")
    if append:
        where = ((pos[0], _I32S, "seq_lens", (B,), False),)
    else:
        where = ((pos[0], _I32S, "cu_seqlens", (B + 1,), False), (pos[1], _I32S, "start_pos", (B,), True))
    if name.endswith("_block"):
        scales = (_block_scales(*scales, num_pages, Hkv, page_size),)
    else:
        scales = _scales(*scales) if fp8 else ()
    (k_p, v_p, q_p, out_p, freq_p, pool_p, table_p, live_p, expected_p, abort_p, pos_p, *rest) = _pointers(
        (k, _BF16S, "k", (T, Hkv, D), False), (v, _BF16S, "v", (T, Hkv, D), False),
        (q, _BF16S, "q", (T, Hq, D), True), (q_out, _BF16S, "q_out", (T, Hq, D) if Hq else None, True),
        (inv_freq, _F32S, "inv_freq", (rot_dim // 2,) if rot_dim else None, rot_dim == 0),
        (kv_pool, _U8S if fp8 else _BF16_LIKE, "kv_pool", 2 * num_pages * Hkv * page_size * D, False),
        (page_table, _I32S, "page_table", None, False), (live_tags, _TAGS, "live_tags", (num_pages,), True),
        (expected_tags, _TAGS, "expected_tags", (B, max_pages), True),
        (abort_mask, _U8S, "abort_mask", (B,), True), *where, *scales)
    fn = getattr(_lib or load_library(), name)
    last = (live_p, expected_p, abort_p, rot_dim, int(interleaved), rot_scale, B, Hq, Hkv, D, page_size,
            num_pages, _launch_stream(stream, kv_pool.get_device()))
    if append:
        _check(fn(q_p, k_p, v_p, freq_p, out_p, pool_p, *rest, table_p, max_pages, pos_p, *last), name)
    else:
        _check(fn(q_p, k_p, v_p, pos_p, T, rest[0], freq_p, out_p, pool_p, *rest[1:], table_p, max_pages, *last), name)


def fpk_rope_append_fp8(q, k_new, v_new, inv_freq, q_out, kv_pool, k_scale, v_scale, page_table,
                        seq_lens, live_tags=None, expected_tags=None, abort_mask=None, *, Hkv,
                        page_size, num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    _rope("fpk_rope_append_fp8", True, q, k_new, v_new, (seq_lens,), inv_freq, q_out, kv_pool,
          (k_scale, v_scale), page_table, live_tags, expected_tags, abort_mask, Hkv, page_size,
          num_pages, rot_dim, interleaved, rot_scale, stream)


def fpk_rope_append_bf16(q, k_new, v_new, inv_freq, q_out, kv_pool, page_table, seq_lens,
                         live_tags=None, expected_tags=None, abort_mask=None, *, Hkv, page_size,
                         num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    _rope("fpk_rope_append_bf16", False, q, k_new, v_new, (seq_lens,), inv_freq, q_out, kv_pool, (),
          page_table, live_tags, expected_tags, abort_mask, Hkv, page_size, num_pages, rot_dim,
          interleaved, rot_scale, stream)


def fpk_rope_prefill_fp8(q, k, v, cu_seqlens, start_pos, inv_freq, q_out, kv_pool, k_scale, v_scale,
                         page_table, live_tags=None, expected_tags=None, abort_mask=None, *, Hkv,
                         page_size, num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    _rope("fpk_rope_prefill_fp8", True, q, k, v, (cu_seqlens, start_pos), inv_freq, q_out, kv_pool,
          (k_scale, v_scale), page_table, live_tags, expected_tags, abort_mask, Hkv, page_size,
          num_pages, rot_dim, interleaved, rot_scale, stream)


def fpk_rope_prefill_bf16(q, k, v, cu_seqlens, start_pos, inv_freq, q_out, kv_pool, page_table,
                          live_tags=None, expected_tags=None, abort_mask=None, *, Hkv, page_size,
                          num_pages, rot_dim, interleaved=False, rot_scale=1.0, stream=None):
    _rope("fpk_rope_prefill_bf16", False, q, k, v, (cu_seqlens, start_pos), inv_freq, q_out, kv_pool,
          (), page_table, live_tags, expected_tags, abort_mask, Hkv, page_size, num_pages, rot_dim,
          interleaved, rot_scale, stream)


# ---------------------------------------------------------- forks and moves
def _moves(kv_pool, page_table, expected_tags, seq_lens, live_tags, layers, Hkv, D, page_size, num_pages, *more):
    """(B, max_pages, element bytes, bytes from one layer's pool to the next), addresses"""
    B, max_pages = page_table.shape
    if layers < 1:
        raise FpkError(f"kv_pool has {kv_pool.numel()} elements for {layers} layers")
    one = 2 * num_pages * Hkv * page_size * D
    at = _pointers((kv_pool, (torch.uint8, *_BF16_LIKE), "kv_pool", layers * one, False),
                   (page_table, _I32S, "page_table", None, False),
                   (expected_tags, _TAGS, "expected_tags", (B, max_pages), False),
                   (seq_lens, _I32S, "seq_lens", (B,), False), (live_tags, _TAGS, "live_tags", (num_pages,), False),
                   *more)
    el = kv_pool.element_size()
    return (B, max_pages, el, one * el), at


def fpk_kv_fork(kv_pool, page_table, expected_tags, seq_lens, live_tags, abort_mask, parent, child,
                fresh, *, layers=1, Hkv, D, page_size, num_pages, stream=None):
    """Rows child[i] take over rows parent[i]: full pages shared, the page in use
    copied to fresh[i] in all layers of kv_pool ([layers][one pool], contiguous)."""
    n = parent.numel()
    (B, max_pages, el, stride), (pool_p, table_p, expected_p, lens_p, live_p, abort_p, parent_p, child_p, fresh_p) = _moves(
        kv_pool, page_table, expected_tags, seq_lens, live_tags, layers, Hkv, D, page_size, num_pages,
        (abort_mask, _U8S, "abort_mask", (page_table.shape[0],), True), (parent, _I32S, "parent", None, False),
        (child, _I32S, "child", (n,), False), (fresh, _I32S, "fresh", (n,), False))
    _check((_lib or load_library()).fpk_kv_fork(
        pool_p, el, layers, stride, table_p, max_pages, expected_p, lens_p, live_p, abort_p, parent_p, child_p,
        fresh_p, n, B, Hkv, D, page_size, num_pages, _launch_stream(stream, kv_pool.get_device())), "fpk_kv_fork")


def fpk_kv_compact(kv_pool, page_table, expected_tags, seq_lens, live_tags, src, dst, *, layers=1,
                   Hkv, D, page_size, num_pages, stream=None):
    """Pages src[i] (ascending) move to dst[i] in all layers of kv_pool; tables and tags follow."""
    n = src.numel()
    (B, max_pages, el, stride), (pool_p, table_p, expected_p, lens_p, live_p, src_p, dst_p) = _moves(
        kv_pool, page_table, expected_tags, seq_lens, live_tags, layers, Hkv, D, page_size, num_pages,
        (src, _I32S, "src", None, False), (dst, _I32S, "dst", (n,), False))
    _check((_lib or load_library()).fpk_kv_compact(
        pool_p, el, layers, stride, table_p, max_pages, expected_p, lens_p, live_p, src_p, dst_p, n, B, Hkv, D,
        page_size, num_pages, _launch_stream(stream, kv_pool.get_device())), "fpk_kv_compact")


def _move_scales(kv_scales, layers, num_pages, Hkv, page_size):
    one = 2 * num_pages * Hkv * (page_size // 16)
    return one, (kv_scales, _U8S, "kv_scales", layers * one, False)


def fpk_kv_fork_block(kv_pool, kv_scales, page_table, expected_tags, seq_lens, live_tags, abort_mask, parent,
                      child, fresh, *, layers=1, Hkv, D, page_size, num_pages, stream=None):
    """fpk_kv_fork of an e4m3 pool with block scales ([layers][one pool's], contiguous)."""
    n, (one, scales) = parent.numel(), _move_scales(kv_scales, layers, num_pages, Hkv, page_size)
    (B, max_pages, _, stride), (pool_p, table_p, expected_p, lens_p, live_p, scales_p, abort_p, parent_p, child_p, fresh_p) = _moves(
        kv_pool, page_table, expected_tags, seq_lens, live_tags, layers, Hkv, D, page_size, num_pages, scales,
        (abort_mask, _U8S, "abort_mask", (page_table.shape[0],), True), (parent, _I32S, "parent", None, False),
        (child, _I32S, "child", (n,), False), (fresh, _I32S, "fresh", (n,), False))
    if kv_pool.dtype != torch.uint8:
        raise FpkError(f"kv_pool has dtype {kv_pool.dtype}: block scales belong to an e4m3 pool")
    _check((_lib or load_library()).fpk_kv_fork_block(
        pool_p, layers, stride, scales_p, one, table_p, max_pages, expected_p, lens_p, live_p, abort_p, parent_p,
        child_p, fresh_p, n, B, Hkv, D, page_size, num_pages, _launch_stream(stream, kv_pool.get_device())),
        "fpk_kv_fork_block")


def fpk_kv_compact_block(kv_pool, kv_scales, page_table, expected_tags, seq_lens, live_tags, src, dst, *,
                         layers=1, Hkv, D, page_size, num_pages, stream=None):
    """fpk_kv_compact of an e4m3 pool with block scales ([layers][one pool's], contiguous)."""
    n, (one, scales) = src.numel(), _move_scales(kv_scales, layers, num_pages, Hkv, page_size)
    (B, max_pages, _, stride), (pool_p, table_p, expected_p, lens_p, live_p, scales_p, src_p, dst_p) = _moves(
        kv_pool, page_table, expected_tags, seq_lens, live_tags, layers, Hkv, D, page_size, num_pages, scales,
        (src, _I32S, "src", None, False), (dst, _I32S, "dst", (n,), False))
    if kv_pool.dtype != torch.uint8:
        raise FpkError(f"kv_pool has dtype {kv_pool.dtype}: block scales belong to an e4m3 pool")
    _check((_lib or load_library()).fpk_kv_compact_block(
        pool_p, layers, stride, scales_p, one, table_p, max_pages, expected_p, lens_p, live_p, src_p, dst_p, n, B,
        Hkv, D, page_size, num_pages, _launch_stream(stream, kv_pool.get_device())), "fpk_kv_compact_block")


def fpk_decode_status(workspace, stream=None) -> int:
    """Status word of an attention workspace; workspace=None reads the one of the
    last allocation-free call on the current device."""
    v = ctypes.c_int32(0)
    _check(load_library().fpk_decode_status(_ptr(workspace, _U8, "workspace", allow_none=True),
                                            ctypes.byref(v), _stream(stream)), "fpk_decode_status")
    return int(v.value)


def fpk_selftest_bounded_wait(status, elapsed_ns, stream=None):
    """One CTA waits on an mbarrier nothing arrives on; the bounded wait gives up
    after its limit and reports it in status[0] (elapsed time in elapsed_ns[0])."""
    _check(load_library().fpk_selftest_bounded_wait(_ptr(status, torch.int32, "status"),
                                                    _ptr(elapsed_ns, torch.int64, "elapsed_ns"),
                                                    _stream(stream)), "fpk_selftest_bounded_wait")


# ---------------------------------------------------------------- weight GEMV
def fpk_w4_quantize(w, codes, scales, stream=None):
    N, K = w.shape
    _check(load_library().fpk_w4_quantize(_ptr(w, _BF16_LIKE, "w"), _ptr(codes, _U8, "codes"),
                                          _ptr(scales, _BF16_LIKE, "scales"), N, K, _stream(stream)),
           "fpk_w4_quantize")


def fpk_w4_gemv(x, codes, scales, y, stream=None):
    B, K = x.shape
    N = y.shape[1]
    _check(load_library().fpk_w4_gemv(_ptr(x, _BF16_LIKE, "x"), _ptr(codes, _U8, "codes"),
                                      _ptr(scales, _BF16_LIKE, "scales"), _ptr(y, _F32, "y"), B, N, K,
                                      _stream(stream)), "fpk_w4_gemv")


def fpk_w8_quantize(w, codes, row_scales, stream=None):
    N, K = w.shape
    _check(load_library().fpk_w8_quantize(_ptr(w, _BF16_LIKE, "w"), _ptr(codes, _U8, "codes"),
                                          _ptr(row_scales, _F32, "row_scales"), N, K, _stream(stream)),
           "fpk_w8_quantize")


def fpk_w8_gemv(x, codes, row_scales, y, stream=None):
    B, K = x.shape
    N = y.shape[1]
    _check(load_library().fpk_w8_gemv(_ptr(x, _BF16_LIKE, "x"), _ptr(codes, _U8, "codes"),
                                      _ptr(row_scales, _F32, "row_scales"), _ptr(y, _F32, "y"), B, N, K,
                                      _stream(stream)), "fpk_w8_gemv")
