"""Thin ctypes binding of libbsp.so (include/bsp.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels. The functions
mirror the C entry points by name; torch tensors supply device memory, pinned
host staging and the current CUDA stream. If the native library is missing or
fails to load, every call raises ``NativeLibraryError``: there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import numpy as np
import torch

from . import build as _build

BSP_OK = 0
STATUS_NAMES = {0: "BSP_OK", 1: "BSP_ERR_INVALID_ARG", 2: "BSP_ERR_UNSUPPORTED", 3: "BSP_ERR_PAGE_INDEX",
                4: "BSP_ERR_CAPACITY", 5: "BSP_ERR_STALE_PLAN", 6: "BSP_ERR_CUDA", 7: "BSP_ERR_DEVICE_TIMEOUT"}
DTYPES = {"bf16": 0, "fp16": 1, torch.bfloat16: 0, torch.float16: 1}
FLAG_LSE_BASE2 = 1
FLAG_CHECK = 2
FLAG_GRAPH = 4
FLAG_ACCUMULATE = 8
MAX_TAIL = 8
MAX_GROUP = 8
STATUS_BYTES = 256  # device status words ahead of the plan image in the workspace
DEVFLAG_PAGE_INDEX = 1
DEVFLAG_TIMEOUT = 2
DEVFLAG_POSITION = 4
DEVFLAG_GRAPH = 8
DEVFLAG_PAGES = 16


class NativeLibraryError(RuntimeError):
    pass


class BspError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Geometry(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("geo", Geometry)] + [(n, ctypes.c_int32) for n in (
        "batch", "beam_width", "max_tail", "prefix_pages_stride", "num_units", "num_parts", "row_blocks",
        "beams_per_block", "tile_keys", "max_prefix_len", "max_total_len", "num_sms", "max_tail_len",
        "prefix_ctas")] + [
        ("generation", ctypes.c_uint64), ("ws_device", ctypes.c_void_p), ("ws_device_bytes", ctypes.c_uint64),
        ("ws_host", ctypes.c_void_p), ("image_bytes", ctypes.c_uint64), ("off_req", ctypes.c_uint64),
        ("off_units", ctypes.c_uint64), ("off_pages", ctypes.c_uint64), ("off_part_lse", ctypes.c_uint64),
        ("off_part_o", ctypes.c_uint64), ("device_bytes_used", ctypes.c_uint64),
        ("tail_requests", ctypes.c_int32), ("total_rows", ctypes.c_int32), ("kind", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("off_cta", ctypes.c_uint64), ("max_splits", ctypes.c_int32),
        ("reserved", ctypes.c_int32)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_position", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class TokenMask(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_void_p), ("stride", ctypes.c_int64), ("index", ctypes.c_void_p),
                ("rows", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _LogitsParams(ctypes.Structure):
    _fields_ = [("prompt_tokens", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p), ("prompt_stride", ctypes.c_int64),
                ("tokens", ctypes.c_void_p), ("token_len", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p), ("bias_len", ctypes.c_void_p),
                ("bias_stride", ctypes.c_int64), ("repetition_penalty", ctypes.c_void_p),
                ("frequency_penalty", ctypes.c_void_p), ("presence_penalty", ctypes.c_void_p),
                ("temperature", ctypes.c_void_p), ("mask", TokenMask), ("prompt_cols", ctypes.c_int32),
                ("token_cols", ctypes.c_int32), ("bias_cols", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None
EXPORTS = ["bsp_status_string", "bsp_bucket_rows", "bsp_workspace_size", "bsp_plan_build", "bsp_plan",
           "bsp_append_kv", "bsp_decode_attn", "bsp_read_device_status", "bsp_decode_attn_noalloc",
           "bsp_plan_prefill_build", "bsp_plan_prefill", "bsp_prefill_attn", "bsp_rope_cos_sin",
           "bsp_rope_append_kv", "bsp_append_kv_fp8", "bsp_rope_append_kv_fp8", "bsp_plan_update_tails",
           "bsp_decode_attn_fp8", "bsp_process_logits", "bsp_beam_select_workspace_size", "bsp_beam_select",
           "bsp_beam_advance", "bsp_key_weights", "bsp_key_weights_fp8", "bsp_evict_prefix",
           "bsp_decode_attn_fp8_blocks", "bsp_append_kv_fp8_blocks", "bsp_norm_rope_append_kv",
           "bsp_norm_rope_append_kv_fp8", "bsp_rope_cos_sin_scaled", "bsp_fork_workspace_size", "bsp_fork_tables",
           "bsp_fork_rows", "bsp_free_pages", "bsp_compact_tables", "bsp_copy_pages"]
NOALLOC_SCRATCH_MIB = 32


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libbsp.so (building it first only when asked)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise NativeLibraryError(
            f"{_build.LIB} is missing: build it with beam_search_shared_gb300.build.build() "
            "(there is no fallback path)")
    try:
        lib = ctypes.CDLL(_build.LIB)
    except OSError as e:  # pragma: no cover - depends on the box
        raise NativeLibraryError(f"cannot load {_build.LIB}: {e}") from e
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    lib.bsp_status_string.restype = ctypes.c_char_p
    lib.bsp_status_string.argtypes = [i32]
    lib.bsp_bucket_rows.restype = i32
    lib.bsp_bucket_rows.argtypes = [i32, i32]
    lib.bsp_workspace_size.restype = i32
    lib.bsp_workspace_size.argtypes = [P(Geometry), i32, i32, i32, P(sz), P(sz)]
    lib.bsp_plan_build.restype = i32
    lib.bsp_plan_build.argtypes = [P(Geometry), i32, i32, vp, vp, vp, i32, i32, i32, vp, sz, P(Plan)]
    lib.bsp_plan.restype = i32
    lib.bsp_plan.argtypes = [P(Geometry), i32, i32, vp, vp, vp, i32, i32, vp, sz, vp, sz, vp, P(Plan)]
    lib.bsp_plan_update_tails.restype = i32
    lib.bsp_plan_update_tails.argtypes = [P(Plan), vp, vp]
    lib.bsp_append_kv.restype = i32
    lib.bsp_append_kv.argtypes = [P(Plan), vp, vp, i64, vp, i32, vp, vp, vp, vp]
    lib.bsp_decode_attn.restype = i32
    lib.bsp_decode_attn.argtypes = [P(Plan), vp, vp, vp, vp, i32, vp, i32, ctypes.c_float, i32, vp, vp, vp, vp]
    f32 = ctypes.c_float
    lib.bsp_decode_attn_fp8.restype = i32
    lib.bsp_decode_attn_fp8.argtypes = [P(Plan), vp, vp, vp, vp, i32, vp, i32, f32, f32, f32, i32, vp, vp, vp, vp]
    lib.bsp_plan_prefill_build.restype = i32
    lib.bsp_plan_prefill_build.argtypes = [P(Geometry), i32, vp, vp, vp, i32, i32, i32, vp, sz, P(Plan)]
    lib.bsp_plan_prefill.restype = i32
    lib.bsp_plan_prefill.argtypes = [P(Geometry), i32, vp, vp, vp, i32, i32, vp, sz, vp, sz, vp, P(Plan)]
    lib.bsp_prefill_attn.restype = i32
    lib.bsp_prefill_attn.argtypes = [P(Plan), vp, vp, vp, ctypes.c_float, i32, vp, vp, vp, vp]
    lib.bsp_rope_cos_sin.restype = i32
    lib.bsp_rope_cos_sin.argtypes = [i32, i32, ctypes.c_double, vp, vp]
    lib.bsp_rope_append_kv.restype = i32
    lib.bsp_rope_append_kv.argtypes = [P(Plan), P(RopeConfig), vp, vp, i64, vp, vp, i64, vp, i32, vp, vp, vp, vp]
    lib.bsp_rope_append_kv_fp8.restype = i32
    lib.bsp_rope_append_kv_fp8.argtypes = [P(Plan), P(RopeConfig), vp, vp, i64, vp, vp, i64, ctypes.c_float,
                                           ctypes.c_float, vp, i32, vp, vp, vp, vp]
    lib.bsp_append_kv_fp8.restype = i32
    lib.bsp_append_kv_fp8.argtypes = [P(Plan), vp, vp, i64, i32, ctypes.c_float, ctypes.c_float, vp, i32, vp, vp, vp, vp]
    lib.bsp_read_device_status.restype = i32
    lib.bsp_read_device_status.argtypes = [P(Plan), vp, i32, P(i32)]
    lib.bsp_decode_attn_noalloc.restype = i32
    lib.bsp_decode_attn_noalloc.argtypes = [P(Geometry), i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, i32, vp, i32,
                                            ctypes.c_float, i32, vp, vp, vp]
    lib.bsp_process_logits.restype = i32
    lib.bsp_process_logits.argtypes = [P(Plan), vp, i32, i64, i32, P(_LogitsParams), vp, i64, vp, vp]
    lib.bsp_beam_select_workspace_size.restype = i32
    lib.bsp_beam_select_workspace_size.argtypes = [i32, i32, i32, i32, P(sz)]
    lib.bsp_beam_select.restype = i32
    lib.bsp_beam_select.argtypes = [P(Plan), vp, i32, i64, i32, vp, vp, i64, P(TokenMask), i32, vp, vp, vp, vp, sz, vp]
    lib.bsp_beam_advance.restype = i32
    lib.bsp_beam_advance.argtypes = [P(Plan), vp, vp, i64, vp, vp, i32, vp, vp, i64, i32, vp, vp]
    lib.bsp_key_weights.restype = i32
    lib.bsp_key_weights.argtypes = [P(Plan), vp, vp, vp, f32, i32, i32, vp, i64, vp]
    lib.bsp_key_weights_fp8.restype = i32
    lib.bsp_key_weights_fp8.argtypes = [P(Plan), vp, vp, vp, f32, f32, i32, i32, vp, i64, vp]
    lib.bsp_evict_prefix.restype = i32
    lib.bsp_evict_prefix.argtypes = [P(Plan), vp, i64, vp, vp, i32, i32, vp, vp, vp, vp, vp, i64, vp]
    lib.bsp_rope_cos_sin_scaled.restype = i32
    lib.bsp_rope_cos_sin_scaled.argtypes = [i32, i32, ctypes.c_double, P(_RopeScaling), vp, vp]
    head = [P(Plan), P(_QkNorm), P(RopeConfig), vp, vp, i64, vp, i64, vp, vp, i64]
    for fn, args in (("bsp_norm_rope_append_kv", [vp, i32, vp, vp, vp, vp]),
                     ("bsp_norm_rope_append_kv_fp8", [f32, f32, vp, i32, vp, vp, vp, vp]),
                     ("bsp_append_kv_fp8_blocks", [vp, i32, vp, vp, P(_BlockScales), vp, vp])):
        getattr(lib, fn).restype = i32
        getattr(lib, fn).argtypes = head + args
    lib.bsp_fork_workspace_size.restype = i32
    lib.bsp_fork_workspace_size.argtypes = [i32, i32, P(sz)]
    lib.bsp_fork_tables.restype = i32
    lib.bsp_fork_tables.argtypes = [P(Plan), vp, i64, i32, vp, vp, vp, i64, i32, vp, sz, vp]
    lib.bsp_fork_rows.restype = i32
    lib.bsp_fork_rows.argtypes = [P(Plan), vp, i64, i32, vp, i64, i32, vp, i32, vp, i32, vp, vp, P(_BlockScales), vp]
    lib.bsp_free_pages.restype = i32
    lib.bsp_free_pages.argtypes = [P(Plan), vp, i64, i32, i32, vp, vp, vp]
    lib.bsp_compact_tables.restype = i32
    lib.bsp_compact_tables.argtypes = [P(Plan), vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, vp]
    lib.bsp_copy_pages.restype = i32
    lib.bsp_copy_pages.argtypes = [P(Plan), vp, vp, i32, vp, vp, P(_BlockScales), vp]
    lib.bsp_decode_attn_fp8_blocks.restype = i32
    lib.bsp_decode_attn_fp8_blocks.argtypes = [P(Plan), vp, vp, vp, P(_BlockScales), vp, i32, vp, i32, f32, i32, vp, vp,
                                               vp, vp]
    _lib = lib
    return lib


def _check(fn: str, st: int):
    if st != BSP_OK:
        raise BspError(fn, st)


def status_string(status: int) -> str:
    return load().bsp_status_string(int(status)).decode()


KV_DTYPE_SAME, KV_DTYPE_E4M3 = 0, 1


def geometry(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, dtype, kv_dtype: int = KV_DTYPE_SAME) -> Geometry:
    """kv_dtype: KV_DTYPE_SAME (the pools hold `dtype`) or KV_DTYPE_E4M3 (one-byte E4M3 pools)."""
    return Geometry(int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size), int(num_pages),
                    DTYPES[dtype], int(kv_dtype))


def bucket_rows(valid_rows: int, capacity: int) -> int:
    return int(load().bsp_bucket_rows(int(valid_rows), int(capacity)))


def workspace_size(geo: Geometry, max_batch: int, max_beam: int, max_prefix_pages: int):
    d, h = ctypes.c_size_t(), ctypes.c_size_t()
    _check("bsp_workspace_size", load().bsp_workspace_size(ctypes.byref(geo), int(max_batch), int(max_beam),
                                                           int(max_prefix_pages), ctypes.byref(d), ctypes.byref(h)))
    return d.value, h.value


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def _ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if torch.cuda.is_initialized():  # the raw handle, without building a Stream object for each call
            return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def plan_build(geo: Geometry, batch, beam_width, prefix_len, tail_len, prefix_pages, max_tail, num_sms,
               image_bytes: int = 1 << 24):
    """Host-only planning. Returns (Plan, image bytes as a numpy uint8 array)."""
    pl, tl = _i32(prefix_len), _i32(tail_len)
    pp = _i32(prefix_pages).reshape(int(batch), -1) if int(batch) else np.zeros((0, 1), np.int32)
    img = np.zeros(int(image_bytes), np.uint8)
    plan = Plan()
    _check("bsp_plan_build", load().bsp_plan_build(
        ctypes.byref(geo), int(batch), int(beam_width), _ptr(pl), _ptr(tl), _ptr(pp), pp.shape[1], int(max_tail),
        int(num_sms), _ptr(img), img.nbytes, ctypes.byref(plan)))
    return plan, img[:plan.image_bytes]


REQ_FIELDS = 12  # int32 per request record of a plan image


def plan_requests(plan_: Plan, img: np.ndarray) -> np.ndarray:
    """Per-request records of a host plan image (``plan_build``), int32 [batch, 12]: prompt length,
    tail length, prompt partial states, first partial slot, first page entry, finished by the
    prompt kernel (1) or by the tail kernel (0), two unused, query rows per head, causal base (-1:
    none), first query row, one unused."""
    lo = plan_.off_req - STATUS_BYTES
    return img[lo:lo + plan_.batch * REQ_FIELDS * 4].view(np.int32).reshape(plan_.batch, REQ_FIELDS)


def plan_prefill_build(geo: Geometry, batch, cached_len, prompt_len, pages, causal, num_sms,
                       image_bytes: int = 1 << 24):
    """Host-only prefill planning. Returns (Plan, image bytes as a numpy uint8 array)."""
    cl, pl = _i32(cached_len), _i32(prompt_len)
    pg = _i32(pages).reshape(int(batch), -1) if int(batch) else np.zeros((0, 1), np.int32)
    img = np.zeros(int(image_bytes), np.uint8)
    plan = Plan()
    _check("bsp_plan_prefill_build", load().bsp_plan_prefill_build(
        ctypes.byref(geo), int(batch), _ptr(cl), _ptr(pl), _ptr(pg), pg.shape[1], 1 if causal else 0,
        int(num_sms), _ptr(img), img.nbytes, ctypes.byref(plan)))
    return plan, img[:plan.image_bytes]


def plan_prefill(geo: Geometry, batch, cached_len, prompt_len, pages, causal, ws: "Workspace",
                 stream=None) -> Plan:
    """bsp_plan_prefill: host arrays in, plan staged into ``ws`` on ``stream`` (no sync)."""
    cl, pl = _i32(cached_len), _i32(prompt_len)
    pg = _i32(pages).reshape(int(batch), -1) if int(batch) else np.zeros((0, 1), np.int32)
    out = Plan()
    _check("bsp_plan_prefill", load().bsp_plan_prefill(
        ctypes.byref(geo), int(batch), _ptr(cl), _ptr(pl), _ptr(pg), pg.shape[1], 1 if causal else 0,
        _dptr(ws.device), ws.device.numel(), _dptr(ws.host), ws.host.numel(), _stream(stream), ctypes.byref(out)))
    return out


def prefill_attn(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, softmax_scale: float,
                 o: torch.Tensor, lse: torch.Tensor, flags: int = 0, events=None, stream=None):
    """bsp_prefill_attn: writes o [total_rows,Hq,D] and lse [total_rows,Hq] (fp32)."""
    _check("bsp_prefill_attn", load().bsp_prefill_attn(
        ctypes.byref(plan_), _dptr(q), _dptr(k_pool), _dptr(v_pool), float(softmax_scale), int(flags), _dptr(o),
        _dptr(lse), _events(events, 3), _stream(stream)))


class Workspace:
    """A device workspace and its pinned host staging buffer, sized by bsp_workspace_size."""

    def __init__(self, geo: Geometry, max_batch: int, max_beam: int, max_prefix_pages: int, device=None):
        dev_bytes, host_bytes = workspace_size(geo, max_batch, max_beam, max_prefix_pages)
        device = torch.device("cuda") if device is None else torch.device(device)
        self.device = torch.empty(dev_bytes, dtype=torch.uint8, device=device)
        self.device.zero_()
        self.host = torch.empty(host_bytes, dtype=torch.uint8, pin_memory=True)
        self.host.zero_()

    def plan(self, geo: Geometry, batch, beam_width, prefix_len, tail_len, prefix_pages, max_tail=MAX_TAIL,
             stream=None) -> Plan:
        return plan(geo, batch, beam_width, prefix_len, tail_len, prefix_pages, max_tail, self, stream)


def plan(geo: Geometry, batch, beam_width, prefix_len, tail_len, prefix_pages, max_tail, ws: Workspace,
         stream=None) -> Plan:
    """bsp_plan: host arrays in, plan staged into ``ws`` on ``stream`` (no sync)."""
    pl, tl = _i32(prefix_len), _i32(tail_len)
    pp = _i32(prefix_pages).reshape(int(batch), -1) if int(batch) else np.zeros((0, 1), np.int32)
    out = Plan()
    _check("bsp_plan", load().bsp_plan(
        ctypes.byref(geo), int(batch), int(beam_width), _ptr(pl), _ptr(tl), _ptr(pp), pp.shape[1], int(max_tail),
        _dptr(ws.device), ws.device.numel(), _dptr(ws.host), ws.host.numel(), _stream(stream), ctypes.byref(out)))
    return out


def plan_update_tails(plan_: Plan, tail_len, stream=None) -> Plan:
    """bsp_plan_update_tails: new tail lengths for a current decode plan, in place (no sync)."""
    tl = _i32(tail_len)
    if tl.shape[0] != plan_.batch:
        raise ValueError(f"tail_len has {tl.shape[0]} entries for a batch of {plan_.batch}")
    _check("bsp_plan_update_tails", load().bsp_plan_update_tails(ctypes.byref(plan_), _ptr(tl), _stream(stream)))
    return plan_


def _events(events, n):
    if events is None:
        return None
    assert len(events) == n
    for e in events:
        if e.cuda_event == 0:
            e.record()  # materialise the underlying cudaEvent_t
    return (ctypes.c_void_p * n)(*[e.cuda_event for e in events])


def append_kv(plan_: Plan, k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor,
              k_pool: torch.Tensor, v_pool: torch.Tensor, src_row_stride: Optional[int] = None, events=None,
              stream=None):
    """bsp_append_kv: k_new/v_new rows [n, Hkv*D] (row stride in elements), out_cache_loc int32 [n].

    ``events``: optional 2 timing events recorded before and after the append kernel.
    """
    n = int(out_cache_loc.numel())
    if src_row_stride is None:
        src_row_stride = int(k_new.stride(0)) if k_new.dim() >= 1 and n else plan_.geo.num_kv_heads * plan_.geo.head_dim
    _check("bsp_append_kv", load().bsp_append_kv(
        ctypes.byref(plan_), _dptr(k_new), _dptr(v_new), int(src_row_stride), _dptr(out_cache_loc), n,
        _dptr(k_pool), _dptr(v_pool), _events(events, 2), _stream(stream)))


FP8_SRC_16BIT, FP8_SRC_E4M3 = 0, 1


def append_kv_fp8(plan_: Plan, k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor,
                  k_pool: torch.Tensor, v_pool: torch.Tensor, k_mul: float = 1.0, v_mul: float = 1.0,
                  src_row_stride: Optional[int] = None, events=None, stream=None):
    """bsp_append_kv_fp8: uint8 (E4M3) pools; k_new/v_new rows [n, Hkv*D] of the geometry's 16-bit dtype
    (quantised with the multipliers) or of E4M3 bytes (torch.float8_e4m3fn or uint8, copied)."""
    n = int(out_cache_loc.numel())
    src = FP8_SRC_E4M3 if k_new.dtype in (torch.uint8, torch.float8_e4m3fn) else FP8_SRC_16BIT
    if src_row_stride is None:
        src_row_stride = int(k_new.stride(0)) if k_new.dim() >= 1 and n else plan_.geo.num_kv_heads * plan_.geo.head_dim
    _check("bsp_append_kv_fp8", load().bsp_append_kv_fp8(
        ctypes.byref(plan_), _dptr(k_new), _dptr(v_new), int(src_row_stride), src, float(k_mul), float(v_mul),
        _dptr(out_cache_loc), n, _dptr(k_pool), _dptr(v_pool), _events(events, 2), _stream(stream)))


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("original_positions", ctypes.c_int32), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class RopeScaling:
    """Frequencies of a model stretched beyond its trained length (bsp_rope_scaling). kind: "linear", "base", "bands" or
    "ramp"; bands and ramp go by original_positions and the turns low < high; amplitude multiplies cos and sin."""

    KINDS = {"linear": 1, "base": 2, "bands": 3, "ramp": 4}

    def __init__(self, kind: str, factor: float, original_positions: int = 0, low: float = 0.0, high: float = 0.0,
                 amplitude: float = 1.0):
        if kind not in self.KINDS:
            raise ValueError(f"kind {kind!r} is none of {sorted(self.KINDS)}")
        self.kind = kind
        self.c = _RopeScaling(self.KINDS[kind], int(original_positions), float(factor), float(low), float(high),
                              float(amplitude))


class Rope:
    """A RoPE table (device fp32 [max_position][rotary_dim], filled by bsp_rope_cos_sin, with ``scaling`` by
    bsp_rope_cos_sin_scaled) and its layout."""

    def __init__(self, max_position: int, rotary_dim: int, base: float, interleaved: bool = False, device="cuda",
                 stream=None, scaling: Optional[RopeScaling] = None):
        self.cos_sin = torch.empty((int(max_position), int(rotary_dim)), dtype=torch.float32, device=device)
        self.base = float(base)
        if scaling is None:
            _check("bsp_rope_cos_sin", load().bsp_rope_cos_sin(int(max_position), int(rotary_dim), self.base,
                                                                _dptr(self.cos_sin), _stream(stream)))
        else:
            _check("bsp_rope_cos_sin_scaled", load().bsp_rope_cos_sin_scaled(
                int(max_position), int(rotary_dim), self.base, ctypes.byref(scaling.c), _dptr(self.cos_sin),
                _stream(stream)))
        self.config = RopeConfig(self.cos_sin.data_ptr(), int(max_position), int(rotary_dim), 1 if interleaved else 0, 0)

    @property
    def rotary_dim(self) -> int:
        return int(self.config.rotary_dim)

    @property
    def interleaved(self) -> bool:
        return bool(self.config.interleaved)

    @property
    def max_position(self) -> int:
        return int(self.config.max_position)


def rope_append_kv(plan_: Plan, rope: Rope, positions: torch.Tensor, q: Optional[torch.Tensor], k_new: torch.Tensor,
                   v_new: torch.Tensor, out_cache_loc: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                   src_row_stride: Optional[int] = None, q_row_stride: Optional[int] = None, events=None,
                   stream=None):
    """bsp_rope_append_kv: rotated K and plain V rows into the pools, q [n, Hq*D] rotated in place (or None).
    positions, out_cache_loc: int32 [n] on the device."""
    n = int(out_cache_loc.numel())
    row = plan_.geo.num_kv_heads * plan_.geo.head_dim
    if src_row_stride is None:
        src_row_stride = int(k_new.stride(0)) if k_new.dim() >= 1 and n else row
    if q is not None and q_row_stride is None:
        q_row_stride = int(q.stride(0)) if q.dim() >= 1 and n else plan_.geo.num_q_heads * plan_.geo.head_dim
    _check("bsp_rope_append_kv", load().bsp_rope_append_kv(
        ctypes.byref(plan_), ctypes.byref(rope.config), _dptr(positions), _dptr(q), int(q_row_stride or 0),
        _dptr(k_new), _dptr(v_new), int(src_row_stride), _dptr(out_cache_loc), n, _dptr(k_pool), _dptr(v_pool),
        _events(events, 2), _stream(stream)))


def rope_append_kv_fp8(plan_: Plan, rope: Rope, positions: torch.Tensor, q: Optional[torch.Tensor],
                       k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor, k_pool: torch.Tensor,
                       v_pool: torch.Tensor, k_mul: float = 1.0, v_mul: float = 1.0,
                       src_row_stride: Optional[int] = None, q_row_stride: Optional[int] = None, events=None,
                       stream=None):
    """bsp_rope_append_kv_fp8: rotated K and V quantised into uint8 (E4M3) pools, q rotated in place."""
    n = int(out_cache_loc.numel())
    row = plan_.geo.num_kv_heads * plan_.geo.head_dim
    if src_row_stride is None:
        src_row_stride = int(k_new.stride(0)) if k_new.dim() >= 1 and n else row
    if q is not None and q_row_stride is None:
        q_row_stride = int(q.stride(0)) if q.dim() >= 1 and n else plan_.geo.num_q_heads * plan_.geo.head_dim
    _check("bsp_rope_append_kv_fp8", load().bsp_rope_append_kv_fp8(
        ctypes.byref(plan_), ctypes.byref(rope.config), _dptr(positions), _dptr(q), int(q_row_stride or 0),
        _dptr(k_new), _dptr(v_new), int(src_row_stride), float(k_mul), float(v_mul), _dptr(out_cache_loc), n,
        _dptr(k_pool), _dptr(v_pool), _events(events, 2), _stream(stream)))


def decode_attn(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                beam_pages: Optional[torch.Tensor], cache_indirection: Optional[torch.Tensor], softmax_scale: float,
                o: torch.Tensor, lse: torch.Tensor, flags: int = 0, events=None, stream=None):
    """bsp_decode_attn: writes o [R,Hq,D] and lse [R,Hq] (fp32).

    ``events``: optional 3 torch.cuda.Event(enable_timing=True) recorded around the prompt and tail kernels.
    """
    bps = int(beam_pages.shape[-1]) if beam_pages is not None else 0
    max_seq = int(cache_indirection.shape[-1]) if cache_indirection is not None else 0
    ev = _events(events, 3)
    _check("bsp_decode_attn", load().bsp_decode_attn(
        ctypes.byref(plan_), _dptr(q), _dptr(k_pool), _dptr(v_pool), _dptr(beam_pages), bps,
        _dptr(cache_indirection), max_seq, float(softmax_scale), int(flags), _dptr(o), _dptr(lse), ev,
        _stream(stream)))


def read_device_status(plan_: Plan, clear: bool = True, stream=None):
    """Synchronises the stream; returns (status, device flag bits)."""
    flags = ctypes.c_int32(0)
    st = load().bsp_read_device_status(ctypes.byref(plan_), _stream(stream), int(bool(clear)), ctypes.byref(flags))
    return int(st), int(flags.value)


def decode_attn_fp8(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                    beam_pages: Optional[torch.Tensor], cache_indirection: Optional[torch.Tensor], softmax_scale: float,
                    k_scale: float, v_scale: float, o: torch.Tensor, lse: torch.Tensor, flags: int = 0, events=None,
                    stream=None):
    """bsp_decode_attn_fp8: decode attention over uint8 E4M3 pools (key = code x k_scale, value = code x
    v_scale); writes o [R,Hq,D] in the q dtype and lse [R,Hq] (fp32)."""
    bps = int(beam_pages.shape[-1]) if beam_pages is not None else 0
    max_seq = int(cache_indirection.shape[-1]) if cache_indirection is not None else 0
    ev = _events(events, 3)
    _check("bsp_decode_attn_fp8", load().bsp_decode_attn_fp8(
        ctypes.byref(plan_), _dptr(q), _dptr(k_pool), _dptr(v_pool), _dptr(beam_pages), bps,
        _dptr(cache_indirection), max_seq, float(softmax_scale), float(k_scale), float(v_scale), int(flags),
        _dptr(o), _dptr(lse), ev, _stream(stream)))


class _BlockScales(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class BlockScales:
    """Scales of E4M3 pools, one for each block of ``block`` slots of a (page, kv head): exponent bytes E of 2^(E - 127)
    in uint8 tables k and v [num_pages, num_kv_heads, page_size // block] (made zeroed, or the given ones). Pools that have
    them go through append_kv_fp8_blocks, decode_attn_fp8_blocks and, with ``scales``, fork_rows and copy_pages; no other
    call knows of the scales, and none can tell."""

    def __init__(self, geo: Geometry, block: int, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                 device="cuda"):
        self.block = int(block)
        if self.block < 1 or geo.page_size % self.block:
            raise ValueError(f"blocks of {block} slots in pages of {geo.page_size}")
        self.shape = (geo.num_pages, geo.num_kv_heads, geo.page_size // self.block)
        new = lambda: torch.zeros(self.shape, dtype=torch.uint8, device=device)  # noqa: E731
        self.k, self.v = new() if k is None else k, new() if v is None else v
        for name, t in (("k", self.k), ("v", self.v)):
            if t.dtype is not torch.uint8 or tuple(t.shape) != self.shape or not t.is_contiguous():
                raise ValueError(f"the {name} scales must be contiguous uint8 {list(self.shape)}, not {t.dtype} "
                                 f"{list(t.shape)}")
        self.c = _BlockScales(self.k.data_ptr(), self.v.data_ptr(), self.block, 0)

    def _of(self, plan_: Plan):
        """For a call on the plan's pools: its tables must be theirs."""
        g = plan_.geo
        if self.shape != (g.num_pages, g.num_kv_heads, g.page_size // self.block):
            raise ValueError(f"scales {list(self.shape)} in blocks of {self.block} for pools of {g.num_pages} pages, "
                             f"{g.num_kv_heads} heads, {g.page_size} slots")
        return ctypes.byref(self.c)


def _buffer(name: str, t: torch.Tensor, dtype, rows: int, row):
    """A contiguous buffer of at least ``rows`` rows of shape ``row`` (or flat), whatever dimensions count the rows."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}, not {t.dtype} of strides {t.stride()}")
    shape, width = tuple(t.shape), math.prod(row)
    fits = shape[-len(row):] == row or shape[-1:] == (width,) or len(shape) == 1
    if not fits or t.numel() < rows * width:
        raise ValueError(f"{name} has shape {shape}, not [{rows}, {', '.join(map(str, row))}]")


def decode_attn_fp8_blocks(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           scales: BlockScales, beam_pages: Optional[torch.Tensor],
                           cache_indirection: Optional[torch.Tensor], softmax_scale: float, o: torch.Tensor,
                           lse: torch.Tensor, flags: int = 0, events=None, stream=None):
    """bsp_decode_attn_fp8_blocks: decode attention over uint8 E4M3 pools with block scales; writes o [R,Hq,D] in
    the q dtype and lse [R,Hq] (fp32)."""
    g, rows = plan_.geo, plan_.total_rows
    heads = (g.num_q_heads, g.head_dim)
    _buffer("q", q, _ELEMENT[g.dtype], rows, heads)
    _buffer("o", o, _ELEMENT[g.dtype], rows, heads)
    _buffer("lse", lse, torch.float32, rows, heads[:1])
    bps = int(beam_pages.shape[-1]) if beam_pages is not None else 0
    max_seq = int(cache_indirection.shape[-1]) if cache_indirection is not None else 0
    if plan_.max_tail_len > 0 or flags & FLAG_GRAPH:  # (they are read)
        for name, t, width in (("beam_pages", beam_pages, bps), ("cache_indirection", cache_indirection, max_seq)):
            if t is not None:
                _buffer(name, t, torch.int32, rows, (width,))
    _pools_ok(plan_, k_pool, v_pool)
    _check("bsp_decode_attn_fp8_blocks", load().bsp_decode_attn_fp8_blocks(
        ctypes.byref(plan_), _dptr(q), _dptr(k_pool), _dptr(v_pool), scales._of(plan_), _dptr(beam_pages), bps,
        _dptr(cache_indirection), max_seq, float(softmax_scale), int(flags), _dptr(o), _dptr(lse), _events(events, 3),
        _stream(stream)))


# ---------------------------------------------------------------- appends of normalised rows

class _QkNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("weight_fp32", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QkNorm:
    """The RMS norm of queries and keys per head: q_weight, k_weight [head_dim], both in the geometry's dtype or both
    fp32 (None: ones), eps, and what is added to the weights (1 for weights stored as their distance from one)."""

    def __init__(self, q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 weight_offset: float = 0.0):
        given = [w for w in (q_weight, k_weight) if w is not None]
        if any(w.dim() != 1 or not w.is_contiguous() or w.dtype != given[0].dtype or w.shape != given[0].shape
               for w in given):
            raise ValueError("q_weight and k_weight must be contiguous vectors of one type and length")
        self.dtype = given[0].dtype if given else None
        self.dim = given[0].shape[0] if given else None
        if self.dtype not in (None, torch.float32, torch.bfloat16, torch.float16):
            raise ValueError(f"weights are {self.dtype}")
        self.c = _QkNorm(_address(q_weight), _address(k_weight), float(eps), float(weight_offset),
                         int(self.dtype is torch.float32), 0)
        self._keep = (q_weight, k_weight)

    def _of(self, plan_: Plan):
        g = plan_.geo
        if self.dim not in (None, g.head_dim) or self.dtype not in (None, torch.float32, _ELEMENT[g.dtype]):
            raise ValueError(f"norm weights {self.dtype} [{self.dim}] for heads of {g.head_dim} {_ELEMENT[g.dtype]}")
        return ctypes.byref(self.c)


_ELEMENT = (torch.bfloat16, torch.float16)


def _token_rows(name: str, t: torch.Tensor, dtype, n: int, width: int) -> int:
    """Rows of tokens [n, width] or [n, heads, dim], contiguous in a token; their stride in elements."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if not n:
        return width + 7 & ~7
    shape, step = t.shape, t.stride()
    if len(shape) == 2:
        fits, packed = shape[1] == width, width == 1 or step[1] == 1
    else:
        fits = len(shape) == 3 and shape[1] * shape[2] == width
        packed = fits and step[2] == 1 and (shape[1] == 1 or step[1] == shape[2])
    if not fits or shape[0] < n:
        raise ValueError(f"{name} has shape {tuple(shape)}, not [{n}, {width}]")
    if not packed:
        raise ValueError(f"the rows of {name} are not contiguous")
    return step[0] if n > 1 else width + 7 & ~7


def _norm_append_args(plan_: Plan, norm, rope, positions, q, q_out, k_new, v_new, out_cache_loc):
    """The arguments that the appends of normalised rows have in common, checked: (.., n) as the library takes them."""
    g = plan_.geo
    dt = _ELEMENT[g.dtype]
    n = out_cache_loc.numel()
    row = g.num_kv_heads * g.head_dim
    stride = _token_rows("k_new", k_new, dt, n, row)
    if _token_rows("v_new", v_new, dt, n, row) != stride:
        raise ValueError("k_new and v_new must have the same row stride")
    if out_cache_loc.dtype is not torch.int32 or not out_cache_loc.is_contiguous():
        raise ValueError("out_cache_loc must be contiguous int32")
    q_stride = out_stride = 0
    if q is not None:
        q_out = q if q_out is None else q_out
        q_stride = _token_rows("q", q, dt, n, g.num_q_heads * g.head_dim)
        out_stride = q_stride if q_out is q else _token_rows("q_out", q_out, dt, n, g.num_q_heads * g.head_dim)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rope is not None:
        if (positions is None or positions.dtype is not torch.int32 or positions.numel() < n or
                not positions.is_contiguous()):
            raise ValueError(f"positions must be contiguous int32 [{n}]")
    return (ctypes.byref(plan_), None if norm is None else norm._of(plan_),
            None if rope is None else ctypes.byref(rope.config), None if rope is None else positions.data_ptr(),
            _address(q), q_stride, _address(q_out), out_stride, k_new.data_ptr(), v_new.data_ptr(), stride), n


def norm_rope_append_kv(plan_: Plan, norm: QkNorm, rope: Optional[Rope], positions: Optional[torch.Tensor],
                        q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor,
                        k_pool: torch.Tensor, v_pool: torch.Tensor, q_out: Optional[torch.Tensor] = None, events=None,
                        stream=None):
    """bsp_norm_rope_append_kv: K rows normalised per head, rotated (rope None: not) and written to their slots, V rows
    written, query rows normalised and rotated into q_out (None: in place). q, k_new, v_new: [n, heads * head_dim] or
    [n, heads, head_dim], tokens any stride apart (column slices of one projection's output)."""
    args, n = _norm_append_args(plan_, norm, rope, positions, q, q_out, k_new, v_new, out_cache_loc)
    _pools_ok(plan_, k_pool, v_pool)
    _check("bsp_norm_rope_append_kv", load().bsp_norm_rope_append_kv(
        *args, out_cache_loc.data_ptr(), n, k_pool.data_ptr(), v_pool.data_ptr(), _events(events, 2), _stream(stream)))


def _pools8_ok(plan_: Plan, *pools: torch.Tensor):
    """E4M3 pools of the plan's geometry, whatever its kv_dtype."""
    g = plan_.geo
    shape = (g.num_pages, g.num_kv_heads, g.page_size, g.head_dim)
    for t in pools:
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"a pool must be contiguous uint8 {list(shape)}, not {t.dtype} {list(t.shape)}")


def norm_rope_append_kv_fp8(plan_: Plan, norm: QkNorm, rope: Optional[Rope], positions: Optional[torch.Tensor],
                            q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                            out_cache_loc: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, k_mul: float = 1.0,
                            v_mul: float = 1.0, q_out: Optional[torch.Tensor] = None, events=None, stream=None):
    """bsp_norm_rope_append_kv_fp8: norm_rope_append_kv into uint8 (E4M3) pools with one multiplier per tensor."""
    args, n = _norm_append_args(plan_, norm, rope, positions, q, q_out, k_new, v_new, out_cache_loc)
    _pools8_ok(plan_, k_pool, v_pool)
    _check("bsp_norm_rope_append_kv_fp8", load().bsp_norm_rope_append_kv_fp8(
        *args, float(k_mul), float(v_mul), out_cache_loc.data_ptr(), n, k_pool.data_ptr(), v_pool.data_ptr(),
        _events(events, 2), _stream(stream)))


def append_kv_fp8_blocks(plan_: Plan, k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor,
                         k_pool: torch.Tensor, v_pool: torch.Tensor, scales: BlockScales, norm: Optional[QkNorm] = None,
                         rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                         q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, events=None,
                         stream=None):
    """bsp_append_kv_fp8_blocks: K rows (normalised with norm, rotated with rope) and V rows into uint8 (E4M3) pools with
    block scales, query rows into q_out (None: in place). Tokens whose slots are in one block stand next to one another
    in ascending order of their slots."""
    args, n = _norm_append_args(plan_, norm, rope, positions, q, q_out, k_new, v_new, out_cache_loc)
    _pools8_ok(plan_, k_pool, v_pool)
    _check("bsp_append_kv_fp8_blocks", load().bsp_append_kv_fp8_blocks(
        *args, out_cache_loc.data_ptr(), n, k_pool.data_ptr(), v_pool.data_ptr(), scales._of(plan_), _events(events, 2),
        _stream(stream)))


def decode_attn_noalloc(geo: Geometry, batch, beam_width, prefix_len, tail_len, prefix_pages, max_tail,
                        q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                        beam_pages: Optional[torch.Tensor], cache_indirection: Optional[torch.Tensor],
                        softmax_scale: float, o: torch.Tensor, lse: torch.Tensor, flags: int = 0, stream=None):
    """bsp_decode_attn_noalloc: plan + cascade attention with the library's fixed device scratch.

    For callers that cannot allocate device memory: no workspace is passed and nothing is allocated.
    Calls share one scratch array per GPU; calls whose GPU work overlaps race on it.
    """
    pl, tl = _i32(prefix_len), _i32(tail_len)
    pp = _i32(prefix_pages).reshape(int(batch), -1) if int(batch) else np.zeros((0, 1), np.int32)
    bps = int(beam_pages.shape[-1]) if beam_pages is not None else 0
    max_seq = int(cache_indirection.shape[-1]) if cache_indirection is not None else 0
    _check("bsp_decode_attn_noalloc", load().bsp_decode_attn_noalloc(
        ctypes.byref(geo), int(batch), int(beam_width), _ptr(pl), _ptr(tl), _ptr(pp), pp.shape[1], int(max_tail),
        _dptr(q), _dptr(k_pool), _dptr(v_pool), _dptr(beam_pages), bps, _dptr(cache_indirection), max_seq,
        float(softmax_scale), int(flags), _dptr(o), _dptr(lse), _stream(stream)))


# ---------------------------------------------------------------- around the attention of a step

LOGITS_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _table(name: str, t: torch.Tensor, dtype, shape, exact_last: bool = True):
    """Checks a table's type and shape (None: any extent) and that its rows are contiguous and evenly spaced;
    returns the row stride in elements."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    s = t.shape
    if t.is_contiguous():  # the usual case
        if s == shape:
            return s[-1]
        n = len(s)
        if n == len(shape):
            for i in range(n):
                w = shape[i]
                if w is not None and s[i] != w and (exact_last or i < n - 1 or s[i] < w):
                    break
            else:
                return s[-1]
    n = t.dim()
    if n != len(shape) or any(w is not None and (t.shape[i] != w if exact_last or i < n - 1 else t.shape[i] < w)
                              for i, w in enumerate(shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the rows of {name} are not contiguous")
    # the stride of a dimension of one entry says nothing: torch leaves it arbitrary
    steps = [(t.stride(i), t.shape[i]) for i in range(n - 1) if t.shape[i] > 1]
    for (outer, _), (inner, count) in zip(steps, steps[1:]):
        if outer != inner * count:
            raise ValueError(f"the rows of {name} are not evenly spaced")
    return steps[-1][0] if steps else t.shape[-1]


def token_mask(bits: Optional[torch.Tensor], index: Optional[torch.Tensor]) -> TokenMask:
    """Grammar masks: ``bits`` int32 [states, words] (bit t % 32 of word t // 32: token t is allowed), ``index``
    int32 [batch * beam_width], the row's state or -1."""
    if bits is None:
        return TokenMask()
    stride = _table("mask", bits, torch.int32, (None, None))
    if index is None:
        raise ValueError("a mask needs mask_index")
    _table("mask_index", index, torch.int32, (None,))
    return TokenMask(bits.data_ptr(), stride, index.data_ptr(), bits.shape[0], 0)


class LogitsParams:
    """What ``process_logits`` does to a row, checked once; tensors' contents may change between calls, the
    tensors may not. prompt_tokens int32 [batch, n] with prompt_token_len [batch]; tokens int32
    [batch * beam_width, n] with token_len [batch * beam_width]; bias_tokens int32 and bias_values fp32
    [batch, n], bias_len int32 [batch] or None (all n); penalties and temperature fp32 [batch]; mask,
    mask_index as ``token_mask``. None leaves a step out."""

    def __init__(self, prompt_tokens=None, prompt_token_len=None, tokens=None, token_len=None,
                 repetition_penalty=None, frequency_penalty=None, presence_penalty=None, temperature=None,
                 bias_tokens=None, bias_values=None, bias_len=None, mask=None, mask_index=None):
        c = _LogitsParams()
        i32, f32 = torch.int32, torch.float32
        self.batch, self.rows = None, None

        def lead(what, n):
            old = getattr(self, what)
            if old is not None and old != n:
                raise ValueError(f"lists for {n} and for {old} {what}")
            setattr(self, what, n)

        for name, t, lens, what in (("prompt_tokens", prompt_tokens, prompt_token_len, "batch"),
                                    ("tokens", tokens, token_len, "rows")):
            if t is None:
                continue
            short = "prompt" if what == "batch" else "token"
            setattr(c, short + "_stride", _table(name, t, i32, (None, None)))
            setattr(c, short + "_cols", t.shape[1])
            if lens is None:
                raise ValueError(f"{name} need their lengths")
            _table(short + "_len", lens, i32, (t.shape[0],))
            lead(what, t.shape[0])
            setattr(c, name, t.data_ptr())
            setattr(c, short + "_len", lens.data_ptr())
        if bias_tokens is not None:
            c.bias_stride = _table("bias_tokens", bias_tokens, i32, (None, None))
            if bias_values is None or _table("bias_values", bias_values, f32, tuple(bias_tokens.shape)) != c.bias_stride:
                raise ValueError("bias_values must be laid out as bias_tokens")
            lead("batch", bias_tokens.shape[0])
            c.bias_cols = bias_tokens.shape[1]
            c.bias_tokens, c.bias_values = bias_tokens.data_ptr(), bias_values.data_ptr()
            if bias_len is not None:
                _table("bias_len", bias_len, i32, (bias_tokens.shape[0],))
                c.bias_len = bias_len.data_ptr()
        for name, t in (("repetition_penalty", repetition_penalty), ("frequency_penalty", frequency_penalty),
                        ("presence_penalty", presence_penalty), ("temperature", temperature)):
            if t is not None:
                _table(name, t, f32, (None,))
                lead("batch", t.shape[0])
                setattr(c, name, t.data_ptr())
        if mask is not None:
            c.mask = token_mask(mask, mask_index)
            lead("rows", mask_index.shape[0])
            self.mask_tokens = 32 * mask.shape[1]
        else:
            self.mask_tokens = None
        self.c = c
        self._keep = (prompt_tokens, prompt_token_len, tokens, token_len, repetition_penalty, frequency_penalty,
                      presence_penalty, temperature, bias_tokens, bias_values, bias_len, mask, mask_index)


def process_logits(plan_: Plan, logits: torch.Tensor, params: LogitsParams, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, stream=None):
    """bsp_process_logits: logits [batch * beam_width, vocab] (bf16, fp16 or fp32) into ``out`` (None: in place),
    and each processed row's log-sum-exp into lse fp32 [batch * beam_width]."""
    rows = plan_.total_rows
    out = logits if out is None else out
    if logits.dtype not in LOGITS_DTYPES:
        raise ValueError(f"logits are {logits.dtype}")
    stride = _table("logits", logits, logits.dtype, (rows, None))
    out_stride = stride if out is logits else _table("out", out, logits.dtype, tuple(logits.shape))
    if params.rows not in (None, rows) or params.batch not in (None, plan_.batch):
        raise ValueError(f"lists for {params.batch} requests and {params.rows} rows, a plan of {plan_.batch} and {rows}")
    if params.mask_tokens is not None and params.mask_tokens < logits.shape[1]:
        raise ValueError(f"a mask of {params.mask_tokens} tokens for a vocabulary of {logits.shape[1]}")
    if lse is not None:
        _table("lse", lse, torch.float32, (rows,))
    _check("bsp_process_logits", load().bsp_process_logits(
        ctypes.byref(plan_), logits.data_ptr(), LOGITS_DTYPES[logits.dtype], stride, logits.shape[1],
        ctypes.byref(params.c), out.data_ptr(), out_stride, _address(lse), _stream(stream)))


def beam_select_workspace(batch: int, beam_width: int, vocab: int, num_candidates: int, device="cuda") -> torch.Tensor:
    """Device workspace of ``beam_select`` (bsp_beam_select_workspace_size bytes)."""
    n = ctypes.c_size_t()
    _check("bsp_beam_select_workspace_size", load().bsp_beam_select_workspace_size(
        int(batch), int(beam_width), int(vocab), int(num_candidates), ctypes.byref(n)))
    return torch.empty(max(16, n.value), dtype=torch.uint8, device=device)


def beam_select(plan_: Plan, logits: torch.Tensor, lse: torch.Tensor, cum_scores: torch.Tensor, scores: torch.Tensor,
                parents: torch.Tensor, tokens: torch.Tensor, workspace: torch.Tensor,
                mask: Optional[torch.Tensor] = None, mask_index: Optional[torch.Tensor] = None, stream=None):
    """bsp_beam_select: the best continuations of each request over its beams' vocabularies, into scores fp32,
    parents int32 and tokens int32 [batch, num_candidates], best first. lse fp32 [batch * beam_width],
    cum_scores fp32 [batch, beam_width] (or wider rows, the first beam_width read)."""
    rows, batch = plan_.total_rows, plan_.batch
    if logits.dtype not in LOGITS_DTYPES:
        raise ValueError(f"logits are {logits.dtype}")
    stride = _table("logits", logits, logits.dtype, (rows, None))
    _table("lse", lse, torch.float32, (rows,))
    cum_stride = _table("cum_scores", cum_scores, torch.float32, (batch, plan_.beam_width), exact_last=False)
    num = scores.shape[-1]
    for name, t, dt in (("scores", scores, torch.float32), ("parents", parents, torch.int32),
                        ("tokens", tokens, torch.int32)):
        if _table(name, t, dt, (batch, num)) != num:
            raise ValueError(f"{name} must be contiguous")
    m = None
    if mask is not None:
        m = token_mask(mask, mask_index)
        if 32 * mask.shape[1] < logits.shape[1] or mask_index.shape[0] != rows:
            raise ValueError("the mask does not cover the vocabulary, or its index the rows")
        m = ctypes.byref(m)
    _check("bsp_beam_select", load().bsp_beam_select(
        ctypes.byref(plan_), logits.data_ptr(), LOGITS_DTYPES[logits.dtype], stride, logits.shape[1], lse.data_ptr(),
        cum_scores.data_ptr(), cum_stride, m, num, scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)))


def beam_advance(plan_: Plan, parents: torch.Tensor, chosen: torch.Tensor,
                 cache_indirection: Optional[torch.Tensor] = None, cache_indirection_out: Optional[torch.Tensor] = None,
                 tokens: Optional[torch.Tensor] = None, tokens_out: Optional[torch.Tensor] = None,
                 token_len: Optional[torch.Tensor] = None, stream=None):
    """bsp_beam_advance: cache_indirection int32 [batch, beam_width, max_seq] and tokens int32
    [batch * beam_width, n] re-ordered by the chosen parents and extended by the new position (outputs None: in
    place). parents, chosen: int32 [batch, >= beam_width], the first beam_width of a row read."""
    batch, W, rows = plan_.batch, plan_.beam_width, plan_.total_rows
    i32 = torch.int32
    stride = _table("parents", parents, i32, (batch, W), exact_last=False)
    if _table("chosen", chosen, i32, (batch, W), exact_last=False) != stride:
        raise ValueError("parents and chosen must have the same row stride")
    max_seq = token_stride = token_cols = 0
    if cache_indirection is not None:
        cache_indirection_out = cache_indirection if cache_indirection_out is None else cache_indirection_out
        max_seq = cache_indirection.shape[-1]
        for name, t in (("cache_indirection", cache_indirection), ("cache_indirection_out", cache_indirection_out)):
            if _table(name, t, i32, (batch, W, max_seq)) != max_seq:
                raise ValueError(f"{name} must be contiguous")
    if tokens is not None:
        tokens_out = tokens if tokens_out is None else tokens_out
        token_cols = tokens.shape[-1]
        token_stride = _table("tokens", tokens, i32, (rows, token_cols))
        if _table("tokens_out", tokens_out, i32, (rows, token_cols)) != token_stride:
            raise ValueError("tokens and tokens_out must have the same row stride")
    if token_len is not None:
        _table("token_len", token_len, i32, (rows,))
    _check("bsp_beam_advance", load().bsp_beam_advance(
        ctypes.byref(plan_), parents.data_ptr(), chosen.data_ptr(), stride, _address(cache_indirection),
        _address(cache_indirection_out), max_seq, _address(tokens), _address(tokens_out), token_stride, token_cols,
        _address(token_len), _stream(stream)))


def _key_table(plan_: Plan, name: str, t: torch.Tensor, dtype):
    return _table(name, t, dtype, (plan_.batch, plan_.geo.num_kv_heads, plan_.max_prefix_len), exact_last=False)


def _rows_ok(plan_: Plan, q: torch.Tensor, lse: torch.Tensor):
    want = torch.bfloat16 if plan_.geo.dtype == 0 else torch.float16
    if q.dtype != want or q.numel() != plan_.total_rows * plan_.geo.num_q_heads * plan_.geo.head_dim or not q.is_contiguous():
        raise ValueError(f"q must be contiguous {want} [{plan_.total_rows}, {plan_.geo.num_q_heads}, {plan_.geo.head_dim}]")
    if lse.dtype != torch.float32 or lse.numel() != plan_.total_rows * plan_.geo.num_q_heads or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous fp32 [{plan_.total_rows}, {plan_.geo.num_q_heads}]")


_POOL_TYPES = {(KV_DTYPE_SAME, 0): (torch.bfloat16,), (KV_DTYPE_SAME, 1): (torch.float16,),
               (KV_DTYPE_E4M3, 0): (torch.uint8, torch.float8_e4m3fn), (KV_DTYPE_E4M3, 1): (torch.uint8, torch.float8_e4m3fn)}


def _pools_ok(plan_: Plan, *pools: torch.Tensor):
    """Pools of the plan's geometry: its element type, all of its pages, contiguous (the calls go by their addresses)."""
    g = plan_.geo
    heads, slots, dim, types = g.num_kv_heads, g.page_size, g.head_dim, _POOL_TYPES[g.kv_dtype, g.dtype]
    shape = (g.num_pages, heads, slots, dim)
    for t in pools:
        if t.dtype in types and t.is_contiguous() and (t.shape == shape or (  # (the usual case first)
                t.numel() >= shape[0] * heads * slots * dim and (t.dim() != 4 or t.shape[1:] == shape[1:]))):
            continue
        raise ValueError(f"a pool must be contiguous {types[0]} {list(shape)}, not {t.dtype} {list(t.shape)}")


def key_weights(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, lse: torch.Tensor, softmax_scale: float,
                weights: torch.Tensor, window: int = 0, flags: int = 0, stream=None):
    """bsp_key_weights: the attention weight each prompt key received from the plan's query rows, into weights
    fp32 [batch, num_kv_heads, >= longest prompt] (flags FLAG_ACCUMULATE: added to it)."""
    _rows_ok(plan_, q, lse)
    _pools_ok(plan_, k_pool)
    stride = _key_table(plan_, "weights", weights, torch.float32)
    _check("bsp_key_weights", load().bsp_key_weights(
        ctypes.byref(plan_), q.data_ptr(), k_pool.data_ptr(), lse.data_ptr(), float(softmax_scale), int(window),
        int(flags), weights.data_ptr(), stride, _stream(stream)))


def key_weights_fp8(plan_: Plan, q: torch.Tensor, k_pool: torch.Tensor, lse: torch.Tensor, softmax_scale: float,
                    k_scale: float, weights: torch.Tensor, window: int = 0, flags: int = 0, stream=None):
    """bsp_key_weights_fp8: key_weights over a uint8 E4M3 pool (key = code x k_scale; not one with BlockScales, whose
    exponents it would pass over)."""
    _rows_ok(plan_, q, lse)
    _pools_ok(plan_, k_pool)
    stride = _key_table(plan_, "weights", weights, torch.float32)
    _check("bsp_key_weights_fp8", load().bsp_key_weights_fp8(
        ctypes.byref(plan_), q.data_ptr(), k_pool.data_ptr(), lse.data_ptr(), float(softmax_scale), float(k_scale),
        int(window), int(flags), weights.data_ptr(), stride, _stream(stream)))


def evict_prefix(plan_: Plan, weights: torch.Tensor, keep_len: torch.Tensor, sinks: int, recent: int,
                 k_pool: torch.Tensor, v_pool: torch.Tensor, kept: torch.Tensor,
                 positions: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                 positions_out: Optional[torch.Tensor] = None, stream=None):
    """bsp_evict_prefix: per (request, kv head) the keep_len[b] rows of largest weight move to the front of the
    request's pages, in place. weights fp32, positions and kept int32 [batch, num_kv_heads, >= longest prompt]. Not for
    pools with BlockScales: rows would leave their blocks' scales behind."""
    i32 = torch.int32
    stride = _key_table(plan_, "weights", weights, torch.float32)
    out_stride = _key_table(plan_, "kept", kept, i32)
    _table("keep_len", keep_len, i32, (plan_.batch,))
    _pools_ok(plan_, k_pool, v_pool)
    if positions is not None and _key_table(plan_, "positions", positions, i32) != stride:
        raise ValueError("positions must have the row stride of weights")
    for name, t, dt in (("weights_out", weights_out, torch.float32), ("positions_out", positions_out, i32)):
        if t is not None and _key_table(plan_, name, t, dt) != out_stride:
            raise ValueError(f"{name} must have the row stride of kept")
    _check("bsp_evict_prefix", load().bsp_evict_prefix(
        ctypes.byref(plan_), weights.data_ptr(), stride, _address(positions), keep_len.data_ptr(), int(sinks), int(recent),
        k_pool.data_ptr(), v_pool.data_ptr(), kept.data_ptr(), _address(weights_out), _address(positions_out), out_stride,
        _stream(stream)))


# ---------------------------------------------------------------- pages of the cache

def fork_workspace(batch: int, num_forks: int, device="cuda") -> torch.Tensor:
    """Device workspace of ``fork_tables`` (bsp_fork_workspace_size bytes)."""
    n = ctypes.c_size_t()
    _check("bsp_fork_workspace_size", load().bsp_fork_workspace_size(int(batch), int(num_forks), ctypes.byref(n)))
    return torch.empty(max(16, n.value), dtype=torch.uint8, device=device)


def _counts(plan_: Plan, *refs: torch.Tensor):
    for t in refs:
        _table("refs", t, torch.int32, (plan_.geo.num_pages,))


def fork_tables(plan_: Plan, beams: torch.Tensor, refs: torch.Tensor, refs_out: torch.Tensor, pages_out: torch.Tensor,
                workspace: torch.Tensor, stream=None):
    """bsp_fork_tables: tables of the beams (int32 [batch, num_forks], -1: none) that go on as sequences of their own:
    full prompt pages shared, fresh ones for the rest, in pages_out int32 [batch * num_forks, columns]. refs, refs_out:
    int32 [num_pages], the counts before and after (may be one tensor)."""
    i32 = torch.int32
    forks = beams.shape[-1]
    stride = _table("beams", beams, i32, (plan_.batch, forks))
    _counts(plan_, refs, refs_out)
    out_stride = _table("pages_out", pages_out, i32, (plan_.batch * forks, None))
    _check("bsp_fork_tables", load().bsp_fork_tables(
        ctypes.byref(plan_), beams.data_ptr(), stride, forks, refs.data_ptr(), refs_out.data_ptr(), pages_out.data_ptr(),
        out_stride, pages_out.shape[1], workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def _captured(t: torch.Tensor) -> bool:
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


def fork_rows(plan_: Plan, beams: torch.Tensor, pages_out: torch.Tensor, beam_pages: Optional[torch.Tensor],
              cache_indirection: Optional[torch.Tensor], k_pool: torch.Tensor, v_pool: torch.Tensor,
              scales: Optional[BlockScales] = None, stream=None):
    """bsp_fork_rows: the prompt's last rows and the beams' tail rows into the fresh pages of ``fork_tables``."""
    i32 = torch.int32
    forks = beams.shape[-1]
    stride = _table("beams", beams, i32, (plan_.batch, forks))
    out_stride = _table("pages_out", pages_out, i32, (plan_.batch * forks, None))
    cols = max_seq = 0
    if beam_pages is not None:
        cols = _table("beam_pages", beam_pages, i32, (plan_.total_rows, None))
        if plan_.max_tail_len > 0 and beam_pages.shape[1] * plan_.geo.page_size < plan_.max_total_len:
            raise ValueError(f"beam_pages has {beam_pages.shape[1]} columns for {plan_.max_total_len} positions")
        if cols != beam_pages.shape[1] and _captured(beam_pages):
            # (a replay reads as far as its plan's sequences and the stride allow)
            end = beam_pages.storage_offset() + plan_.total_rows * cols
            if 4 * end > beam_pages.untyped_storage().nbytes():
                raise ValueError("the last row of beam_pages ends before its stride")
        if cache_indirection is not None:
            max_seq = cache_indirection.shape[-1]
            if _table("cache_indirection", cache_indirection, i32, (plan_.batch, plan_.beam_width, max_seq)) != max_seq:
                raise ValueError("cache_indirection must be contiguous")
    _pools_ok(plan_, k_pool, v_pool)
    _check("bsp_fork_rows", load().bsp_fork_rows(
        ctypes.byref(plan_), beams.data_ptr(), stride, forks, pages_out.data_ptr(), out_stride, pages_out.shape[1],
        _address(beam_pages), cols, _address(cache_indirection), max_seq, k_pool.data_ptr(), v_pool.data_ptr(),
        None if scales is None else scales._of(plan_), _stream(stream)))


def free_pages(plan_: Plan, tables: torch.Tensor, refs: torch.Tensor, refs_out: torch.Tensor, stream=None):
    """bsp_free_pages: one reference less for every page in tables (int32 [rows, columns], -1: none)."""
    stride = _table("tables", tables, torch.int32, (None, None))
    _counts(plan_, refs, refs_out)
    _check("bsp_free_pages", load().bsp_free_pages(
        ctypes.byref(plan_), tables.data_ptr(), stride, tables.shape[0], tables.shape[1], refs.data_ptr(),
        refs_out.data_ptr(), _stream(stream)))


class PageMoves:
    """Buffers of a compaction: pairs int32 [num_pages // 2, 2] (from, to), count int32 [2] (pairs, live pages), remap
    int32 [num_pages]; or with ``pairs`` and ``count`` given, a list of copies of the caller's."""

    def __init__(self, num_pages: int, device="cuda", pairs: Optional[torch.Tensor] = None,
                 count: Optional[torch.Tensor] = None):
        i32 = torch.int32
        self.pairs = torch.empty((num_pages // 2, 2), dtype=i32, device=device) if pairs is None else pairs
        self.count = torch.zeros(2, dtype=i32, device=device) if count is None else count
        self.remap = torch.empty(num_pages, dtype=i32, device=device) if pairs is None else None
        if _table("pairs", self.pairs, i32, (None, 2)) != 2:
            raise ValueError("pairs must be contiguous")
        _table("count", self.count, i32, (None,))


def compact_tables(plan_: Plan, refs: torch.Tensor, refs_out: torch.Tensor, moves: PageMoves,
                   tables: Optional[torch.Tensor] = None, tables_out: Optional[torch.Tensor] = None, stream=None):
    """bsp_compact_tables: the live pages' new places, the lowest ids, into ``moves``, refs_out and tables_out (None: in
    place). tables: int32 [rows, columns], every live sequence's pages (-1: none)."""
    _counts(plan_, refs, refs_out)
    if moves.remap is None or moves.remap.shape[0] != plan_.geo.num_pages:
        raise ValueError(f"moves are not made for {plan_.geo.num_pages} pages")
    if moves.count.shape[0] < 2 or moves.pairs.shape[0] < plan_.geo.num_pages // 2:
        raise ValueError(f"count {list(moves.count.shape)} and pairs {list(moves.pairs.shape)} for two counts and "
                         f"{plan_.geo.num_pages // 2} pairs")
    stride = rows = cols = 0
    if tables is not None:
        tables_out = tables if tables_out is None else tables_out
        rows, cols = tables.shape
        stride = _table("tables", tables, torch.int32, (rows, cols))
        if _table("tables_out", tables_out, torch.int32, (rows, cols)) != stride:
            raise ValueError("tables and tables_out must have the same row stride")
    _check("bsp_compact_tables", load().bsp_compact_tables(
        ctypes.byref(plan_), refs.data_ptr(), refs_out.data_ptr(), moves.pairs.data_ptr(), moves.count.data_ptr(),
        moves.remap.data_ptr(), _address(tables), _address(tables_out), stride, rows, cols, _stream(stream)))


def copy_pages(plan_: Plan, moves: PageMoves, k_pool: torch.Tensor, v_pool: torch.Tensor,
               scales: Optional[BlockScales] = None, stream=None):
    """bsp_copy_pages: the first count[0] pairs of ``moves``, whole pages of both pools (and their scales)."""
    if moves.count.shape[0] < 1:
        raise ValueError("count is empty")
    _pools_ok(plan_, k_pool, v_pool)
    _check("bsp_copy_pages", load().bsp_copy_pages(
        ctypes.byref(plan_), moves.pairs.data_ptr(), moves.count.data_ptr(), moves.pairs.shape[0], k_pool.data_ptr(),
        v_pool.data_ptr(), None if scales is None else scales._of(plan_), _stream(stream)))
