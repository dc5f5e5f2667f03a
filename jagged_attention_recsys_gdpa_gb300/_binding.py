"""ctypes binding of libjattn (argument marshalling only).

Every computation runs in the CUDA library; this module only converts torch
tensors to raw pointers and sizes, passes the current CUDA stream, and turns
non-zero return codes into exceptions. The library must exist: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

from . import build as _build

SOFTMAX, SILU, GELU_TANH, GELU_POLY = 0, 1, 2, 3
MASK_NONE, MASK_CAUSAL, MASK_WINDOW, MASK_BLOCK = 0, 1, 2, 4

EXPORTED = (
    "jattn_workspace_size",
    "jattn_fwd",
    "jattn_fwd_noalloc",
    "jattn_bwd",
    "jattn_bwd_rope",
    "jattn_bwd_rope_workspace_size",
    "jattn_rope",
    "jattn_mxfp8_scale_rows",
    "jattn_mxfp8_quantize",
    "jattn_fwd_mxfp8",
    "jattn_bwd_mxfp8",
    "jattn_cache_append",
    "jattn_cache_read",
    "jattn_decode",
    "jattn_decode_scratch_size",
    "jattn_layer_norm",
    "jattn_layer_norm_bwd",
    "jattn_layer_norm_bwd_scratch_size",
    "jattn_rotary",
    "jattn_rotary_tables",
    "jattn_page_assign",
    "jattn_page_release",
    "jattn_page_scratch_size",
    "jattn_schedule",
    "jattn_partition",
    "jattn_max_tiles",
    "jattn_get_status",
    "jattn_error_string",
    "jattn_last_error",
    "jattn_profile_events",
    "jattn_debug_set",
)


class Params(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int64),
        ("total_q", ctypes.c_int64),
        ("total_kv", ctypes.c_int64),
        ("H", ctypes.c_int),
        ("D", ctypes.c_int),
        ("act", ctypes.c_int),
        ("mask", ctypes.c_int),
        ("window", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("norm_by_lkv", ctypes.c_int),
    ]


CACHE_BF16, CACHE_MXFP8 = 0, 1


class Cache(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int),
        ("H", ctypes.c_int),
        ("D", ctypes.c_int),
        ("format", ctypes.c_int),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


F32, BF16, F16 = 0, 1, 2
ROTARY_INTERLEAVED, ROTARY_HALF = 0, 1
SCALE_NONE, SCALE_LINEAR, SCALE_NTK, SCALE_YARN = 0, 1, 2, 3


class Norm(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("heads", ctypes.c_int),
        ("N", ctypes.c_int),
        ("type", ctypes.c_int),
        ("weight_type", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("zero_behind", ctypes.c_int),
        ("x_strides", ctypes.c_int64 * 2),
        ("y_strides", ctypes.c_int64 * 2),
        ("dy_strides", ctypes.c_int64 * 2),
        ("zero_stats", ctypes.c_int),
    ]


class Rotary(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int64),
        ("total", ctypes.c_int64),
        ("heads", ctypes.c_int),
        ("D", ctypes.c_int),
        ("half", ctypes.c_int),
        ("type", ctypes.c_int),
        ("layout", ctypes.c_int),
        ("inverse", ctypes.c_int),
        ("zero_behind", ctypes.c_int),
        ("table_rows", ctypes.c_int64),
        ("x_strides", ctypes.c_int64 * 2),
        ("y_strides", ctypes.c_int64 * 2),
    ]


class RotaryTables(ctypes.Structure):
    _fields_ = [
        ("first", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("half", ctypes.c_int),
        ("scaling", ctypes.c_int),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original", ctypes.c_double),
        ("beta_fast", ctypes.c_double),
        ("beta_slow", ctypes.c_double),
    ]


class PagePool(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int),
        ("free_pages", ctypes.c_void_p),
        ("count", ctypes.c_void_p),
    ]


class JattnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = ""
        if code in (2, 8):
            detail = " [" + load().jattn_last_error().decode() + "]"
        super().__init__(f"{where}: {error_string(code)} (code {code}){detail}")


_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libjattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"libjattn.so not found at {path}; build it with "
            "`python -m jagged_attention_recsys_gdpa_gb300.build` (no CPU fallback exists)"
        )
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Params)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.jattn_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
    lib.jattn_workspace_size.restype = i32
    lib.jattn_fwd.argtypes = [P] + [vp] * 7 + [vp, ctypes.c_size_t, vp]
    lib.jattn_fwd.restype = i32
    lib.jattn_fwd_noalloc.argtypes = [P] + [vp] * 8 + [vp]
    lib.jattn_fwd_noalloc.restype = i32
    lib.jattn_bwd.argtypes = [P] + [vp] * 11 + [vp, ctypes.c_size_t, vp]
    lib.jattn_bwd.restype = i32
    lib.jattn_bwd_rope.argtypes = [P] + [vp] * 10 + [i64] + [vp] * 3 + [vp, ctypes.c_size_t, vp]
    lib.jattn_bwd_rope.restype = i32
    lib.jattn_rope.argtypes = [P, vp, vp, i32, i32, vp, vp, vp, vp, i64, vp, ctypes.c_size_t, vp]
    lib.jattn_rope.restype = i32
    lib.jattn_mxfp8_scale_rows.argtypes = [i64, i64]
    lib.jattn_mxfp8_scale_rows.restype = i64
    lib.jattn_mxfp8_quantize.argtypes = [i64, i64, i32, i32] + [vp] * 5 + [vp, ctypes.c_size_t, vp]
    lib.jattn_mxfp8_quantize.restype = i32
    lib.jattn_fwd_mxfp8.argtypes = [P] + [vp] * 12 + [vp, ctypes.c_size_t, vp]
    lib.jattn_fwd_mxfp8.restype = i32
    lib.jattn_bwd_mxfp8.argtypes = [P] + [vp] * 17 + [vp, ctypes.c_size_t, vp]
    lib.jattn_bwd_mxfp8.restype = i32
    lib.jattn_bwd_rope_workspace_size.argtypes = [P, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.jattn_bwd_rope_workspace_size.restype = i32
    C = ctypes.POINTER(Cache)
    lib.jattn_cache_append.argtypes = [C, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp, i64, vp, ctypes.c_size_t, vp]
    lib.jattn_cache_append.restype = i32
    lib.jattn_cache_read.argtypes = [C, i64, i64, vp, vp, vp, i64, vp, vp, vp, ctypes.c_size_t, vp]
    lib.jattn_cache_read.restype = i32
    lib.jattn_decode_scratch_size.argtypes = [P, C, ctypes.POINTER(ctypes.c_size_t)]
    lib.jattn_decode_scratch_size.restype = i32
    lib.jattn_decode.argtypes = [P, C, vp, vp, vp, i64, vp, vp, vp, vp, ctypes.c_size_t, vp, ctypes.c_size_t, vp]
    lib.jattn_decode.restype = i32
    N, Z = ctypes.POINTER(Norm), ctypes.c_size_t
    lib.jattn_layer_norm.argtypes = [N] + [vp] * 8 + [Z, vp]
    lib.jattn_layer_norm.restype = i32
    lib.jattn_layer_norm_bwd_scratch_size.argtypes = [N, ctypes.POINTER(Z)]
    lib.jattn_layer_norm_bwd_scratch_size.restype = i32
    lib.jattn_layer_norm_bwd.argtypes = [N] + [vp] * 10 + [Z, vp, Z, vp]
    lib.jattn_layer_norm_bwd.restype = i32
    lib.jattn_rotary.argtypes = [ctypes.POINTER(Rotary)] + [vp] * 7 + [Z, vp]
    lib.jattn_rotary.restype = i32
    lib.jattn_rotary_tables.argtypes = [ctypes.POINTER(RotaryTables), vp, vp, vp]
    lib.jattn_rotary_tables.restype = i32
    G = ctypes.POINTER(PagePool)
    lib.jattn_page_scratch_size.argtypes = [i64, i64, i64, ctypes.POINTER(Z)]
    lib.jattn_page_scratch_size.restype = i32
    lib.jattn_page_assign.argtypes = [G, i64, i64, vp, vp, vp, i64, vp, vp, Z, vp, Z, vp]
    lib.jattn_page_assign.restype = i32
    lib.jattn_page_release.argtypes = [G, i64, vp, vp, vp, i64, vp, Z, vp, Z, vp]
    lib.jattn_page_release.restype = i32
    lib.jattn_schedule.argtypes = [P, vp, vp, i32, i32, i32, vp, i64, vp, vp, ctypes.c_size_t, vp]
    lib.jattn_schedule.restype = i32
    lib.jattn_partition.argtypes = [i64, vp, vp, i32, i32, i32, vp, vp]
    lib.jattn_partition.restype = i32
    lib.jattn_max_tiles.argtypes = [P, i32, i32]
    lib.jattn_max_tiles.restype = i64
    lib.jattn_get_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
    lib.jattn_get_status.restype = i32
    lib.jattn_error_string.argtypes = [i32]
    lib.jattn_error_string.restype = ctypes.c_char_p
    lib.jattn_last_error.argtypes = []
    lib.jattn_last_error.restype = ctypes.c_char_p
    lib.jattn_profile_events.argtypes = [ctypes.POINTER(vp)]
    lib.jattn_profile_events.restype = None
    lib.jattn_debug_set.argtypes = [i32, ctypes.c_uint64]
    lib.jattn_debug_set.restype = None
    _lib = lib
    return lib


_host = None


def host():
    """The extension module of the row operators' and the page pool's calls, bound to the loaded library."""
    global _host
    if _host is None:
        from .paged import status_address

        path = _build.HOST
        if not os.path.exists(path):
            raise RuntimeError(f"_host.so not found at {path}; build it with "
                               "`python -m jagged_attention_recsys_gdpa_gb300.build` (no other path exists)")
        built = _build.host_misfit()
        if built:
            raise RuntimeError(f"_host.so was built for {built}, which is not what is installed; build it again with "
                               "`python -m jagged_attention_recsys_gdpa_gb300.build`")
        spec = importlib.util.spec_from_file_location("_host", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(load()._handle, check, status_address)
        _host = module
    return _host


def error_string(code: int) -> str:
    return load().jattn_error_string(int(code)).decode()


def check(code: int, where: str):
    if code != 0:
        raise JattnError(code, where)


def params(B, total_q, total_kv, H, D, act, mask, window, scale, norm_by_lkv) -> Params:
    return Params(int(B), int(total_q), int(total_kv), int(H), int(D), int(act), int(mask), int(window),
                  float(scale or 0.0), int(bool(norm_by_lkv)))


def workspace_size(p: Params) -> int:
    n = ctypes.c_size_t(0)
    check(load().jattn_workspace_size(ctypes.byref(p), ctypes.byref(n)), "jattn_workspace_size")
    return int(n.value)


def bwd_rope_workspace_size(p: Params, rope_rows: int) -> int:
    n = ctypes.c_size_t(0)
    check(load().jattn_bwd_rope_workspace_size(ctypes.byref(p), int(rope_rows), ctypes.byref(n)),
          "jattn_bwd_rope_workspace_size")
    return int(n.value)


def ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def fwd(p: Params, q_off, kv_off, q, k, v, o, lse, ws, ws_bytes: int, stream: int):
    check(load().jattn_fwd(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(k), ptr(v), ptr(o), ptr(lse),
                           ws, ws_bytes, stream), "jattn_fwd")


def fwd_noalloc(p: Params, q_off, kv_off, q, k, v, o, lse, device_status, stream: int):
    """Forward without a workspace (scratch held by the library); see jattn_fwd_noalloc."""
    check(load().jattn_fwd_noalloc(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(k), ptr(v), ptr(o),
                                   ptr(lse), ptr(device_status), stream), "jattn_fwd_noalloc")


def bwd(p: Params, q_off, kv_off, q, k, v, o, lse, do, dq, dk, dv, ws, ws_bytes: int, stream: int):
    check(load().jattn_bwd(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(k), ptr(v), ptr(o), ptr(lse),
                           ptr(do), ptr(dq), ptr(dk), ptr(dv), ws, ws_bytes, stream), "jattn_bwd")


def bwd_rope(p: Params, q_off, kv_off, q, k, v, o, lse, do, rope_cos, rope_sin, dq, dk, dv, ws, ws_bytes: int,
             stream: int):
    """jattn_bwd_rope: q and k are the rotated inputs; dq and dk come back rotated by R^T."""
    check(load().jattn_bwd_rope(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(k), ptr(v), ptr(o),
                                ptr(lse), ptr(do), ptr(rope_cos), ptr(rope_sin), int(rope_cos.shape[0]), ptr(dq),
                                ptr(dk), ptr(dv), ws, ws_bytes, stream), "jattn_bwd_rope")


def mxfp8_scale_rows(B: int, total: int) -> int:
    return int(load().jattn_mxfp8_scale_rows(int(B), int(total)))


def mxfp8_quantize(B: int, total: int, H: int, D: int, off, x, codes, scales, block_start, ws, ws_bytes: int,
                   stream: int):
    check(load().jattn_mxfp8_quantize(int(B), int(total), int(H), int(D), ptr(off), ptr(x), ptr(codes), ptr(scales),
                                      ptr(block_start), ws, ws_bytes, stream), "jattn_mxfp8_quantize")


def fwd_mxfp8(p: Params, q_off, kv_off, q, q_scales, q_bs, k, k_scales, v, v_scales, kv_bs, o, lse, ws,
              ws_bytes: int, stream: int):
    check(load().jattn_fwd_mxfp8(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(q_scales), ptr(q_bs), ptr(k),
                                 ptr(k_scales), ptr(v), ptr(v_scales), ptr(kv_bs), ptr(o), ptr(lse), ws, ws_bytes,
                                 stream), "jattn_fwd_mxfp8")


def bwd_mxfp8(p: Params, q_off, kv_off, q, q_scales, q_bs, k, k_scales, v, v_scales, kv_bs, o, lse, dout,
              dout_scales, dq, dk, dv, ws, ws_bytes: int, stream: int):
    check(load().jattn_bwd_mxfp8(ctypes.byref(p), ptr(q_off), ptr(kv_off), ptr(q), ptr(q_scales), ptr(q_bs), ptr(k),
                                 ptr(k_scales), ptr(v), ptr(v_scales), ptr(kv_bs), ptr(o), ptr(lse), ptr(dout),
                                 ptr(dout_scales), ptr(dq), ptr(dk), ptr(dv), ws, ws_bytes, stream),
          "jattn_bwd_mxfp8")


def rope(p: Params, q_off, kv_off, keys: bool, inverse: bool, x, y, rope_cos, rope_sin, ws, ws_bytes: int,
         stream: int):
    """jattn_rope: y = R(pos) x (or R(pos)^T x) on query (keys=False) or key rows."""
    check(load().jattn_rope(ctypes.byref(p), ptr(q_off), ptr(kv_off), int(bool(keys)), int(bool(inverse)), ptr(x),
                            ptr(y), ptr(rope_cos), ptr(rope_sin), int(rope_cos.shape[0]), ws, ws_bytes, stream),
          "jattn_rope")


def cache(n_pages, page_size, H, D, fmt, k, v, k_scales, v_scales) -> Cache:
    return Cache(int(n_pages), int(page_size), int(H), int(D), int(fmt), ptr(k), ptr(v), ptr(k_scales), ptr(v_scales))


# The paged-cache calls serve single tokens, where the host's time counts: they take the cache as a reference made
# once (byref) and addresses of required tensors directly.
def cache_append(c, B: int, total: int, off, start, page_table, k, v, cos, sin, ws: int, ws_bytes: int, stream: int):
    rc = (_lib or load()).jattn_cache_append(c, B, total, ptr(off), start.data_ptr(), page_table.data_ptr(),
                                             page_table.shape[1], k.data_ptr(), v.data_ptr(), ptr(cos), ptr(sin),
                                             0 if cos is None else cos.shape[0], ws, ws_bytes, stream)
    if rc:
        check(rc, "jattn_cache_append")


def cache_read(c, B: int, total: int, off, start, page_table, k, v, ws: int, ws_bytes: int, stream: int):
    rc = (_lib or load()).jattn_cache_read(c, B, total, off.data_ptr(), ptr(start), page_table.data_ptr(),
                                           page_table.shape[1], k.data_ptr(), v.data_ptr(), ws, ws_bytes, stream)
    if rc:
        check(rc, "jattn_cache_read")


def decode_scratch_size(p, c) -> int:
    n = ctypes.c_size_t(0)
    check((_lib or load()).jattn_decode_scratch_size(p, c, ctypes.byref(n)), "jattn_decode_scratch_size")
    return n.value


def decode(p, c, q_off, kv_lens, page_table, q, o, lse, scratch: int, scratch_bytes: int, ws: int, ws_bytes: int,
           stream: int):
    rc = (_lib or load()).jattn_decode(p, c, ptr(q_off), kv_lens.data_ptr(), page_table.data_ptr(),
                                       page_table.shape[1], q.data_ptr(), o.data_ptr(), ptr(lse), scratch,
                                       scratch_bytes, ws, ws_bytes, stream)
    if rc:
        check(rc, "jattn_decode")


def schedule(p: Params, q_off, kv_off, row_tile, col_tile, transposed, tiles, max_tiles, n_tiles, ws, ws_bytes,
             stream):
    check(load().jattn_schedule(ctypes.byref(p), ptr(q_off), ptr(kv_off), int(row_tile), int(col_tile),
                                int(bool(transposed)), ptr(tiles), int(max_tiles), ptr(n_tiles), ws, ws_bytes,
                                stream), "jattn_schedule")


def partition(q_off, kv_off, mask: int, window: int, n_ranks: int, rank_of, rank_pairs):
    """Host arrays (numpy): q_off, kv_off int64 [B+1]; rank_of int32 [B], rank_pairs int64 [n_ranks] out."""
    B = len(q_off) - 1
    check(load().jattn_partition(B, q_off.ctypes.data, kv_off.ctypes.data, int(mask), int(window), int(n_ranks),
                                 rank_of.ctypes.data, rank_pairs.ctypes.data), "jattn_partition")


def max_tiles(p: Params, row_tile: int, transposed: bool) -> int:
    return int(load().jattn_max_tiles(ctypes.byref(p), int(row_tile), int(bool(transposed))))


def get_status(ws, stream) -> int:
    s = ctypes.c_int(0)
    check(load().jattn_get_status(ws, stream, ctypes.byref(s)), "jattn_get_status")
    return int(s.value)


def debug_set(flags: int, timeout_ns: int):
    load().jattn_debug_set(int(flags), int(timeout_ns))


def profile_events(events):
    """Record the six given torch.cuda.Event objects around the main kernels (None: off)."""
    if events is None:
        load().jattn_profile_events(None)
        return
    arr = (ctypes.c_void_p * 6)(*[e.cuda_event for e in events])
    load().jattn_profile_events(arr)
