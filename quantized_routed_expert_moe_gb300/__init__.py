"""Python binding of the GB300 routed-MoE library (ctypes over ``include/moe.h``).

Argument marshalling only: every step of the computation runs in the CUDA
library ``_build/libmoe_gb300.so``. Importing this module does not build or
fall back to anything; calling into it without the built library raises.

Functions keep the C names (``moe_layer_create``, ``moe_route``,
``moe_decode``, ``moe_prefill_chunk``, ``moe_decode_tokens_host``,
``moe_cache_stage`` ...). Pointer arguments accept a torch tensor (its
``data_ptr()``), a numpy array, a raw integer address or None.

``MoELayer``, ``BlockNorm`` and ``KVCache`` own a handle or weights and take
tensors; the latter two check shapes, types and devices before a call, and run on
torch's current stream where none is given. Elsewhere stream=None is the legacy
default stream, as in C.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libmoe_gb300.so")

MOE_ABI_VERSION = 1
MOE_F32, MOE_BF16, MOE_E4M3 = 0, 1, 2
MOE_W_F32, MOE_W_Q8G64, MOE_W_Q4G64, MOE_W_Q2G64 = 0, 1, 2, 3
STATUS = {0: "MOE_OK", 1: "MOE_E_INVALID", 2: "MOE_E_UNSUPPORTED", 3: "MOE_E_NOMEM",
          4: "MOE_E_CUDA", 5: "MOE_E_TIMEOUT", 6: "MOE_E_STATE", 7: "MOE_E_SOURCE"}

# every symbol include/moe.h declares
EXPORTS = ("moe_layer_create", "moe_layer_destroy", "moe_expert_record_bytes", "moe_pack_expert_record",
           "moe_layer_device_bytes", "moe_layer_set_next", "moe_layer_set_router_scoring", "moe_route", "moe_layer_selection", "moe_decode", "moe_decode_static_scratch", "moe_prefill_chunk",
           "moe_decode_tokens_host", "moe_cache_stage", "moe_cache_prefetch", "moe_cache_prefetch_stats", "moe_cache_stats", "moe_cache_residency", "moe_cache_usage", "moe_cache_pin", "moe_hottest", "moe_cache_pin_hottest", "moe_lfu_trace", "moe_lfu_trace_pinned",
           "moe_profile_start", "moe_profile_stop", "moe_layer_set_option", "moe_layer_check", "moe_trace_read_split",
           "moe_block_norm", "moe_block_norm_check", "moe_kv_create", "moe_kv_destroy", "moe_kv_device_bytes", "moe_kv_append", "moe_kv_attend",
           "moe_kv_append_check", "moe_kv_attend_check", "moe_kv_locate", "moe_kv_health", "moe_kv_set_option",
           "moe_status_str", "moe_last_error")

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_STATIC_SCRATCH_BYTES = 256 * 1024
MOE_OPT_TEST_STALL_SHARED, MOE_OPT_TRACE = 2, 3
MOE_OPT_HOST_TIMEOUT_MS, MOE_OPT_TEST_STALL_COPIES_MS, MOE_OPT_CACHE_DEVICE = 4, 5, 6
MOE_MAX_TOP_K = 8
MOE_KV_BAD_SEQ, MOE_KV_BAD_LENGTH, MOE_KV_BAD_PAGE, MOE_KV_TIMEOUT = 1, 2, 4, 8
MOE_KV_OPT_TEST_STALL = 1


class MoEError(RuntimeError):
    def __init__(self, status: int, call: str, detail: str):
        self.status = status
        super().__init__(f"{call}: {STATUS.get(status, status)}: {detail}")


class moe_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class moe_expert(ctypes.Structure):
    _fields_ = [("gate", moe_qmat), ("up", moe_qmat), ("down", moe_qmat)]


class moe_router(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("q", moe_qmat)]


class moe_layer_desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("router_fmt", ctypes.c_int32), ("expert_fmt", ctypes.c_int32), ("group", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("cache_slots", ctypes.c_int32)]


class moe_cache_stats_t(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_uint64), ("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64),
                ("bytes_h2d", ctypes.c_uint64), ("stage_ns", ctypes.c_uint64)]


class moe_block_norm_desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("hidden", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("block_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("weight_offset", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("o_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64),
                ("h_stride", ctypes.c_int64)]


class moe_kv_desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("rotary_adjacent", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class moe_kv_append_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("seq", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("T", ctypes.c_int32),
                ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("q_out", ctypes.c_void_p)]


class moe_kv_attend_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("block_table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class moe_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_uint64), ("total_ms", ctypes.c_double)]


SOURCE_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t)

_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library not built ({LIB_PATH} missing): run "
                    "`python -m quantized_routed_expert_moe_gb300.build` or __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            st = ctypes.c_int
            L.moe_layer_create.restype = st
            L.moe_layer_create.argtypes = [ctypes.POINTER(moe_layer_desc), ctypes.POINTER(moe_router), vp,
                                           ctypes.POINTER(moe_expert), ctypes.POINTER(moe_expert), vp,
                                           SOURCE_FN, vp, i32, ctypes.POINTER(vp)]
            L.moe_layer_destroy.restype = None
            L.moe_layer_destroy.argtypes = [vp]
            L.moe_expert_record_bytes.restype = sz
            L.moe_expert_record_bytes.argtypes = [ctypes.POINTER(moe_layer_desc)]
            L.moe_pack_expert_record.restype = st
            L.moe_pack_expert_record.argtypes = [ctypes.POINTER(moe_layer_desc), ctypes.POINTER(moe_expert), vp]
            L.moe_layer_device_bytes.restype = sz
            L.moe_layer_device_bytes.argtypes = [vp]
            L.moe_route.restype = st
            L.moe_route.argtypes = [vp, vp, i32, vp, vp, vp]
            L.moe_decode.restype = st
            L.moe_decode.argtypes = [vp, vp, vp, vp, vp]
            L.moe_decode_static_scratch.restype = st
            L.moe_decode_static_scratch.argtypes = [vp, vp, vp, vp, vp]
            L.moe_prefill_chunk.restype = st
            L.moe_prefill_chunk.argtypes = [vp, vp, i32, vp, vp, vp]
            L.moe_decode_tokens_host.restype = st
            L.moe_decode_tokens_host.argtypes = [vp, vp, i32, vp, vp]
            L.moe_cache_stage.restype = st
            L.moe_cache_stage.argtypes = [vp, vp, i32, vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.moe_cache_prefetch.restype = st
            L.moe_cache_prefetch.argtypes = [vp, vp, vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.moe_cache_prefetch_stats.restype = st
            L.moe_cache_prefetch_stats.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64)]
            L.moe_cache_stats.restype = st
            L.moe_cache_stats.argtypes = [vp, ctypes.POINTER(moe_cache_stats_t)]
            L.moe_cache_residency.restype = st
            L.moe_cache_residency.argtypes = [vp, vp]
            L.moe_cache_usage.restype = st
            L.moe_cache_usage.argtypes = [vp, vp]
            L.moe_cache_pin.restype = st
            L.moe_cache_pin.argtypes = [vp, vp, ctypes.c_int32]
            L.moe_hottest.restype = st
            L.moe_hottest.argtypes = [vp, i32, i32, vp]
            L.moe_cache_pin_hottest.restype = st
            L.moe_cache_pin_hottest.argtypes = [vp, i32]
            L.moe_lfu_trace.restype = st
            L.moe_lfu_trace.argtypes = [i32, i32, i32, i32, vp, vp, vp]
            L.moe_lfu_trace_pinned.restype = st
            L.moe_lfu_trace_pinned.argtypes = [i32, i32, i32, i32, vp, vp, i32, vp, vp, vp]
            L.moe_profile_start.restype = st
            L.moe_profile_start.argtypes = [vp, i32]
            L.moe_profile_stop.restype = st
            L.moe_profile_stop.argtypes = [vp, ctypes.POINTER(moe_kernel_time), i32, ctypes.POINTER(i32)]
            L.moe_layer_set_option.restype = st
            L.moe_layer_set_option.argtypes = [vp, i32, ctypes.c_int64]
            L.moe_layer_set_next.restype = st
            L.moe_layer_set_next.argtypes = [vp, vp]
            L.moe_layer_set_router_scoring.restype = st
            L.moe_layer_set_router_scoring.argtypes = [vp, i32, ctypes.c_float]
            L.moe_layer_check.restype = st
            L.moe_layer_check.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
            L.moe_layer_selection.restype = st
            L.moe_layer_selection.argtypes = [vp, i32, vp, vp, vp]
            L.moe_trace_read_split.restype = st
            L.moe_trace_read_split.argtypes = [vp, vp, i32]
            nd, kd = ctypes.POINTER(moe_block_norm_desc), ctypes.POINTER(moe_kv_desc)
            ap, at = ctypes.POINTER(moe_kv_append_args), ctypes.POINTER(moe_kv_attend_args)
            L.moe_block_norm.restype = st
            L.moe_block_norm.argtypes = [nd, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp]
            L.moe_block_norm_check.restype = st
            L.moe_block_norm_check.argtypes = [nd, vp, vp, vp, vp, vp, vp, vp, i32]
            L.moe_kv_create.restype = st
            L.moe_kv_create.argtypes = [kd, vp, vp, vp, vp, vp, i32, ctypes.POINTER(vp)]
            L.moe_kv_destroy.restype = None
            L.moe_kv_destroy.argtypes = [vp]
            L.moe_kv_device_bytes.restype = sz
            L.moe_kv_device_bytes.argtypes = [vp]
            L.moe_kv_append.restype = st
            L.moe_kv_append.argtypes = [vp, ap, vp]
            L.moe_kv_attend.restype = st
            L.moe_kv_attend.argtypes = [vp, at, vp]
            L.moe_kv_append_check.restype = st
            L.moe_kv_append_check.argtypes = [kd, ap]
            L.moe_kv_attend_check.restype = st
            L.moe_kv_attend_check.argtypes = [kd, at]
            L.moe_kv_locate.restype = st
            L.moe_kv_locate.argtypes = [kd, vp, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int64),
                                        ctypes.POINTER(ctypes.c_uint32)]
            L.moe_kv_health.restype = st
            L.moe_kv_health.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
            L.moe_kv_set_option.restype = st
            L.moe_kv_set_option.argtypes = [vp, i32, ctypes.c_int64]
            L.moe_status_str.restype = ctypes.c_char_p
            L.moe_status_str.argtypes = [st]
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_last_error.argtypes = []
            _lib = L
    return _lib


def _addr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        return a.data_ptr()
    if hasattr(a, "ctypes"):
        return a.ctypes.data
    raise TypeError(f"cannot take the address of {type(a)}")


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def _stream_on(s, current, device: int):
    """The handle of a stream, or of torch's current one on a device."""
    if s is None:
        s = current(device)
    try:
        return s.cuda_stream
    except AttributeError:
        return _stream(s)


def _check(status: int, call: str):
    if status != 0:
        raise MoEError(status, call, moe_last_error())


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


# ---------------------------------------------------------------------------
# marshalling of canonical weights
# ---------------------------------------------------------------------------

def _qmat(m) -> moe_qmat:
    for a in (m.codes, m.scale, m.bias):
        assert a.flags["C_CONTIGUOUS"]
    return moe_qmat(_addr(m.codes), _addr(m.scale), _addr(m.bias))


def _expert(e) -> moe_expert:
    return moe_expert(_qmat(e.gate), _qmat(e.up), _qmat(e.down))


def make_desc(hidden, inter, n_experts, top_k=8, n_shared=1, router_fmt="f32", act="bf16",
              max_tokens=1, cache_slots=0, expert_bits=4) -> moe_layer_desc:
    return moe_layer_desc(MOE_ABI_VERSION, hidden, inter, n_experts, top_k, n_shared,
                          MOE_W_F32 if router_fmt == "f32" else MOE_W_Q8G64,
                          MOE_W_Q2G64 if expert_bits == 2 else MOE_W_Q4G64, 64,
                          MOE_BF16 if act == "bf16" else MOE_F32, max_tokens, cache_slots)


def desc_from_spec(spec, max_tokens=1, cache_slots=0) -> moe_layer_desc:
    return make_desc(spec.hidden, spec.inter, spec.n_experts, spec.top_k, spec.n_shared,
                     spec.router_fmt, spec.act, max_tokens, cache_slots, getattr(spec, "expert_bits", 4))


def moe_expert_record_bytes(desc: moe_layer_desc) -> int:
    return int(lib().moe_expert_record_bytes(ctypes.byref(desc)))


def moe_pack_expert_record(desc: moe_layer_desc, expert, dst) -> None:
    ce = _expert(expert)
    _check(lib().moe_pack_expert_record(ctypes.byref(desc), ctypes.byref(ce), _addr(dst)),
           "moe_pack_expert_record")


def moe_layer_create(desc: moe_layer_desc, router, router_bias=None, shared=None, experts=None,
                     records=None, source=None, source_user=None, device: int = 0) -> int:
    """Create a layer from canonical host arrays; returns the opaque handle."""
    r = moe_router()
    if router.fmt == "f32":
        assert router.w.flags["C_CONTIGUOUS"]
        r.w = _addr(router.w)
    else:
        r.q = _qmat(router.q)
    sh = _expert(shared) if shared is not None else None
    ex_arr = None
    if experts is not None:
        ex_arr = (moe_expert * len(experts))(*[_expert(e) for e in experts])
    rec_arr = None
    if records is not None:
        rec_arr = (ctypes.c_void_p * len(records))(*[_addr(p) for p in records])
    src = source if source is not None else SOURCE_FN()
    out = ctypes.c_void_p()
    st = lib().moe_layer_create(ctypes.byref(desc), ctypes.byref(r), _addr(router_bias),
                                ctypes.byref(sh) if sh is not None else None, ex_arr,
                                ctypes.cast(rec_arr, ctypes.c_void_p) if rec_arr is not None else None,
                                src, _addr(source_user), device, ctypes.byref(out))
    _check(st, "moe_layer_create")
    return out.value


def moe_layer_destroy(handle) -> None:
    lib().moe_layer_destroy(handle)


def moe_layer_device_bytes(handle) -> int:
    return int(lib().moe_layer_device_bytes(handle))


def moe_route(handle, x, T, ids, w, stream=None) -> None:
    _check(lib().moe_route(handle, _addr(x), T, _addr(ids), _addr(w), _stream(stream)), "moe_route")


def moe_decode(handle, x, y, y_f32=None, stream=None) -> None:
    _check(lib().moe_decode(handle, _addr(x), _addr(y), _addr(y_f32), _stream(stream)), "moe_decode")


def moe_decode_static_scratch(handle, x, y, y_f32=None, stream=None) -> None:
    """moe_decode over the library's fixed per-device scratch region; the
    library allocates nothing (the caller passes buffers it already owns)."""
    _check(lib().moe_decode_static_scratch(handle, _addr(x), _addr(y), _addr(y_f32), _stream(stream)),
           "moe_decode_static_scratch")


def moe_prefill_chunk(handle, x, T, y, y_f32=None, stream=None) -> None:
    _check(lib().moe_prefill_chunk(handle, _addr(x), T, _addr(y), _addr(y_f32), _stream(stream)),
           "moe_prefill_chunk")


def moe_decode_tokens_host(handle, x_host, T, y_host, stream=None) -> None:
    _check(lib().moe_decode_tokens_host(handle, _addr(x_host), T, _addr(y_host), _stream(stream)),
           "moe_decode_tokens_host")


def moe_cache_prefetch(handle, x, stream=None) -> tuple[int, int]:
    """Router lookahead on a streamed layer; returns (predicted already resident, fills issued)."""
    r, f = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_cache_prefetch(handle, _addr(x), _stream(stream), ctypes.byref(r), ctypes.byref(f)),
           "moe_cache_prefetch")
    return r.value, f.value


def moe_cache_prefetch_stats(handle) -> dict:
    out = (ctypes.c_uint64 * 4)()
    _check(lib().moe_cache_prefetch_stats(handle, out), "moe_cache_prefetch_stats")
    return {"calls": out[0], "resident": out[1], "fills": out[2], "bytes_h2d": out[3]}


def moe_cache_stage(handle, ids, n, stream=None) -> tuple[int, int]:
    h, m = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_cache_stage(handle, _addr(ids), n, _stream(stream), ctypes.byref(h), ctypes.byref(m)),
           "moe_cache_stage")
    return h.value, m.value


def moe_cache_stats(handle) -> dict:
    s = moe_cache_stats_t()
    _check(lib().moe_cache_stats(handle, ctypes.byref(s)), "moe_cache_stats")
    return {f: int(getattr(s, f)) for f, _ in moe_cache_stats_t._fields_}


def moe_lfu_trace(slots: int, n_experts: int, ids):
    """Host-only run of the cache policy: ids int32 [n_tokens][k] -> (slot, hit) arrays."""
    import numpy as _np
    ids = _np.ascontiguousarray(ids, dtype=_np.int32)
    n_tokens, k = ids.shape
    slot = _np.empty((n_tokens, k), _np.int32)
    hit = _np.empty((n_tokens, k), _np.uint8)
    _check(lib().moe_lfu_trace(slots, n_experts, k, n_tokens, ids.ctypes.data, slot.ctypes.data, hit.ctypes.data),
           "moe_lfu_trace")
    return slot, hit


def moe_lfu_trace_pinned(slots: int, n_experts: int, ids, pinned):
    """Host-only run of the cache policy with pinned experts: -> (slot, hit, usage)."""
    import numpy as _np
    ids = _np.ascontiguousarray(ids, dtype=_np.int32)
    pin = _np.ascontiguousarray(_np.asarray(pinned, dtype=_np.int32))
    n_tokens, k = ids.shape
    slot = _np.empty((n_tokens, k), _np.int32)
    hit = _np.empty((n_tokens, k), _np.uint8)
    usage = _np.zeros(n_experts, _np.uint64)
    _check(lib().moe_lfu_trace_pinned(slots, n_experts, k, n_tokens, ids.ctypes.data,
                                      pin.ctypes.data if len(pin) else None, len(pin), slot.ctypes.data,
                                      hit.ctypes.data, usage.ctypes.data), "moe_lfu_trace_pinned")
    return slot, hit, usage


def moe_cache_residency(handle, slots: int) -> list[int]:
    arr = (ctypes.c_int32 * slots)()
    _check(lib().moe_cache_residency(handle, ctypes.cast(arr, ctypes.c_void_p)), "moe_cache_residency")
    return list(arr)


def moe_cache_usage(handle, n_experts: int):
    """Per-expert selection counts of a streamed layer (numpy uint64 [n_experts])."""
    import numpy as np
    out = np.zeros(n_experts, np.uint64)
    _check(lib().moe_cache_usage(handle, ctypes.c_void_p(out.ctypes.data)), "moe_cache_usage")
    return out


def moe_cache_pin(handle, experts) -> None:
    """Pin these experts (the learning cache); an empty list unpins all."""
    import numpy as np
    ids = np.ascontiguousarray(np.asarray(experts, dtype=np.int32))
    _check(lib().moe_cache_pin(handle, ctypes.c_void_p(ids.ctypes.data) if len(ids) else None, len(ids)),
           "moe_cache_pin")


def moe_hottest(counts, n: int):
    """The n experts with the largest counts, the lower id first among equal
    counts (the library's ordering, host only)."""
    import numpy as np
    c = np.ascontiguousarray(np.asarray(counts, dtype=np.uint64))
    out = np.zeros(max(n, 0), np.int32)
    _check(lib().moe_hottest(ctypes.c_void_p(c.ctypes.data), len(c), n, ctypes.c_void_p(out.ctypes.data)),
           "moe_hottest")
    return out


def moe_cache_pin_hottest(handle, n: int) -> None:
    """Pin the n most used experts of a streamed layer so far."""
    _check(lib().moe_cache_pin_hottest(handle, n), "moe_cache_pin_hottest")


def moe_profile_start(handle, max_launches: int) -> None:
    _check(lib().moe_profile_start(handle, max_launches), "moe_profile_start")


def moe_profile_stop(handle) -> dict:
    """{kernel name: (launches, total_ms)} since moe_profile_start."""
    cap = 32
    arr = (moe_kernel_time * cap)()
    n = ctypes.c_int32()
    _check(lib().moe_profile_stop(handle, arr, cap, ctypes.byref(n)), "moe_profile_stop")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(min(n.value, cap))}


def moe_layer_set_option(handle, option: int, value: int) -> None:
    _check(lib().moe_layer_set_option(handle, option, value), "moe_layer_set_option")


def moe_layer_set_next(handle, next_handle) -> None:
    _check(lib().moe_layer_set_next(handle, next_handle), "moe_layer_set_next")


def moe_layer_set_router_scoring(handle, scoring: int, routed_scaling: float = 1.0) -> None:
    _check(lib().moe_layer_set_router_scoring(handle, scoring, routed_scaling), "moe_layer_set_router_scoring")


def moe_layer_check(handle) -> tuple[int, int]:
    """(status, error bits) of device-side bounded waits since the last check."""
    bits = ctypes.c_uint32()
    st = lib().moe_layer_check(handle, ctypes.byref(bits))
    return st, bits.value


def moe_layer_selection(handle, T, ids, w, stream=None):
    """Copy the selection the last route / decode / prefill call used into
    device buffers ids int32 [T][k] and w fp32 [T][k] (enqueued on stream)."""
    _check(lib().moe_layer_selection(handle, T, _addr(ids), _addr(w), _stream(stream)), "moe_layer_selection")


# ---------------------------------------------------------------------------
# the rest of a decoder layer: block norms, paged key-value cache
# ---------------------------------------------------------------------------

def moe_block_norm(desc, x, o, gate, w_post, w_pre, r, h, T, device=0, stream=None) -> None:
    _check(lib().moe_block_norm(ctypes.byref(desc), _addr(x), _addr(o), _addr(gate), _addr(w_post), _addr(w_pre),
                                _addr(r), _addr(h), T, device, _stream(stream)), "moe_block_norm")


def moe_block_norm_check(desc, x, o, gate, w_post, w_pre, r, h, T) -> None:
    """The argument checks of moe_block_norm alone (host only)."""
    _check(lib().moe_block_norm_check(ctypes.byref(desc), _addr(x), _addr(o), _addr(gate), _addr(w_post),
                                      _addr(w_pre), _addr(r), _addr(h), T), "moe_block_norm_check")


def moe_kv_create(desc, k_pages, v_pages, inv_freq=None, k_scale=None, v_scale=None, device: int = 0) -> int:
    """Create a cache handle over two borrowed page pools; inv_freq float64 and
    the scales float32 are host arrays, copied."""
    out = ctypes.c_void_p()
    _check(lib().moe_kv_create(ctypes.byref(desc), _addr(k_pages), _addr(v_pages), _addr(inv_freq), _addr(k_scale),
                               _addr(v_scale), device, ctypes.byref(out)), "moe_kv_create")
    return out.value


def moe_kv_destroy(handle) -> None:
    lib().moe_kv_destroy(handle)


def moe_kv_device_bytes(handle) -> int:
    return int(lib().moe_kv_device_bytes(handle))


def moe_kv_append(handle, args: moe_kv_append_args, stream=None) -> None:
    _check(lib().moe_kv_append(handle, ctypes.byref(args), _stream(stream)), "moe_kv_append")


def moe_kv_attend(handle, args: moe_kv_attend_args, stream=None) -> None:
    _check(lib().moe_kv_attend(handle, ctypes.byref(args), _stream(stream)), "moe_kv_attend")


def moe_kv_append_check(desc, args) -> None:
    """The argument checks of moe_kv_append alone (host only)."""
    _check(lib().moe_kv_append_check(ctypes.byref(desc), ctypes.byref(args)), "moe_kv_append_check")


def moe_kv_attend_check(desc, args) -> None:
    """The argument checks of moe_kv_attend alone (host only)."""
    _check(lib().moe_kv_attend_check(ctypes.byref(desc), ctypes.byref(args)), "moe_kv_attend_check")


def moe_kv_locate(desc, block_table, seq: int, position: int, head: int = 0) -> int:
    """Element offset of a cached row in a pool; block_table: host int32 [n_seqs][max_pages]."""
    import numpy as np
    t = np.ascontiguousarray(block_table, dtype=np.int32)
    off, bits = ctypes.c_int64(), ctypes.c_uint32()
    _check(lib().moe_kv_locate(ctypes.byref(desc), t.ctypes.data, t.shape[0], t.shape[1], seq, position, head,
                               ctypes.byref(off), ctypes.byref(bits)), "moe_kv_locate")
    return off.value


def moe_kv_health(handle) -> tuple[int, int]:
    """(status, health bits) of what the handle's kernels refused since the last call."""
    bits = ctypes.c_uint32()
    st = lib().moe_kv_health(handle, ctypes.byref(bits))
    return st, bits.value


def moe_kv_set_option(handle, option: int, value: int) -> None:
    _check(lib().moe_kv_set_option(handle, option, value), "moe_kv_set_option")


MOE_TRACE_MAX_CTAS = 1024
MOE_TRACE_KERNELS = 5
SPLIT_TRACE_KERNELS = ("router", "gateup", "down", "prefill_gemm_gateup", "prefill_gemm_down")
SPLIT_TRACE_POINTS = ("start", "dependency", "main_done", "end")
PREFILL_WAIT_ROLES = ("copy", "dequant", "mma", "total")


def moe_trace_read_split(handle):
    """[kernel][cta][4]: decode stamps (ns) for kernels 0..2; for the prefill
    GEMMs (kernels 3..4) the cycles the copy, dequantiser and MMA roles waited
    and the CTA's total cycles."""
    cap = MOE_TRACE_KERNELS * MOE_TRACE_MAX_CTAS * 4
    buf = (ctypes.c_uint64 * cap)()
    _check(lib().moe_trace_read_split(handle, ctypes.cast(buf, ctypes.c_void_p), cap), "moe_trace_read_split")
    v = list(buf)
    return [[v[(kk * MOE_TRACE_MAX_CTAS + c) * 4:(kk * MOE_TRACE_MAX_CTAS + c) * 4 + 4]
             for c in range(MOE_TRACE_MAX_CTAS)] for kk in range(MOE_TRACE_KERNELS)]


class MoELayer:
    """Owns one layer handle; ``layer`` is any object with ``spec``, ``router``,
    ``router_bias``, ``shared`` and ``experts`` attributes in canonical form."""

    def __init__(self, layer, device: int = 0, max_tokens: int = 1, cache_slots: int = 0,
                 records=None, source=None):
        self.spec = layer.spec
        self.desc = desc_from_spec(layer.spec, max_tokens=max_tokens, cache_slots=cache_slots)
        self._records = records
        self._source = source
        self.handle = moe_layer_create(self.desc, layer.router, layer.router_bias, layer.shared,
                                       None if cache_slots else layer.experts, records=records,
                                       source=source, device=device)
        if getattr(layer.spec, "router_score", "softmax") == "sigmoid":
            moe_layer_set_router_scoring(self.handle, MOE_SCORE_SIGMOID, layer.spec.routed_scaling)

    def close(self):
        if getattr(self, "handle", None):
            moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def route(self, x, T, ids, w, stream=None):
        moe_route(self.handle, x, T, ids, w, stream)

    def decode(self, x, y, y_f32=None, stream=None):
        moe_decode(self.handle, x, y, y_f32, stream)

    def selection(self, T, ids, w, stream=None):
        moe_layer_selection(self.handle, T, ids, w, stream)

    def decode_static_scratch(self, x, y, y_f32=None, stream=None):
        moe_decode_static_scratch(self.handle, x, y, y_f32, stream)

    def prefill_chunk(self, x, T, y, y_f32=None, stream=None):
        moe_prefill_chunk(self.handle, x, T, y, y_f32, stream)

    def decode_tokens_host(self, x_host, T, y_host, stream=None):
        moe_decode_tokens_host(self.handle, x_host, T, y_host, stream)

    def cache_stage(self, ids, n, stream=None):
        return moe_cache_stage(self.handle, ids, n, stream)

    def cache_prefetch(self, x, stream=None):
        return moe_cache_prefetch(self.handle, x, stream)

    def prefetch_stats(self):
        return moe_cache_prefetch_stats(self.handle)

    def cache_stats(self):
        return moe_cache_stats(self.handle)

    def residency(self):
        return moe_cache_residency(self.handle, self.desc.cache_slots)

    def cache_usage(self):
        return moe_cache_usage(self.handle, self.desc.n_experts)

    def cache_pin(self, experts):
        moe_cache_pin(self.handle, experts)

    def pin_hottest(self, n):
        """Pin the n most used experts so far (ties: the lower id first)."""
        moe_cache_pin_hottest(self.handle, n)

    def set_option(self, option, value):
        moe_layer_set_option(self.handle, option, value)

    def set_next(self, other):
        moe_layer_set_next(self.handle, other.handle if other is not None else None)

    def set_router_scoring(self, scoring, routed_scaling=1.0):
        moe_layer_set_router_scoring(self.handle, scoring, routed_scaling)

    def check(self):
        return moe_layer_check(self.handle)

    @property
    def device_bytes(self):
        return moe_layer_device_bytes(self.handle)


def _refuse(t, name: str, shape, dtype, device: int):
    raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{device}, last dimensions contiguous; got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {tuple(t.stride())}")


def _dense(t, name: str, shape, dtype, device: int) -> int:
    """Address of a contiguous tensor of this shape, type and CUDA device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(t, name, shape, dtype, device)
    return t.data_ptr()


def _rows(t, name: str, shape, dtype, device: int) -> int:
    """Elements between the rows (first dimension) of a tensor of this shape,
    type and CUDA device whose other dimensions are contiguous."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    if len(shape) == 3:
        return _token_stride(t, name, *shape)
    if st[1] != 1:
        _refuse(t, name, shape, dtype, device)
    return st[0] if shape[0] > 1 else shape[1]   # a single row has no stride of its own


def _token_stride(t, name: str, rows: int, heads: int, width: int) -> int:
    """Elements between the tokens of t [rows, heads, width]; heads must be contiguous."""
    token, head, one = t.stride()
    if one != 1 or (head != width and heads != 1):
        _refuse(t, name, (rows, heads, width), t.dtype, t.get_device())
    return token if rows > 1 else heads * width


class BlockNorm:
    """The norms between two blocks of a decoder layer (moe_block_norm): keeps
    the weights, fp32 [hidden] on the device; w_post and w_pre may be None. One
    object serves one host thread at a time."""

    # moe_block_norm_desc, packed in place: the fields a call sets cost it one pack
    _desc = struct.Struct("Iiiiifffqqqqq")

    def __init__(self, hidden: int, w_post=None, w_pre=None, eps: float = 1e-6, scale: float = 1.0,
                 weight_offset: float = 0.0):
        import torch
        self.hidden, self.eps, self.scale, self.weight_offset = hidden, eps, scale, weight_offset
        self.w_post, self.w_pre, self._f32 = w_post, w_pre, torch.float32
        self._bind(next((w.get_device() for w in (w_post, w_pre) if w is not None), None))
        self._ids = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
        self._buf = ctypes.create_string_buffer(ctypes.sizeof(moe_block_norm_desc))
        self._buf_addr = ctypes.addressof(self._buf)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        self._call = ctypes.CFUNCTYPE(ctypes.c_int, *[vp] * 8, i32, i32, vp)(("moe_block_norm", lib()))
        self._current_stream = torch.cuda.current_stream

    def _bind(self, device):
        """Take the weights' addresses. They hold while the aliases keep that memory from other
        use, so that a call only looks whether an address is still the weight's (moving a module
        gives its weights new memory)."""
        at = []
        for name, w in (("w_post", self.w_post), ("w_pre", self.w_pre)):
            at.append((w, None if w is None else w.detach(),
                       None if w is None else _dense(w, name, (self.hidden,), self._f32, device)))
        (self._post_of, self._post_alias, self._post), (self._pre_of, self._pre_alias, self._pre) = at
        self.device = device

    def run(self, x, o=None, r=None, h=None, gate=None, stream=None):
        """x [T, H] residual, o [T, H] the block's output or None, r [T, H]
        (may be x) and h [T, H] the outputs (either may be None), gate [T, H],
        [1, H] or [H] of o's type. stream: torch's current one on x's device by default."""
        ids, H, dev = self._ids, self.hidden, x.get_device()
        shape, res = x.shape, x.dtype
        if len(shape) != 2 or shape[1] != H or res not in ids or dev < 0:
            raise ValueError("x must be a float32 or bfloat16 CUDA tensor [T, hidden]")
        post, pre = self.w_post, self.w_pre
        if (post is not self._post_of or pre is not self._pre_of or (post is not None and post.data_ptr() != self._post)
                or (pre is not None and pre.data_ptr() != self._pre) or self.device != dev):
            self._bind(dev)
        blk = res if o is None else o.dtype
        out = res if h is None else h.dtype
        if blk not in ids or out not in ids:
            raise TypeError("o and h must be float32 or bfloat16")
        # rows without gaps, as almost every call has them, or the stride of each
        xs = H if x.is_contiguous() else _rows(x, "x", shape, res, dev)
        os_ = gs = rs = hs = 0
        op = gp = rp = hp = wp = wn = None
        if o is not None:
            plain = o.shape == shape and o.get_device() == dev and o.is_contiguous()
            os_, op, wp = H if plain else _rows(o, "o", shape, blk, dev), o.data_ptr(), self._post
        if r is not None:
            plain = r.shape == shape and r.dtype is res and r.get_device() == dev and r.is_contiguous()
            rs, rp = H if plain else _rows(r, "r", shape, res, dev), r.data_ptr()
        if h is not None:
            plain = h.shape == shape and h.get_device() == dev and h.is_contiguous()
            hs, hp, wn = H if plain else _rows(h, "h", shape, out, dev), h.data_ptr(), self._pre
        if gate is not None:
            if o is None:
                raise ValueError("gate needs o")
            if gate.dim() < 2:
                _dense(gate, "gate", (H,), blk, dev)
            elif gate.shape[0] == 1:
                _dense(gate, "gate", (1, H), blk, dev)
            else:
                gs = _rows(gate, "gate", shape, blk, dev)
            gp = gate.data_ptr()
        try:
            self._desc.pack_into(self._buf, 0, MOE_ABI_VERSION, H, ids[res], ids[blk], ids[out], self.eps, self.scale,
                                 self.weight_offset, xs, os_, gs, rs, hs)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"eps, scale or weight_offset is not a number of fp32's range: {e}") from None
        st = self._call(self._buf_addr, x.data_ptr(), op, gp, wp, wn, rp, hp, shape[0], dev,
                        _stream_on(stream, self._current_stream, dev))
        if st:
            _check(st, "moe_block_norm")


class KVCache:
    """Owns one cache handle over two page pools, tensors [n_pages, n_kv_heads,
    page_size, head_dim] of bfloat16 or float8_e4m3fn in any memory order whose
    last dimension is contiguous (token-major pages: a permuted view). The handle is
    bound to the pools' memory: pools that get new memory need a new object."""

    # moe_kv_append_args and moe_kv_attend_args, packed in place
    _append_args = struct.Struct("PPPqqqPPPiiiP")
    _attend_args = struct.Struct("PqPPiiffiPP")

    def __init__(self, k_pages, v_pages, n_heads: int, inv_freq=None, interleaved: bool = False, k_scale=None,
                 v_scale=None, max_batch: int = 1):
        import numpy as np
        import torch
        kinds = {torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_E4M3}
        n_pages, hk, page, d = k_pages.shape
        if k_pages.dtype not in kinds:
            raise TypeError("the pools must be bfloat16 or float8_e4m3fn")
        if not k_pages.is_cuda or v_pages.device != k_pages.device:
            raise ValueError("k_pages and v_pages must be CUDA tensors on one device")
        if v_pages.shape != k_pages.shape or v_pages.stride() != k_pages.stride() or v_pages.dtype != k_pages.dtype:
            raise ValueError("k_pages and v_pages must have one shape, type and memory order")
        if k_pages.stride(3) != 1:
            raise ValueError("the last dimension of the pools must be contiguous")
        freq = None if inv_freq is None else np.ascontiguousarray(inv_freq, dtype=np.float64)
        scales = [None if s is None else np.ascontiguousarray(s, dtype=np.float32) for s in (k_scale, v_scale)]
        for s in scales:
            if s is not None and s.shape != (hk,):
                raise ValueError("k_scale and v_scale hold one value per key-value head")
        self.k_pages, self.v_pages = k_pages, v_pages
        self._k_at, self._v_at = k_pages.data_ptr(), v_pages.data_ptr()
        self.device = k_pages.get_device()
        self.desc = moe_kv_desc(MOE_ABI_VERSION, n_heads, hk, d, page, n_pages, kinds[k_pages.dtype],
                                0 if freq is None else 2 * freq.size, int(interleaved), max_batch,
                                k_pages.stride(0), k_pages.stride(1), k_pages.stride(2))
        self.handle = moe_kv_create(self.desc, k_pages, v_pages, freq if freq is None or freq.size else None,
                                    scales[0], scales[1], self.device)
        self._bf16, self._f32, self._i32 = torch.bfloat16, torch.float32, torch.int32
        self._heads = (n_heads, hk, d)
        self._buf = ctypes.create_string_buffer(max(self._append_args.size, self._attend_args.size))
        self._buf_addr = ctypes.addressof(self._buf)
        proto = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)
        self._append_call = proto(("moe_kv_append", lib()))
        self._attend_call = proto(("moe_kv_attend", lib()))
        self._current_stream = torch.cuda.current_stream

    def close(self):
        if getattr(self, "handle", None):
            moe_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def _pools_moved(self):
        raise ValueError("k_pages or v_pages has new memory: the handle is bound to that of its construction")

    def append(self, q, k, v, positions, block_table, q_out=None, seq=None, stream=None):
        """Rotate and cache T tokens: q [T, n_heads, d] (or None with q_out), k
        and v [T, n_kv_heads, d], positions and seq int32 [T], block_table int32
        [n_seqs, max_pages]. stream: torch's current one on the pools' device by default."""
        hq, hk, d = self._heads
        dev, bf16, i32 = self.device, self._bf16, self._i32
        if self.k_pages.data_ptr() != self._k_at or self.v_pages.data_ptr() != self._v_at:
            self._pools_moved()
        shape, table = k.shape, block_table.shape
        T = shape[0]
        # one condition for what almost every call passes; the refusals are worked out after it
        if not (shape == (T, hk, d) and v.shape == shape and positions.shape == (T,) and len(table) == 2
                and k.dtype is bf16 and v.dtype is bf16 and positions.dtype is i32 and block_table.dtype is i32
                and k.get_device() == dev and v.get_device() == dev and positions.get_device() == dev
                and block_table.get_device() == dev and positions.is_contiguous() and block_table.is_contiguous()):
            _rows(k, "k", (T, hk, d), bf16, dev)
            _rows(v, "v", (T, hk, d), bf16, dev)
            _dense(positions, "positions", (T,), i32, dev)
            if len(table) != 2:
                raise ValueError("block_table must be [n_seqs, max_pages]")
            _dense(block_table, "block_table", table, i32, dev)
        ks, vs = _token_stride(k, "k", T, hk, d), _token_stride(v, "v", T, hk, d)
        qs = qp = op = sp = 0
        if q is not None:
            if not (q.shape == (T, hq, d) and q.dtype is bf16 and q.get_device() == dev):
                _rows(q, "q", (T, hq, d), bf16, dev)
            qs, qp = _token_stride(q, "q", T, hq, d), q.data_ptr()
        if q_out is not None:
            op = _dense(q_out, "q_out", (T, hq, d), bf16, dev)
        if seq is not None:
            sp = _dense(seq, "seq", (T,), i32, dev)
        self._append_args.pack_into(self._buf, 0, qp, k.data_ptr(), v.data_ptr(), qs, ks, vs, positions.data_ptr(), sp,
                                    block_table.data_ptr(), T, table[0], table[1], op)
        st = self._append_call(self.handle, self._buf_addr, _stream_on(stream, self._current_stream, dev))
        if st:
            _check(st, "moe_kv_append")

    def attend(self, q, block_table, lens, out, lse=None, scale=None, softcap: float = 0.0, window: int = 0,
               stream=None):
        """Attention of one new token per sequence: q and out [B, n_heads, d]
        bf16, lens int32 [B], block_table int32 [B, max_pages], lse fp32
        [B, n_heads] or None; scale defaults to 1 / sqrt(d). stream: torch's current one on the
        pools' device by default."""
        hq, _, d = self._heads
        dev, bf16, i32 = self.device, self._bf16, self._i32
        if self.k_pages.data_ptr() != self._k_at or self.v_pages.data_ptr() != self._v_at:
            self._pools_moved()
        shape, table = q.shape, block_table.shape
        B = shape[0]
        if not (shape == (B, hq, d) and out.shape == shape and lens.shape == (B,) and len(table) == 2 and table[0] == B
                and q.dtype is bf16 and out.dtype is bf16 and lens.dtype is i32 and block_table.dtype is i32
                and q.get_device() == dev and out.get_device() == dev and lens.get_device() == dev
                and block_table.get_device() == dev and out.is_contiguous() and lens.is_contiguous()
                and block_table.is_contiguous()):
            _rows(q, "q", (B, hq, d), bf16, dev)
            _dense(out, "out", (B, hq, d), bf16, dev)
            _dense(lens, "lens", (B,), i32, dev)
            if len(table) != 2:
                raise ValueError("block_table must be [B, max_pages]")
            _dense(block_table, "block_table", (B, table[1]), i32, dev)
        try:
            self._attend_args.pack_into(
                self._buf, 0, q.data_ptr(), _token_stride(q, "q", B, hq, d), block_table.data_ptr(), lens.data_ptr(), B,
                table[1], d ** -0.5 if scale is None else scale, softcap, window, out.data_ptr(),
                0 if lse is None else _dense(lse, "lse", (B, hq), self._f32, dev))
        except (struct.error, OverflowError) as e:
            raise ValueError(f"scale, softcap or window is not a number of its type's range: {e}") from None
        st = self._attend_call(self.handle, self._buf_addr, _stream_on(stream, self._current_stream, dev))
        if st:
            _check(st, "moe_kv_attend")

    def locate(self, block_table, seq: int, position: int, head: int = 0) -> int:
        """Element offset of a cached row in a pool (block_table on the host)."""
        return moe_kv_locate(self.desc, block_table, seq, position, head)

    def health(self):
        return moe_kv_health(self.handle)

    def set_option(self, option: int, value: int):
        moe_kv_set_option(self.handle, option, value)

    @property
    def device_bytes(self):
        return moe_kv_device_bytes(self.handle)
