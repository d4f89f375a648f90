"""ctypes binding of the C ABI in ``include/fa.h``, ``include/fa_paged.h`` and
``include/fa_packed.h`` (argument marshalling only).

The functions here carry the C names and take raw device pointers (ints),
sizes and a CUDA stream handle; every step of the computation runs in the
CUDA library.  If ``libfa_gb300.so`` has not been built this module raises on
first use: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa_gb300.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_WORKSPACE = 4
FA_ERR_LAUNCH = 5
FA_ERR_DEVICE_TIMEOUT = 6

FA_FWD_MAX_SPLITS = 64

FA_BWD_AUTO = 0
FA_BWD_5GEMM = 5
FA_BWD_7GEMM = 7

# Every symbol the header declares, with its ctypes signature.
_VP = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_LL = ctypes.c_longlong
_ARGS = ctypes.c_char_p  # the bytes of a structure of arguments
SIGNATURES = {
    "fa_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _I, _VP]),
    "fa_fwd_splitkv_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_fwd_splitkv": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _I, _I, _VP, _SZ, _VP]),
    "fa_fwd_choose_splits": (_I, [_I, _I, _I, _I, _I]),
    "fa_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_bwd": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                    _I, _I, _I, _I, _F, _I, _I, _VP, _SZ, _VP]),
    "fa_bwd_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                            _I, _I, _I, _I, _F, _I, _I, _VP]),
    "fa_bwd_noalloc_device_error": (_I, [_VP, ctypes.POINTER(_I)]),
    "fa_bwd_noalloc_watchdog_selftest": (_I, [_VP]),
    "fa_bwd_query_parts": (_I, [_I, _I, _I, _I, _I, _I]),
    "fa_bwd_force_query_parts": (_I, [_I]),
    "fa_bwd_key_parts": (_I, [_I, _I, _I, _I, _I, _I]),
    "fa_bwd_force_key_parts": (_I, [_I]),
    "fa_bwd_choose": (_I, [_I, _I, _I, _I, _I]),
    "fa_get_device_error": (_I, [_VP, ctypes.POINTER(_I)]),
    "fa_watchdog_selftest": (_I, [_VP]),
    "fa_last_cuda_error": (_I, []),
    "fa_strerror": (ctypes.c_char_p, [_I]),
    "fa_profile_start": (_I, []),
    "fa_profile_stop": (_I, [_VP]),
    "fa_profile_stop_kinds": (_I, [_I, _VP, _VP]),
    "fa_kernel_name": (ctypes.c_char_p, [_I]),
    "fa_ex2_probe": (_I, [_VP, _I, _I, ctypes.POINTER(ctypes.c_longlong), _VP]),
    "fa_fwd_launches": (_I, [_I, _I, _I, _I]),
    "fa_fwd_splitkv_launches": (_I, [_I, _I, _I, _I, _I]),
    "fa_bwd_launches": (_I, [_I, _I, _I, _I, _I, _I]),
    # include/fa_paged.h
    "fa_page_grow": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP, _I, _VP, _I, _VP, _VP, _VP, _VP, _VP]),
    "fa_page_slots": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP]),
    "fa_kv4_store": (_I, [_VP, _VP, _VP, _LL, _LL, _LL, _LL, _VP, _I, _VP]),
    "fa_kv4_load": (_I, [_VP, _VP, _I, _VP, _VP, _VP]),
    "fa_kv4_attn": (_I, [_VP, _VP, _LL, _LL, _I, _VP, _I, _VP, _I, _VP, _I, _I, _F, _VP, _LL, _LL, _VP, _VP, _SZ, _VP]),
    "fa_kv4_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    # include/fa_packed.h
    "fa_packed_fwd": (_I, [_ARGS]),
    "fa_packed_fwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_packed_bwd": (_I, [_ARGS]),
    "fa_packed_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "fa_qk_norm_rope": (_I, [_ARGS]),
    "fa_qk_norm_rope_bwd": (_I, [_ARGS]),
    "fa_qk_norm_rope_bwd_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "fa_kv4_append": (_I, [_ARGS]),
}

_lib = None
_lock = threading.Lock()


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_strerror(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Loads the shared library once; raises if it is missing."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with tiled_attention_tmem_gb300.build "
                        "(or __graft_entry__.build()); there is no CPU fallback")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def fa_strerror(status: int) -> str:
    return lib().fa_strerror(status).decode()


def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream) -> int:
    return lib().fa_fwd(q, k, v, o, lse, B, H, N, d, float(scale), int(causal), stream)


def fa_fwd_splitkv_workspace_size(B, H, N, d, splits) -> int:
    return lib().fa_fwd_splitkv_workspace_size(B, H, N, d, splits)


def fa_fwd_splitkv(q, k, v, o, lse, B, H, N, d, scale, causal, splits, workspace, workspace_bytes,
                   stream) -> int:
    return lib().fa_fwd_splitkv(q, k, v, o, lse, B, H, N, d, float(scale), int(causal), int(splits),
                                workspace, workspace_bytes, stream)


def fa_fwd_choose_splits(B, H, N, d, causal) -> int:
    return lib().fa_fwd_choose_splits(B, H, N, d, int(causal))


def fa_bwd_workspace_size(B, H, N, d, variant) -> int:
    return lib().fa_bwd_workspace_size(B, H, N, d, variant)


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, variant,
           workspace, workspace_bytes, stream) -> int:
    return lib().fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, float(scale), int(causal),
                        variant, workspace, workspace_bytes, stream)


def fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, variant, stream) -> int:
    """The backward without a workspace: scratch lives in the library's static device array."""
    return lib().fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, float(scale), int(causal),
                                variant, stream)


FA_NOALLOC_SCRATCH_BYTES = 64 << 20


def fa_bwd_noalloc_device_error(stream) -> tuple[int, int]:
    """(status, site) of the no-alloc backward's own error word; reading clears it."""
    site = _I(0)
    status = lib().fa_bwd_noalloc_device_error(stream, ctypes.byref(site))
    return status, site.value


def fa_bwd_noalloc_watchdog_selftest(stream) -> int:
    return lib().fa_bwd_noalloc_watchdog_selftest(stream)


def fa_bwd_query_parts(B, H, N, d, causal, variant) -> int:
    return lib().fa_bwd_query_parts(B, H, N, d, int(causal), variant)


def fa_bwd_force_query_parts(parts) -> int:
    return lib().fa_bwd_force_query_parts(int(parts))


def fa_bwd_key_parts(B, H, N, d, causal, variant) -> int:
    return lib().fa_bwd_key_parts(B, H, N, d, int(causal), variant)


def fa_bwd_force_key_parts(parts) -> int:
    return lib().fa_bwd_force_key_parts(int(parts))


def fa_bwd_choose(B, H, N, d, causal) -> int:
    return lib().fa_bwd_choose(B, H, N, d, int(causal))


def fa_get_device_error(stream) -> tuple[int, int]:
    site = _I(0)
    status = lib().fa_get_device_error(stream, ctypes.byref(site))
    return status, site.value


def fa_watchdog_selftest(stream) -> int:
    return lib().fa_watchdog_selftest(stream)


def fa_last_cuda_error() -> int:
    return lib().fa_last_cuda_error()


def fa_ex2_probe(sink, blocks, iters, stream) -> tuple[int, int]:
    """Launches the exponential-unit probe; returns (status, ex2 evaluations launched)."""
    count = ctypes.c_longlong(0)
    status = lib().fa_ex2_probe(sink, blocks, iters, ctypes.byref(count), stream)
    return status, count.value


def fa_fwd_launches(B, H, N, d) -> int:
    return lib().fa_fwd_launches(B, H, N, d)


def fa_fwd_splitkv_launches(B, H, N, d, splits) -> int:
    return lib().fa_fwd_splitkv_launches(B, H, N, d, splits)


def fa_bwd_launches(B, H, N, d, variant, causal=0) -> int:
    return lib().fa_bwd_launches(B, H, N, d, variant, int(causal))


def fa_page_grow(lengths, new_tokens, table, B, width, page, free_pages, free_size, free_count, T, slots, cu,
                 lengths_out, count_out, stream) -> int:
    return lib().fa_page_grow(lengths, new_tokens, table, B, width, page, free_pages, free_size, free_count, T,
                              slots, cu, lengths_out, count_out, stream)


def fa_page_slots(first, count, table, B, width, page, T, slots, cu, stream) -> int:
    return lib().fa_page_slots(first, count, table, B, width, page, T, slots, cu, stream)


class FaKv4Cache(ctypes.Structure):
    """fa_kv4_cache; ``address`` is what the calls take (the structure must outlive them)."""
    _fields_ = [("k_codes", _VP), ("k_scales", _VP), ("v_codes", _VP), ("v_scales", _VP), ("pages", _I), ("page", _I),
                ("Hkv", _I), ("d", _I), ("k_gain", _F), ("v_gain", _F)]

    @property
    def address(self) -> int:
        return ctypes.addressof(self)


def fa_kv4_store(cache, k, v, k_token, k_head, v_token, v_head, slots, T, stream) -> int:
    return lib().fa_kv4_store(cache, k, v, k_token, k_head, v_token, v_head, slots, T, stream)


def fa_kv4_load(cache, slots, T, k, v, stream) -> int:
    return lib().fa_kv4_load(cache, slots, T, k, v, stream)


def fa_kv4_attn(cache, q, q_token, q_head, T, cu, max_q, table, width, lengths, B, H, scale, o, o_token, o_head, lse,
                workspace, workspace_bytes, stream) -> int:
    return lib().fa_kv4_attn(cache, q, q_token, q_head, T, cu, max_q, table, width, lengths, B, H, scale, o, o_token,
                             o_head, lse, workspace, workspace_bytes, stream)


def fa_kv4_attn_workspace_size(B, H, Hkv, d, max_q, page, width) -> int:
    return lib().fa_kv4_attn_workspace_size(B, H, Hkv, d, max_q, page, width)


# The structures of include/fa_packed.h, field by field (fa_rows: address, token and head strides; a
# NULL pointer is 0).  Packing one and passing its bytes takes a fraction of what ctypes does
# to convert as many arguments: 0.4 us instead of 2.8 for 27.
_ROWS = "Pqq"
_PACKED_FWD = struct.Struct(_ROWS * 4 + "PP" + "iiiii" + "fi" + "PNP")
_PACKED_BWD = struct.Struct(_ROWS * 5 + "P" + _ROWS * 3 + "P" + "iiiii" + "fii" + "PNP")
_QK_NORM_ROPE = struct.Struct(_ROWS * 4 + "PPPP" + "iifi" + "iiii" + "P")
_QK_NORM_ROPE_BWD = struct.Struct(_ROWS * 6 + "PPPPPP" + "iifi" + "iiii" + "PNP")
_KV4_APPEND = struct.Struct("P" + _ROWS * 5 + "PPPPP" + "iifi" + "ii" + "P")


def fa_packed_fwd(*fields) -> int:
    return lib().fa_packed_fwd(_PACKED_FWD.pack(*fields))


def fa_packed_fwd_workspace_size(B, T, H, Hkv, d) -> int:
    return lib().fa_packed_fwd_workspace_size(B, T, H, Hkv, d)


def fa_packed_bwd(*fields) -> int:
    return lib().fa_packed_bwd(_PACKED_BWD.pack(*fields))


def fa_packed_bwd_workspace_size(B, T, H, Hkv, d, variant) -> int:
    return lib().fa_packed_bwd_workspace_size(B, T, H, Hkv, d, variant)


def fa_qk_norm_rope(*fields) -> int:
    return lib().fa_qk_norm_rope(_QK_NORM_ROPE.pack(*fields))


def fa_qk_norm_rope_bwd(*fields) -> int:
    return lib().fa_qk_norm_rope_bwd(_QK_NORM_ROPE_BWD.pack(*fields))


def fa_qk_norm_rope_bwd_workspace_size(T, H, Hkv, d) -> int:
    return lib().fa_qk_norm_rope_bwd_workspace_size(T, H, Hkv, d)


def fa_kv4_append(*fields) -> int:
    return lib().fa_kv4_append(_KV4_APPEND.pack(*fields))


FA_KERNEL_ALL_KINDS = 19


def fa_profile_start() -> int:
    return lib().fa_profile_start()


def fa_profile_stop() -> dict:
    """Returns {kernel name: (launches, total ms)} for the kernels launched since start."""
    launches, ms = (_I * FA_KERNEL_ALL_KINDS)(), (ctypes.c_double * FA_KERNEL_ALL_KINDS)()
    st = lib().fa_profile_stop_kinds(FA_KERNEL_ALL_KINDS, launches, ms)
    if st != FA_OK:
        raise FaError(st, "fa_profile_stop")
    return {lib().fa_kernel_name(k).decode(): (launches[k], ms[k]) for k in range(FA_KERNEL_ALL_KINDS)}
