"""ctypes binding of the C ABI in include/gdn.h, include/gdn_conv.h,
include/gdn_pool.h and include/gdn_attn.h (same entry-point names).

Tensors are torch tensors on the current HIP device; torch only provides the
device memory and the stream. Shapes are read from the tensors, checked for
consistency (the C ABI sees bare pointers and cannot), and passed as sizes.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libgdn.so"

GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_ALIAS = 0, 1, 2, 3, 4
GDN_ERR_CAPACITY, GDN_ERR_WORKSPACE, GDN_ERR_PLAN, GDN_ERR_RULE, GDN_ERR_HIP = 5, 6, 7, 8, 9
GDN_ERR_SCRATCH = 10
NO_ALLOC_SCRATCH_BYTES = 128 << 20   # GDN_NO_ALLOC_SCRATCH_BYTES
GDN_F32, GDN_F16, GDN_BF16 = 0, 1, 2
PLAN_AUTO, PLAN_RECURRENT, PLAN_CHUNK = 0, 1, 2
RULE_GATED_DELTA, RULE_DELTA, RULE_GATED, RULE_LINEAR = 0, 1, 2, 3
GATE_RAW, GATE_NONE = 0, 1
STATE_V_MAJOR, STATE_K_MAJOR = 0, 1
ABI_VERSION = 7          # the struct layouts below match this version of include/gdn.h
CONV_SILU, CONV_NONE = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALING_NONE, ROPE_SCALING_LINEAR, ROPE_SCALING_NTK, ROPE_SCALING_YARN = 0, 1, 2, 3
CACHE_IO, CACHE_E4M3, CACHE_E2M1 = 0, 1, 4


class LibraryNotBuilt(RuntimeError):
    pass


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({gdn_strerror(status)})")


class GdnParams(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
        ("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
        ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("chunk", ctypes.c_int32),
        ("state_update_capacity", ctypes.c_int32), ("plan", ctypes.c_int32),
        ("update_rule", ctypes.c_int32), ("gate_activation", ctypes.c_int32),
        ("state_layout", ctypes.c_int32),
    ]


class GdnTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "k", "v", "a", "b", "A_log", "dt_bias", "cu_seqlens", "cu_seqlens_host",
        "initial_state", "final_state", "output", "state_update", "capture_count")]


class GdnConvParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "num_reqs", "channels", "kernel_size", "io_dtype", "activation",
        "state_update_capacity")]


class GdnConvTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "x", "weight", "bias", "cu_seqlens", "cu_seqlens_host", "initial_state", "final_state",
        "output", "state_update", "capture_count")]


class GdnConvFused(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("mixed", "weight", "bias", "initial_state", "final_state")] + \
               [("kernel_size", ctypes.c_int32), ("activation", ctypes.c_int32)]


class GdnSlots(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("read_slots", ctypes.c_void_p),
                ("write_slots", ctypes.c_void_p), ("read_slots_host", ctypes.c_void_p),
                ("write_slots_host", ctypes.c_void_p)]


class GdnKvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_scales", "v_scales", "page_table",
                                               "page_table_host")] + \
               [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "max_pages", "num_kv_heads", "head_dim",
                                              "io_dtype", "format")]


class GdnRopeParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_q_heads", "num_k_heads", "head_dim", "io_dtype",
                                              "rotary_dim", "layout")] + \
               [("factor", ctypes.c_float), ("q_stride", ctypes.c_int32), ("k_stride", ctypes.c_int32)]


class GdnRopeTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "positions", "inv_freq", "q_out", "k_out")]


class GdnKvParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_reqs", "num_q_heads", "rotary_dim",
                                              "rope_layout")] + \
               [("rope_factor", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("q_stride", "k_stride", "v_stride")]


class GdnKvTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "cu_seqlens", "cu_seqlens_host", "seq_lens",
                                               "seq_lens_host", "q", "q_out", "positions", "inv_freq")]


class GdnAttnParams(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_reqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("scale", ctypes.c_float), ("window", ctypes.c_int32), ("q_stride", ctypes.c_int32)]


class GdnAttnTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "cu_seqlens", "cu_seqlens_host", "seq_lens", "seq_lens_host",
                                               "output")]


class GdnSelectParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_reqs", "num_q_heads", "list_len", "first_pages",
                                              "newest_pages", "q_stride")]


class GdnSelectTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "cu_seqlens", "cu_seqlens_host", "seq_lens", "seq_lens_host",
                                               "bounds", "pages", "counts")]


class GdnSparseParams(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_reqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("list_len", ctypes.c_int32), ("scale", ctypes.c_float), ("q_stride", ctypes.c_int32)]


class GdnSparseTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "cu_seqlens", "cu_seqlens_host", "seq_lens", "seq_lens_host",
                                               "pages", "counts", "output")]


def _packer(cls):
    """cls's fields in order -> the bytes of such a struct. Called for every decode step, this
    takes 0.07 us where making the ctypes object takes 0.2."""
    kinds = {ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    s = struct.Struct("@" + "".join(kinds[t] for _, t in cls._fields_))
    if s.size != ctypes.sizeof(cls):
        raise TypeError(f"{cls.__name__} has padding at its end")
    return s.pack


_rope_params, _rope_tensors = _packer(GdnRopeParams), _packer(GdnRopeTensors)
_kv_params, _kv_tensors = _packer(GdnKvParams), _packer(GdnKvTensors)
_attn_params, _attn_tensors = _packer(GdnAttnParams), _packer(GdnAttnTensors)
_select_params, _select_tensors = _packer(GdnSelectParams), _packer(GdnSelectTensors)
_sparse_params, _sparse_tensors = _packer(GdnSparseParams), _packer(GdnSparseTensors)

_lib = None
_calls = None            # the attention layer's calls, taking packed structs


def library_path() -> str:
    """libgdn.so next to this file, or the file named by GDN_LIBRARY."""
    return os.environ.get("GDN_LIBRARY") or os.path.join(PKG, _LIB_NAME)


def _declare(L):
    """Argument and result types of L's functions; the attention layer's calls on packed structs."""
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    L.gdn_forward.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors), vp,
                              ctypes.c_size_t, vp]
    L.gdn_forward.restype = ctypes.c_int
    L.gdn_forward_no_alloc.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors), vp]
    L.gdn_forward_no_alloc.restype = ctypes.c_int
    L.gdn_forward_workspace_bytes.argtypes = [ctypes.POINTER(GdnParams), vp,
                                              ctypes.POINTER(ctypes.c_size_t)]
    L.gdn_forward_workspace_bytes.restype = ctypes.c_int
    L.gdn_resolve_plan.argtypes = [ctypes.POINTER(GdnParams), vp, ctypes.POINTER(i32)]
    L.gdn_resolve_plan.restype = ctypes.c_int
    L.gdn_replay.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.gdn_replay.restype = ctypes.c_int
    L.gdn_replay_forward.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors), vp, vp, vp,
                                     vp, vp]
    L.gdn_replay_forward.restype = ctypes.c_int
    L.gdn_conv_forward.argtypes = [ctypes.POINTER(GdnConvParams),
                                   ctypes.POINTER(GdnConvTensors), vp]
    L.gdn_conv_forward.restype = ctypes.c_int
    L.gdn_conv_replay.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.gdn_conv_replay.restype = ctypes.c_int
    sp = ctypes.POINTER(GdnSlots)
    L.gdn_forward_pooled.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors), sp, vp,
                                     ctypes.c_size_t, vp]
    L.gdn_forward_pooled.restype = ctypes.c_int
    L.gdn_replay_pooled.argtypes = [ctypes.POINTER(GdnParams), vp, vp, vp, vp, vp, sp, vp]
    L.gdn_replay_pooled.restype = ctypes.c_int
    L.gdn_replay_forward_pooled.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors), sp, vp,
                                            vp, vp, vp, vp]
    L.gdn_replay_forward_pooled.restype = ctypes.c_int
    L.gdn_conv_forward_pooled.argtypes = [ctypes.POINTER(GdnConvParams),
                                          ctypes.POINTER(GdnConvTensors), sp, vp]
    L.gdn_conv_forward_pooled.restype = ctypes.c_int
    L.gdn_conv_replay_pooled.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, sp, vp]
    L.gdn_conv_replay_pooled.restype = ctypes.c_int
    L.gdn_conv_decode_forward.argtypes = [ctypes.POINTER(GdnParams), ctypes.POINTER(GdnTensors),
                                          ctypes.POINTER(GdnConvFused), vp]
    L.gdn_conv_decode_forward.restype = ctypes.c_int
    L.gdn_publish_slots.argtypes = [i32, vp, vp, vp]
    L.gdn_publish_slots.restype = ctypes.c_int
    dbl, cp = ctypes.c_double, ctypes.POINTER(GdnKvCache)
    L.gdn_rope_frequencies.argtypes = [i32, dbl, i32, dbl, dbl, dbl, dbl, vp, ctypes.POINTER(ctypes.c_float)]
    L.gdn_rope_forward.argtypes = [ctypes.POINTER(GdnRopeParams), ctypes.POINTER(GdnRopeTensors), vp]
    for fn in (L.gdn_kv_write, L.gdn_kv_read):
        fn.argtypes = [ctypes.POINTER(GdnKvParams), ctypes.POINTER(GdnKvTensors), cp, vp]
    L.gdn_attn_forward.argtypes = [ctypes.POINTER(GdnAttnParams), ctypes.POINTER(GdnAttnTensors), cp, vp,
                                   ctypes.c_size_t, vp]
    L.gdn_attn_workspace_bytes.argtypes = [ctypes.POINTER(GdnAttnParams), cp, ctypes.POINTER(ctypes.c_size_t)]
    L.gdn_kv_bounds.argtypes = [ctypes.POINTER(GdnKvParams), ctypes.POINTER(GdnKvTensors), cp, vp, vp]
    L.gdn_attn_select.argtypes = [ctypes.POINTER(GdnSelectParams), ctypes.POINTER(GdnSelectTensors), cp, vp,
                                  ctypes.c_size_t, vp]
    L.gdn_attn_sparse_forward.argtypes = [ctypes.POINTER(GdnSparseParams), ctypes.POINTER(GdnSparseTensors), cp, vp,
                                          ctypes.c_size_t, vp]
    L.gdn_attn_select_workspace_bytes.argtypes = [ctypes.POINTER(GdnSelectParams), cp, ctypes.POINTER(ctypes.c_size_t)]
    L.gdn_attn_sparse_workspace_bytes.argtypes = [ctypes.POINTER(GdnSparseParams), cp, ctypes.POINTER(ctypes.c_size_t)]
    for fn in (L.gdn_rope_frequencies, L.gdn_rope_forward, L.gdn_kv_write, L.gdn_kv_read, L.gdn_attn_forward,
               L.gdn_attn_workspace_bytes, L.gdn_kv_bounds, L.gdn_attn_select, L.gdn_attn_sparse_forward,
               L.gdn_attn_select_workspace_bytes, L.gdn_attn_sparse_workspace_bytes):
        fn.restype = ctypes.c_int
    chars = ctypes.c_char_p
    calls = {n: L[n] for n in ("gdn_rope_forward", "gdn_kv_write", "gdn_kv_read", "gdn_attn_forward", "gdn_kv_bounds",
                               "gdn_attn_select", "gdn_attn_sparse_forward")}
    calls["gdn_rope_forward"].argtypes = [chars, chars, vp]
    calls["gdn_kv_write"].argtypes = calls["gdn_kv_read"].argtypes = [chars, chars, vp, vp]
    for n in ("gdn_attn_forward", "gdn_attn_select", "gdn_attn_sparse_forward"):
        calls[n].argtypes = [chars, chars, vp, vp, ctypes.c_size_t, vp]
    calls["gdn_kv_bounds"].argtypes = [chars, chars, vp, vp, vp]
    for fn in calls.values():
        fn.restype = ctypes.c_int
    L.gdn_strerror.argtypes = [ctypes.c_int]
    L.gdn_strerror.restype = ctypes.c_char_p
    return calls


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so; raises LibraryNotBuilt when it has not been built, or is not of this version."""
    global _lib, _calls
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise LibraryNotBuilt(f"{path} is missing: build it with "
                                  "`python -m gateddeltanet_recurrence_amd.build`")
        L = ctypes.CDLL(path)
        try:
            L.gdn_abi_version.argtypes = []
            L.gdn_abi_version.restype = ctypes.c_int
            if L.gdn_abi_version() != ABI_VERSION:
                raise LibraryNotBuilt(f"{path} has ABI version {L.gdn_abi_version()}, this binding "
                                      f"needs {ABI_VERSION}: rebuild it")
            calls = _declare(L)
        except AttributeError as e:                          # a function that a library of this version may lack
            raise LibraryNotBuilt(f"{path} is older than this binding ({e}): rebuild it") from e
        _lib, _calls = L, calls
    return _lib


def _call(name):
    if _calls is None:
        lib()
    return _calls[name]


def gdn_abi_version() -> int:
    return int(lib().gdn_abi_version())


def gdn_strerror(status: int) -> str:
    return lib().gdn_strerror(int(status)).decode()


def capsule_width(Hk: int, Hv: int, Dk: int, Dv: int) -> int:
    """Floats per capsule row: Hv decays, Hk*Dk unit keys, Hv*Dv deltas."""
    return Hv + Hk * Dk + Hv * Dv


def make_params(N, R, Hk, Hv, Dk, Dv, io_dtype, *, scale=0.0, chunk=0, capacity=0,
                plan=PLAN_AUTO, update_rule=RULE_GATED_DELTA, gate_activation=GATE_RAW,
                state_layout=STATE_V_MAJOR) -> GdnParams:
    return GdnParams(int(N), int(R), int(Hk), int(Hv), int(Dk), int(Dv), int(io_dtype),
                     float(scale), int(chunk), int(capacity), int(plan), int(update_rule),
                     int(gate_activation), int(state_layout))


# ------------------------------------------------------------------ helpers
_numpy_module = None
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _numpy():
    global _numpy_module
    if _numpy_module is None:
        import numpy
        _numpy_module = numpy
    return _numpy_module


def _io_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return GDN_F32
    if dtype == torch.float16:
        return GDN_F16
    if dtype == torch.bfloat16:
        return GDN_BF16                      # passed through so the library rejects it
    raise ValueError(f"unsupported io dtype {dtype}")


def _ptr(x) -> Optional[int]:
    return None if x is None else int(x.data_ptr())


def _need(x, name, shape, dtype=None):
    if x is None:
        return
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(x.shape)} != expected {tuple(shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name}: dtype {x.dtype} != expected {dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _stream_handle(stream, index: Optional[int] = None) -> Optional[int]:
    """The handle of `stream`; of None, the current stream's on GPU `index` (default: the current one)."""
    if stream is None:
        # the raw handle: making the Stream object of torch.cuda.current_stream() takes 2.7 us
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice() if index is None else index)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _host_i32(arr):
    """Keep-alive int32 host buffer and its address, from a sequence / numpy / CPU tensor."""
    if arr is None:
        return None, None
    np = _numpy()
    if type(arr) is np.ndarray and arr.dtype == np.int32 and arr.flags.c_contiguous:
        try:                                                 # through the buffer: 0.2 us instead of 0.6
            return arr, ctypes.addressof(ctypes.c_char.from_buffer(arr))
        except (TypeError, ValueError):                      # read-only, empty
            return arr, arr.ctypes.data
    if hasattr(arr, "numpy") and hasattr(arr, "is_cuda"):
        if arr.is_cuda:
            raise ValueError("host mirrors must be CPU data")
        arr = arr.numpy()
    a = np.ascontiguousarray(np.asarray(arr, dtype=np.int32))
    return a, a.ctypes.data


def _slots(R, num_slots, read_slots, write_slots, read_slots_host, write_slots_host):
    """GdnSlots for R requests plus the host arrays it points to (kept alive by the caller)."""
    torch = _torch()
    _need(read_slots, "read_slots", (R,), torch.int32)
    _need(write_slots, "write_slots", (R,), torch.int32)
    rh, rh_ptr = _host_i32(read_slots_host)
    wh, wh_ptr = _host_i32(write_slots_host)
    for h, name in ((rh, "read_slots_host"), (wh, "write_slots_host")):
        if h is not None and h.shape != (R,):
            raise ValueError(f"{name} must have R entries")
    sl = GdnSlots(int(num_slots), _ptr(read_slots), _ptr(write_slots), rh_ptr, wh_ptr)
    return sl, (rh, wh)


# ------------------------------------------------------------- entry points
def gdn_forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, **kw) -> int:
    """gdn_forward of include/gdn.h on torch tensors; returns the status code.
    Keywords as _forward."""
    return _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, **kw)


def gdn_forward_no_alloc(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, **kw) -> int:
    """gdn_forward_no_alloc of include/gdn.h: gdn_forward whose workspace is the
    library's static scratch array on the current GPU (no workspace argument).
    Keywords as _forward, without workspace."""
    if kw.get("workspace") is not None:
        raise ValueError("gdn_forward_no_alloc takes no workspace")
    return _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, no_alloc=True, **kw)


def gdn_replay_forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, *, prev_state_update,
                       accepted, replay_state, accepted_host=None, **kw) -> int:
    """gdn_replay_forward of include/gdn.h: replay of the previous step's accepted
    capsule prefix onto initial_state (the committed bank) into replay_state (the
    inactive bank) and the verify of this step's tokens from that state, in one
    pass. prev_state_update [R, capacity, W] float32, accepted [R] int32 (GPU
    tensors), accepted_host a host int32 mirror or None, replay_state
    [R, Hv, Dv, Dk] float32; the other keywords as _forward."""
    return _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output,
                    replay=dict(prev=prev_state_update, accepted=accepted, state=replay_state,
                                accepted_host=accepted_host), **kw)


def gdn_replay_forward_pooled(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, *, num_slots: int,
                              prev_state_update, accepted, replay_pool, read_slots=None, write_slots=None,
                              read_slots_host=None, write_slots_host=None, accepted_host=None, **kw) -> int:
    """gdn_replay_forward_pooled of include/gdn_pool.h: initial_state and replay_pool
    are pools [P, Hv, Dv, Dk] (may be one tensor); request r replays from slot
    read_slots[r] into slot write_slots[r] and verifies from it."""
    pool = dict(num_slots=num_slots, read_slots=read_slots, write_slots=write_slots,
                read_slots_host=read_slots_host, write_slots_host=write_slots_host)
    return _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, pool=pool,
                    replay=dict(prev=prev_state_update, accepted=accepted, state=replay_pool,
                                accepted_host=accepted_host), **kw)


def gdn_forward_pooled(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, *, num_slots: int,
                       read_slots=None, write_slots=None, read_slots_host=None,
                       write_slots_host=None, **kw) -> int:
    """gdn_forward_pooled of include/gdn_pool.h: initial_state and final_state are
    pools [P, Hv, Dv, Dk]; request r reads slot read_slots[r] and writes slot
    write_slots[r] (int32 GPU tensors [R], None for slot r)."""
    pool = dict(num_slots=num_slots, read_slots=read_slots, write_slots=write_slots,
                read_slots_host=read_slots_host, write_slots_host=write_slots_host)
    return _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, pool=pool, **kw)


def _forward(q, k, v, a, b, A_log, dt_bias, cu_seqlens, output, *, initial_state=None,
             final_state=None, state_update=None, capture_count=None, cu_seqlens_host=None,
             scale: float = 0.0, chunk: int = 0, state_update_capacity: int = 0,
             plan: int = PLAN_AUTO, update_rule: int = RULE_GATED_DELTA,
             gate_activation: int = GATE_RAW, num_reqs: Optional[int] = None, workspace=None,
             stream=None, check: bool = True, pool=None, state_layout: int = STATE_V_MAJOR,
             no_alloc: bool = False, replay=None) -> int:
    """One forward call on torch tensors; returns the status code.

    q, k [N, Hk, Dk], v and output [N, Hv, Dv] in float16 or float32 (for the
    dense rank-4 layout, cu_seqlens None: [R, S, H, D] tensors, or the same
    flattened; R from num_reqs or the leading dim); a, b [N, Hv] float32 (raw
    gate inputs, or alpha and beta with gate_activation GATE_NONE, when A_log
    and dt_bias may be None); A_log, dt_bias [Hv] float32; cu_seqlens [R+1]
    int32 or None; states [R, Hv, Dv, Dk] float32; state_update
    [R, capacity, W] float32; capture_count [R] int32; workspace a uint8 GPU
    tensor (CHUNK plan).
    """
    torch = _torch()
    if cu_seqlens is None and q.dim() == 4:
        if num_reqs is None:
            num_reqs = q.shape[0]
        q, k, v, output = (x.reshape(-1, x.shape[2], x.shape[3]) for x in (q, k, v, output))
        a, b = (x.reshape(-1, x.shape[-1]) for x in (a, b))
    N, Hk, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[2]
    if cu_seqlens is None:
        if num_reqs is None:
            raise ValueError("the dense layout (cu_seqlens None) needs num_reqs or [R, S, H, D] inputs")
        R = int(num_reqs)
    else:
        R = cu_seqlens.shape[0] - 1
    io = q.dtype
    _need(q, "q", (N, Hk, Dk))
    _need(k, "k", (N, Hk, Dk), io)
    _need(v, "v", (N, Hv, Dv), io)
    _need(output, "output", (N, Hv, Dv), io)
    _need(a, "a", (N, Hv), torch.float32)
    _need(b, "b", (N, Hv), torch.float32)
    _need(A_log, "A_log", (Hv,), torch.float32)
    _need(dt_bias, "dt_bias", (Hv,), torch.float32)
    _need(cu_seqlens, "cu_seqlens", (R + 1,), torch.int32)
    S = int(pool["num_slots"]) if pool is not None else R
    st_shape = (S, Hv, Dk, Dv) if state_layout == STATE_K_MAJOR else (S, Hv, Dv, Dk)
    _need(initial_state, "initial_state", st_shape, torch.float32)
    _need(final_state, "final_state", st_shape, torch.float32)
    if state_update is not None:
        _need(state_update, "state_update",
              (R, state_update_capacity, capsule_width(Hk, Hv, Dk, Dv)), torch.float32)
    _need(capture_count, "capture_count", (R,), torch.int32)
    host_cu, host_cu_ptr = _host_i32(cu_seqlens_host)
    if host_cu is not None and host_cu.shape != (R + 1,):
        raise ValueError("cu_seqlens_host must have R + 1 entries")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous GPU tensor")
        ws_ptr, ws_bytes = int(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    params = make_params(N, R, Hk, Hv, Dk, Dv, _io_code(io), scale=scale, chunk=chunk,
                         capacity=state_update_capacity, plan=plan, update_rule=update_rule,
                         gate_activation=gate_activation,
                         state_layout=state_layout)
    tens = GdnTensors(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                      _ptr(cu_seqlens), host_cu_ptr, _ptr(initial_state), _ptr(final_state),
                      _ptr(output), _ptr(state_update), _ptr(capture_count))
    where = "gdn_forward_pooled" if pool is not None else "gdn_forward"
    if replay is not None:
        if no_alloc or workspace is not None:
            raise ValueError("gdn_replay_forward takes no workspace")
        where = "gdn_replay_forward" if pool is None else "gdn_replay_forward_pooled"
        _need(replay["prev"], "prev_state_update",
              (R, state_update_capacity, capsule_width(Hk, Hv, Dk, Dv)), torch.float32)
        _need(replay["accepted"], "accepted", (R,), torch.int32)
        _need(replay["state"], "replay_state", st_shape, torch.float32)
        acc_host, acc_host_ptr = _host_i32(replay["accepted_host"])
        if acc_host is not None and acc_host.shape != (R,):
            raise ValueError("accepted_host must have R entries")
        if pool is None:
            st = lib().gdn_replay_forward(ctypes.byref(params), ctypes.byref(tens), _ptr(replay["prev"]),
                                          _ptr(replay["accepted"]), acc_host_ptr, _ptr(replay["state"]),
                                          _stream_handle(stream))
        else:
            sl, keep = _slots(R, **pool)
            st = lib().gdn_replay_forward_pooled(ctypes.byref(params), ctypes.byref(tens), ctypes.byref(sl),
                                                 _ptr(replay["prev"]), _ptr(replay["accepted"]), acc_host_ptr,
                                                 _ptr(replay["state"]), _stream_handle(stream))
            del keep
        del acc_host
    elif no_alloc:
        where = "gdn_forward_no_alloc"
        st = lib().gdn_forward_no_alloc(ctypes.byref(params), ctypes.byref(tens), _stream_handle(stream))
    elif pool is None:
        st = lib().gdn_forward(ctypes.byref(params), ctypes.byref(tens), ws_ptr,
                               ctypes.c_size_t(ws_bytes), _stream_handle(stream))
    else:
        sl, keep = _slots(R, **pool)
        st = lib().gdn_forward_pooled(ctypes.byref(params), ctypes.byref(tens), ctypes.byref(sl), ws_ptr,
                                      ctypes.c_size_t(ws_bytes), _stream_handle(stream))
        del keep
    del host_cu
    if check and st != GDN_OK:
        raise GDNError(st, where)
    return st


def gdn_forward_workspace_bytes(N, R, Hk, Hv, Dk, Dv, io_dtype=GDN_F16, *, capacity=0,
                                plan=PLAN_AUTO, cu_seqlens_host=None, chunk=0) -> int:
    """Workspace bytes gdn_forward needs (0 for the recurrent plan)."""
    params = make_params(N, R, Hk, Hv, Dk, Dv, io_dtype, chunk=chunk, capacity=capacity, plan=plan)
    host_cu, host_ptr = _host_i32(cu_seqlens_host)
    out = ctypes.c_size_t(0)
    st = lib().gdn_forward_workspace_bytes(ctypes.byref(params), host_ptr, ctypes.byref(out))
    del host_cu
    if st != GDN_OK:
        raise GDNError(st, "gdn_forward_workspace_bytes")
    return int(out.value)


def gdn_resolve_plan(N, R, Hk, Hv, Dk, Dv, io_dtype=GDN_F16, *, capacity=0, plan=PLAN_AUTO,
                     cu_seqlens_host=None) -> int:
    params = make_params(N, R, Hk, Hv, Dk, Dv, io_dtype, capacity=capacity, plan=plan)
    host_cu, host_ptr = _host_i32(cu_seqlens_host)
    out = ctypes.c_int32(0)
    st = lib().gdn_resolve_plan(ctypes.byref(params), host_ptr, ctypes.byref(out))
    del host_cu
    if st != GDN_OK:
        raise GDNError(st, "gdn_resolve_plan")
    return int(out.value)


def gdn_replay(src_state, state_update, accepted, dst_state, *, num_k_heads: int,
               state_update_capacity: int, accepted_host=None, stream=None,
               check: bool = True) -> int:
    """gdn_replay of include/gdn.h: dst = src advanced by the accepted capsule prefix."""
    return _replay(src_state, state_update, accepted, dst_state, num_k_heads=num_k_heads,
                   state_update_capacity=state_update_capacity, accepted_host=accepted_host,
                   stream=stream, check=check)


def gdn_replay_pooled(src_pool, state_update, accepted, dst_pool, *, num_k_heads: int,
                      state_update_capacity: int, read_slots=None, write_slots=None,
                      read_slots_host=None, write_slots_host=None, accepted_host=None,
                      state_layout: int = STATE_V_MAJOR, pooled: bool = True, stream=None,
                      check: bool = True) -> int:
    """gdn_replay_pooled of include/gdn_pool.h: pools [P, Hv, Dv, Dk] (K-major
    [P, Hv, Dk, Dv]); the request count is accepted's length. pooled=False passes
    no slot description: the states are then [R, ...], indexed by request."""
    pool = None
    if pooled:
        pool = dict(num_slots=src_pool.shape[0], read_slots=read_slots, write_slots=write_slots,
                    read_slots_host=read_slots_host, write_slots_host=write_slots_host)
    return _replay(src_pool, state_update, accepted, dst_pool, num_k_heads=num_k_heads,
                   state_update_capacity=state_update_capacity, accepted_host=accepted_host,
                   stream=stream, check=check, pool=pool, state_layout=state_layout, via_params=True)


def _replay(src_state, state_update, accepted, dst_state, *, num_k_heads, state_update_capacity,
            accepted_host, stream, check, pool=None, state_layout=STATE_V_MAJOR, via_params=False):
    torch = _torch()
    if state_layout == STATE_K_MAJOR:
        S, Hv, Dk, Dv = src_state.shape
    else:
        S, Hv, Dv, Dk = src_state.shape
    R = accepted.shape[0]
    Hk = int(num_k_heads)
    cap = int(state_update_capacity)
    st_shape = tuple(src_state.shape)
    _need(dst_state, "dst_state", st_shape, torch.float32)
    _need(src_state, "src_state", st_shape, torch.float32)
    if pool is None and S != R:
        raise ValueError("request-indexed states need one state per request")
    _need(accepted, "accepted", (R,), torch.int32)
    if cap > 0:
        _need(state_update, "state_update", (R, cap, capsule_width(Hk, Hv, Dk, Dv)), torch.float32)
    host_acc, host_ptr = _host_i32(accepted_host)
    if host_acc is not None and host_acc.shape != (R,):
        raise ValueError("accepted_host must have R entries")
    if not via_params:
        st = lib().gdn_replay(R, Hk, Hv, Dk, Dv, cap, _ptr(src_state), _ptr(state_update),
                              _ptr(accepted), host_ptr, _ptr(dst_state), _stream_handle(stream))
    else:
        params = make_params(0, R, Hk, Hv, Dk, Dv, GDN_F32, capacity=cap, state_layout=state_layout)
        sl, keep = _slots(R, **pool) if pool is not None else (None, None)
        st = lib().gdn_replay_pooled(ctypes.byref(params), _ptr(src_state), _ptr(state_update),
                                     _ptr(accepted), host_ptr, _ptr(dst_state),
                                     ctypes.byref(sl) if sl is not None else None, _stream_handle(stream))
        del keep
    del host_acc
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_replay_pooled" if via_params else "gdn_replay")
    return st


def gdn_conv_forward(x, weight, bias, cu_seqlens, output, **kw) -> int:
    """gdn_conv_forward of include/gdn_conv.h on torch tensors; returns the status.
    Keywords as _conv_forward."""
    return _conv_forward(x, weight, bias, cu_seqlens, output, **kw)


def gdn_conv_forward_pooled(x, weight, bias, cu_seqlens, output, *, num_slots: int, read_slots=None,
                            write_slots=None, read_slots_host=None, write_slots_host=None,
                            **kw) -> int:
    """gdn_conv_forward_pooled of include/gdn_pool.h: states are pools [P, C, K - 1]."""
    pool = dict(num_slots=num_slots, read_slots=read_slots, write_slots=write_slots,
                read_slots_host=read_slots_host, write_slots_host=write_slots_host)
    return _conv_forward(x, weight, bias, cu_seqlens, output, pool=pool, **kw)


def _conv_forward(x, weight, bias, cu_seqlens, output, *, initial_state=None,
                  final_state=None, state_update=None, capture_count=None,
                  cu_seqlens_host=None, activation: int = CONV_SILU,
                  state_update_capacity: int = 0, num_reqs: Optional[int] = None,
                  stream=None, check: bool = True, pool=None) -> int:
    """One convolution forward call on torch tensors; returns the status.

    x and output [N, C] float16 or float32 (dense layout, cu_seqlens None:
    [R, S, C] or [N, C] with num_reqs); weight [C, K] and bias [C] float32;
    cu_seqlens [R + 1] int32; states [R, C, K - 1] float32; state_update
    [R, capacity, C] float32; capture_count [R] int32.
    """
    torch = _torch()
    if cu_seqlens is None and x.dim() == 3:
        if num_reqs is None:
            num_reqs = x.shape[0]
        x, output = x.reshape(-1, x.shape[2]), output.reshape(-1, output.shape[2])
    N, C = x.shape
    K = weight.shape[1]
    if cu_seqlens is None:
        if num_reqs is None:
            raise ValueError("the dense layout (cu_seqlens None) needs num_reqs or [R, S, C] inputs")
        R = int(num_reqs)
    else:
        R = cu_seqlens.shape[0] - 1
    io = x.dtype
    _need(x, "x", (N, C))
    _need(output, "output", (N, C), io)
    _need(weight, "weight", (C, K), torch.float32)
    _need(bias, "bias", (C,), torch.float32)
    _need(cu_seqlens, "cu_seqlens", (R + 1,), torch.int32)
    S = int(pool["num_slots"]) if pool is not None else R
    _need(initial_state, "initial_state", (S, C, K - 1), torch.float32)
    _need(final_state, "final_state", (S, C, K - 1), torch.float32)
    if state_update is not None:
        _need(state_update, "state_update", (R, state_update_capacity, C), torch.float32)
    _need(capture_count, "capture_count", (R,), torch.int32)
    host_cu, host_cu_ptr = _host_i32(cu_seqlens_host)
    if host_cu is not None and host_cu.shape != (R + 1,):
        raise ValueError("cu_seqlens_host must have R + 1 entries")
    params = GdnConvParams(N, R, C, K, _io_code(io), int(activation), int(state_update_capacity))
    tens = GdnConvTensors(_ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), host_cu_ptr,
                          _ptr(initial_state), _ptr(final_state), _ptr(output),
                          _ptr(state_update), _ptr(capture_count))
    if pool is None:
        st = lib().gdn_conv_forward(ctypes.byref(params), ctypes.byref(tens), _stream_handle(stream))
    else:
        sl, keep = _slots(R, **pool)
        st = lib().gdn_conv_forward_pooled(ctypes.byref(params), ctypes.byref(tens), ctypes.byref(sl),
                                           _stream_handle(stream))
        del keep
    del host_cu
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_conv_forward_pooled" if pool is not None else "gdn_conv_forward")
    return st


def gdn_conv_decode_forward(mixed, conv_weight, conv_bias, a, b, A_log, dt_bias, cu_seqlens, output, *,
                            num_k_heads: int, head_k_dim: int, conv_initial_state=None, conv_final_state=None,
                            conv_activation: int = CONV_SILU, initial_state=None, final_state=None,
                            cu_seqlens_host=None, scale: float = 0.0, plan: int = PLAN_AUTO,
                            update_rule: int = RULE_GATED_DELTA, gate_activation: int = GATE_RAW,
                            num_reqs: Optional[int] = None, stream=None, check: bool = True) -> int:
    """gdn_conv_decode_forward of include/gdn_conv.h on torch tensors; returns the status.

    mixed [N, Cm] (dense layout, cu_seqlens None: [R, S, Cm]) float16 or float32,
    Cm = 2 Hk Dk + Hv Dv with the channels [q | k | v]; conv_weight [Cm, K] and
    conv_bias [Cm] float32; conv states [R, Cm, K - 1] float32; output [N, Hv, Dv]
    (or [R, S, Hv, Dv]) gives Hv and Dv; the rest as gdn_forward (V-major states).
    """
    torch = _torch()
    if cu_seqlens is None and mixed.dim() == 3:
        if num_reqs is None:
            num_reqs = mixed.shape[0]
        mixed = mixed.reshape(-1, mixed.shape[2])
        output = output.reshape(-1, output.shape[2], output.shape[3])
        a, b = (x.reshape(-1, x.shape[-1]) if x is not None else None for x in (a, b))
    N, Cm = mixed.shape
    Hv, Dv = output.shape[1], output.shape[2]
    Hk, Dk = int(num_k_heads), int(head_k_dim)
    if Cm != 2 * Hk * Dk + Hv * Dv:
        raise ValueError(f"mixed has {Cm} channels, expected 2 Hk Dk + Hv Dv = {2 * Hk * Dk + Hv * Dv}")
    K = conv_weight.shape[1]
    if cu_seqlens is None:
        if num_reqs is None:
            raise ValueError("the dense layout (cu_seqlens None) needs num_reqs or [R, S, Cm] inputs")
        R = int(num_reqs)
    else:
        R = cu_seqlens.shape[0] - 1
    io = mixed.dtype
    _need(mixed, "mixed", (N, Cm))
    _need(output, "output", (N, Hv, Dv), io)
    _need(conv_weight, "conv_weight", (Cm, K), torch.float32)
    _need(conv_bias, "conv_bias", (Cm,), torch.float32)
    _need(conv_initial_state, "conv_initial_state", (R, Cm, K - 1), torch.float32)
    _need(conv_final_state, "conv_final_state", (R, Cm, K - 1), torch.float32)
    _need(a, "a", (N, Hv), torch.float32)
    _need(b, "b", (N, Hv), torch.float32)
    _need(A_log, "A_log", (Hv,), torch.float32)
    _need(dt_bias, "dt_bias", (Hv,), torch.float32)
    _need(cu_seqlens, "cu_seqlens", (R + 1,), torch.int32)
    _need(initial_state, "initial_state", (R, Hv, Dv, Dk), torch.float32)
    _need(final_state, "final_state", (R, Hv, Dv, Dk), torch.float32)
    host_cu, host_cu_ptr = _host_i32(cu_seqlens_host)
    if host_cu is not None and host_cu.shape != (R + 1,):
        raise ValueError("cu_seqlens_host must have R + 1 entries")
    params = make_params(N, R, Hk, Hv, Dk, Dv, _io_code(io), scale=scale, plan=plan, update_rule=update_rule,
                         gate_activation=gate_activation)
    tens = GdnTensors(None, None, None, _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(cu_seqlens),
                      host_cu_ptr, _ptr(initial_state), _ptr(final_state), _ptr(output), None, None)
    conv = GdnConvFused(_ptr(mixed), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_initial_state),
                        _ptr(conv_final_state), int(K), int(conv_activation))
    st = lib().gdn_conv_decode_forward(ctypes.byref(params), ctypes.byref(tens), ctypes.byref(conv),
                                       _stream_handle(stream))
    del host_cu
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_conv_decode_forward")
    return st


def gdn_conv_replay(src_state, state_update, accepted, dst_state, *, state_update_capacity: int,
                    accepted_host=None, stream=None, check: bool = True) -> int:
    """gdn_conv_replay of include/gdn_conv.h: dst = the last K - 1 of [src, accepted inputs]."""
    return _conv_replay(src_state, state_update, accepted, dst_state,
                        state_update_capacity=state_update_capacity, accepted_host=accepted_host,
                        stream=stream, check=check)


def gdn_conv_replay_pooled(src_pool, state_update, accepted, dst_pool, *, state_update_capacity: int,
                           read_slots=None, write_slots=None, read_slots_host=None,
                           write_slots_host=None, accepted_host=None, stream=None,
                           check: bool = True) -> int:
    """gdn_conv_replay_pooled of include/gdn_pool.h: pools [P, C, K - 1]."""
    pool = dict(num_slots=src_pool.shape[0], read_slots=read_slots, write_slots=write_slots,
                read_slots_host=read_slots_host, write_slots_host=write_slots_host)
    return _conv_replay(src_pool, state_update, accepted, dst_pool,
                        state_update_capacity=state_update_capacity, accepted_host=accepted_host,
                        stream=stream, check=check, pool=pool)


def _conv_replay(src_state, state_update, accepted, dst_state, *, state_update_capacity,
                 accepted_host, stream, check, pool=None):
    torch = _torch()
    S, C, Km1 = src_state.shape
    R = accepted.shape[0] if pool is not None else S
    cap = int(state_update_capacity)
    _need(src_state, "src_state", (S, C, Km1), torch.float32)
    _need(dst_state, "dst_state", (S, C, Km1), torch.float32)
    _need(accepted, "accepted", (R,), torch.int32)
    if cap > 0:
        _need(state_update, "state_update", (R, cap, C), torch.float32)
    host_acc, host_ptr = _host_i32(accepted_host)
    if host_acc is not None and host_acc.shape != (R,):
        raise ValueError("accepted_host must have R entries")
    if pool is None:
        st = lib().gdn_conv_replay(R, C, Km1 + 1, cap, _ptr(src_state), _ptr(state_update),
                                   _ptr(accepted), host_ptr, _ptr(dst_state), _stream_handle(stream))
    else:
        sl, keep = _slots(R, **pool)
        st = lib().gdn_conv_replay_pooled(R, C, Km1 + 1, cap, _ptr(src_state), _ptr(state_update),
                                          _ptr(accepted), host_ptr, _ptr(dst_state), ctypes.byref(sl),
                                          _stream_handle(stream))
        del keep
    del host_acc
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_conv_replay_pooled" if pool is not None else "gdn_conv_replay")
    return st


def gdn_publish_slots(committed_slots, inactive_slots, *, stream=None, check: bool = True) -> int:
    """gdn_publish_slots of include/gdn_pool.h: exchanges the two int32 GPU slot arrays."""
    torch = _torch()
    R = committed_slots.shape[0]
    _need(committed_slots, "committed_slots", (R,), torch.int32)
    _need(inactive_slots, "inactive_slots", (R,), torch.int32)
    st = lib().gdn_publish_slots(R, _ptr(committed_slots), _ptr(inactive_slots), _stream_handle(stream))
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_publish_slots")
    return st


# ------------------------------------------------- the attention layer (gdn_attn.h)
class KVCache:
    """The paged key-value cache of one layer (gdn_kv_cache of include/gdn_attn.h): a
    description of tensors that the caller owns, made once and passed to every call.

    k_pages, v_pages [num_pages, Hk, page_size, D] float16 or float32; for the 8-bit
    format float8_e4m3fn or uint8, with k_scales, v_scales [num_pages, Hk, page_size]
    uint8 (the exponent bytes; I/O is then float16). For the 4-bit format k_pages, v_pages
    are [num_pages, Hk, page_size, D / 2] uint8, two e2m1 codes a byte, and the scales
    [num_pages, Hk, D / 32, page_size]. page_table [R, max_pages] int32;
    page_table_host an optional host mirror, checked on every call: a contiguous int32
    array or CPU tensor is read in place, so that a program can change it along with
    page_table; anything else is copied once, here.

    format is CACHE_IO, CACHE_E4M3 or CACHE_E2M1 (e4m3: whether it is the second; a 4-bit
    cache has scales, too), io_dtype the type of q, k, v and outputs.
    """

    def __init__(self, k_pages, v_pages, page_table, *, k_scales=None, v_scales=None, page_table_host=None):
        torch = _torch()
        if k_pages.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k_pages must be [num_pages, Hk, page_size, D] and page_table [R, max_pages]")
        P, Hk, page_size, D = k_pages.shape
        row = D                                              # a row's columns in the pages
        self.format, self.io_dtype = CACHE_IO, k_pages.dtype
        if k_scales is not None or v_scales is not None:
            if k_scales is None or v_scales is None:
                raise ValueError("the 8-bit and 4-bit formats need k_scales and v_scales")
            self.io_dtype = torch.float16
            if k_scales.dim() == 4:
                self.format, D = CACHE_E2M1, 2 * D
                if k_pages.dtype is not torch.uint8:
                    raise ValueError(f"k_pages: dtype {k_pages.dtype} is not a 4-bit cache (uint8)")
                scales = (P, Hk, D // 32, page_size)
            else:
                self.format, scales = CACHE_E4M3, (P, Hk, page_size)
                if k_pages.dtype not in (torch.uint8, torch.float8_e4m3fn):
                    raise ValueError(f"k_pages: dtype {k_pages.dtype} is not an 8-bit cache")
            _need(k_scales, "k_scales", scales, torch.uint8)
            _need(v_scales, "v_scales", scales, torch.uint8)
        self.e4m3 = self.format == CACHE_E4M3
        _need(k_pages, "k_pages", (P, Hk, page_size, row))
        _need(v_pages, "v_pages", (P, Hk, page_size, row), k_pages.dtype)
        _need(page_table, "page_table", tuple(page_table.shape), torch.int32)
        for x, name in ((v_pages, "v_pages"), (page_table, "page_table"), (k_scales, "k_scales"),
                        (v_scales, "v_scales")):
            if x is not None and x.device != k_pages.device:
                raise ValueError(f"{name} is on {x.device}, k_pages on {k_pages.device}")
        host, host_ptr = _host_i32(page_table_host)
        if host is not None and host.shape != tuple(page_table.shape):
            raise ValueError("page_table_host must have page_table's shape")
        self.num_reqs, max_pages = page_table.shape
        self.num_kv_heads, self.head_dim, self.index = Hk, D, k_pages.get_device()
        self.num_pages, self.page_size = P, page_size
        self._keep = (k_pages, v_pages, k_scales, v_scales, page_table, host)
        self.struct = GdnKvCache(_ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), _ptr(page_table),
                                 host_ptr, P, page_size, max_pages, Hk, D, _io_code(self.io_dtype),
                                 self.format)
        self.address = ctypes.addressof(self.struct)


# Decode calls take a few microseconds on the GPU, so the checks below are written to
# be cheap: one attribute each, no helper objects.
def _token_rows(x, name, heads, D, io, index):
    """Token stride of x [N, heads, D] of type io on GPU `index`, whose tokens may lie apart
    (0: dense): a slice of a wider projection's output is taken as it is."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{name}: shape {tuple(shape)} != expected (N, {heads}, {D})")
    if x.dtype is not io:
        raise ValueError(f"{name}: dtype {x.dtype} != expected {io}")
    if x.get_device() != index:
        raise ValueError(f"{name} is on {x.device}, expected GPU {index}")
    if x.is_contiguous():
        return 0
    st = x.stride()
    if st[2] == 1 and (heads <= 1 or st[1] == D):
        if shape[0] <= 1:
            return 0
        if heads * D <= st[0] < 1 << 31:
            return st[0]
    raise ValueError(f"{name}: only the token dimension may be strided, by less than 2^31 elements")


def _out_rows(out, of, name):
    """An output of the rotation: dense, or `of` itself."""
    if out is of:
        return
    if out is None or out.shape != of.shape or out.dtype is not of.dtype or out.get_device() != of.get_device():
        raise ValueError(f"{name} must have its input's shape, type and device")
    if out.data_ptr() == of.data_ptr():
        # the library takes equal addresses for in place, and then the input's strides for the output's
        if any(n > 1 and a != b for n, a, b in zip(of.shape, out.stride(), of.stride())):
            raise ValueError(f"{name} begins where its input does, but its rows lie elsewhere")
    elif not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or its input itself")


def _int_vector(x, name, n, index):
    if x.shape != (n,) or x.dtype is not _torch().int32 or x.get_device() != index or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] on GPU {index}")
    return x.data_ptr()


def _frequencies(x, index):
    if x is None or x.dtype is not _torch().float64 or x.dim() != 1 or x.get_device() != index or \
            not x.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 [rotary_dim / 2] on GPU {index}")
    return x.data_ptr()


def _on_current_device(index):
    if index < 0:
        raise ValueError("tensors must be GPU tensors")
    current = _torch()._C._cuda_getDevice()
    if index != current:
        raise ValueError(f"tensors are on GPU {index}, the current device is {current}")


def _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host, seq_lens_host):
    """(R, seq_lens, cu_seqlens, their host mirrors as addresses, the mirrors to keep alive)."""
    R = num_reqs if num_reqs is not None else \
        cu_seqlens.shape[0] - 1 if cu_seqlens is not None else seq_lens.shape[0]
    index = cache.index
    if R > cache.num_reqs:
        raise ValueError(f"{R} requests, but page_table has {cache.num_reqs} rows")
    lens = _int_vector(seq_lens, "seq_lens", R, index)
    cu = 0 if cu_seqlens is None else _int_vector(cu_seqlens, "cu_seqlens", R + 1, index)
    cu_h, cu_ptr = _host_i32(cu_seqlens_host)
    len_h, len_ptr = _host_i32(seq_lens_host)
    if cu_h is not None and cu_h.shape != (R + 1,):
        raise ValueError("cu_seqlens_host must have R + 1 entries")
    if len_h is not None and len_h.shape != (R,):
        raise ValueError("seq_lens_host must have R entries")
    _on_current_device(index)
    return R, lens, cu, len_ptr or 0, cu_ptr or 0, (cu_h, len_h)


def gdn_rope_frequencies(rotary_dim: int, *, base: float = 10000.0, scaling: int = ROPE_SCALING_NONE,
                         scale: float = 1.0, trained_length: float = 0.0, beta_fast: float = 0.0,
                         beta_slow: float = 0.0):
    """gdn_rope_frequencies of include/gdn_attn.h: (inv_freq, a float64 numpy array
    [rotary_dim / 2], the factor of cos and sin)."""
    import numpy as np
    out = np.empty(max(int(rotary_dim) // 2, 1), np.float64)
    factor = ctypes.c_float(0.0)
    st = lib().gdn_rope_frequencies(int(rotary_dim), float(base), int(scaling), float(scale), float(trained_length),
                                    float(beta_fast), float(beta_slow), out.ctypes.data, ctypes.byref(factor))
    if st != GDN_OK:
        raise GDNError(st, "gdn_rope_frequencies")
    return out, float(factor.value)


def gdn_rope_forward(q, k, positions, inv_freq, q_out, k_out, *, rope_layout: int = ROPE_HALF,
                     rope_factor: float = 1.0, stream=None, check: bool = True) -> int:
    """gdn_rope_forward of include/gdn_attn.h on torch tensors; returns the status.

    q [N, Hq, D] and k [N, Hk, D] float16 or float32 (either may be None; the token
    dimension may be strided), positions [N] int32, inv_freq [rotary_dim / 2] float64;
    q_out, k_out dense, or q, k themselves.
    """
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        raise ValueError("q or k [N, heads, D] is needed")
    N, _, D = x.shape
    index, io = x.get_device(), x.dtype
    Hq = Hk = qs = ks = 0
    qp = kp = qop = kop = 0
    if q is not None:
        Hq, qp = q.shape[1], q.data_ptr()
        qs = _token_rows(q, "q", Hq, D, io, index)
        _out_rows(q_out, q, "q_out")
        qop = q_out.data_ptr()
    if k is not None:
        if k.shape[0] != N:
            raise ValueError("q and k must have the same tokens")
        Hk, kp = k.shape[1], k.data_ptr()
        ks = _token_rows(k, "k", Hk, D, io, index)
        _out_rows(k_out, k, "k_out")
        kop = k_out.data_ptr()
    pos, freq = _int_vector(positions, "positions", N, index), _frequencies(inv_freq, index)
    _on_current_device(index)
    st = _call("gdn_rope_forward")(
        _rope_params(N, Hq, Hk, D, _io_code(io), 2 * inv_freq.shape[0], rope_layout, rope_factor, qs, ks),
        _rope_tensors(qp, kp, pos, freq, qop, kop), _stream_handle(stream, index))
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_rope_forward")
    return st


def gdn_kv_write(k, v, cache: KVCache, seq_lens, cu_seqlens=None, *, q=None, q_out=None, inv_freq=None,
                 positions=None, rope_layout: int = ROPE_HALF, rope_factor: float = 1.0,
                 num_reqs: Optional[int] = None, cu_seqlens_host=None, seq_lens_host=None, stream=None,
                 check: bool = True) -> int:
    """gdn_kv_write of include/gdn_attn.h on torch tensors; returns the status.

    k, v [N, Hk, D] in the cache's I/O type (the token dimension may be strided);
    seq_lens [R] int32, the cached tokens with these included; cu_seqlens [R + 1] int32
    or None for N / R tokens each. With inv_freq [rotary_dim / 2] float64 k is rotated
    as it is written, and q [N, Hq, D], when given, into q_out; positions [N] int32
    default to the positions in the cache.
    """
    Hk, D, index, io = cache.num_kv_heads, cache.head_dim, cache.index, cache.io_dtype
    N = k.shape[0]
    ks, vs = _token_rows(k, "k", Hk, D, io, index), _token_rows(v, "v", Hk, D, io, index)
    if v.shape[0] != N:
        raise ValueError("k and v must have the same tokens")
    Hq = qs = rot = 0
    qp = qop = pos = freq = 0
    if inv_freq is not None:
        freq = _frequencies(inv_freq, index)
        rot = 2 * inv_freq.shape[0]
        if positions is not None:
            pos = _int_vector(positions, "positions", N, index)
        if q is not None:
            if q.shape[0] != N:
                raise ValueError("q and k must have the same tokens")
            Hq, qp = q.shape[1], q.data_ptr()
            qs = _token_rows(q, "q", Hq, D, io, index)
            _out_rows(q_out, q, "q_out")
            qop = q_out.data_ptr()
    elif q is not None or positions is not None:
        raise ValueError("q and positions go with a rotation (inv_freq)")
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_kv_write")(_kv_params(N, R, Hq, rot, rope_layout, rope_factor, qs, ks, vs),
                               _kv_tensors(k.data_ptr(), v.data_ptr(), cu, cu_h, lens, len_h, qp, qop, pos, freq),
                               cache.address, _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_kv_write")
    return st


def gdn_kv_read(k, v, cache: KVCache, seq_lens, cu_seqlens=None, *, num_reqs: Optional[int] = None,
                cu_seqlens_host=None, seq_lens_host=None, stream=None, check: bool = True) -> int:
    """gdn_kv_read of include/gdn_attn.h: the newest T_r of every request's seq_lens[r]
    cached tokens into k, v [N, Hk, D] (dense, the cache's I/O type); returns the status."""
    Hk, D, index, io = cache.num_kv_heads, cache.head_dim, cache.index, cache.io_dtype
    N = k.shape[0]
    if _token_rows(k, "k", Hk, D, io, index) or _token_rows(v, "v", Hk, D, io, index) or v.shape[0] != N or \
            not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("k and v must be contiguous and have the same tokens")
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_kv_read")(_kv_params(N, R, 0, 0, 0, 0.0, 0, 0, 0),
                              _kv_tensors(k.data_ptr(), v.data_ptr(), cu, cu_h, lens, len_h, 0, 0, 0, 0),
                              cache.address, _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_kv_read")
    return st


def gdn_attn_workspace_bytes(N: int, R: int, Hq: int, cache: KVCache) -> int:
    """Workspace bytes gdn_attn_forward needs for these sizes, whatever the lengths."""
    params = GdnAttnParams(int(N), int(R), int(Hq), 0.0, 0, 0)
    out = ctypes.c_size_t(0)
    st = lib().gdn_attn_workspace_bytes(ctypes.byref(params), ctypes.byref(cache.struct), ctypes.byref(out))
    if st != GDN_OK:
        raise GDNError(st, "gdn_attn_workspace_bytes")
    return int(out.value)


def gdn_attn_forward(q, cache: KVCache, seq_lens, cu_seqlens, output, *, scale: float = 0.0, window: int = 0,
                     num_reqs: Optional[int] = None, cu_seqlens_host=None, seq_lens_host=None, workspace=None,
                     stream=None, check: bool = True) -> int:
    """gdn_attn_forward of include/gdn_attn.h on torch tensors; returns the status.

    q [N, Hq, D] in the cache's I/O type (the token dimension may be strided), output
    [N, Hq, D] dense; seq_lens [R] int32; cu_seqlens [R + 1] int32 or None for N / R
    tokens each; workspace a uint8 GPU tensor of gdn_attn_workspace_bytes().
    """
    index, io = cache.index, cache.io_dtype
    shape = q.shape
    N, Hq = shape[0], shape[1]
    qs = _token_rows(q, "q", Hq, cache.head_dim, io, index)
    if output.shape != shape or output.dtype is not io or output.get_device() != index or not output.is_contiguous():
        raise ValueError("output must be contiguous and have q's shape, type and device")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's GPU")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_attn_forward")(_attn_params(N, R, Hq, scale, window, qs),
                                   _attn_tensors(q.data_ptr(), cu, cu_h, lens, len_h, output.data_ptr()),
                                   cache.address, ws, ws_bytes, _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_attn_forward")
    return st


def gdn_kv_bounds(bounds, cache: KVCache, seq_lens, cu_seqlens=None, *, num_tokens: int, num_reqs: Optional[int] = None,
                  cu_seqlens_host=None, seq_lens_host=None, stream=None, check: bool = True) -> int:
    """gdn_kv_bounds of include/gdn_attn.h: the lowest and highest key, channel by channel, of
    every page that holds one of the newest num_tokens tokens (as in gdn_kv_write) into bounds
    [num_pages, Hk, 2, D] (the cache's I/O type); returns the status."""
    index = cache.index
    _page_bounds(bounds, cache, index)
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_kv_bounds")(_kv_params(num_tokens, R, 0, 0, 0, 0.0, 0, 0, 0),
                                _kv_tensors(0, 0, cu, cu_h, lens, len_h, 0, 0, 0, 0), cache.address, bounds.data_ptr(),
                                _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_kv_bounds")
    return st


def _page_bounds(x, cache, index):
    if x.shape != (cache.num_pages, cache.num_kv_heads, 2, cache.head_dim) or x.dtype is not cache.io_dtype or \
            x.get_device() != index or not x.is_contiguous():
        raise ValueError("bounds must be contiguous [num_pages, Hk, 2, D] in the cache's I/O type, on its GPU")


def _page_lists(pages, counts, N, cache, index):
    """K of lists [N, Hk, K] and their counts [N]."""
    shape, i32 = pages.shape, _torch().int32
    if len(shape) != 3 or shape[0] != N or shape[1] != cache.num_kv_heads or pages.dtype is not i32 or \
            pages.get_device() != index or not pages.is_contiguous():
        raise ValueError(f"pages must be a contiguous int32 [{N}, {cache.num_kv_heads}, K] on GPU {index}")
    if counts is not None:
        _int_vector(counts, "counts", N, index)
    return shape[2]


def _workspace(workspace, index):
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's GPU")
    return workspace.data_ptr(), workspace.nbytes


def gdn_attn_select_workspace_bytes(N: int, R: int, Hq: int, K: int, cache: KVCache) -> int:
    """Workspace bytes gdn_attn_select needs for these sizes, whatever the lengths."""
    params = GdnSelectParams(int(N), int(R), int(Hq), int(K), 0, 0, 0)
    out = ctypes.c_size_t(0)
    st = lib().gdn_attn_select_workspace_bytes(ctypes.byref(params), ctypes.byref(cache.struct), ctypes.byref(out))
    if st != GDN_OK:
        raise GDNError(st, "gdn_attn_select_workspace_bytes")
    return int(out.value)


def gdn_attn_select(q, bounds, cache: KVCache, seq_lens, cu_seqlens, pages, counts, *, first_pages: int = 1,
                    newest_pages: int = 1, num_reqs: Optional[int] = None, cu_seqlens_host=None, seq_lens_host=None,
                    workspace=None, stream=None, check: bool = True) -> int:
    """gdn_attn_select of include/gdn_attn.h on torch tensors; returns the status.

    q [N, Hq, D] in the cache's I/O type (the token dimension may be strided); bounds
    [num_pages, Hk, 2, D] of gdn_kv_bounds; pages [N, Hk, K] int32 receives the selected
    entries of the page table, ascending and -1 behind them, counts [N] int32 their number.
    The first first_pages and the newest newest_pages are always in. workspace: a uint8 GPU
    tensor of gdn_attn_select_workspace_bytes().
    """
    index, io = cache.index, cache.io_dtype
    N, Hq = q.shape[0], q.shape[1]
    qs = _token_rows(q, "q", Hq, cache.head_dim, io, index)
    _page_bounds(bounds, cache, index)
    K = _page_lists(pages, counts, N, cache, index)
    ws, ws_bytes = _workspace(workspace, index)
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_attn_select")(_select_params(N, R, Hq, K, first_pages, newest_pages, qs),
                                  _select_tensors(q.data_ptr(), cu, cu_h, lens, len_h, bounds.data_ptr(),
                                                  pages.data_ptr(), counts.data_ptr()),
                                  cache.address, ws, ws_bytes, _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_attn_select")
    return st


def gdn_attn_sparse_workspace_bytes(N: int, R: int, Hq: int, K: int, cache: KVCache) -> int:
    """Workspace bytes gdn_attn_sparse_forward needs for these sizes, whatever the lists."""
    params = GdnSparseParams(int(N), int(R), int(Hq), int(K), 0.0, 0)
    out = ctypes.c_size_t(0)
    st = lib().gdn_attn_sparse_workspace_bytes(ctypes.byref(params), ctypes.byref(cache.struct), ctypes.byref(out))
    if st != GDN_OK:
        raise GDNError(st, "gdn_attn_sparse_workspace_bytes")
    return int(out.value)


def gdn_attn_sparse_forward(q, cache: KVCache, seq_lens, cu_seqlens, pages, counts, output, *, scale: float = 0.0,
                            num_reqs: Optional[int] = None, cu_seqlens_host=None, seq_lens_host=None, workspace=None,
                            stream=None, check: bool = True) -> int:
    """gdn_attn_sparse_forward of include/gdn_attn.h on torch tensors; returns the status.

    q, output, seq_lens and cu_seqlens as in gdn_attn_forward; pages [N, Hk, K] int32 the
    entries of its request's page table that each token and key head attends, counts [N]
    int32 how many of them (None: K); workspace a uint8 GPU tensor of
    gdn_attn_sparse_workspace_bytes().
    """
    index, io = cache.index, cache.io_dtype
    shape = q.shape
    N, Hq = shape[0], shape[1]
    qs = _token_rows(q, "q", Hq, cache.head_dim, io, index)
    if output.shape != shape or output.dtype is not io or output.get_device() != index or not output.is_contiguous():
        raise ValueError("output must be contiguous and have q's shape, type and device")
    K = _page_lists(pages, counts, N, cache, index)
    ws, ws_bytes = _workspace(workspace, index)
    R, lens, cu, len_h, cu_h, keep = _cache_rows(cache, seq_lens, cu_seqlens, num_reqs, cu_seqlens_host,
                                                 seq_lens_host)
    st = _call("gdn_attn_sparse_forward")(_sparse_params(N, R, Hq, K, scale, qs),
                                          _sparse_tensors(q.data_ptr(), cu, cu_h, lens, len_h, pages.data_ptr(),
                                                          0 if counts is None else counts.data_ptr(), output.data_ptr()),
                                          cache.address, ws, ws_bytes, _stream_handle(stream, index))
    del keep
    if check and st != GDN_OK:
        raise GDNError(st, "gdn_attn_sparse_forward")
    return st
