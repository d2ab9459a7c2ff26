"""Host-side checks of the 4-bit cache format and of the sparse attention's entry points: every bad
argument is rejected with the documented status before anything is enqueued.

As in test_attn_host.py, no call here launches a kernel, and the module runs only where no GPU is visible.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import gateddeltanet_recurrence_amd as gdn
from gateddeltanet_recurrence_amd import binding


def _gpu_visible() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:
        return False


pytestmark = [
    pytest.mark.skipif(not os.path.exists(gdn.library_path()), reason="libgdn.so not built (run the build first)"),
    pytest.mark.skipif(_gpu_visible(), reason="fake-pointer host checks run only without a GPU"),
]

FAKE = 1 << 40          # 16-byte aligned, never dereferenced
N, R, HQ, HK, D, PAGES, PAGE, MAXP, K = 8, 2, 4, 2, 64, 10, 16, 4, 3
CU_BAD = np.array([0, 3, 7], np.int32)     # cu[R] != N: a call that passes every other check still ends here
CU = np.array([0, 3, 8], np.int32)
IO, E4M3, E2M1 = gdn.CACHE_IO, gdn.CACHE_E4M3, gdn.CACHE_E2M1


class Fields:
    """Fake, disjoint device addresses of one call."""

    def __init__(self, fmt=IO, io=2):
        at = FAKE
        rows = PAGES * HK * PAGE
        row = D * io if fmt == IO else D if fmt == E4M3 else D // 2
        scale = 0 if fmt == IO else 1 if fmt == E4M3 else D // 32
        for name, size in dict(k_pages=rows * row, v_pages=rows * row, k_scales=rows * scale, v_scales=rows * scale, table=R * MAXP * 4,
                               q=N * HQ * D * io, k=N * HK * D * io, v=N * HK * D * io, bounds=PAGES * HK * 2 * D * io,
                               pages=N * HK * K * 4, counts=N * 4, cu=(R + 1) * 4, lens=R * 4, output=N * HQ * D * io,
                               ws=1 << 24).items():
            setattr(self, name, at)
            at += (size + 4095) // 4096 * 4096 + 4096


def _cache(f, fmt=IO, *, io=gdn.GDN_F16, **over):
    coded = fmt != IO
    c = gdn.GdnKvCache(f.k_pages, f.v_pages, f.k_scales if coded else None, f.v_scales if coded else None, f.table, None, PAGES, PAGE,
                       MAXP, HK, D, io, fmt)
    for name, v in over.items():
        setattr(c, name, v)
    return c


def _fill(struct, over):
    for name, v in over.items():
        setattr(struct, name, v)
    return struct


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _write(f, cache, params=None, **over):
    p = _fill(gdn.GdnKvParams(N, R, 0, 0, 0, 0.0, 0, 0, 0), params or {})
    t = _fill(gdn.GdnKvTensors(f.k, f.v, f.cu, CU_BAD.ctypes.data, f.lens, None, None, None, None, None), over)
    return gdn.lib().gdn_kv_write(ctypes.byref(p), ctypes.byref(t), _ref(cache), None)


def _read(f, cache, params=None, **over):
    p = _fill(gdn.GdnKvParams(N, R, 0, 0, 0, 0.0, 0, 0, 0), params or {})
    t = _fill(gdn.GdnKvTensors(f.k, f.v, f.cu, CU_BAD.ctypes.data, f.lens, None, None, None, None, None), over)
    return gdn.lib().gdn_kv_read(ctypes.byref(p), ctypes.byref(t), _ref(cache), None)


def _attn(f, cache, params=None, ws_bytes=1 << 24, **over):
    p = _fill(gdn.GdnAttnParams(N, R, HQ, 0.0, 0, 0), params or {})
    ws = over.pop("ws", f.ws)
    t = _fill(gdn.GdnAttnTensors(f.q, f.cu, CU_BAD.ctypes.data, f.lens, None, f.output), over)
    return gdn.lib().gdn_attn_forward(ctypes.byref(p), ctypes.byref(t), _ref(cache), ws, ws_bytes, None)


def _bounds(f, cache, params=None, **over):
    p = _fill(gdn.GdnKvParams(N, R, 0, 0, 0, 0.0, 0, 0, 0), params or {})
    out = over.pop("bounds", f.bounds)
    t = _fill(gdn.GdnKvTensors(None, None, f.cu, CU_BAD.ctypes.data, f.lens, None, None, None, None, None), over)
    return gdn.lib().gdn_kv_bounds(ctypes.byref(p), ctypes.byref(t), _ref(cache), out, None)


def _select(f, cache, params=None, ws_bytes=1 << 24, **over):
    p = _fill(gdn.GdnSelectParams(N, R, HQ, K, 1, 1, 0), params or {})
    ws = over.pop("ws", f.ws)
    t = _fill(gdn.GdnSelectTensors(f.q, f.cu, CU_BAD.ctypes.data, f.lens, None, f.bounds, f.pages, f.counts), over)
    return gdn.lib().gdn_attn_select(ctypes.byref(p), ctypes.byref(t), _ref(cache), ws, ws_bytes, None)


def _sparse(f, cache, params=None, ws_bytes=1 << 24, **over):
    p = _fill(gdn.GdnSparseParams(N, R, HQ, K, 0.0, 0), params or {})
    ws = over.pop("ws", f.ws)
    t = _fill(gdn.GdnSparseTensors(f.q, f.cu, CU_BAD.ctypes.data, f.lens, None, f.pages, f.counts, f.output), over)
    return gdn.lib().gdn_attn_sparse_forward(ctypes.byref(p), ctypes.byref(t), _ref(cache), ws, ws_bytes, None)


ALL = [_write, _read, _attn, _bounds, _select, _sparse]
NEW = [_bounds, _select, _sparse]
DENSE = dict(cu_seqlens=None, cu_seqlens_host=None)


@pytest.mark.parametrize("call", ALL)
def test_the_4_bit_format_needs_scales_and_fp16(call):
    f = Fields(E2M1)
    assert call(f, _cache(f, E2M1)) == gdn.GDN_ERR_SHAPE                    # the malformed mirror: all else is taken
    assert call(f, _cache(f, E2M1, v_scales=None)) == gdn.GDN_ERR_NULL
    assert call(f, _cache(f, E2M1, io_dtype=gdn.GDN_F32)) == gdn.GDN_ERR_DTYPE
    assert call(f, _cache(f, E2M1, k_scales=f.k_scales + 8)) == gdn.GDN_ERR_SHAPE
    assert call(f, _cache(f, E2M1, format=3)) == gdn.GDN_ERR_DTYPE


def test_4_bit_pools_may_not_overlap():
    """Pages of D / 2 bytes a row and scales of D / 32: a pool ends where its last byte does."""
    f = Fields(E2M1)
    scales, pages = PAGES * HK * PAGE * (D // 32), PAGES * HK * PAGE * D // 2
    assert _write(f, _cache(f, E2M1, v_scales=f.k_scales + scales - 16), **DENSE) == gdn.GDN_ERR_ALIAS
    assert _write(f, _cache(f, E2M1, v_pages=f.k_pages + pages - 16), **DENSE) == gdn.GDN_ERR_ALIAS


def test_outputs_may_not_touch_the_4_bit_pool():
    f = Fields(E2M1)
    last = PAGES * HK * PAGE * (D // 32) - 16
    c = _cache(f, E2M1)
    assert _read(f, c, k=f.k_scales + last, **DENSE) == gdn.GDN_ERR_ALIAS
    assert _attn(f, c, output=f.v_scales + last, **DENSE) == gdn.GDN_ERR_ALIAS
    assert _bounds(f, c, bounds=f.k_scales + last, **DENSE) == gdn.GDN_ERR_ALIAS
    assert _bounds(f, c, bounds=f.k_pages + PAGES * HK * PAGE * D // 2 - 16, **DENSE) == gdn.GDN_ERR_ALIAS


@pytest.mark.parametrize("call", NEW)
@pytest.mark.parametrize("field,value,code", [
    ("io_dtype", gdn.GDN_BF16, gdn.GDN_ERR_DTYPE), ("format", 2, gdn.GDN_ERR_DTYPE), ("num_pages", 0, gdn.GDN_ERR_SHAPE),
    ("max_pages", 0, gdn.GDN_ERR_SHAPE), ("num_kv_heads", 0, gdn.GDN_ERR_SHAPE), ("page_size", 48, gdn.GDN_ERR_SHAPE),
    ("head_dim", 96, gdn.GDN_ERR_SHAPE), ("max_pages", 1 << 27, gdn.GDN_ERR_SHAPE), ("k_pages", None, gdn.GDN_ERR_NULL),
    ("page_table", None, gdn.GDN_ERR_NULL), ("k_pages", FAKE + 8, gdn.GDN_ERR_SHAPE), ("k_scales", FAKE, gdn.GDN_ERR_SHAPE),
])
def test_cache_validation(call, field, value, code):
    f = Fields()
    assert call(f, _cache(f, **{field: value})) == code
    assert call(f, None) == gdn.GDN_ERR_NULL


@pytest.mark.parametrize("call", NEW)
def test_row_validation(call):
    f = Fields()
    c = _cache(f)
    assert call(f, c) == gdn.GDN_ERR_SHAPE
    for lens in ([2, 8], [3, 4], [3, MAXP * PAGE + 1]):
        assert call(f, c, cu_seqlens_host=CU.ctypes.data, seq_lens_host=np.array(lens, np.int32).ctypes.data) == gdn.GDN_ERR_CAPACITY
    assert call(f, c, cu_seqlens=None) == gdn.GDN_ERR_SHAPE
    assert call(f, c, **DENSE, params=dict(num_tokens=7)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, cu_seqlens_host=CU.ctypes.data, seq_lens=None) == gdn.GDN_ERR_NULL
    assert call(f, c, params=dict(num_tokens=-1)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, params=dict(num_reqs=-1)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, params=dict(num_reqs=0)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, params=dict(num_reqs=0, num_tokens=0)) == gdn.GDN_OK
    assert call(f, c, **DENSE, params=dict(num_tokens=0)) == gdn.GDN_OK


@pytest.mark.parametrize("call", NEW)
@pytest.mark.parametrize("bad", [-2, PAGES])
def test_page_numbers_are_checked_where_the_host_has_them(call, bad):
    f = Fields()
    table = np.full((R, MAXP), -1, np.int32)
    table[1, 2] = bad
    assert call(f, _cache(f, page_table_host=table.ctypes.data), cu_seqlens_host=CU.ctypes.data) == gdn.GDN_ERR_SHAPE


@pytest.mark.parametrize("params,over,code", [
    (dict(num_q_heads=1), {}, gdn.GDN_ERR_SHAPE), (dict(rotary_dim=32), {}, gdn.GDN_ERR_SHAPE), (dict(k_stride=128), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(bounds=None), gdn.GDN_ERR_NULL), ({}, dict(bounds=FAKE + 4), gdn.GDN_ERR_SHAPE), ({}, dict(bounds="k_pages"), gdn.GDN_ERR_ALIAS),
    ({}, dict(bounds="v_pages"), gdn.GDN_ERR_ALIAS), ({}, dict(bounds="table"), gdn.GDN_ERR_ALIAS), ({}, dict(bounds="lens"), gdn.GDN_ERR_ALIAS),
])
def test_bounds_arguments(params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _bounds(f, _cache(f), params, **{**DENSE, **over}) == code


def test_two_requests_may_not_bound_one_page():
    f = Fields()
    table = np.array([[0, 1, 2, -1], [3, 1, 4, -1]], np.int32)
    lens = np.array([20, 20], np.int32)
    c = _cache(f, page_table_host=table.ctypes.data)
    assert _bounds(f, c, cu_seqlens_host=CU.ctypes.data, seq_lens_host=lens.ctypes.data) == gdn.GDN_ERR_ALIAS


@pytest.mark.parametrize("call", [_select, _sparse])
@pytest.mark.parametrize("params,over,code", [
    (dict(num_q_heads=3), {}, gdn.GDN_ERR_SHAPE), (dict(num_q_heads=0), {}, gdn.GDN_ERR_SHAPE), (dict(list_len=0), {}, gdn.GDN_ERR_SHAPE),
    (dict(list_len=-1), {}, gdn.GDN_ERR_SHAPE), (dict(list_len=(1 << 26) + 1), {}, gdn.GDN_ERR_SHAPE),
    (dict(q_stride=HQ * D - 8), {}, gdn.GDN_ERR_SHAPE), (dict(q_stride=HQ * D + 4), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(q=None), gdn.GDN_ERR_NULL), ({}, dict(pages=None), gdn.GDN_ERR_NULL), ({}, dict(q=FAKE + 4), gdn.GDN_ERR_SHAPE),
    ({}, dict(ws=None), gdn.GDN_ERR_WORKSPACE), ({}, dict(ws=FAKE + 8), gdn.GDN_ERR_WORKSPACE), ({}, dict(ws_bytes=15), gdn.GDN_ERR_WORKSPACE),
    ({}, dict(ws="q"), gdn.GDN_ERR_ALIAS), ({}, dict(ws="k_pages"), gdn.GDN_ERR_ALIAS), ({}, dict(ws="lens"), gdn.GDN_ERR_ALIAS),
    ({}, dict(ws="pages"), gdn.GDN_ERR_ALIAS), ({}, dict(ws="counts"), gdn.GDN_ERR_ALIAS),
])
def test_arguments_of_lists(call, params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert call(f, _cache(f), params, **{**DENSE, **over}) == code


@pytest.mark.parametrize("params,over,code", [
    (dict(first_pages=-1), {}, gdn.GDN_ERR_SHAPE), (dict(newest_pages=-1), {}, gdn.GDN_ERR_SHAPE),
    (dict(first_pages=2, newest_pages=2), {}, gdn.GDN_ERR_SHAPE), (dict(first_pages=(1 << 31) - 1, newest_pages=1), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(bounds=None), gdn.GDN_ERR_NULL), ({}, dict(counts=None), gdn.GDN_ERR_NULL), ({}, dict(bounds=FAKE + 4), gdn.GDN_ERR_SHAPE),
    ({}, dict(pages="q"), gdn.GDN_ERR_ALIAS), ({}, dict(pages="bounds"), gdn.GDN_ERR_ALIAS), ({}, dict(pages="counts"), gdn.GDN_ERR_ALIAS),
    ({}, dict(pages="table"), gdn.GDN_ERR_ALIAS), ({}, dict(counts="lens"), gdn.GDN_ERR_ALIAS),
    ({}, dict(ws="bounds"), gdn.GDN_ERR_ALIAS),
])
def test_select_arguments(params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _select(f, _cache(f), params, **{**DENSE, **over}) == code


@pytest.mark.parametrize("params,over,code", [
    (dict(scale=float("nan")), {}, gdn.GDN_ERR_SHAPE), (dict(scale=float("inf")), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(output=None), gdn.GDN_ERR_NULL), ({}, dict(output=FAKE + 4), gdn.GDN_ERR_SHAPE), ({}, dict(output="q"), gdn.GDN_ERR_ALIAS),
    ({}, dict(output="pages"), gdn.GDN_ERR_ALIAS), ({}, dict(output="counts"), gdn.GDN_ERR_ALIAS), ({}, dict(output="v_pages"), gdn.GDN_ERR_ALIAS),
    ({}, dict(output="ws"), gdn.GDN_ERR_ALIAS),
])
def test_sparse_arguments(params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _sparse(f, _cache(f), params, **{**DENSE, **over}) == code


@pytest.mark.parametrize("name,params", [("gdn_attn_select_workspace_bytes", gdn.GdnSelectParams(N, R, HQ, K, 1, 1, 0)),
                                         ("gdn_attn_sparse_workspace_bytes", gdn.GdnSparseParams(N, R, HQ, K, 0.0, 0))])
def test_workspace_queries(name, params):
    f, out = Fields(), ctypes.c_size_t(0)
    call = lambda p, c, o: getattr(gdn.lib(), name)(_ref(p), _ref(c), o)  # noqa: E731
    assert call(params, _cache(f), ctypes.byref(out)) == gdn.GDN_OK and out.value > 0
    assert call(None, _cache(f), ctypes.byref(out)) == gdn.GDN_ERR_NULL
    assert call(params, None, ctypes.byref(out)) == gdn.GDN_ERR_NULL
    assert call(params, _cache(f), None) == gdn.GDN_ERR_NULL
    bad = type(params)(*(getattr(params, n) for n, _ in params._fields_))
    bad.list_len = 0
    assert call(bad, _cache(f), ctypes.byref(out)) == gdn.GDN_ERR_SHAPE
    none = type(params)(*(getattr(params, n) for n, _ in params._fields_))
    none.num_tokens = none.num_reqs = 0
    assert call(none, _cache(f), ctypes.byref(out)) == gdn.GDN_OK and out.value == 0


def test_sizes_past_what_is_counted():
    f, out = Fields(), ctypes.c_size_t(0)
    huge = gdn.GdnSelectParams(1 << 30, 1, HQ, K, 1, 1, 0)                  # 2^31 lists
    assert gdn.lib().gdn_attn_select_workspace_bytes(ctypes.byref(huge), _ref(_cache(f)), ctypes.byref(out)) == gdn.GDN_ERR_SHAPE
    wide = gdn.GdnSelectParams(1 << 15, 1, HQ, K, 1, 1, 0)                  # 2^16 lists of 2^26 entries
    assert gdn.lib().gdn_attn_select_workspace_bytes(ctypes.byref(wide), _ref(_cache(f, max_pages=1 << 26)),
                                                     ctypes.byref(out)) == gdn.GDN_ERR_SHAPE
    rows = gdn.GdnSparseParams(1 << 28, 1, HQ, K, 0.0, 0)
    assert gdn.lib().gdn_attn_sparse_workspace_bytes(ctypes.byref(rows), _ref(_cache(f)), ctypes.byref(out)) == gdn.GDN_ERR_SHAPE


@pytest.mark.parametrize("cls,pack,values", [
    (gdn.GdnSelectParams, "_select_params", (7, 3, 4, 64, 1, 2, 24)), (gdn.GdnSparseParams, "_sparse_params", (9, 2, 8, 100, 0.125, 4096)),
    (gdn.GdnSelectTensors, "_select_tensors", tuple(FAKE + 64 * i for i in range(8))),
    (gdn.GdnSparseTensors, "_sparse_tensors", tuple(FAKE + 64 * i for i in range(8))),
])
def test_packed_structs_are_the_ctypes_ones(cls, pack, values):
    assert getattr(binding, pack)(*values) == bytes(cls(*values))


class _Cache:
    num_pages, num_kv_heads, page_size, head_dim, index = 5, 2, 16, 64, -1

    def __init__(self, io):
        self.io_dtype = io


def test_what_the_binding_refuses():
    torch = pytest.importorskip("torch")
    c = _Cache(torch.float16)
    binding._page_bounds(torch.zeros(5, 2, 2, 64, dtype=torch.float16), c, -1)
    for bad in (torch.zeros(5, 2, 2, 64), torch.zeros(4, 2, 2, 64, dtype=torch.float16), torch.zeros(5, 2, 64, 2, dtype=torch.float16).transpose(2, 3)):
        with pytest.raises(ValueError, match="bounds"):
            binding._page_bounds(bad, c, -1)
    i32 = torch.int32
    assert binding._page_lists(torch.zeros(3, 2, 7, dtype=i32), torch.zeros(3, dtype=i32), 3, c, -1) == 7
    assert binding._page_lists(torch.zeros(3, 2, 7, dtype=i32), None, 3, c, -1) == 7
    for bad in (torch.zeros(3, 2, 7), torch.zeros(2, 2, 7, dtype=i32), torch.zeros(3, 1, 7, dtype=i32), torch.zeros(3, 7, dtype=i32),
                torch.zeros(3, 7, 2, dtype=i32).transpose(1, 2)):
        with pytest.raises(ValueError, match="pages"):
            binding._page_lists(bad, None, 3, c, -1)
    for bad in (torch.zeros(3), torch.zeros(4, dtype=i32), torch.zeros(3, 2, dtype=i32), torch.zeros(6, dtype=i32)[::2]):
        with pytest.raises(ValueError, match="counts"):
            binding._page_lists(torch.zeros(3, 2, 7, dtype=i32), bad, 3, c, -1)
