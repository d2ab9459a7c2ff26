"""Host-side checks of the attention layer's entry points (include/gdn_attn.h):
every bad argument is rejected on the host with the documented status before
anything is enqueued, and the rotary frequencies against their formulas.

As in test_abi_host.py, no call here launches a kernel: each one is built to
fail a host check (the fake device addresses are never dereferenced), or has no
work, and the module runs only where no GPU is visible.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import pytest

import gateddeltanet_recurrence_amd as gdn


def _gpu_visible() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0        # counts devices without initialising HIP
    except Exception:
        return False


pytestmark = [
    pytest.mark.skipif(not os.path.exists(gdn.library_path()),
                       reason="libgdn.so not built (run the build first)"),
    pytest.mark.skipif(_gpu_visible(), reason="fake-pointer host checks run only without a GPU"),
]

FAKE = 1 << 40          # 16-byte aligned, never dereferenced
N, R, HQ, HK, D, PAGES, PAGE, MAXP = 8, 2, 4, 2, 64, 10, 16, 4
CU_BAD = np.array([0, 3, 7], np.int32)     # cu[R] != N: a call that passes every other check still ends here


class Fields:
    """Fake, disjoint device addresses of one call."""

    def __init__(self, io=2, e4m3=False):
        self.at = FAKE
        eb = 1 if e4m3 else io
        rows = PAGES * HK * PAGE
        for name, size in dict(k_pages=rows * D * eb, v_pages=rows * D * eb, k_scales=rows, v_scales=rows,
                               table=R * MAXP * 4, q=N * HQ * D * io, k=N * HK * D * io, v=N * HK * D * io,
                               q_out=N * HQ * D * io, k_out=N * HK * D * io, cu=(R + 1) * 4, lens=R * 4,
                               positions=N * 4, inv_freq=16 * 8, output=N * HQ * D * io, ws=1 << 24).items():
            setattr(self, name, self.at)
            self.at += (size + 4095) // 4096 * 4096 + 4096


def _cache(f, *, io=gdn.GDN_F16, e4m3=False, **over):
    c = gdn.GdnKvCache(f.k_pages, f.v_pages, f.k_scales if e4m3 else None, f.v_scales if e4m3 else None, f.table,
                       None, PAGES, PAGE, MAXP, HK, D, io, gdn.CACHE_E4M3 if e4m3 else gdn.CACHE_IO)
    for name, v in over.items():
        setattr(c, name, v)
    return c


def _write(f, cache, params=None, **over):
    p = gdn.GdnKvParams(N, R, HQ, 32, gdn.ROPE_HALF, 1.0, 0, 0, 0)
    for name, v in (params or {}).items():
        setattr(p, name, v)
    t = gdn.GdnKvTensors(f.k, f.v, f.cu, CU_BAD.ctypes.data, f.lens, None, f.q, f.q_out, None, f.inv_freq)
    for name, v in over.items():
        setattr(t, name, v)
    return gdn.lib().gdn_kv_write(ctypes.byref(p), ctypes.byref(t), ctypes.byref(cache) if cache else None, None)


def _read(f, cache, params=None, **over):
    p = gdn.GdnKvParams(N, R, 0, 0, 0, 0.0, 0, 0, 0)
    for name, v in (params or {}).items():
        setattr(p, name, v)
    t = gdn.GdnKvTensors(f.k, f.v, f.cu, CU_BAD.ctypes.data, f.lens, None, None, None, None, None)
    for name, v in over.items():
        setattr(t, name, v)
    return gdn.lib().gdn_kv_read(ctypes.byref(p), ctypes.byref(t), ctypes.byref(cache) if cache else None, None)


def _attn(f, cache, params=None, ws_bytes=1 << 24, **over):
    p = gdn.GdnAttnParams(N, R, HQ, 0.0, 0, 0)
    for name, v in (params or {}).items():
        setattr(p, name, v)
    ws = over.pop("ws", f.ws)
    t = gdn.GdnAttnTensors(f.q, f.cu, CU_BAD.ctypes.data, f.lens, None, f.output)
    for name, v in over.items():
        setattr(t, name, v)
    return gdn.lib().gdn_attn_forward(ctypes.byref(p), ctypes.byref(t), ctypes.byref(cache) if cache else None, ws,
                                      ws_bytes, None)


def _rope(f, params=None, **over):
    p = gdn.GdnRopeParams(N, HQ, HK, D, gdn.GDN_F16, 32, gdn.ROPE_HALF, 1.0, 0, 0)
    for name, v in (params or {}).items():
        setattr(p, name, v)
    t = gdn.GdnRopeTensors(f.q, f.k, f.positions, f.inv_freq, f.q_out, f.k_out)
    for name, v in over.items():
        setattr(t, name, v)
    return gdn.lib().gdn_rope_forward(ctypes.byref(p), ctypes.byref(t), None)


ALL = [_write, _read, _attn]


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("field,value,code", [
    ("io_dtype", gdn.GDN_BF16, gdn.GDN_ERR_DTYPE),
    ("format", 2, gdn.GDN_ERR_DTYPE),
    ("num_pages", 0, gdn.GDN_ERR_SHAPE),
    ("max_pages", 0, gdn.GDN_ERR_SHAPE),
    ("num_kv_heads", 0, gdn.GDN_ERR_SHAPE),
    ("page_size", 8, gdn.GDN_ERR_SHAPE),
    ("page_size", 48, gdn.GDN_ERR_SHAPE),
    ("page_size", 2048, gdn.GDN_ERR_SHAPE),
    ("head_dim", 96, gdn.GDN_ERR_SHAPE),
    ("max_pages", 1 << 27, gdn.GDN_ERR_SHAPE),         # more than 2^30 positions
    ("k_pages", None, gdn.GDN_ERR_NULL),
    ("v_pages", None, gdn.GDN_ERR_NULL),
    ("page_table", None, gdn.GDN_ERR_NULL),
    ("k_pages", FAKE + 8, gdn.GDN_ERR_SHAPE),          # alignment
    ("k_scales", FAKE, gdn.GDN_ERR_SHAPE),             # scales without the 8-bit format
])
def test_cache_validation(call, field, value, code):
    f = Fields()
    assert call(f, _cache(f, **{field: value})) == code


@pytest.mark.parametrize("call", ALL)
def test_cache_is_required(call):
    assert call(Fields(), None) == gdn.GDN_ERR_NULL


@pytest.mark.parametrize("call", ALL)
def test_e4m3_needs_scales_and_fp16(call):
    f = Fields(e4m3=True)
    assert call(f, _cache(f, e4m3=True, k_scales=None)) == gdn.GDN_ERR_NULL
    assert call(f, _cache(f, e4m3=True, io_dtype=gdn.GDN_F32)) == gdn.GDN_ERR_DTYPE
    assert call(f, _cache(f, e4m3=True, v_scales=f.v_scales + 8)) == gdn.GDN_ERR_SHAPE       # alignment


@pytest.mark.parametrize("call", ALL)
def test_row_validation(call):
    f = Fields()
    c = _cache(f)
    assert call(f, c) == gdn.GDN_ERR_SHAPE                                  # the malformed mirror itself
    good = np.array([0, 3, 8], np.int32)
    for lens in ([2, 8], [3, 4], [3, MAXP * PAGE + 1]):                     # fewer than the new tokens; past the table
        assert call(f, c, cu_seqlens_host=good.ctypes.data,
                    seq_lens_host=np.array(lens, np.int32).ctypes.data) == gdn.GDN_ERR_CAPACITY
    assert call(f, c, cu_seqlens=None) == gdn.GDN_ERR_SHAPE                 # a mirror without its array
    assert call(f, c, cu_seqlens=None, cu_seqlens_host=None, params=dict(num_tokens=7)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, cu_seqlens_host=good.ctypes.data, seq_lens=None) == gdn.GDN_ERR_NULL
    assert call(f, c, params=dict(num_tokens=-1)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, params=dict(num_reqs=-1)) == gdn.GDN_ERR_SHAPE
    assert call(f, c, params=dict(num_reqs=0)) == gdn.GDN_ERR_SHAPE         # tokens without a request
    assert call(f, c, params=dict(num_reqs=0, num_tokens=0)) == gdn.GDN_OK  # nothing to do, nothing launched


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("bad", [-2, PAGES])
def test_page_numbers_are_checked_where_the_host_has_them(call, bad):
    f = Fields()
    table = np.full((R, MAXP), -1, np.int32)
    table[1, 2] = bad
    good = np.array([0, 3, 8], np.int32)
    c = _cache(f, page_table_host=table.ctypes.data)
    assert call(f, c, cu_seqlens_host=good.ctypes.data) == gdn.GDN_ERR_SHAPE


def test_two_requests_may_not_write_one_page():
    f = Fields()
    table = np.array([[0, 1, 2, -1], [3, 1, 4, -1]], np.int32)              # page 1 shared
    good, lens = np.array([0, 3, 8], np.int32), np.array([20, 20], np.int32)
    c = _cache(f, page_table_host=table.ctypes.data)
    over = dict(cu_seqlens_host=good.ctypes.data, seq_lens_host=lens.ctypes.data)
    assert _write(f, c, **over) == gdn.GDN_ERR_ALIAS                        # positions 17.. and 15.. : entry 1 of both


@pytest.mark.parametrize("field,value,code", [
    ("rotary_dim", 24, gdn.GDN_ERR_SHAPE), ("rotary_dim", 80, gdn.GDN_ERR_SHAPE), ("rotary_dim", -16, gdn.GDN_ERR_SHAPE),
    ("rotary_dim", 0, gdn.GDN_ERR_SHAPE),                                   # q without a rotation
    ("rope_layout", 2, gdn.GDN_ERR_RULE), ("rope_factor", float("inf"), gdn.GDN_ERR_RULE),
    ("num_q_heads", -1, gdn.GDN_ERR_SHAPE),
    ("q_stride", HQ * D - 8, gdn.GDN_ERR_SHAPE), ("k_stride", HK * D + 4, gdn.GDN_ERR_SHAPE),
    ("v_stride", -8, gdn.GDN_ERR_SHAPE),
])
def test_write_params(field, value, code):
    f = Fields()
    assert _write(f, _cache(f), params={field: value}) == code


def _aliases(f):
    return dict(cu_seqlens=None, cu_seqlens_host=None)


@pytest.mark.parametrize("over,code", [
    (dict(k=None), gdn.GDN_ERR_NULL), (dict(v=None), gdn.GDN_ERR_NULL), (dict(inv_freq=None), gdn.GDN_ERR_NULL),
    (dict(q=None), gdn.GDN_ERR_NULL), (dict(q_out=None), gdn.GDN_ERR_NULL),
    (dict(k=FAKE + 4), gdn.GDN_ERR_SHAPE),
    (dict(k="k_pages"), gdn.GDN_ERR_ALIAS), (dict(v="v_pages"), gdn.GDN_ERR_ALIAS),
    (dict(q="k_pages"), gdn.GDN_ERR_ALIAS), (dict(q_out="table"), gdn.GDN_ERR_ALIAS),
    (dict(q_out="k"), gdn.GDN_ERR_ALIAS), (dict(q_out="lens"), gdn.GDN_ERR_ALIAS),
    (dict(positions="k_pages"), gdn.GDN_ERR_ALIAS), (dict(inv_freq="q_out"), gdn.GDN_ERR_ALIAS),
])
def test_write_tensors(over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _write(f, _cache(f), **{**_aliases(f), **over}) == code


def test_pools_may_not_overlap():
    f = Fields()
    assert _write(f, _cache(f, v_pages=f.k_pages), **_aliases(f)) == gdn.GDN_ERR_ALIAS


@pytest.mark.parametrize("over,code", [
    (dict(k=None), gdn.GDN_ERR_NULL), (dict(v=None), gdn.GDN_ERR_NULL),
    (dict(k="v"), gdn.GDN_ERR_ALIAS), (dict(k="k_pages"), gdn.GDN_ERR_ALIAS), (dict(v="table"), gdn.GDN_ERR_ALIAS),
    (dict(v="lens"), gdn.GDN_ERR_ALIAS), (dict(v=FAKE + 4), gdn.GDN_ERR_SHAPE),
])
def test_read_tensors(over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _read(f, _cache(f), **{**_aliases(f), **over}) == code


@pytest.mark.parametrize("field,value", [("num_q_heads", 4), ("rotary_dim", 32), ("k_stride", 1024)])
def test_read_takes_no_rotation_or_strides(field, value):
    f = Fields()
    assert _read(f, _cache(f), params={field: value}) == gdn.GDN_ERR_SHAPE


@pytest.mark.parametrize("params,over,code", [
    (dict(num_q_heads=3), {}, gdn.GDN_ERR_SHAPE), (dict(num_q_heads=0), {}, gdn.GDN_ERR_SHAPE),
    (dict(window=-1), {}, gdn.GDN_ERR_SHAPE), (dict(scale=float("nan")), {}, gdn.GDN_ERR_SHAPE),
    (dict(q_stride=HQ * D + 4), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(q=None), gdn.GDN_ERR_NULL), ({}, dict(output=None), gdn.GDN_ERR_NULL),
    ({}, dict(q=FAKE + 4), gdn.GDN_ERR_SHAPE),
    ({}, dict(output="q"), gdn.GDN_ERR_ALIAS), ({}, dict(output="v_pages"), gdn.GDN_ERR_ALIAS),
    ({}, dict(output="table"), gdn.GDN_ERR_ALIAS), ({}, dict(output="lens"), gdn.GDN_ERR_ALIAS),
])
def test_attention_arguments(params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _attn(f, _cache(f), params, **{**_aliases(f), **over}) == code


@pytest.mark.parametrize("params,over,code", [
    (dict(layout=2), {}, gdn.GDN_ERR_RULE), (dict(factor=float("nan")), {}, gdn.GDN_ERR_RULE),
    (dict(io_dtype=gdn.GDN_BF16), {}, gdn.GDN_ERR_DTYPE), (dict(head_dim=80), {}, gdn.GDN_ERR_SHAPE),
    (dict(rotary_dim=0), {}, gdn.GDN_ERR_SHAPE), (dict(rotary_dim=72), {}, gdn.GDN_ERR_SHAPE),
    (dict(num_tokens=-1), {}, gdn.GDN_ERR_SHAPE), (dict(num_k_heads=-1), {}, gdn.GDN_ERR_SHAPE),
    (dict(q_stride=8), {}, gdn.GDN_ERR_SHAPE),
    ({}, dict(q=None), gdn.GDN_ERR_NULL), ({}, dict(k_out=None), gdn.GDN_ERR_NULL),
    ({}, dict(positions=None), gdn.GDN_ERR_NULL), ({}, dict(inv_freq=None), gdn.GDN_ERR_NULL),
    ({}, dict(q=FAKE + 2), gdn.GDN_ERR_SHAPE),
    ({}, dict(q_out="k"), gdn.GDN_ERR_ALIAS), ({}, dict(k_out="q"), gdn.GDN_ERR_ALIAS),
    ({}, dict(q_out="k_out"), gdn.GDN_ERR_ALIAS), ({}, dict(q_out="positions"), gdn.GDN_ERR_ALIAS),
])
def test_rope_arguments(params, over, code):
    f = Fields()
    over = {n: getattr(f, v) if isinstance(v, str) else v for n, v in over.items()}
    assert _rope(f, params, **over) == code


def test_rope_without_work():
    f = Fields()
    assert _rope(f, dict(num_tokens=0)) == gdn.GDN_OK
    assert _rope(f, dict(num_q_heads=0, num_k_heads=0)) == gdn.GDN_OK


def test_rows_side_by_side_in_one_buffer_do_not_alias():
    """q in place beside k and v in one projection's output: refused only where they touch."""
    f = Fields()
    row = (HQ + 2 * HK) * D
    base = f.ws
    over = dict(q=base, q_out=base, k=base + HQ * D * 2, v=base + (HQ + HK) * D * 2)
    p = dict(q_stride=row, k_stride=row, v_stride=row)
    # the malformed mirror is what ends the call once the overlap rules are passed... they come later, so a
    # page that two requests write ends it instead
    table = np.array([[0, 1, 2, -1], [3, 1, 4, -1]], np.int32)
    good, lens = np.array([0, 3, 8], np.int32), np.array([20, 20], np.int32)
    c = _cache(f, page_table_host=table.ctypes.data)
    rows = dict(cu_seqlens_host=good.ctypes.data)
    assert _write(f, c, p, **{**over, **rows, "seq_lens_host": lens.ctypes.data}) == gdn.GDN_ERR_ALIAS
    over["k"] = base + HQ * D * 2 - 16
    assert _write(f, _cache(f), p, **{**over, **rows}) == gdn.GDN_ERR_ALIAS


def test_workspace_query():
    f = Fields()
    p, out = gdn.GdnAttnParams(N, R, HQ, 0.0, 0, 0), ctypes.c_size_t(0)
    call = lambda p, c, o: gdn.lib().gdn_attn_workspace_bytes(p and ctypes.byref(p), c and ctypes.byref(c), o)  # noqa: E731
    assert call(p, _cache(f), ctypes.byref(out)) == gdn.GDN_OK
    assert call(None, _cache(f), ctypes.byref(out)) == gdn.GDN_ERR_NULL
    assert call(p, None, ctypes.byref(out)) == gdn.GDN_ERR_NULL
    assert call(p, _cache(f), None) == gdn.GDN_ERR_NULL
    assert call(gdn.GdnAttnParams(N, R, 3, 0.0, 0, 0), _cache(f), ctypes.byref(out)) == gdn.GDN_ERR_SHAPE


# ------------------------------------------------------------- frequencies
def test_frequencies_plain_linear_ntk():
    i = np.arange(32)
    base = 1e6 ** (-2.0 * i / 64)
    f, m = gdn.gdn_rope_frequencies(64, base=1e6)
    np.testing.assert_allclose(f, base, rtol=1e-14)
    assert m == 1.0
    f, m = gdn.gdn_rope_frequencies(64, base=1e6, scaling=gdn.ROPE_SCALING_LINEAR, scale=8.0)
    np.testing.assert_allclose(f, base / 8, rtol=1e-14)
    f, m = gdn.gdn_rope_frequencies(64, base=1e6, scaling=gdn.ROPE_SCALING_NTK, scale=8.0)
    np.testing.assert_allclose(f, (1e6 * 8 ** (64 / 62)) ** (-2.0 * i / 64), rtol=1e-13)
    # what the changed base is for: the slowest pair is interpolated in full, the fastest not at all
    assert f[0] == 1.0 and math.isclose(f[31], base[31] / 8, rel_tol=1e-12) and m == 1.0


def test_frequencies_yarn():
    r, base, s, n = 128, 10000.0, 4.0, 4096.0
    f, m = gdn.gdn_rope_frequencies(r, base=base, scaling=gdn.ROPE_SCALING_YARN, scale=s, trained_length=n)
    plain = base ** (-2.0 * np.arange(r // 2) / r)
    turns = n * plain / (2 * math.pi)                    # rotations of a pair within the trained length
    assert np.allclose(f[turns > 33], plain[turns > 33], rtol=1e-13)        # fast pairs as they are (ramp starts at 32)
    assert np.allclose(f[turns < 0.9], plain[turns < 0.9] / s, rtol=1e-13)  # slow ones interpolated
    w = (plain - f) / (plain - plain / s)
    assert np.all(np.diff(w) > -1e-12) and np.any((w > 0.01) & (w < 0.99))
    assert math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-7)
    assert gdn.gdn_rope_frequencies(r, scaling=gdn.ROPE_SCALING_YARN, scale=1.0, trained_length=n)[1] == 1.0


@pytest.mark.parametrize("kw,code", [
    (dict(scaling=4), gdn.GDN_ERR_RULE), (dict(scaling=-1), gdn.GDN_ERR_RULE),
    (dict(rotary_dim=0), gdn.GDN_ERR_SHAPE), (dict(rotary_dim=7), gdn.GDN_ERR_SHAPE),
    (dict(base=1.0), gdn.GDN_ERR_SHAPE), (dict(base=float("nan")), gdn.GDN_ERR_SHAPE),
    (dict(scaling=gdn.ROPE_SCALING_LINEAR, scale=0.0), gdn.GDN_ERR_SHAPE),
    (dict(scaling=gdn.ROPE_SCALING_LINEAR, scale=float("inf")), gdn.GDN_ERR_SHAPE),
    (dict(scaling=gdn.ROPE_SCALING_NTK, scale=2.0, rotary_dim=2), gdn.GDN_ERR_SHAPE),
    (dict(scaling=gdn.ROPE_SCALING_YARN, scale=2.0), gdn.GDN_ERR_SHAPE),
])
def test_frequency_refusals(kw, code):
    kw = {"rotary_dim": 64, **kw}
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_rope_frequencies(kw.pop("rotary_dim"), **kw)
    assert e.value.status == code


@pytest.mark.parametrize("cls,pack,values", [
    (gdn.GdnRopeParams, "_rope_params", (7, 4, 2, 64, 1, 32, 1, 1.25, 256, 128)),
    (gdn.GdnRopeTensors, "_rope_tensors", (FAKE, FAKE + 16, 3 << 33, 0, 5, 6)),
    (gdn.GdnKvParams, "_kv_params", (7, 3, 4, 64, 1, 0.5, 8, 16, 24)),
    (gdn.GdnKvTensors, "_kv_tensors", tuple(FAKE + 64 * i for i in range(10))),
    (gdn.GdnAttnParams, "_attn_params", (9, 2, 8, 0.125, 100, 4096)),
    (gdn.GdnAttnTensors, "_attn_tensors", (FAKE, 0, 0, FAKE + 32, 0, FAKE + 64)),
])
def test_packed_structs_are_the_ctypes_ones(cls, pack, values):
    from gateddeltanet_recurrence_amd import binding
    assert getattr(binding, pack)(*values) == bytes(cls(*values))
