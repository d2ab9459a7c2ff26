"""GPU parity of the 4-bit cache (GDN_CACHE_E2M1): written, read back and attended, against the
float64 oracle, called through the C ABI.

Codes and exponent bytes are compared exactly: what is quantised is the key or value in the type it
is given in, and the format says what its code is. Unused slots hold 0xff, codes and scales, so a
masked position that has any influence shows.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, oracle_attention, page_table, run_attention
from gpu_helpers import dev
from long_helpers import any_device_cache, cu_of, make_cache4, queries, transposed

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import attn_oracle as AO                 # noqa: E402
from oracle import sparse_oracle as SO               # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _empty(lens, Hk, D, page, seed=0, fill=0xa5):
    table, P = page_table(lens, page, np.random.default_rng(seed))
    arrays = {n: np.full((P, Hk, page, D // 2) if "pages" in n else (P, Hk, D // 32, page), fill, np.uint8)
              for n in ("k_pages", "v_pages", "k_scales", "v_scales")}
    t = {n: dev(a, torch) for n, a in arrays.items()}
    cache = gdn.KVCache(t["k_pages"], t["v_pages"], dev(table, torch), k_scales=t["k_scales"], v_scales=t["v_scales"])
    return cache, t, arrays, table


def _written(rows, pages, scales, table, cu, lens):
    """The pool after a write of rows [N, Hk, D]."""
    codes, s = SO.quantise(rows)
    return (AO.cache_write(SO.pack(codes), pages, table, cu, lens),
            transposed(AO.cache_write(s, transposed(scales), table, cu, lens)))


def _check_write(k, v, lens, T, page, *, seed=0, mirrors=True, dense=False, **rot):
    Hk, D = k.shape[1:]
    cache, t, a, table = _empty(lens, Hk, D, page, seed)
    cu, lens32 = cu_of(T), np.asarray(lens, np.int32)
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), cache, dev(lens32, torch), None if dense else dev(cu, torch), num_reqs=len(lens),
                     seq_lens_host=lens32 if mirrors else None, cu_seqlens_host=cu if mirrors and not dense else None, **rot)
    torch.cuda.synchronize()
    return cache, t, a, table, cu, lens32


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("order", ["sorted", "mixed"])
def test_every_fp16_value_gets_its_code(D, order):
    """All finite halves: in order, so that a block's values are near its largest, and mixed."""
    _case(f"all halves, D={D}, {order}")
    x = np.arange(1 << 16, dtype=np.uint16).view(np.float16)
    x = x[np.isfinite(x)]
    x = x[np.argsort(np.abs(x.astype(np.float64)), kind="stable")]
    rng = np.random.default_rng(3)
    if order == "mixed":
        # blocks of a few binades each, so that all codes appear
        x = np.concatenate([rng.permutation(p) for p in np.array_split(x, 40)])
    x = np.concatenate([x, np.zeros(-len(x) % (2 * D), np.float16)]).reshape(-1, 2, D)
    N = len(x)
    back = x[::-1].copy()
    _, t, a, table, cu, lens = _check_write(x, back, [N], [N], 64)
    for name, rows in (("k", x), ("v", back)):
        pages, scales = _written(rows, a[name + "_pages"], a[name + "_scales"], table, cu, lens)
        assert (t[name + "_scales"].cpu().numpy() == scales).all()
        assert (t[name + "_pages"].cpu().numpy() == pages).all()


def test_blocks_with_something_not_finite():
    _case("inf and NaN")
    x = np.random.default_rng(0).standard_normal((40, 2, 128)).astype(np.float16)
    x[3, 0, 5], x[7, 1, 127], x[9, 0, 64] = np.inf, np.nan, -np.inf
    v = x[::-1].copy()
    cache, t, a, table, cu, lens = _check_write(x, v, [40], [40], 16)
    for name, rows in (("k", x), ("v", v)):
        pages, scales = _written(rows, a[name + "_pages"], a[name + "_scales"], table, cu, lens)
        assert (t[name + "_scales"].cpu().numpy() == scales).all() and (t[name + "_pages"].cpu().numpy() == pages).all()
    out_k, out_v = (torch.empty((40, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    gdn.gdn_kv_read(out_k, out_v, cache, dev(lens, torch))
    got = out_k.cpu().numpy()
    assert np.isnan(got[3, 0, :32]).all() and np.isfinite(got[3, 0, 32:]).all() and np.isfinite(got[3, 1]).all()
    assert np.isnan(got[7, 1, 96:]).all() and np.isnan(got[9, 0, 64:96]).all()
    want = SO.dequantise(*SO.quantise(x))
    assert np.array_equal(got.astype(np.float64), want, equal_nan=True)


@pytest.mark.parametrize("lens,T,page", [([1], [1], 16), ([16], [16], 16), ([17, 1, 300], [1, 1, 33], 16), ([64, 5, 0, 65], [64, 2, 0, 1], 64),
                                         ([500, 33], [7, 7], 128), ([1030], [1030], 1024)])
@pytest.mark.parametrize("D,Hk", [(64, 1), (128, 3), (256, 2)])
def test_write_and_read(lens, T, page, D, Hk):
    _case(f"write/read lens={lens} T={T} page={page} D={D} Hk={Hk}")
    rng = np.random.default_rng(1)
    N = sum(T)
    k, v = (rng.standard_normal((N, Hk, D)) * 10.0 ** rng.integers(-6, 4, (N, Hk, 1))).astype(np.float16), \
        rng.standard_normal((N, Hk, D)).astype(np.float16)
    v[::3, :, 32:64] = 0                                     # blocks of zeros
    cache, t, a, table, cu, lens32 = _check_write(k, v, lens, T, page, dense=len(set(T)) == 1)
    for name, rows in (("k", k), ("v", v)):
        pages, scales = _written(rows, a[name + "_pages"], a[name + "_scales"], table, cu, lens)
        assert (t[name + "_pages"].cpu().numpy() == pages).all() and (t[name + "_scales"].cpu().numpy() == scales).all()
    out = [torch.full((N + 2, Hk, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    gdn.gdn_kv_read(out[0], out[1], cache, dev(lens32, torch), dev(cu, torch))          # two tokens behind the last request
    for o, rows in zip(out, (k, v)):
        got = o.cpu().numpy()
        assert np.array_equal(got[:N].astype(np.float64), SO.dequantise(*SO.quantise(rows))) and (got[N:] == 9).all()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 48), (128, 128), (256, 64), (256, 240), (256, 256)])
def test_rotated_keys_are_the_rotations(layout, D, rot):
    """The bytes of gdn_rope_forward followed by a write without a rotation, strided rows, in place and not."""
    _case(f"rotated layout={layout} D={D} rot={rot}")
    rng = np.random.default_rng(rot)
    T, lens, Hq, Hk, page = [5, 1, 20], [9, 301, 20], 4, 2, 16
    N, cu, lens32 = sum(T), cu_of(T), np.asarray(lens, np.int32)
    wide = dev(rng.standard_normal((N, (Hq + 2 * Hk) * D)).astype(np.float16), torch)
    q, k, v = (wide[:, a * D:b * D].view(N, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    freq = dev(AO.frequencies(rot), torch)
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(T, lens)]).astype(np.int32)
    qr, kr = (torch.empty((N, h, D), dtype=torch.float16, device="cuda") for h in (Hq, Hk))
    gdn.gdn_rope_forward(q, k, dev(pos, torch), freq, qr, kr, rope_layout=layout, rope_factor=1.25)
    pools = []
    for rotate in (True, False):
        cache, t, _, _ = _empty(lens, Hk, D, page)
        kw = dict(q=q, q_out=torch.empty_like(qr), inv_freq=freq, rope_layout=layout, rope_factor=1.25) if rotate else {}
        gdn.gdn_kv_write(k if rotate else kr, v, cache, dev(lens32, torch), dev(cu, torch), cu_seqlens_host=cu, seq_lens_host=lens32, **kw)
        torch.cuda.synchronize()
        if rotate:
            assert torch.equal(kw["q_out"], qr)
        pools.append(t)
    for name in pools[0]:
        assert torch.equal(pools[0][name], pools[1][name]), name
    pages, _ = _written(kr.cpu().numpy(), np.full(pools[0]["k_pages"].shape, 0xa5, np.uint8), pools[0]["k_scales"].cpu().numpy(),
                        page_table(lens, page, np.random.default_rng(0))[0], cu, lens)
    assert (pools[0]["k_pages"].cpu().numpy() == pages).all()


def test_pages_that_are_not_there():
    """Writes to no page are dropped, reads give zeros, a padded batch's last tokens are left alone."""
    _case("no page")
    D, Hk, page, lens, T = 128, 2, 16, [40, 20], [40, 4]
    rng = np.random.default_rng(0)
    N = sum(T) + 3
    k, v = (rng.standard_normal((N, Hk, D)).astype(np.float16) for _ in range(2))
    cache, t, a, table = _empty(lens, Hk, D, page)
    table[0, 1], table[1, 1] = -1, 1 << 20
    cache = gdn.KVCache(t["k_pages"], t["v_pages"], dev(table, torch), k_scales=t["k_scales"], v_scales=t["v_scales"])
    cu, lens32 = cu_of(T), np.asarray(lens, np.int32)
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), cache, dev(lens32, torch), dev(cu, torch))
    for name, rows in (("k", k), ("v", v)):
        pages, scales = _written(rows[:sum(T)], a[name + "_pages"], a[name + "_scales"], table, cu, lens)
        assert (t[name + "_pages"].cpu().numpy() == pages).all() and (t[name + "_scales"].cpu().numpy() == scales).all()
    out = [torch.full((N, Hk, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    gdn.gdn_kv_read(out[0], out[1], cache, dev(lens32, torch), dev(cu, torch))
    got = out[1].cpu().numpy()
    want = SO.dequantise(*SO.quantise(v))
    want[16:32], want[40:44] = 0, 0
    assert np.array_equal(got[:44].astype(np.float64), want[:44]) and (got[44:] == 9).all()


# ------------------------------------------------------------------------------------------------ attention
def _check(lens, T, *, Hk, G, D, page, seed=0, dense=False, mirrors=True, scale=1.0, **kw):
    what = f"lens={lens[:8]} T={T[:8]} Hk={Hk} G={G} D={D} page={page} {kw}"
    _case(what)
    c = make_cache4(lens, Hk=Hk, D=D, page=page, seed=seed, scale=scale)
    cu = cu_of(T)
    q = queries(cu[-1], Hk * G, D, "f16", seed)
    want, tol = oracle_attention(c, q, cu, **kw)
    got = run_attention(c, q, cu, torch, gdn, dense=dense, mirrors=mirrors, cache=any_device_cache(c, torch, gdn), **kw)
    assert_within(got, want, tol, what)
    return got


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 6, 16, 20, 33])
def test_decode_heads(D, G):
    _check([1, 15, 16, 17, 100, 333], [1] * 6, Hk=2, G=G, D=D, page=16, dense=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("n", [31, 32, 33, 127, 128, 129, 700])
def test_lengths(D, page, n):
    _check([n], [1], Hk=1, G=4, D=D, page=page)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_drafts_windows_and_empty_rows(D):
    _check([50, 3, 400, 7], [5, 3, 1, 0], Hk=2, G=6, D=D, page=32)
    _check([500, 90, 33], [4, 4, 4], Hk=1, G=6, D=D, page=16, window=40, dense=True)
    _check([5000], [3], Hk=2, G=4, D=D, page=64, window=1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 512])
@pytest.mark.parametrize("window", [7, 33, 100, 1000])
def test_windows_end_inside_pages_and_tiles(D, page, window):
    _check([700, 33, 1, 90], [3, 1, 1, 5], Hk=2, G=4, D=D, page=page, window=window, seed=window)


@pytest.mark.parametrize("D,Hk,G", [(64, 1, 4), (128, 2, 8), (256, 1, 6)])
@pytest.mark.parametrize("mirrors", [True, False])
def test_split_lengths(D, Hk, G, mirrors):
    """Requests whose length several workgroups share, joined by a second launch; several row tiles and segments."""
    _check([9000, 77, 4097], [1, 1, 1], Hk=Hk, G=G, D=D, page=64, dense=True, mirrors=mirrors)
    _check([6000, 2050], [5, 2], Hk=Hk, G=G, D=D, page=128, mirrors=mirrors)


@pytest.mark.parametrize("D,Hk", [(64, 16), (128, 12), (256, 8)])
@pytest.mark.parametrize("page", [16, 64])
def test_split_of_many_segments(D, Hk, page):
    """As many units as make a segment's fixed part count in the split: a share may begin, or lie, within one."""
    lens = [6000, 4000, 2500, 2000, 1, 129, 0, 1500, 1300]
    _check(lens, [1, 1, 1, 1, 1, 1, 0, 1, 1], Hk=Hk, G=2, D=D, page=page)
    _check(lens[::-1], [1, 1, 0, 1, 1, 1, 1, 1, 1], Hk=Hk, G=2, D=D, page=page, window=5500, seed=1)


@pytest.mark.parametrize("D,Hk", [(64, 8), (128, 8), (256, 4)])
def test_split_of_many_segments_of_drafts(D, Hk):
    lens = [6000, 4000, 2500, 2000, 1, 129, 0, 1500, 1300]
    _check(lens, [4, 3, 1, 4, 1, 4, 0, 2, 4], Hk=Hk, G=6, D=D, page=64)
    _check(lens, [9, 3, 1, 4, 1, 4, 0, 2, 8], Hk=Hk, G=6, D=D, page=32, seed=1)     # two segments of 32 rows


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_short_requests_share_workgroups(D):
    rng = np.random.default_rng(D)
    lens = rng.integers(1, 120, 300).tolist()
    _check(lens, [1] * 300, Hk=4, G=2, D=D, page=16, dense=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -8, 3000.0])
def test_small_and_large_values(D, scale):
    """Rows near fp16's smallest and largest values: subnormal halves on the way to the matrix cores keep their digits."""
    what = f"scale={scale} D={D}"
    _case(what)
    c = make_cache4([300, 40], Hk=1, D=D, page=16, seed=4, scale=scale)
    q = queries(2, 4, D, "f16", 5, scale=min(1.0, 1.0 / scale))
    kw = dict(scale=D ** -0.5 if scale < 1000 else D ** -0.5 / 16)
    want, tol = oracle_attention(c, q, [0, 1, 2], **kw)
    assert np.abs(want).max() > 0
    got = run_attention(c, q, [0, 1, 2], torch, gdn, cache=any_device_cache(c, torch, gdn), **kw)
    assert_within(got, want, tol, what)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_blocks_show_where_they_are_attended_only(D):
    _case(f"NaN blocks D={D}")
    lens, T, Hk, G, page = [40, 300], [3, 2], 1, 4, 16
    c = make_cache4(lens, Hk=Hk, D=D, page=page, seed=8)
    cu, q = cu_of(T), queries(5, 4, D, "f16", 9)
    clean = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn))
    # the value of request 0's last position, which only its third token attends; of request 1's position 7, under a window
    for r, pos in ((0, 39), (1, 7)):
        page_no, slot = AO.places(c["table"], page, c["P"], r, [pos])
        c["v_scales"][page_no[0], 0, 1, slot[0]] = 255
    got = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn), window=250)
    full = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn))
    assert np.array_equal(full[:2], clean[:2]) and np.isfinite(got[:2]).all()
    assert np.isnan(full[2, :, 32:64]).all() and np.isfinite(full[2, :, :32]).all() and np.isfinite(full[2, :, 64:]).all()
    assert np.isfinite(got[3:]).all()                        # masked by the window
    assert np.isnan(full[3:, :, 32:64]).all() and np.isfinite(full[3:, :, :32]).all()
    # a NaN key: the whole row, and only where it is attended
    page_no, slot = AO.places(c["table"], page, c["P"], 0, [38])
    c["k_scales"][page_no[0], 0, 0, slot[0]] = 255
    bad = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn))
    assert np.array_equal(bad[0], clean[0]) and np.isnan(bad[1]).all() and np.isnan(bad[2]).all()


def test_pages_left_out():
    _case("missing pages")
    c = make_cache4([100, 64, 20], Hk=2, D=128, page=16, seed=1)
    table = c["table"].copy()
    table[0, 2], table[1, :], table[2, 0] = -1, -1, c["P"]
    c["table"] = table
    q, cu = queries(4, 8, 128, "f16", 3), cu_of([2, 1, 1])
    want, tol = oracle_attention(c, q, cu)
    got = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn))
    assert_within(got, want, tol, "missing pages")
    assert not got[2].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_strided_q_and_the_ends_of_int32(D):
    """q as a slice of a projection's output; lengths at the ends of int32, of which the table holds what it holds."""
    _case(f"strided q, int32 lengths D={D}")
    c = make_cache4([64, 64], Hk=2, D=D, page=16, seed=1)
    c["table"] = c["table"][:, :4]
    q = queries(2, 8, D, "f16", 2)
    wide = torch.zeros((2, 8 * D + 64), dtype=torch.float16, device="cuda")
    wide[:, :8 * D] = dev(q, torch).view(2, -1)
    cache = any_device_cache(c, torch, gdn)
    ws = torch.empty(gdn.gdn_attn_workspace_bytes(2, 2, 8, cache), dtype=torch.uint8, device="cuda")
    out = torch.full((2, 8, D), -7.75, dtype=torch.float16, device="cuda")
    for lens in ([64, 64], [(1 << 31) - 1, -(1 << 31)]):
        c["lens"] = np.asarray(lens, np.int32)
        gdn.gdn_attn_forward(wide[:, :8 * D].view(2, 8, D), cache, dev(c["lens"], torch), None, out, workspace=ws)
        torch.cuda.synchronize()
        want, tol = oracle_attention({**c, "lens": np.clip(np.asarray(lens, np.int64), 0, 64)}, q, [0, 1, 2])
        if lens[1] < 0:
            want[1], tol[1] = 0, 0
        assert_within(out.double().cpu().numpy(), want, tol, f"lens {lens}")
