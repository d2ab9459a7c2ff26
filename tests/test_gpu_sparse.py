"""GPU parity of sparse attention (gdn_kv_bounds, gdn_attn_select, gdn_attn_sparse_forward) against
the float64 oracle, called through the C ABI.

Bounds are values of the I/O type and compared exactly, as are the selections: the scores are summed
in 64 bits, and the inputs' last selected and first left out scores are 1e-12 of their size apart or
equal. Attention's tolerance is the oracle's bound plus half a step of the I/O type.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, half_step, io_np, run_attention
from gpu_helpers import dev
from long_helpers import FORMATS, any_cache, any_device_cache, cu_of, queries, run_select, run_sparse

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


# --------------------------------------------------------------------------------------------------- bounds
def _run_bounds(c, T, old, *, dense=False, mirrors=True, N=None):
    cu = cu_of(T)
    d = dev(old, torch)
    gdn.gdn_kv_bounds(d, any_device_cache(c, torch, gdn), dev(c["lens"], torch), None if dense else dev(cu, torch),
                      num_tokens=int(cu[-1]) if N is None else N, num_reqs=len(T),
                      cu_seqlens_host=cu if mirrors and not dense else None, seq_lens_host=c["lens"] if mirrors else None)
    torch.cuda.synchronize()
    return d.cpu().numpy()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,T,page", [([1], [1], 16), ([16, 17, 33, 700], [1, 1, 1, 1], 16), ([100, 64, 65, 9], [5, 1, 65, 0], 64),
                                         ([300, 40], [300, 3], 32), ([1030], [700], 1024)])
def test_bounds(fmt, D, lens, T, page):
    _case(f"bounds {fmt} D={D} lens={lens} T={T} page={page}")
    c = any_cache(lens, fmt=fmt, Hk=2, D=D, page=page, seed=D)
    old = queries(c["P"] * 2, 2, D, fmt, 3).reshape(c["P"], 2, 2, D)
    want = SO.bounds(c["k"], c["table"], cu_of(T), lens, old)
    got = _run_bounds(c, T, old, dense=len(set(T)) == 1, mirrors=page != 64)
    assert np.array_equal(got.astype(np.float64), want)


def test_bounds_of_prompts_of_many_tokens():
    """More than 4,096 tokens: a workgroup looks at 16 of them; requests end inside."""
    lens, T = [3000, 1, 2, 1, 1500, 40, 7, 5], [2990, 1, 2, 1, 1500, 37, 7, 5]
    _case(f"bounds lens={lens} T={T}")
    for page in (16, 64):
        c = any_cache(lens, fmt="f16", Hk=3, D=64, page=page, seed=1)
        old = np.zeros((c["P"], 3, 2, 64), np.float16)
        want = SO.bounds(c["k"], c["table"], cu_of(T), lens, old)
        assert np.array_equal(_run_bounds(c, T, old).astype(np.float64), want)
        assert np.array_equal(_run_bounds(c, T, old, N=4800, mirrors=False).astype(np.float64), want)    # a padded batch


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bounds_of_many_pages(fmt, D):
    """Enough short pages for a wave each."""
    lens, T = [1500, 3, 1, 900, 40], [1500, 2, 1, 890, 17]
    _case(f"bounds of many pages {fmt} D={D}")
    for page, Hk in ((16, 8), (32, 16)):
        c = any_cache(lens, fmt=fmt, Hk=Hk, D=D, page=page, seed=1)
        old = queries(c["P"] * Hk, 2, D, fmt, 3).reshape(c["P"], Hk, 2, D)
        want = SO.bounds(c["k"], c["table"], cu_of(T), lens, old)
        assert np.array_equal(_run_bounds(c, T, old).astype(np.float64), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_bounds_of_every_code(fmt):
    """Every code beside every exponent byte that a cache holds, one key a page: what gdn_kv_read gives for it."""
    _case(f"bounds of every code {fmt}")
    scales = np.array([0, *range(95, 136)] if fmt == "e4m3" else [0, *range(101, 141), 255], np.uint8)
    R, D = len(scales), 256
    c = any_cache([1] * R, fmt=fmt, Hk=1, D=D, page=16, seed=0)
    page = c["table"][:, 0]
    codes = np.arange(256, dtype=np.uint8) if fmt == "e4m3" else np.arange(128, dtype=np.uint8) * 2 + 1
    c["k_codes"][page, 0, 0] = codes
    if fmt == "e4m3":
        c["k_scales"][page, 0, 0] = scales
    else:
        c["k_scales"][page, 0, :, 0] = scales[:, None]
    if fmt == "e2m1":
        c["k_codes"][page[0], 0, 0] = 0                      # a block of scale 0 is zero
    else:
        c["k_codes"][page[0], 0, 0] = np.where((codes & 127) == 127, codes, 0)
    old = np.zeros((c["P"], 1, 2, D), np.float16)
    got = _run_bounds(c, [1] * R, old, dense=True)[page, 0]
    k, v = (torch.empty((R, 1, D), dtype=torch.float16, device="cuda") for _ in range(2))
    gdn.gdn_kv_read(k, v, any_device_cache(c, torch, gdn), dev(c["lens"], torch))
    want = k.cpu().numpy()[:, 0]
    with np.errstate(over="ignore"):
        exact = AO.dequantise(c["k_codes"][page, 0, 0], scales) if fmt == "e4m3" else \
            SO.dequantise(SO.unpack(c["k_codes"][page, 0, 0]), np.repeat(scales[:, None], D // 32, 1))
        half = exact.astype(np.float16)
    inside = (np.abs(exact) >= 2.0 ** -24) | (exact == 0) | np.isnan(exact)
    assert np.array_equal(np.where(inside, want, 0), np.where(inside, half, 0), equal_nan=True)
    assert np.array_equal(got[:, 0], want, equal_nan=True) and np.array_equal(got[:, 1], want, equal_nan=True)


def test_bounds_without_pages_and_with_nan_keys():
    c = any_cache([50, 33, 20], fmt="f16", Hk=2, D=64, page=16, seed=2)
    _case("bounds: no page, NaN, infinity")
    page, slot = AO.places(c["table"], 16, c["P"], 0, [40, 41])
    c["k"][page[0], 1, slot[0], 7], c["k"][page[1], 0, slot[1], 9] = np.nan, -np.inf
    c["table"][1, 1], c["table"][2, 0], c["table"][2, 1] = -1, c["P"], -5
    old = np.full((c["P"], 2, 2, 64), 3.0, np.float16)
    T = [30, 20, 20]
    want = SO.bounds(c["k"], c["table"], cu_of(T), c["lens"], old)
    got = _run_bounds(c, T, old, mirrors=False)
    assert np.array_equal(got.astype(np.float64), want, equal_nan=True)
    assert np.isnan(got[page[0], 1, :, 7]).all() and np.isfinite(got[page[0], 1, :, 8]).all() and got[page[1], 0, 0, 9] == -np.inf


def test_tokens_that_were_not_accepted_leave_no_trace():
    c = any_cache([40], fmt="f16", Hk=1, D=64, page=16, seed=2)
    _case("bounds after rejected drafts")
    old = np.zeros((c["P"], 1, 2, 64), np.float16)
    first = _run_bounds(c, [8], old)
    c["lens"] = np.array([35], np.int32)                     # 5 of the 8 newest dropped, two new ones in their place
    rows = queries(2, 1, 64, "f16", 0)
    c["k"] = AO.cache_write(rows, c["k"], c["table"], [0, 2], c["lens"])
    want = SO.bounds(c["k"], c["table"], [0, 2], c["lens"], first)
    assert np.array_equal(_run_bounds(c, [2], first).astype(np.float64), want)


# ------------------------------------------------------------------------------------------------- selection
def _bounds_of(c, seed, D, Hk, wide=1.0):
    rng = np.random.default_rng(seed)
    mid, reach = rng.standard_normal((c["P"], Hk, D)) * 0.5 * wide, 2 + np.abs(rng.standard_normal((c["P"], Hk, D)))
    return np.stack((mid - reach, mid + reach), 2).astype(io_np(c["fmt"]))


def _check_select(lens, T, *, Hk, G, D, page, fmt="f16", K=8, first=1, newest=1, seed=0, bounds=None, table=None, **kw):
    what = f"select lens={lens[:8]} T={T[:8]} Hk={Hk} G={G} D={D} page={page} {fmt} K={K} first={first} newest={newest} {kw}"
    _case(what)
    c = any_cache(lens, fmt=fmt, Hk=Hk, D=D, page=page, seed=seed)
    if table is not None:
        c["table"] = table(c["table"])
    b = _bounds_of(c, seed + 1, D, Hk) if bounds is None else bounds(c)
    cu, q = cu_of(T), queries(sum(T), Hk * G, D, fmt, seed + 2)
    lists, counts, gaps = SO.select(q, b, c["table"], page, cu, lens, K, first, newest)
    assert gaps.min(initial=1.0) > 1e-12, what
    got, n = run_select(c, q, b, cu, torch, gdn, K=K, first=first, newest=newest, **kw)
    assert np.array_equal(n, counts), what
    assert np.array_equal(got, lists), what


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 6, 16])
def test_select_heads(fmt, D, G):
    _check_select([1, 16, 17, 500, 2000], [1] * 5, Hk=2, G=G, D=D, page=16, fmt=fmt, dense=True)


@pytest.mark.parametrize("K", [1, 2, 7, 64, 65, 300])
@pytest.mark.parametrize("first,newest", [(0, 0), (1, 0), (0, 1)])
def test_select_counts(K, first, newest):
    _check_select([1040, 1041, 16 * 64, 40], [1, 2, 3, 1], Hk=1, G=4, D=64, page=16, K=K, first=first, newest=newest, mirrors=K % 2 == 0)


@pytest.mark.parametrize("first,newest", [(3, 5), (8, 0), (0, 8), (1, 1)])
def test_pages_that_are_always_in(first, newest):
    _check_select([64, 500, 3000], [1, 4, 1], Hk=2, G=3, D=64, page=16, K=8, first=first, newest=newest)


@pytest.mark.parametrize("page,n", [(16, 131072), (16, 40000), (64, 70001), (1024, 5000)])
@pytest.mark.parametrize("mirrors", [True, False])
def test_select_among_many(page, n, mirrors):
    _check_select([n, n // 3], [1, 2], Hk=1, G=2, D=64, page=page, K=33, mirrors=mirrors)


def test_select_for_many_tokens():
    _check_select([900, 77, 300], [600, 20, 300], Hk=2, G=2, D=64, page=16, K=5)


def test_equal_scores_go_to_the_lower_entry():
    """The same bounds everywhere, and pages that several entries share."""
    def same(c):
        b = _bounds_of(c, 5, 64, 2)
        b[:] = b[0]
        return b
    _check_select([1600, 333], [1, 1], Hk=2, G=2, D=64, page=16, K=9, bounds=same)

    def shared(t):
        t = t.copy()
        t[0, 30:60] = t[0, 0:30]
        return t
    _check_select([1600, 333], [2, 1], Hk=2, G=2, D=64, page=16, K=21, table=shared)


def test_select_over_wide_ranges_and_infinities():
    def wide(c):
        b = _bounds_of(c, 5, 64, 1).astype(np.float32)
        scale = np.float32(10.0) ** np.random.default_rng(0).integers(-30, 30, c["P"]).astype(np.float32)
        b *= scale[:, None, None, None]
        b[3], b[4, 0, 1, 5], b[5, 0, 0, 6], b[6, 0, 1, 2] = 0, np.inf, -np.inf, np.nan
        return b
    with np.errstate(all="ignore"):
        _check_select([1000], [3], Hk=1, G=2, D=64, page=16, fmt="f32", K=7, bounds=wide)
        _check_select([1000], [3], Hk=1, G=2, D=64, page=16, fmt="f32", K=40, bounds=wide)


def test_select_without_pages():
    def holes(t):
        t = t.copy()
        t[0, 0], t[0, 4:20], t[0, 40], t[1, :] = -1, -1, 1 << 30, -1
        return t
    for K in (3, 40, 60):
        _check_select([1000, 200], [2, 1], Hk=2, G=2, D=64, page=16, K=K, first=1, newest=2, table=holes, mirrors=False)


def test_padded_batches_and_tokens_before_the_cache():
    """Tokens behind the last request keep their lists; one whose position is negative selects nothing."""
    _case("padded batch")
    c = any_cache([100, 20], fmt="f16", Hk=2, D=64, page=16, seed=0)
    b, q, cu = _bounds_of(c, 1, 64, 2), queries(6, 4, 64, "f16", 2), cu_of([2, 1])
    lists, counts, _ = SO.select(q[:3], b, c["table"], 16, cu, c["lens"], 3, 1, 1)
    got, n = run_select(c, q, b, cu, torch, gdn, K=3, mirrors=False)
    assert np.array_equal(got[:3], lists) and np.array_equal(n[:3], counts) and (got[3:] == -77).all() and (n[3:] == -77).all()
    c["lens"] = np.array([1, 20], np.int32)                  # two tokens, of which the first would be at -1
    got, n = run_select(c, q[:3], b, cu, torch, gdn, K=3, mirrors=False)
    assert n.tolist() == [0, 1, 2] and (got[0] == -1).all() and (got[1] == [0, -1, -1]).all()


# ------------------------------------------------------------------------------------------------- attention
def _some_lists(c, T, K, seed, Hk):
    """Random lists in random order, fewer entries than K for some tokens."""
    rng = np.random.default_rng(seed)
    N = sum(T)
    lists, counts, n = np.full((N, Hk, K), -1, np.int32), np.zeros(N, np.int32), 0
    for t, m in zip(T, c["lens"]):
        for j in range(t):
            held = (int(m) - t + j) // c["page"] + 1
            counts[n] = min(K, held)
            for h in range(Hk):
                lists[n, h, :counts[n]] = rng.permutation(held)[:counts[n]]
            n += 1
    return lists, counts


def _check(lens, T, *, Hk, G, D, fmt, page, K, seed=0, lists=None, counts="given", scale=None, table=None, **kw):
    what = f"sparse lens={lens[:8]} T={T[:8]} Hk={Hk} G={G} D={D} {fmt} page={page} K={K} counts={counts} {kw}"
    _case(what)
    c = any_cache(lens, fmt=fmt, Hk=Hk, D=D, page=page, seed=seed)
    if table is not None:
        c["table"] = table(c["table"])
    cu, q = cu_of(T), queries(sum(T), Hk * G, D, fmt, seed + 7)
    l, n = _some_lists(c, T, K, seed, Hk) if lists is None else lists(c)
    if counts == "null":
        n = None
    want, tol = SO.sparse_attention(q, c["k"], c["v"], c["table"], cu, c["lens"], l, n, scale=scale)
    got = run_sparse(c, q, cu, l, n, torch, gdn, **kw, **({} if scale is None else {"scale": scale}))
    assert_within(got, want, tol + half_step(fmt, np.abs(want) + tol), what)
    return c, q, cu, got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 6, 16, 20])
def test_sparse_heads(fmt, D, G):
    _check([1, 16, 17, 100, 700], [1] * 5, Hk=2, G=G, D=D, fmt=fmt, page=16, K=5, dense=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,K", [(16, 3), (32, 4), (64, 9), (256, 2), (1024, 1)])
def test_sparse_pages(fmt, page, K):
    _check([1500, 64, 33, 5], [3, 1, 2, 0], Hk=2, G=4, D=128, fmt=fmt, page=page, K=K, counts="null" if page == 64 else "given")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mirrors", [True, False])
def test_sparse_split(fmt, D, mirrors):
    """Long lists, which several workgroups share."""
    _check([20000, 9000], [1, 3], Hk=2, G=6, D=D, fmt=fmt, page=64, K=100, mirrors=mirrors)


def test_sparse_split_of_many_lists():
    """As many lists as make a list's fixed part count in the split."""
    _check([2100], [16], Hk=8, G=2, D=64, fmt="e2m1", page=64, K=32)


@pytest.mark.parametrize("fmt", FORMATS)
def test_sparse_many(fmt):
    """More segments than get a workgroup each, of a prompt and of a batch."""
    _check([900, 40], [300, 40], Hk=4, G=2, D=64, fmt=fmt, page=16, K=4)
    _check([200] * 150, [1] * 150, Hk=8, G=1, D=128, fmt=fmt, page=16, K=6, dense=True, scale=0.3)


@pytest.mark.parametrize("fmt", FORMATS)
def test_entries_that_hold_nothing(fmt):
    """-1 anywhere, entries past the token, past the table or without a page, one twice, lists of nothing."""
    def lists(c):
        l = np.array([[5, -1, 0, 70, 2, 2, 1 << 27], [-1] * 7, [-5, 3, 3, -1, -1, -1, 0], [-(1 << 31), (1 << 31) - 1, 1, 1, 1, 1, 1],
                      [6, 6, 6, 6, 6, 6, 6]], np.int64).astype(np.int32)
        l = np.repeat(l[:, None], 2, 1)
        l[2, 1] = [1, 0, 4, -1, 2, 3, 9]
        return l, np.array([7, 7, 7, 4, 100], np.int32)

    def holes(t):
        t = t.copy()
        t[0, 2], t[1, 1] = -1, 1 << 29
        return t
    for table in (None, holes):
        c, q, cu, got = _check([95, 60], [3, 2], Hk=2, G=3, D=64, fmt=fmt, page=16, K=7, lists=lists, table=table, mirrors=False)
        assert not got[1].any()                              # a list of nothing
        assert not got[4].any()                              # past the token's own position
    zero = run_sparse(c, q, cu, lists(c)[0], np.array([0, -3, 0, 0, 0], np.int32), torch, gdn)
    assert not zero.any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_sparse_over_all_pages_is_attention(fmt):
    """The same positions in the same order are the same sums where nothing is split."""
    _case(f"sparse over all pages {fmt}")
    lens, T = [300, 20, 77], [1, 1, 1]
    c = any_cache(lens, fmt=fmt, Hk=2, D=128, page=16, seed=3)
    cu, q = cu_of(T), queries(3, 8, 128, fmt, 4)
    lists = np.repeat(np.arange(20, dtype=np.int32)[None, None], 3, 0).repeat(2, 1)
    got = run_sparse(c, q, cu, lists, None, torch, gdn)
    want = run_attention(c, q, cu, torch, gdn, cache=any_device_cache(c, torch, gdn))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_what_lies_behind_the_token_has_no_influence(fmt):
    """NaN behind a draft's own position, in its page and in the next; attended, it shows."""
    _case(f"NaN behind {fmt}")
    c = any_cache([40], fmt=fmt, Hk=1, D=64, page=16, seed=3)
    cu, q = cu_of([3]), queries(3, 4, 64, fmt, 4)
    lists = np.repeat(np.array([[2, 0, 1]], np.int32)[None], 3, 0)
    clean = run_sparse(c, q, cu, lists, None, torch, gdn)
    page, slot = AO.places(c["table"], 16, c["P"], 0, [39])
    if fmt == "e2m1":
        c["v_scales"][page[0], 0, :, slot[0]] = 255
    elif fmt == "e4m3":
        c["v_codes"][page[0], 0, slot[0], :] = 0x7f
    else:
        c["v"][page[0], 0, slot[0], :] = np.nan
    got = run_sparse(c, q, cu, lists, None, torch, gdn)
    assert np.array_equal(got[:2], clean[:2]) and np.isnan(got[2]).all()


@pytest.mark.parametrize("fmt", ["f16", "e2m1"])
def test_sparse_padded_batch(fmt):
    """Tokens behind the last request keep their output, also where parts are joined."""
    _case(f"sparse padded {fmt}")
    for lens, K in (([300, 50], 4), ([20000, 9000], 90)):
        c = any_cache(lens, fmt=fmt, Hk=1, D=64, page=64, seed=0)
        cu, q = cu_of([1, 2]), queries(7, 4, 64, fmt, 1)
        l3, n3 = _some_lists(c, [1, 2], K, 0, 1)
        lists, counts = np.zeros((7, 1, K), np.int32), np.full(7, K, np.int32)
        lists[:3], counts[:3] = l3, n3
        want, tol = SO.sparse_attention(q[:3], c["k"], c["v"], c["table"], cu, c["lens"], l3, n3)
        for mirrors in (False,):
            got = run_sparse(c, q, cu, lists, counts, torch, gdn, mirrors=mirrors)
            assert_within(got[:3], want, tol + half_step(fmt, np.abs(want) + tol), f"padded {lens}")
            assert (got[3:] == -7.75).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3])
def test_strided_q(fmt, T):
    """q as a slice of a projection's output, of the selection and of the attention."""
    _case(f"strided q {fmt} T={T}")
    lens, Hk, Hq, D, K = [300, 77], 2, 8, 128, 5
    c = any_cache(lens, fmt=fmt, Hk=Hk, D=D, page=16, seed=3)
    b, N = _bounds_of(c, 4, D, Hk), 2 * T
    cu, q = cu_of([T, T]), queries(N, Hq, D, fmt, 5)
    wide = torch.full((N, Hq * D + 256), float("nan"), dtype=dev(q, torch).dtype, device="cuda")
    wide[:, 64:64 + Hq * D] = dev(q, torch).view(N, -1)
    dq, cache, dlens = wide[:, 64:64 + Hq * D].view(N, Hq, D), any_device_cache(c, torch, gdn), dev(c["lens"], torch)
    lists, counts = torch.empty((N, Hk, K), dtype=torch.int32, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
    out = torch.empty((N, Hq, D), dtype=dq.dtype, device="cuda")
    ws = torch.empty(max(gdn.gdn_attn_select_workspace_bytes(N, 2, Hq, K, cache), gdn.gdn_attn_sparse_workspace_bytes(N, 2, Hq, K, cache)),
                     dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_select(dq, dev(b, torch), cache, dlens, None, lists, counts, num_reqs=2, workspace=ws)
    gdn.gdn_attn_sparse_forward(dq, cache, dlens, None, lists, counts, out, num_reqs=2, workspace=ws)
    torch.cuda.synchronize()
    want_l, want_n, gaps = SO.select(q, b, c["table"], 16, cu, lens, K, 1, 1)
    assert gaps.min() > 1e-12
    assert np.array_equal(lists.cpu().numpy(), want_l) and np.array_equal(counts.cpu().numpy(), want_n)
    want, tol = SO.sparse_attention(q, c["k"], c["v"], c["table"], cu, lens, want_l, want_n)
    assert_within(out.double().cpu().numpy(), want, tol + half_step(fmt, np.abs(want) + tol), "strided q")


def test_a_nan_query_selects_the_lowest_entries():
    _case("NaN q")
    c = any_cache([700, 700], fmt="f16", Hk=2, D=64, page=16, seed=0)
    b, q = _bounds_of(c, 1, 64, 2), queries(2, 4, 64, "f16", 2)
    q[0, 1, 5] = np.nan                                      # of key head 0
    want, counts, _ = SO.select(q, b, c["table"], 16, [0, 1, 2], c["lens"], 6, 1, 1)
    got, n = run_select(c, q, b, [0, 1, 2], torch, gdn, K=6)
    assert np.array_equal(got, want) and np.array_equal(n, counts)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 4, 43]


@pytest.mark.parametrize("fmt", ["f16", "e2m1"])
def test_lengths_at_the_ends_of_int32(fmt):
    """The table's positions are all there are, and a negative length has none."""
    _case(f"int32 lengths {fmt}")
    c = any_cache([64, 64], fmt=fmt, Hk=1, D=64, page=16, seed=1)
    c["table"] = c["table"][:, :4]
    c["lens"] = np.array([(1 << 31) - 1, -(1 << 31)], np.int32)
    cu, q, b = cu_of([2, 2]), queries(4, 4, 64, fmt, 2), _bounds_of(c, 1, 64, 1)
    lists, counts = run_select(c, q, b, cu, torch, gdn, K=3, mirrors=False)
    assert counts.tolist() == [3, 3, 0, 0] and (lists[2:] == -1).all()
    got = run_sparse(c, q, cu, lists, counts, torch, gdn, mirrors=False)
    want, tol = SO.sparse_attention(q[:2], c["k"], c["v"], c["table"], [0, 2], [(1 << 31) - 1], lists[:2], counts[:2])
    assert_within(got[:2], want, tol + half_step(fmt, np.abs(want) + tol), "int32 lengths")
    assert not got[2:].any()
    old = np.full((c["P"], 1, 2, 64), 3.0, io_np(fmt))
    assert np.array_equal(_run_bounds(c, [2, 2], old, mirrors=False), old)    # no new token lies on a page


def test_many_lists_whose_lengths_the_host_says_are_none():
    """A mirror of zeros with the device's lengths: lists in two launches, over what the device says."""
    _case("mirror of zeros")
    R = 160
    c = any_cache([200] * R, fmt="f16", Hk=8, D=64, page=16, seed=0)
    b, q, cu = _bounds_of(c, 1, 64, 8), queries(R, 8, 64, "f16", 2), np.arange(R + 1, dtype=np.int32)
    want, counts, gaps = SO.select(q, b, c["table"], 16, cu, c["lens"], 5, 1, 1)
    assert gaps.min() > 1e-12
    lists = torch.full((R, 8, 5), -77, dtype=torch.int32, device="cuda")
    n = torch.full((R,), -77, dtype=torch.int32, device="cuda")
    cache = any_device_cache(c, torch, gdn)
    ws = torch.full((gdn.gdn_attn_select_workspace_bytes(R, R, 8, 5, cache),), 0xff, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_select(dev(q, torch), dev(b, torch), cache, dev(c["lens"], torch), dev(cu, torch), lists, n,
                        seq_lens_host=np.zeros(R, np.int32), workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(lists.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), counts)
