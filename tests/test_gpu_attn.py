"""GPU parity of the attention over a paged cache (gdn_attn_forward) against the
float64 oracle, called through the C ABI.

The tolerance of every element is oracle.attn_oracle.attention's bound (roundings of
the scores, the weights and the sums, counted from the inputs) plus half a step of
the I/O type. Unused slots of the pool hold NaN, so a masked position that has any
influence shows.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import (FORMATS, assert_within, device_cache, half_step, io_np, make_cache, oracle_attention,
                          run_attention)
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import attn_oracle as AO                 # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def _q(N, Hq, D, fmt, seed, scale=1.5):
    return (np.random.default_rng(seed + 1000).standard_normal((N, Hq, D)) * scale).astype(io_np(fmt))


def _check(lens, new, *, Hk, G, D, fmt, page, seed=0, **kw):
    what = f"lens={lens} new={new} Hk={Hk} G={G} D={D} {fmt} page={page} {kw}"
    _case(what)
    run = {n: kw.pop(n) for n in ("dense", "mirrors") if n in kw}
    c = make_cache(lens, Hk=Hk, D=D, fmt=fmt, page=page, seed=seed)
    cu = _cu(new)
    q = _q(cu[-1], Hk * G, D, fmt, seed)
    want, tol = oracle_attention(c, q, cu, **kw)
    got = run_attention(c, q, cu, torch, gdn, **run, **kw)
    assert_within(got, want, tol, what)
    return got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 6, 16, 20])
def test_decode_heads(fmt, D, G):
    _check([77, 1, 200], [1, 1, 1], Hk=2, G=G, D=D, fmt=fmt, page=32, seed=D + G, dense=True)


# around the tile sizes of the kernel, a page's end and one token
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("lens", [[1, 2, 15, 16, 17], [31, 32, 33, 63, 64, 65], [127, 128, 129], [255, 256, 257, 3], [1000, 1, 511]])
def test_lengths(fmt, page, lens):
    _check(lens, [1] * len(lens), Hk=2, G=4, D=64, fmt=fmt, page=page, seed=len(lens) + page)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,new", [([9, 40, 4], [4, 4, 4]), ([130, 5, 64, 700], [3, 5, 1, 4]), ([50, 90], [50, 33]),
                                      ([33, 200], [17, 40])])
@pytest.mark.parametrize("G", [1, 4, 5])
def test_draft_tokens_and_prompts(fmt, lens, new, G):
    _check(lens, new, Hk=2, G=G, D=128, fmt=fmt, page=16, seed=G)


@pytest.mark.parametrize("D", [64, 256])
def test_drafts_of_large_heads(D):
    _check([300, 77], [4, 3], Hk=1, G=6, D=D, fmt="f16", page=16, seed=D)
    _check([300, 77], [4, 3], Hk=1, G=6, D=D, fmt="f32", page=16, seed=D)
    _check([300, 77], [4, 3], Hk=1, G=6, D=D, fmt="e4m3", page=16, seed=D)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 7, 64, 129, 5000])
def test_window(fmt, window):
    _check([300, 40, 129, 3], [1, 4, 3, 2], Hk=2, G=2, D=64, fmt=fmt, page=32, window=window, seed=window)


def test_scale():
    _check([70, 9], [1, 2], Hk=2, G=2, D=64, fmt="f16", page=16, scale=0.05)


@pytest.mark.parametrize("mirrors", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
def test_long_caches_are_split_and_joined(fmt, mirrors):
    """One and a few requests over thousands of positions: the length is all there is to split."""
    _check([9001], [1], Hk=2, G=6, D=128, fmt=fmt, page=64, dense=True, mirrors=mirrors, seed=3)
    _check([5000, 3, 7777], [4, 2, 1], Hk=1, G=4, D=256, fmt=fmt, page=256, mirrors=mirrors, seed=4)


def test_many_requests():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 400, 300)]
    _check(lens, [1] * 300, Hk=2, G=2, D=64, fmt="f16", page=16, seed=6, dense=True)
    new = [int(min(x, n)) for x, n in zip(rng.integers(0, 5, 300), lens)]
    _check(lens, new, Hk=2, G=2, D=64, fmt="f16", page=16, seed=7, mirrors=False)


@pytest.mark.parametrize("fmt", FORMATS)
def test_requests_without_tokens_and_empty_rows(fmt):
    """Length zero with a token (an empty row: zeros), requests without new tokens, tokens older than the cache."""
    got = _check([0, 20, 0, 5], [1, 0, 0, 5], Hk=2, G=2, D=64, fmt=fmt, page=16, mirrors=False)
    assert np.all(got[0] == 0)
    got = _check([2, 3], [4, 3], Hk=2, G=2, D=64, fmt=fmt, page=16, mirrors=False)     # two rows before position 0
    assert np.all(got[:2] == 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_that_name_nothing(fmt):
    """-1 and numbers past the pool inside the length: those positions are left out."""
    c = make_cache([100, 90, 40], Hk=2, D=64, fmt=fmt, page=16, seed=8)
    c["table"][0, 2] = -1
    c["table"][0, 0] = c["P"]
    c["table"][1, 5] = 2 ** 31 - 1
    c["table"][2, :] = -5
    cu = _cu([2, 3, 1])
    q = _q(cu[-1], 4, 64, fmt, 8)
    want, tol = oracle_attention(c, q, cu)
    got = run_attention(c, q, cu, torch, gdn)
    assert_within(got, want, tol, fmt)
    assert np.all(got[-1] == 0)


def test_lengths_past_the_table():
    """seq_lens beyond max_pages * page_size (no host mirror): the positions the table holds count."""
    c = make_cache([64, 64], Hk=2, D=64, fmt="f16", page=16, seed=9)
    c["table"] = np.ascontiguousarray(c["table"][:, :4])
    c["lens"] = np.array([80, 64], np.int32)
    cu = _cu([1, 1])
    q = _q(2, 4, 64, "f16", 9)
    want, tol = oracle_attention(c, q, cu)
    assert_within(run_attention(c, q, cu, torch, gdn, mirrors=False), want, tol, "past the table")


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_and_infinities_in_later_drafts(fmt):
    """A draft token sees nothing of the drafts after it, whatever their keys and values are."""
    c = make_cache([70, 35], Hk=2, D=64, fmt=fmt, page=16, seed=10)
    cu = _cu([4, 3])
    q = _q(cu[-1], 6, 64, fmt, 10)
    bad = [(0, 69, np.nan), (0, 68, np.inf), (1, 34, -np.inf)]
    for r, pos, x in bad:
        pg, sl = c["table"][r, pos // 16], pos % 16
        for name in ("k", "v"):
            if fmt == "e4m3":
                c[name + "_codes"][pg, :, sl, 3] = 0x7f
                c[name][pg, :, sl, 3] = np.nan
            else:
                c[name][pg, :, sl, 3] = x
    ok = np.array([0, 1, 4, 5])                         # rows before the first bad position
    got = run_attention(c, q, cu, torch, gdn)
    clean = {**c, "k": np.nan_to_num(c["k"].astype(np.float64), posinf=0, neginf=0),
             "v": np.nan_to_num(c["v"].astype(np.float64), posinf=0, neginf=0)}
    want, tol = oracle_attention(clean, q, cu)
    assert_within(got[ok], want[ok], tol[ok], fmt)
    assert np.all(np.isnan(got[3])), "a NaN that is attended has to show"


def test_nan_in_an_attended_value_stays_in_its_element():
    c = make_cache([40], Hk=1, D=64, fmt="f16", page=16, seed=11)
    c["v"][c["table"][0, 1], 0, 3, 17] = np.nan
    got = run_attention(c, _q(1, 2, 64, "f16", 11), _cu([1]), torch, gdn)
    assert np.all(np.isnan(got[..., 17])) and np.all(np.isfinite(np.delete(got, 17, -1)))


@pytest.mark.parametrize("fmt", ["f16", "f32"])
def test_large_scores(fmt):
    """Scores in the thousands: the running maximum keeps the weights in range, at the first position or the last."""
    for place in (0, 63, 64, 199):
        c = make_cache([200], Hk=1, D=64, fmt=fmt, page=16, seed=12)
        pg, sl = c["table"][0, place // 16], place % 16
        c["k"][pg, 0, sl] = 60.0
        q = np.full((1, 2, 64), 8.0, io_np(fmt))
        want, tol = oracle_attention(c, q, _cu([1]))
        assert_within(run_attention(c, q, _cu([1]), torch, gdn), want, tol, f"{fmt} {place}")


def test_values_over_the_whole_fp16_range():
    """8-bit rows whose scales span 2^-30 .. 2^8: a row of small values keeps its own digits."""
    c = make_cache([150], Hk=2, D=64, fmt="e4m3", page=16, seed=13)
    rng = np.random.default_rng(13)
    c["v_scales"] = np.where(c["v_scales"] == 130, 130, rng.integers(96, 136, c["v_scales"].shape)).astype(np.uint8)
    c["v"] = AO.dequantise(c["v_codes"], c["v_scales"])
    q = _q(1, 4, 64, "f16", 13)
    want, tol = oracle_attention(c, q, _cu([1]))
    assert_within(run_attention(c, q, _cu([1]), torch, gdn), want, tol, "scales")


def test_zero_rows_in_an_8_bit_cache():
    c = make_cache([90], Hk=1, D=128, fmt="e4m3", page=16, seed=14)
    for pos in (0, 5, 50, 89):
        pg, sl = c["table"][0, pos // 16], pos % 16
        for name in ("k", "v"):
            c[name + "_codes"][pg, 0, sl], c[name + "_scales"][pg, 0, sl], c[name][pg, 0, sl] = 0, 0, 0.0
    q = _q(1, 4, 128, "f16", 14)
    want, tol = oracle_attention(c, q, _cu([1]))
    assert_within(run_attention(c, q, _cu([1]), torch, gdn), want, tol, "zero rows")
    c["v_codes"][:], c["v_scales"][:], c["v"] = 0, 0, np.zeros(c["v"].shape)
    assert np.all(run_attention(c, q, _cu([1]), torch, gdn) == 0)


def test_rows_behind_the_last_request_stay():
    """A padded batch: cu_seqlens ends before num_tokens (no host mirror)."""
    c = make_cache([40, 9], Hk=2, D=64, fmt="f16", page=16, seed=15)
    cu = _cu([2, 1])
    q = _q(6, 4, 64, "f16", 15)
    want, tol = oracle_attention(c, q, cu)
    got = run_attention(c, q, cu, torch, gdn, mirrors=False)
    assert_within(got[:3], want[:3], tol[:3], "padded")
    assert np.all(got[3:] == -7.75)


def test_queries_in_a_wider_buffer():
    c = make_cache([40, 300], Hk=2, D=64, fmt="f16", page=16, seed=16)
    cu = _cu([2, 3])
    q = _q(5, 4, 64, "f16", 16)
    wide = torch.full((5, 4 * 64 + 136), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 256] = dev(q, torch).view(5, 256)
    view = wide[:, 8:8 + 256].view(5, 4, 64)
    assert not view.is_contiguous()
    cache = device_cache(c, torch, gdn)
    ws = torch.empty(max(16, gdn.gdn_attn_workspace_bytes(5, 2, 4, cache)), dtype=torch.uint8, device="cuda")
    outs = []
    for x in (dev(q, torch), view):
        out = torch.empty((5, 4, 64), dtype=torch.float16, device="cuda")
        gdn.gdn_attn_forward(x, cache, dev(c["lens"], torch), dev(cu.astype(np.int32), torch), out, workspace=ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_repeats_bit_for_bit():
    c = make_cache([5000, 60], Hk=2, D=128, fmt="f16", page=64, seed=17)
    q = _q(2, 8, 128, "f16", 17)
    a = run_attention(c, q, _cu([1, 1]), torch, gdn)
    assert np.array_equal(a, run_attention(c, q, _cu([1, 1]), torch, gdn))


def test_offsets_past_32_bits():
    """Pages beyond 2^31 elements into the pool."""
    D, Hk, page, P = 128, 8, 256, 9000
    pool = P * Hk * page * D                             # 2.36e9 elements, 4.7 GB each
    assert pool > 2 ** 31
    c = make_cache([700, 130], Hk=Hk, D=D, fmt="f16", page=page, seed=18)
    far = (P - 1 - np.arange(c["P"])).astype(np.int32)
    kp = torch.zeros((P, Hk, page, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    kp[torch.from_numpy(far.astype(np.int64)).cuda()] = dev(c["k"], torch)
    vp[torch.from_numpy(far.astype(np.int64)).cuda()] = dev(c["v"], torch)
    table = np.where(c["table"] >= 0, far[np.clip(c["table"], 0, None)], -1).astype(np.int32)
    q = _q(2, 16, D, "f16", 18)
    want, tol = oracle_attention(c, q, _cu([1, 1]))
    cache = gdn.KVCache(kp, vp, dev(table, torch))
    assert_within(run_attention(c, q, _cu([1, 1]), torch, gdn, cache=cache), want, tol, "far pages")


def test_other_streams_and_two_at_once():
    """Two calls in flight on two streams, each with its own workspace and output."""
    cs = [make_cache([4000 + 100 * i, 50], Hk=2, D=128, fmt="f16", page=64, seed=19 + i) for i in range(2)]
    qs = [_q(2, 8, 128, "f16", 19 + i) for i in range(2)]
    alone = [run_attention(c, q, _cu([1, 1]), torch, gdn) for c, q in zip(cs, qs)]
    dc = [device_cache(c, torch, gdn) for c in cs]
    dq, dl = [dev(q, torch) for q in qs], [dev(c["lens"], torch) for c in cs]
    out = [torch.empty_like(x) for x in dq]
    ws = [torch.empty(gdn.gdn_attn_workspace_bytes(2, 2, 8, x) + 16, dtype=torch.uint8, device="cuda") for x in dc]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            gdn.gdn_attn_forward(dq[i], dc[i], dl[i], None, out[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(out[i].double().cpu().numpy(), alone[i])


def test_workspace_refusal_and_wrong_arguments():
    c = make_cache([4000], Hk=1, D=64, fmt="f16", page=16, seed=21)
    cache = device_cache(c, torch, gdn)
    q = dev(_q(1, 2, 64, "f16", 21), torch)
    out, lens = torch.full_like(q, -7.75), dev(c["lens"], torch)
    if gdn.gdn_attn_workspace_bytes(1, 1, 2, cache) > 0:
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_attn_forward(q, cache, lens, None, out)
        assert e.value.status == gdn.GDN_ERR_WORKSPACE
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q.float(), cache, lens, None, out.float())
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q.transpose(0, 1), cache, lens, None, out)
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q, cache, lens.long(), None, out)
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q, cache, torch.cat([lens, lens]), None, out)        # more requests than table rows
    torch.cuda.synchronize()
    assert bool((out == -7.75).all())
