"""GPU: the ways gdn_attn_forward shares its work out, each asserted to be the one the call takes.

`_path` repeats the host's rule: segments (request, 16 or 32 rows, key head) that are not split
get a workgroup each, are shared out by length over 512, or (past 2^22) by number; else the
positions are split. All ways have to give what the oracle does.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import FORMATS, assert_within, device_cache, io_np, make_cache, oracle_attention, run_attention
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


BYTES = {"f32": 4, "f16": 2, "e4m3": 1}


def _whole(longest, total, Hk, D, fmt):
    size = 2 * D * BYTES[fmt]
    return longest * size / (29e3 if fmt == "e4m3" else 47e3) <= total * Hk * size / 6.4e6 / 2 + 5.0


def _path(lens, new, *, Hk, G, D, fmt, cap, window=0, mirrors=True, dense=False):
    """(path, whether a unit of work is longer than its usual 32 or 128 positions)."""
    N, R, T = sum(new), len(new), max(new) if mirrors or dense else sum(new)
    most = T * G
    rows = 16 if most <= 16 else 32
    segments = ((N * G // rows if most > rows else 0) + R) * Hk
    top = min(cap, window + T) if window else cap
    seen = [min(n, top) for n in lens] if mirrors else []
    if _whole(max(seen) if mirrors else top, sum(seen), Hk, D, fmt):
        if segments <= 1024:
            return "own", False
        if segments > 1 << 22:
            return "number", False
        return "shared", segments * ((cap >> 5) + 1 + 200000 // (64 * D * BYTES[fmt])) > 1 << 30
    return "split", segments * ((cap >> 7) + 1) > 1 << 30


def _cap(c):
    return c["table"].shape[1] * c["page"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [2, 20])
@pytest.mark.parametrize("window", [0, 25])
def test_many_short_segments_are_shared_out(fmt, D, G, window):
    """One request as long as the rule allows among hundreds of short ones, some without tokens or positions."""
    rng = np.random.default_rng(160)
    R, Hk = 600, 2
    lens = [int(x) for x in rng.integers(0, 41, R)]
    new = [int(min(x, n)) for x, n in zip(rng.integers(0, 3, R), lens)]
    lens[200:260], new[200:260] = [5] * 60, [0] * 60
    lens[0], new[0], lens[R - 1], new[R - 1] = 17, 2, 33, 1
    lens[130], new[130] = 2, 2
    while lens[130] < 2000 and _whole(lens[130] + 1, sum(lens) + 1, Hk, D, fmt):
        lens[130] += 1
    c = make_cache(lens, Hk=Hk, D=D, fmt=fmt, page=16, seed=161)
    path = _path(lens, new, Hk=Hk, G=G, D=D, fmt=fmt, cap=_cap(c), window=window)
    _case(f"{fmt} D={D} G={G} window={window} longest {lens[130]}: {path}")
    assert path == ("shared", False)
    q = rng.standard_normal((sum(new), Hk * G, D)).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu(new), window=window)
    assert_within(run_attention(c, q, _cu(new), torch, gdn, window=window), want, tol, f"{fmt} {D} {G}")


def _widened(c, pages):
    """The same cache under a table of `pages` entries a request."""
    wide = np.full((c["table"].shape[0], pages), -1, np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    return {**c, "table": wide}


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_shared_out_under_a_wide_table(fmt):
    """Units of work that are longer than usual, so that their number stays within 32 bits."""
    rng = np.random.default_rng(162)
    R, Hk, G, D = 600, 2, 3, 64
    lens = [int(x) for x in rng.integers(1, 60, R)]
    lens[77] = 300
    new = [int(min(x, n)) for x, n in zip(rng.integers(1, 4, R), lens)]
    c = _widened(make_cache(lens, Hk=Hk, D=D, fmt=fmt, page=1024, seed=163), 1 << 15)
    path = _path(lens, new, Hk=Hk, G=G, D=D, fmt=fmt, cap=_cap(c))
    _case(f"{fmt}: {path}")
    assert path == ("shared", True)
    q = rng.standard_normal((sum(new), Hk * G, D)).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu(new))
    assert_within(run_attention(c, q, _cu(new), torch, gdn), want, tol, fmt)


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("new", [1, 9])
def test_split_under_the_widest_table(fmt, new):
    """2^30 positions a request as far as the table goes, without mirrors."""
    rng = np.random.default_rng(164)
    R, Hk, G, D = 70, 2, 4, 64
    lens = [int(x) for x in rng.integers(9, 900, R)]
    lens[3], lens[69] = 6000, 4097
    c = _widened(make_cache(lens, Hk=Hk, D=D, fmt=fmt, page=1024, seed=165), 1 << 20)
    path = _path(lens, [new] * R, Hk=Hk, G=G, D=D, fmt=fmt, cap=_cap(c), mirrors=False, dense=True)
    _case(f"{fmt} {new}: {path}")
    assert path == ("split", True)
    q = rng.standard_normal((R * new, Hk * G, D)).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu([new] * R))
    assert_within(run_attention(c, q, _cu([new] * R), torch, gdn, mirrors=False, dense=True), want, tol, fmt)


def test_more_segments_than_units_can_be_counted_for():
    """Past 2^22 segments they are shared out by number: the same requests over and over, against one of each."""
    R, kinds, D, G = 4_200_000, 1500, 64, 2
    rng = np.random.default_rng(166)
    lens = [int(x) for x in rng.integers(0, 17, kinds)]
    c = make_cache(lens, Hk=1, D=D, fmt="f16", page=16, seed=167)
    c["table"] = np.ascontiguousarray(c["table"][:, :1])
    q = rng.standard_normal((kinds, G, D)).astype(np.float16)
    assert _path(lens, [1] * kinds, Hk=1, G=G, D=D, fmt="f16", cap=16, mirrors=False, dense=True)[0] == "shared"
    want, tol = oracle_attention(c, q, _cu([1] * kinds))
    one = run_attention(c, q, _cu([1] * kinds), torch, gdn, dense=True, mirrors=False)
    assert_within(one, want, tol, "one of each")

    of = torch.arange(R, device="cuda") % kinds
    cache = device_cache(c, torch, gdn)
    many = gdn.KVCache(cache._keep[0], cache._keep[1], dev(c["table"], torch)[of].contiguous())
    dq, dl = dev(q, torch)[of].contiguous(), dev(c["lens"], torch)[of].contiguous()
    assert _path([16] * R, [1] * R, Hk=1, G=G, D=D, fmt="f16", cap=16, mirrors=False, dense=True)[0] == "number"
    out = torch.full_like(dq, -7.75)
    ws = torch.empty(gdn.gdn_attn_workspace_bytes(R, R, G, many) + 16, dtype=torch.uint8, device="cuda")
    _case("the call over all of them")
    gdn.gdn_attn_forward(dq, many, dl, None, out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, dev(one.astype(np.float16), torch)[of])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("lens,new,G", [([900, 300], [700, 300], 6), ([1100], [1100], 1), ([2500, 1, 64], [520, 1, 64], 17)])
def test_prompts_of_hundreds_of_tokens(fmt, window, lens, new, G):
    """Dozens to hundreds of segments of a request and key head, whose rows attend from their windows to their own
    positions."""
    D = 64
    c = make_cache(lens, Hk=2, D=D, fmt=fmt, page=32, seed=170)
    q = np.random.default_rng(171).standard_normal((sum(new), 2 * G, D)).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu(new), window=window)
    for mirrors in (True, False):
        _case(f"{fmt} window={window} {lens} {new} G={G} mirrors={mirrors}")
        got = run_attention(c, q, _cu(new), torch, gdn, window=window, mirrors=mirrors)
        assert_within(got, want, tol, f"{fmt} {window} {mirrors}")
