"""What is measured of the operators for long contexts: the paged key-value cache in 4 bits (appended to, read back,
attended), and sparse attention (the channel bounds of a page's keys, the selection of pages by them, attention over the
selected pages).

Every case is a dict of plain values; `run` computes it with elementary torch operations where `own` is false and with the
library's entry points where it is true. Layouts (io: float16 or float32):

  q [N, Hq, D], k and v [N, Hk, D]   packed tokens, request r owning cu[r] .. cu[r+1]-1, the newest of its seq_lens[r]
  pages [P, Hk, page, D]             io, or float8_e4m3fn with an exponent byte per row [P, Hk, page], or two e2m1 codes a
                                     byte [P, Hk, page, D / 2] with an exponent byte per 32 elements [P, Hk, D / 32, page]
  page_table [R, M]                  the page of a request's positions page*i .. page*i + page-1 (-1: none)
  bounds [P, Hk, 2, D]               io: the lowest and the highest key of a page, channel by channel
  lists [N, Hk, K]                   which entries of its request's table a token attends, ascending, -1 behind the last
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
IO = {"f16": torch.float16, "f32": torch.float32}
BYTES = {"f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests into 4-bit pages, q and k rotated on the way, and the new rows as the cache now
        # holds them; latency counts
        dict(name="append_decode_e2m1", op="append", reqs=64, new=1, mix=11, past=500, hq=24, hk=4, dim=256, rot=64, layout="half", page=64),
        # ragged prompts into 4-bit pages, whole heads rotated in the interleaved layout, and back for their own attention
        dict(name="append_prompt_e2m1", op="append", reqs=8, new=4096, mix=3, past=0, hq=32, hk=8, dim=128, rot=128, layout="interleaved",
             page=32),
        # a long cached prefix read back for the attention of a further prompt
        dict(name="read_long_e2m1", op="read", reqs=1, len=32768, mix=0, hk=4, dim=256, page=64),
        # short ragged prefixes of small heads
        dict(name="read_ragged_e2m1", op="read", reqs=5, len=1993, mix=5, hk=2, dim=64, page=16),
        # the decode step of a full batch over 4-bit caches of mixed lengths
        dict(name="attn_decode_e2m1", op="attn", reqs=64, new=1, len=16384, mix=21, hq=32, hk=8, dim=128, page=64, window=0),
        # the verify of up to 4 draft tokens for each of 16 requests, large heads in groups of 6, odd lengths
        dict(name="attn_verify_e2m1", op="attn", reqs=16, new=4, len=8191, mix=22, hq=24, hk=4, dim=256, page=64, window=0),
        # the bounds of the pages that a decode step of 64 requests has added a key to; latency counts
        dict(name="bounds_decode_f16", op="bounds", reqs=64, new=1, mix=31, past=4096, hk=8, dim=128, page=64, format="io", dtype="f16"),
        # the bounds of all pages of ragged prompts in 8 bits
        dict(name="bounds_prompt_e4m3", op="bounds", reqs=8, new=8192, mix=36, past=0, hk=4, dim=256, page=64, format="e4m3", dtype="f16"),
        # every request of a decode batch selects 32 of up to 256 pages
        dict(name="select_decode_f16", op="select", reqs=64, new=1, len=16384, mix=21, hq=32, hk=8, dim=128, page=64, pages=32, first=1,
             newest=2, format="io", dtype="f16"),
        # 3 drafts of one long context select 128 of 4,097 pages, in single precision
        dict(name="select_long_f32", op="select", reqs=1, new=3, len=131075, mix=0, hq=24, hk=4, dim=256, page=32, pages=128, first=2,
             newest=4, format="io", dtype="f32"),
        # the decode step of the batch over its 32 selected pages
        dict(name="sparse_decode_f16", op="sparse", reqs=64, new=1, len=16384, mix=21, hq=32, hk=8, dim=128, page=64, pages=32, format="io",
             dtype="f16"),
        # 2 drafts of one long context over 65 selected pages of 4 bits
        dict(name="sparse_long_e2m1", op="sparse", reqs=1, new=2, len=131072, mix=42, hq=24, hk=4, dim=256, page=64, pages=65, format="e2m1",
             dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "read", "attn", "attn", "bounds", "select", "sparse", "sparse"))
    dim = rng.choice((64, 128, 256))
    hk = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    hq = hk * group
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice((16, 32, 64, 128, 256))
    kind = rng.choice((("io", "f16"), ("e4m3", "f16"), ("e2m1", "f16"), ("io", "f32")))
    if op == "append":
        reqs = _log_int(rng, 1, 128)
        return dict(op=op, reqs=reqs, new=_log_int(rng, 1, max(1, min(8192, (1 << 25) // (reqs * (hq + hk) * dim)))), mix=mix,
                    past=_log_int(rng, 1, 1024), hq=hq, hk=hk, dim=dim, rot=rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim]),
                    layout=rng.choice(("half", "interleaved")), page=page)
    if op == "read":
        reqs = _log_int(rng, 1, 64)
        return dict(op=op, reqs=reqs, len=_log_int(rng, 1, min(65536, (1 << 26) // (reqs * hk * dim))), mix=mix, hk=hk, dim=dim, page=page)
    if op == "bounds":
        reqs = _log_int(rng, 1, 128)
        return dict(op=op, reqs=reqs, new=_log_int(rng, 1, min(16384, (1 << 25) // (reqs * hk * dim))), mix=mix, past=_log_int(rng, 1, 2048),
                    hk=hk, dim=dim, page=page, format=kind[0], dtype=kind[1])
    reqs, new, mix = _log_int(rng, 1, 256), rng.choice((1, 1, 1, 2, 3, 4, 5, 8)), rng.choice((0, mix, mix))
    if op == "attn":
        most = int(4.5e8 / (reqs * hk * dim * max(1.0, new * group / 5)))
        return dict(op=op, reqs=reqs, new=new, len=_log_int(rng, 9, min(131072, most)), mix=mix, hq=hq, hk=hk, dim=dim, page=page,
                    window=rng.choice((0, 0, 0, 128, 1000, 4096)))
    if op == "select":
        # bounds in all, and products; contexts of 64 pages and more, at most half of them selected
        most = int(min(6.6e7 / (reqs * hk * dim), 1e8 / (reqs * new * hk * dim)) * page)
        length = _log_int(rng, 64 * page, max(64 * page, min(131072, most)))
        first, newest = rng.choice((0, 1, 2)), rng.choice((0, 1, 2, 4))
        return dict(op=op, reqs=reqs, new=new, len=length, mix=mix, hq=hq, hk=hk, dim=dim, page=page,
                    pages=_log_int(rng, first + newest + 2, max(first + newest + 2, min(256, length // page // 2))), first=first, newest=newest,
                    format=kind[0], dtype=kind[1])
    length = _log_int(rng, 9, min(131072, int(4.5e8 / (reqs * hk * dim))))
    pages = min(_log_int(rng, 1, 256), -(-length // page), max(1, int(2.6e8 / BYTES[kind[1]] / (reqs * new * hk * page * dim))))
    return dict(op=op, reqs=reqs, new=new, len=length, mix=mix, hq=hq, hk=hk, dim=dim, page=page, pages=pages, format=kind[0], dtype=kind[1])


def _ragged(mix, n, most, least=1):
    """n lengths up to `most`, the first of them `most`: spread over their logarithm, or all the same with mix 0."""
    if mix == 0 or most <= least:
        return [most] * n
    rng = random.Random(mix)
    return [most] + [_log_int(rng, max(1, least), most) for _ in range(n - 1)]


def _plan(case):
    """New tokens and cached tokens (the new ones included) of every request."""
    r = case["reqs"]
    if case["op"] == "read":
        lens = _ragged(case["mix"], r, case["len"])
        return lens, lens
    if case["op"] in ("append", "bounds"):
        new = _ragged(case["mix"] if case["new"] > 1 else 0, r, case["new"])
        past = [0] * r if case["past"] == 0 else _ragged(case["mix"] + 1, r, case["past"])
        return new, [n + p for n, p in zip(new, past)]
    # the lengths of a running batch: within a factor of eight of each other
    lens = _ragged(case["mix"], r, case["len"], least=max(case["new"], case["len"] // 8))
    new = _ragged(case["mix"] if case["new"] > 1 else 0, r, case["new"])
    return [min(n, m) for n, m in zip(new, lens)], lens


def _lists(case):
    """Lists [N, Hk, K] and counts [N] of a sparse case: the first and the newest page and others by chance, those of a
    request's drafts mostly the same."""
    new, lens = _plan(case)
    k, ps, hk = case["pages"], case["page"], case["hk"]
    rs = np.random.RandomState(case["mix"] + 17)
    lists, counts = np.full((sum(new), hk, k), -1, np.int32), np.zeros(sum(new), np.int32)
    n = 0
    for t, m in zip(new, lens):
        common = rs.random_sample((hk, -(-m // ps)))
        for j in range(t):
            held = (m - t + j) // ps + 1
            score = common[:, :held] + 0.1 * rs.random_sample((hk, held))
            score[:, 0] = 2.0
            score[:, held - 1] = 3.0
            counts[n] = min(k, held)
            lists[n, :, :counts[n]] = np.sort(np.argsort(-score, axis=1, kind="stable")[:, :counts[n]], axis=1)
            n += 1
    return lists, counts


def _row_bytes(case):
    """Bytes of one head's k or v of one token in the cache."""
    d, kind = case["dim"], case.get("format", "e2m1")
    return d * BYTES[case["dtype"]] if kind == "io" else d + 1 if kind == "e4m3" else d // 2 + d // 32


def work(case):
    d, hk, row, b = case["dim"], case["hk"], _row_bytes(case), BYTES[case.get("dtype", "f16")]
    new, lens = _plan(case)
    n = sum(new)
    if case["op"] == "append":                                 # q, k, v in; q and the rows out; the rows as values
        return {"bytes": n * (2 * case["hq"] * d * b + 4 * hk * d * b + 2 * hk * row), "flops": 3 * n * (case["hq"] + hk) * case["rot"]}
    if case["op"] == "read":
        return {"bytes": sum(lens) * 2 * hk * (row + d * b), "flops": 0}
    ps = case["page"]
    if case["op"] == "bounds":
        pages = sum((m - 1) // ps - (m - t) // ps + 1 for t, m in zip(new, lens))
        keys = sum(m - (m - t) // ps * ps for t, m in zip(new, lens))
        return {"bytes": keys * hk * row + pages * hk * 2 * d * b, "flops": 2 * keys * hk * d}
    hq = case["hq"]
    if case["op"] == "select":
        pages = sum(-(-m // ps) for m in lens)
        pairs = sum((m - t + j) // ps + 1 for t, m in zip(new, lens) for j in range(t))
        return {"bytes": pages * hk * 2 * d * b + n * hq * d * b + 4 * n * hk * case["pages"], "flops": 4 * pairs * hk * d + n * hq * d}
    if case["op"] == "sparse":
        lists, counts = _lists(case)
        read, pairs, at = 0, 0, 0
        for t, m in zip(new, lens):
            held = np.zeros((hk, -(-m // ps)), bool)
            for j in range(t):
                mine = lists[at, :, :counts[at]]
                held[np.arange(hk)[:, None], mine] = True
                pairs += hk * (int(counts[at]) * ps - ps + (m - t + j) % ps + 1)
                at += 1
            read += int(held.sum()) * ps - (hk * (-m % ps) if t else 0)
        return {"bytes": 2 * read * row + 2 * n * hq * d * b + 4 * n * hk * case["pages"], "flops": 4 * pairs * (hq // hk) * d}
    w, read, pairs = case["window"], 0, 0
    for t, m in zip(new, lens):
        read += m - (max(0, m - t + 1 - w) if w and t else 0) if t else 0
        pairs += sum(min(m - t + j + 1, w) if w else m - t + j + 1 for j in range(t))
    return {"bytes": 2 * read * hk * row + 2 * n * hq * d * b, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------- inputs
def _i32(v):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(v, np.int32))).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    io, d, hk, ps = IO[case.get("dtype", "f16")], case["dim"], case["hk"], case["page"]
    kind = case.get("format", "e2m1")

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(io)

    s = {"case": case, "io": io, "kind": kind}
    new, lens = _plan(case)
    r, n = case["reqs"], sum(new)
    cu = np.concatenate([[0], np.cumsum(np.asarray(new, np.int64))]).astype(np.int32)
    s["cu"], s["cu_host"] = _i32(cu), cu
    s["lens"], s["lens_host"] = _i32(lens), np.asarray(lens, np.int32)
    s["same"] = min(new) == max(new)
    # the pages of the requests, scattered over a pool with a few spare ones; a table ends with entries that name no page
    each = np.asarray([-(-m // ps) for m in lens])
    pool = int(each.sum()) + 3
    ids = torch.randperm(pool, generator=g, device=DEV)[: int(each.sum())].to(torch.int32)
    used = torch.from_numpy(np.arange(each.max() + 2)[None, :] < each[:, None]).to(DEV)
    table = torch.full(used.shape, -1, dtype=torch.int32, device=DEV)
    table[used] = ids
    s["table"] = table
    # keys have a few channels well above the others
    wide = torch.where(torch.arange(d, device=DEV) % 37 == 5, 4.0, 1.0)

    def pages(which):
        if case["op"] == "select":                             # the selection reads no page
            empty = {"io": (d, io), "e4m3": (d, torch.float8_e4m3fn), "e2m1": (d // 2, torch.uint8)}[kind]
            scales = {"io": None, "e4m3": (pool, hk, ps), "e2m1": (pool, hk, d // 32, ps)}[kind]
            return (torch.empty((pool, hk, ps, empty[0]), dtype=empty[1], device=DEV),
                    None if scales is None else torch.empty(scales, dtype=torch.uint8, device=DEV))
        x = torch.randn((pool, hk, ps, d), generator=g, device=DEV, dtype=torch.float32)
        x = (x * wide if which == "k" else x).to(io)
        return (x, None) if kind == "io" else _quantise8(x) if kind == "e4m3" else _quantise4(x)

    (s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]) = pages("k"), pages("v")
    if case["op"] == "append":
        i = np.arange(case["rot"] // 2, dtype=np.float64)
        s["inv_freq"] = torch.from_numpy(1e6 ** (-2.0 * i / case["rot"])).to(DEV)
        s["q"], s["k"], s["v"] = normal(n, case["hq"], d), normal(n, hk, d) * wide.to(io), normal(n, hk, d)
        s["q_out"] = torch.empty_like(s["q"])
    if case["op"] in ("append", "read"):
        s["k_out"], s["v_out"] = (torch.empty((n, hk, d), dtype=io, device=DEV) for _ in range(2))
    if case["op"] == "bounds":
        s["bounds"] = normal(pool, hk, 2, d)
        # the entries that hold a new token, and their requests: what a program knows of its batch
        spans = [((m - t) // ps, (m - 1) // ps + 1) for t, m in zip(new, lens)]
        s["touched"] = tuple(torch.from_numpy(x).to(DEV) for x in (
            np.concatenate([np.full(b - a, i) for i, (a, b) in enumerate(spans)]), np.concatenate([np.arange(a, b) for a, b in spans])))
    if case["op"] == "select":
        mid, reach = normal(pool, hk, d).float() * wide * 0.5, 2.3 * wide + 0.4 * normal(pool, hk, d).float().abs()
        s["bounds"] = torch.stack((mid - reach, mid + reach), 2).to(io)
        s["lists"] = torch.empty((n, hk, case["pages"]), dtype=torch.int32, device=DEV)
        s["counts"] = torch.empty(n, dtype=torch.int32, device=DEV)
    if case["op"] == "sparse":
        s["lists"], s["counts"] = (_i32(x) for x in _lists(case))
    if case["op"] in ("attn", "select", "sparse"):
        s["q"] = normal(n, case["hq"], d, scale=1.5)
        s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------------------------------- plain forms
def _power(k):
    """2^k in float32 for whole k in -126 .. 127."""
    return ((k + 127).to(torch.int32) << 23).view(torch.float32)


def _quantise8(x):
    """e4m3 codes of finite x [..., D] and the exponent byte of each row's scale, the smallest power of two that keeps it
    within 448."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                                    # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    k = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), -127)
    return (x * _power((-k).clamp(max=127))).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8).squeeze(-1)


def _blocks4(x):
    """e2m1 codes of finite x [..., D], one a byte, and the exponent bytes [..., D / 32] of the scales of 32 neighbours, the
    smallest power of two up to 2^13 that keeps them within 6: the nearest code, ties to the even one, at most 6."""
    x = x.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                                    # 6 = 0.75 * 2^3
    k = torch.where(amax > 0, (e - 3 + (m > 0.75).to(e.dtype)).clamp(max=13), -127)
    a = (x * _power((-k).clamp(max=127))).abs()
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    return (c + torch.signbit(x).byte() * 8).flatten(-2), (k + 127).to(torch.uint8).squeeze(-1)


def _quantise4(x):
    """Pages of e2m1, two codes a byte, and their exponent bytes: x [P, Hk, page, D]."""
    c, s = _blocks4(x)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.transpose(-1, -2).contiguous()


def _values4(codes, scales):
    """What 4-bit rows hold, in float32: codes [..., D / 2], scales [..., D / 32]."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    return (v[c].unflatten(-1, (-1, 32)) * _power(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _values(s, which, page, slot=None):
    """What pages [...] (or a slot of each) hold, in float32."""
    at = page if slot is None else (page, slice(None), slot)
    pages, scales = s[which + "_pages"], s[which + "_scales"]
    if s["kind"] == "io":
        return pages[at].float()
    if s["kind"] == "e4m3":
        return pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * _power(scales[at].int() - 127).unsqueeze(-1)
    return _values4(pages[at], scales.transpose(-1, -2)[at])


def _rotate(x, positions, inv_freq, rot, layout):
    """x [N, H, D] rotated by its positions: angles in double precision; of the two products that make an element the second
    is rounded to float32, and then the sum, as a fused multiply-add does. A key next to a border of its 4-bit code lands on
    the same side whoever computes it."""
    ang = positions.double()[:, None] * inv_freq[None, :]
    c, s = ang.cos().float()[:, None], ang.sin().float()[:, None]
    xf = x.float()
    a, b = (xf[..., 0:rot:2], xf[..., 1:rot:2]) if layout == "interleaved" else (xf[..., : rot // 2], xf[..., rot // 2:rot])
    ra = (a.double() * c.double() - (b * s).double()).float()
    rb = (b.double() * c.double() + (a * s).double()).float()
    turned = torch.stack((ra, rb), -1).flatten(-2) if layout == "interleaved" else torch.cat((ra, rb), -1)
    return torch.cat((turned, xf[..., rot:]), -1).to(x.dtype)


def _places(s, n):
    """Position, page and slot of every packed token."""
    at = torch.arange(n, device=s["cu"].device, dtype=torch.int32)
    r = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    pos = s["lens"][r] - s["cu"][1:][r] + at
    return pos, s["table"][r, (pos // s["case"]["page"]).long()].long(), (pos % s["case"]["page"]).long()


def _plain_append(s):
    case = s["case"]
    pos, page, slot = _places(s, s["k"].shape[0])
    turn = (pos, s["inv_freq"], case["rot"], case["layout"])
    q, k = _rotate(s["q"], *turn), _rotate(s["k"], *turn)
    for which, x in (("k", k), ("v", s["v"])):
        c, scale = _blocks4(x)
        s[which + "_pages"][page, :, slot] = c[..., 0::2] | (c[..., 1::2] << 4)
        s[which + "_scales"].transpose(-1, -2)[page, :, slot] = scale
    return q, _values(s, "k", page, slot).to(s["io"]), _values(s, "v", page, slot).to(s["io"])


def _plain_read(s):
    _, page, slot = _places(s, s["k_out"].shape[0])
    return _values(s, "k", page, slot).to(s["io"]), _values(s, "v", page, slot).to(s["io"])


def _plain_bounds(s):
    r, i = s["touched"]
    page, ps = s["table"][r, i].long(), s["case"]["page"]
    held = (i[:, None] * ps + torch.arange(ps, device=i.device) < s["lens"][r][:, None])[:, None, :, None]
    k = _values(s, "k", page)
    s["bounds"][page, :, 0] = torch.where(held, k, math.inf).amin(2).to(s["io"])
    s["bounds"][page, :, 1] = torch.where(held, k, -math.inf).amax(2).to(s["io"])
    return s["bounds"]


def _of_tokens(s):
    """Request, newest position and table entries up to it of every packed token."""
    at = torch.arange(s["q"].shape[0], device=s["cu"].device, dtype=torch.int32)
    r = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    pos = s["lens"][r] - s["cu"][1:][r] + at
    return r, pos, pos // s["case"]["page"] + 1


def _plain_select(s):
    case = s["case"]
    (n, hq, d), hk, r, t, most = s["q"].shape, case["hk"], case["reqs"], case["new"], case["pages"]
    new = s["cu"][1:] - s["cu"][:-1]
    j = torch.arange(t, device=new.device)
    token = (s["cu"][:-1, None] + j).clamp(max=n - 1).long()                   # [R, T], past a request's own tokens: any
    q = s["q"][token].double().view(r, t, hk, hq // hk, d)
    w = torch.stack((q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)), 3)         # [R, T, Hk, 2, D]
    b = s["bounds"][s["table"].clamp(min=0).long()].double()                   # [R, M, Hk, 2, D]
    x = torch.matmul(b.permute(0, 2, 1, 3, 4).flatten(3), w.permute(0, 2, 3, 4, 1).flatten(2, 3).contiguous())     # [R, Hk, M, T]
    mine = torch.arange(n, device=new.device, dtype=torch.int32)
    req, _, held = _of_tokens(s)
    x = x[req, :, :, (mine - s["cu"][req]).long()]                             # [N, Hk, M]
    i = torch.arange(x.shape[2], device=x.device, dtype=torch.int32)
    forced = (i < case["first"]) | (i >= held[:, None] - case["newest"])
    x = torch.where(forced[:, None], math.inf, x).masked_fill((i >= held[:, None])[:, None], -math.inf)
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :most]
    if best.shape[2] < most:
        best = torch.cat((best, best.new_zeros(n, hk, most - best.shape[2])), -1)
    counts = held.clamp(max=most).int()
    there = (torch.arange(most, device=x.device) < counts[:, None])[:, None]
    best = torch.sort(best.masked_fill(~there, 1 << 40), dim=-1).values
    s["lists"].copy_(torch.where(there, best, -1))
    s["counts"].copy_(counts)
    return s["lists"], s["counts"]


def _softmax(x):
    """Weights and their sum over the last dimension, zeros where nothing is attended."""
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    return p, p.sum(-1, keepdim=True)


def _plain_sparse(s):
    case = s["case"]
    (n, hq, d), hk, ps = s["q"].shape, case["hk"], case["page"]
    req, pos, _ = _of_tokens(s)
    listed_here = torch.arange(case["pages"], device=pos.device) < s["counts"][:, None]
    entry = torch.where(listed_here[:, None], s["lists"], -1)                  # [N, Hk, K]
    page = s["table"][req[:, None, None], entry.clamp(min=0).long()].long()
    at = entry[..., None] * ps + torch.arange(ps, device=pos.device)
    sees = ((entry[..., None] >= 0) & (at <= pos[:, None, None, None])).view(n, hk, 1, -1)

    def gather(which):
        pages, scales, h = s[which + "_pages"], s[which + "_scales"], torch.arange(hk, device=pos.device)[:, None]
        if s["kind"] == "io":
            x = pages[page, h].float()
        elif s["kind"] == "e4m3":
            x = pages.view(torch.uint8)[page, h].view(torch.float8_e4m3fn).float() * _power(scales[page, h].int() - 127).unsqueeze(-1)
        else:
            x = _values4(pages[page, h], scales.transpose(-1, -2)[page, h])
        return torch.where(sees.view(n, hk, -1, 1), x.view(n, hk, -1, d), 0.0)

    q = s["q"].float().view(n, hk, hq // hk, d)
    x = torch.matmul(q, gather("k").transpose(-1, -2)) * d ** -0.5
    p, total = _softmax(x.masked_fill(~sees, -math.inf))
    o = torch.matmul(p, gather("v"))
    return torch.where(total > 0, o / total, 0.0).view(n, hq, d).to(s["io"])


def _plain_attention(s):
    case = s["case"]
    n, hq, d = s["q"].shape
    hk, r, t = case["hk"], case["reqs"], case["new"]

    def gather(which):
        x = _values(s, which, s["table"].clamp(min=0).long())                  # [R, M, Hk, page, D]
        return x.transpose(1, 2).reshape(r, hk, -1, d)

    k, v = gather("k"), gather("v")
    new = s["cu"][1:] - s["cu"][:-1]
    j, at = torch.arange(t, device=k.device), torch.arange(k.shape[2], device=k.device)
    token = (s["cu"][:-1, None] + j).clamp(max=n - 1).long()
    q = s["q"][token].float().reshape(r, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(r, hk, t * (hq // hk), d)
    last = (s["lens"] - new)[:, None] + j                                      # the newest position that token j attends
    sees = (at <= last[..., None]) & (at < s["lens"][:, None, None])
    if case["window"]:
        sees &= at > last[..., None] - case["window"]
    held = (at < s["lens"][:, None])[:, None, :, None]
    k, v = torch.where(held, k, 0.0), torch.where(held, v, 0.0)
    x = torch.matmul(q, k.transpose(-1, -2)).view(r, hk, t, hq // hk, -1) * d ** -0.5
    p, total = _softmax(x.masked_fill(~sees[:, None, :, None], -math.inf))
    o = torch.matmul(p.view(r, hk, t * (hq // hk), -1), v).view(r, hk, t, hq // hk, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(r, t, hq, d)
    mine = torch.arange(n, device=k.device, dtype=torch.int32)
    req = torch.searchsorted(s["cu"][1:].contiguous(), mine, right=True)
    return o[req, (mine - s["cu"][req]).long()].to(s["io"])


# ---------------------------------------------------------------------------------------------------- run
def _handles(s):
    """The cache's description and the workspace, which a program makes once."""
    import gateddeltanet_recurrence_amd as gdn
    if "cache" not in s:
        case = s["case"]
        cache = s["cache"] = gdn.KVCache(s["k_pages"], s["v_pages"], s["table"], k_scales=s["k_scales"], v_scales=s["v_scales"])
        need = 0
        if case["op"] == "attn":
            need = gdn.gdn_attn_workspace_bytes(s["q"].shape[0], case["reqs"], case["hq"], cache)
        elif case["op"] == "select":
            need = gdn.gdn_attn_select_workspace_bytes(s["q"].shape[0], case["reqs"], case["hq"], case["pages"], cache)
        elif case["op"] == "sparse":
            need = gdn.gdn_attn_sparse_workspace_bytes(s["q"].shape[0], case["reqs"], case["hq"], case["pages"], cache)
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["table"].device)
    return gdn, s["cache"]


def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse,
                "attn": _plain_attention}[case["op"]](s)
    gdn, cache = _handles(s)
    cu = None if s["same"] else s["cu"]
    rows = dict(num_reqs=case["reqs"], seq_lens_host=s["lens_host"], cu_seqlens_host=None if s["same"] else s["cu_host"])
    if case["op"] == "append":
        gdn.gdn_kv_write(s["k"], s["v"], cache, s["lens"], cu, q=s["q"], q_out=s["q_out"], inv_freq=s["inv_freq"],
                         rope_layout=gdn.ROPE_INTERLEAVED if case["layout"] == "interleaved" else gdn.ROPE_HALF, **rows)
        gdn.gdn_kv_read(s["k_out"], s["v_out"], cache, s["lens"], cu, **rows)
        return s["q_out"], s["k_out"], s["v_out"]
    if case["op"] == "read":
        gdn.gdn_kv_read(s["k_out"], s["v_out"], cache, s["lens"], cu, **rows)
        return s["k_out"], s["v_out"]
    if case["op"] == "bounds":
        gdn.gdn_kv_bounds(s["bounds"], cache, s["lens"], cu, num_tokens=int(s["cu_host"][-1]), **rows)
        return s["bounds"]
    if case["op"] == "select":
        gdn.gdn_attn_select(s["q"], s["bounds"], cache, s["lens"], cu, s["lists"], s["counts"], first_pages=case["first"],
                            newest_pages=case["newest"], workspace=s["workspace"], **rows)
        return s["lists"], s["counts"]
    if case["op"] == "sparse":
        gdn.gdn_attn_sparse_forward(s["q"], cache, s["lens"], cu, s["lists"], s["counts"], s["out"], workspace=s["workspace"], **rows)
        return s["out"]
    gdn.gdn_attn_forward(s["q"], cache, s["lens"], cu, s["out"], window=case["window"], workspace=s["workspace"], **rows)
    return s["out"]


# ---------------------------------------------------------------------------------------------------- 64 bits
def _turn_exact(x, pos, case, s):
    """x [N, H, D] as complex numbers, each pair times e^(i pos f)."""
    x = x.double()
    half = case["rot"] // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + half)
    w = torch.polar(torch.ones((len(pos), half), dtype=torch.float64, device=x.device), torch.outer(pos.double(), s["inv_freq"]))[:, None]
    z = torch.complex(x[..., first], x[..., second]) * w
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _rounded_exact(x):
    """x [..., D] as the 4-bit cache holds it, by the format's definition: steps of a half up to 2, then of a quarter of the
    power of two below, half-way values to the even multiple."""
    y = x.double().unflatten(-1, (-1, 32))
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.full_like(amax, 2.0 ** -30)
    for _ in range(43):                                        # from 2^-30 up to the first power of two that keeps amax within 6
        scale = torch.where(amax > 6 * scale, scale * 2, scale)
    y = (y / scale).clamp(-6, 6)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return (torch.round(y / step) * step * scale).flatten(-2)


def _cells_exact(s, which):
    """What the pool holds in 64 bits: [P, Hk, page, D]."""
    pages, scales = s[which + "_pages"], s[which + "_scales"]
    if s["kind"] == "io":
        return pages.double()
    if s["kind"] == "e4m3":
        return pages.double() * torch.exp2(scales.double() - 127)[..., None]
    out = torch.empty((*pages.shape[:-1], 2 * pages.shape[-1]), dtype=torch.float64, device=pages.device)
    for half in range(2):
        code = (pages >> (4 * half)).int() & 15
        e, m = (code >> 1) & 3, (code & 1).double()            # sign, two exponent bits (bias 1), one bit of mantissa
        a = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
        out[..., half::2] = torch.where(code >= 8, -a, a)
    return out * torch.exp2(scales.double() - 127).transpose(-1, -2).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    io, cu, lens, ps, hk, d = s["io"], s["cu_host"], s["lens_host"], case["page"], case["hk"], case["dim"]
    dev = s["table"].device
    if case["op"] == "append":
        pos = torch.cat([torch.arange(int(m) - t, int(m), device=dev) for t, m in zip(np.diff(cu).tolist(), lens)])
        # what is quantised is the key in the type it is given in
        return (_turn_exact(s["q"], pos, case, s), _rounded_exact(_turn_exact(s["k"], pos, case, s).to(io)), _rounded_exact(s["v"]))
    if case["op"] == "select":
        q = s["q"].double().view(-1, hk, case["hq"] // hk, d)
        lists, counts = np.full(tuple(s["lists"].shape), -1, np.int32), np.zeros(q.shape[0], np.int32)
        for r in range(case["reqs"]):
            for n in range(int(cu[r]), int(cu[r + 1])):
                held = (int(lens[r]) - int(cu[r + 1]) + n) // ps + 1
                b = s["bounds"][s["table"][r, :held].long()].double().transpose(0, 1)     # [Hk, held, 2, D]
                x = torch.zeros((hk, held), dtype=torch.float64, device=dev)
                for g in range(q.shape[2]):
                    x += torch.maximum(q[n, :, g, None] * b[..., 0, :], q[n, :, g, None] * b[..., 1, :]).sum(-1)
                x = x.cpu().numpy()
                x[:, :case["first"]] = np.inf
                x[:, max(0, held - case["newest"]):] = np.inf
                counts[n] = min(held, case["pages"])
                lists[n, :, :counts[n]] = np.sort(np.argsort(-x, axis=1, kind="stable")[:, :counts[n]], axis=1)
        return torch.from_numpy(lists), torch.from_numpy(counts)
    kp = _cells_exact(s, "k")
    if case["op"] == "bounds":
        out = s["bounds"].double()
        for r in range(case["reqs"]):
            t, m = int(cu[r + 1] - cu[r]), int(lens[r])
            for i in range((m - t) // ps, (m - 1) // ps + 1):
                page = int(s["table"][r, i])
                k = kp[page, :, :min(ps, m - i * ps)]
                out[page, :, 0], out[page, :, 1] = k.min(1).values, k.max(1).values
        return out
    vp = _cells_exact(s, "v")

    def cells(r, at):
        return s["table"][r].long()[at // ps], at % ps

    if case["op"] == "read":
        both = [cells(r, torch.arange(int(lens[r]), device=dev)) for r in range(case["reqs"])]
        page, slot = torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])
        return kp[page, :, slot], vp[page, :, slot]
    hq, w = case["hq"], case.get("window", 0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)

    def attend(q, k, v):                                       # [H, G, D], [H, L, D]
        return torch.bmm(torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) / math.sqrt(d), -1), v)

    for r in range(case["reqs"]):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if case["op"] == "attn":
            lowest = max(0, m - (b - a) + 1 - w) if w else 0
            page, slot = cells(r, torch.arange(lowest, m, device=dev))
            k, v = kp[page, :, slot].transpose(0, 1).contiguous(), vp[page, :, slot].transpose(0, 1).contiguous()
        for n in range(a, b):
            q, hi = s["q"][n].double().view(hk, hq // hk, d), m - b + n + 1
            if case["op"] == "attn":
                lo = max(0, hi - w) if w else 0
                out[n] = attend(q, k[:, lo - lowest:hi - lowest], v[:, lo - lowest:hi - lowest]).view(hq, d)
                continue
            count = int(s["counts"][n])
            for h in range(hk):
                at = (s["lists"][n, h, :count].long()[:, None] * ps + torch.arange(ps, device=dev)).flatten()
                page, slot = cells(r, at[at < hi])
                o = attend(q[h:h + 1], kp[page, h, slot][None], vp[page, h, slot][None])
                out[n, h * (hq // hk):(h + 1) * (hq // hk)] = o[0]
    return out
