"""What is measured of the attention layer's operators: rotary positions, the paged key-value cache (written, quantised on
request, and read back) and the attention of a request's newest tokens over it.

Every case is a dict of plain values; `run` computes it with elementary torch operations where `own` is false and with the
library's entry points where it is true. Layouts (io: float16 or float32):

  q [N, Hq, D], k and v [N, Hk, D]   packed tokens, request r owning cu[r] .. cu[r+1]-1
  pages [P, Hk, page, D]             io, or float8_e4m3fn with a power-of-two scale per (page, head, token), kept as its exponent byte
  page_table [R, M]                  the page that holds a request's positions page*i .. page*i + page-1 (-1: none)
  seq_lens [R]                       a request's cached tokens, its newest ones included
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
IO = {"f16": torch.float16, "f32": torch.float32}
BYTES = {"f16": 2, "f32": 4}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the rotation of a ragged prompt batch (8 prompts, 15,352 tokens) of a layer that rotates a quarter of its head
        dict(name="rope_prompt_f16", op="rope", tokens=15352, reqs=8, far=4096, hq=24, hk=4, dim=256, rot=64, layout="half", scaling="none",
             dtype="f16"),
        # an odd number of tokens of a long context (positions to a million), whole heads in the interleaved layout
        dict(name="rope_far_f32", op="rope", tokens=2049, reqs=3, far=1 << 20, hq=32, hk=8, dim=128, rot=128, layout="interleaved",
             scaling="yarn", dtype="f32"),
        # one decode step of 64 requests: q and k rotated, k and v into the pages; latency counts
        dict(name="write_decode_f16", op="write", reqs=64, new=1, mix=11, past=500, hq=24, hk=4, dim=256, rot=64, layout="half", page=64,
             format="io", dtype="f16"),
        # draft tokens of a speculative step (up to 4 for each of 16 requests) into an 8-bit cache
        dict(name="write_drafts_e4m3", op="write", reqs=16, new=4, mix=12, past=300, hq=32, hk=8, dim=128, rot=128, layout="half", page=16,
             format="e4m3", dtype="f16"),
        # ragged prompts into an 8-bit cache
        dict(name="write_prompt_e4m3", op="write", reqs=8, new=4096, mix=3, past=0, hq=24, hk=4, dim=256, rot=64, layout="half", page=64,
             format="e4m3", dtype="f16"),
        # a long cached prefix read back for the attention of a further prompt
        dict(name="read_long_e4m3", op="read", reqs=1, len=32768, mix=0, hk=4, dim=256, page=64, format="e4m3", dtype="f16"),
        # short ragged prefixes in single precision
        dict(name="read_ragged_f32", op="read", reqs=5, len=1993, mix=5, hk=2, dim=64, page=16, format="io", dtype="f32"),
        # the smallest step: one request, one token, a short cache
        dict(name="attn_one_short_f16", op="attn", reqs=1, new=1, len=333, mix=0, hq=32, hk=8, dim=128, page=16, format="io", dtype="f16",
             window=0),
        # the decode step of a full batch over caches of mixed lengths
        dict(name="attn_decode_f16", op="attn", reqs=64, new=1, len=16384, mix=21, hq=32, hk=8, dim=128, page=64, format="io", dtype="f16",
             window=0),
        # the verify of up to 4 draft tokens for each of 16 requests, large heads in groups of 6
        dict(name="attn_verify_f16", op="attn", reqs=16, new=4, len=8192, mix=22, hq=24, hk=4, dim=256, page=64, format="io", dtype="f16",
             window=0),
        # one long context over an 8-bit cache: the cache's length is all there is to split
        dict(name="attn_long_e4m3", op="attn", reqs=1, new=1, len=131072, mix=0, hq=24, hk=4, dim=256, page=256, format="e4m3", dtype="f16",
             window=0),
        # a windowed layer in single precision, a head of its own for every query head, odd lengths
        dict(name="attn_window_f32", op="attn", reqs=7, new=3, len=5001, mix=23, hq=6, hk=6, dim=64, page=32, format="io", dtype="f32",
             window=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "write", "write", "read", "attn", "attn", "attn"))
    dim = rng.choice((64, 128, 256))
    hk = rng.choice((1, 2, 3, 4, 8))
    hq = hk * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice((16, 32, 64, 128, 256))
    kind = rng.choice((("io", "f16"), ("e4m3", "f16"), ("io", "f32")))
    layout = rng.choice(("half", "interleaved"))
    rot = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim])
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, min(32768, (1 << 27) // (hq * dim))), reqs=rng.randrange(1, 9), far=_log_int(rng, 64, 1 << 20),
                    hq=hq, hk=hk, dim=dim, rot=rot, layout=layout, scaling=rng.choice(("none", "linear", "ntk", "yarn")), dtype=kind[1])
    if op == "write":
        reqs = _log_int(rng, 1, 128)
        return dict(op=op, reqs=reqs, new=_log_int(rng, 1, max(1, min(8192, (1 << 25) // (reqs * (hq + hk) * dim)))), mix=mix,
                    past=_log_int(rng, 1, 1024), hq=hq, hk=hk, dim=dim, rot=rot, layout=layout, page=page,
                    format=kind[0], dtype=kind[1])
    if op == "read":
        reqs = _log_int(rng, 1, 64)
        return dict(op=op, reqs=reqs, len=_log_int(rng, 1, min(65536, (1 << 26) // (reqs * hk * dim))), mix=mix, hk=hk, dim=dim, page=page,
                    format=kind[0], dtype=kind[1])
    reqs, new = _log_int(rng, 1, 256), rng.choice((1, 1, 1, 2, 3, 4, 5, 8))
    most = int(9e8 / (reqs * hk * dim * BYTES[kind[1]] * max(1.0, new * hq / hk / 50)))      # bytes of keys, or flops
    return dict(op=op, reqs=reqs, new=new, len=_log_int(rng, 9, min(131072, most)), mix=rng.choice((0, mix, mix)), hq=hq, hk=hk, dim=dim, page=page, format=kind[0], dtype=kind[1],
                window=rng.choice((0, 0, 0, 128, 1000, 4096)))


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
    if case["op"] == "write":
        new = _ragged(case["mix"] if case["new"] > 1 else 0, r, case["new"])
        past = [0] * r if case["past"] == 0 else _ragged(case["mix"] + 1, r, case["past"])
        return new, [n + p for n, p in zip(new, past)]
    # the lengths of a running batch: within a factor of eight of each other
    lens = _ragged(case["mix"], r, case["len"], least=max(case["new"], case["len"] // 8))
    new = _ragged(case["mix"] if case["new"] > 1 else 0, r, case["new"])
    return [min(n, m) for n, m in zip(new, lens)], lens


def work(case):
    b, d = BYTES[case["dtype"]], case["dim"]
    if case["op"] == "rope":
        n, h = case["tokens"], case["hq"] + case["hk"]
        return {"bytes": 2 * n * h * d * b + 4 * n, "flops": 3 * n * h * case["rot"]}
    new, lens = _plan(case)
    row = d * b if case["format"] == "io" else d + 1           # one head's k or v of one token in the cache
    hk = case["hk"]
    if case["op"] == "write":
        n = sum(new)
        return {"bytes": n * (2 * case["hq"] * d * b + 2 * hk * d * b + 2 * hk * row), "flops": 3 * n * (case["hq"] + hk) * case["rot"]}
    if case["op"] == "read":
        return {"bytes": sum(lens) * 2 * hk * (row + d * b), "flops": 0}
    w, n, read, pairs = case["window"], sum(new), 0, 0
    for t, m in zip(new, lens):
        read += m - (max(0, m - t + 1 - w) if w and t else 0) if t else 0
        pairs += sum(min(m - t + j + 1, w) if w else m - t + j + 1 for j in range(t))
    return {"bytes": 2 * read * hk * row + 2 * n * case["hq"] * d * b, "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------------------------------------------- inputs
def _frequencies(case):
    """inv_freq [rot / 2] in double precision and the multiplier of cos and sin."""
    r, base = case["rot"], 1e6
    i = np.arange(r // 2, dtype=np.float64)
    scaling = case.get("scaling", "none")
    f = base ** (-2.0 * i / r)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "ntk":
        return (base * 8.0 ** (r / (r - 2.0))) ** (-2.0 * i / r), 1.0
    if scaling == "yarn":                                      # 32 and 1 rotations within 32768 trained positions bound the ramp
        at = lambda turns: r * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / 8.0 * ramp + f * (1 - ramp), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(new):
    return np.concatenate([[0], np.cumsum(np.asarray(new, np.int64))]).astype(np.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    io, d, hk = IO[case["dtype"]], case["dim"], case["hk"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(io)

    s = {"case": case}
    if case.get("rot"):
        f, s["factor"] = _frequencies(case)
        s["inv_freq"] = torch.from_numpy(f).to(DEV)
    if case["op"] == "rope":
        n = case["tokens"]
        s["q"], s["k"] = normal(n, case["hq"], d), normal(n, hk, d)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        # consecutive positions within a request, from a start of its own
        at = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, n + 1, case["reqs"] - 1)) if case["reqs"] > 1 else np.zeros(0, np.int64)
        start = np.concatenate([[0], at])[np.searchsorted(at, np.arange(n), side="right")]
        first = np.random.RandomState((seed + 1) % (1 << 31)).randint(0, max(1, case["far"] - n), n)[start.clip(0, n - 1)]
        s["positions"] = _i32((first + np.arange(n) - start).astype(np.int32))
        return s

    new, lens = _plan(case)
    r, ps, n = case["reqs"], case["page"], sum(new)
    cu = _cu(new)
    s["cu"], s["cu_host"] = torch.from_numpy(cu).to(DEV), cu
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

    def pages(kind):
        x = torch.randn((pool, hk, ps, d), generator=g, device=DEV, dtype=torch.float32)
        x = (x * wide if kind == "k" else x).to(io)
        return _quantise(x) if case["format"] == "e4m3" else (x, None)

    (s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]) = pages("k"), pages("v")
    if case["op"] == "write":
        s["q"], s["k"], s["v"] = normal(n, case["hq"], d), normal(n, hk, d) * wide.to(io), normal(n, hk, d)
        s["q_out"] = torch.empty_like(s["q"])
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty((n, hk, d), dtype=io, device=DEV) for _ in range(2))
    else:
        s["q"] = normal(n, case["hq"], d, scale=1.5)
        s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------------------------------- plain forms
def _power(k):
    """2^k in float32 for whole k in -126 .. 127."""
    return ((k + 127).to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 codes of x [..., D] and the exponent byte of each row's scale, the smallest power of two that keeps it within 448."""
    x = x.float()
    fine = torch.isfinite(x)
    amax = torch.where(fine, x, 0.0).abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                                    # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    k = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), -127)
    y = torch.where(fine, x * _power((-k).clamp(max=127)), float("nan"))
    return y.to(torch.float8_e4m3fn), (k + 127).to(torch.uint8).squeeze(-1)


def _values(pages, scales):
    """What pages hold, in float32."""
    return pages.float() if scales is None else pages.float() * _power(scales.int() - 127).unsqueeze(-1)


def _rotate(x, positions, inv_freq, factor, rot, layout):
    """x [N, H, D] rotated by its positions: angles in double precision, the rotation in float32."""
    ang = positions.double()[:, None] * inv_freq[None, :]
    c, s = (ang.cos() * factor).float()[:, None], (ang.sin() * factor).float()[:, None]
    xf = x.float()
    a, b = (xf[..., 0:rot:2], xf[..., 1:rot:2]) if layout == "interleaved" else (xf[..., : rot // 2], xf[..., rot // 2:rot])
    ra, rb = a * c - b * s, b * c + a * s
    turned = torch.stack((ra, rb), -1).flatten(-2) if layout == "interleaved" else torch.cat((ra, rb), -1)
    return torch.cat((turned, xf[..., rot:]), -1).to(x.dtype)


def _places(s, n):
    """Request, cache position and page-table entry of every packed token."""
    at = torch.arange(n, device=s["cu"].device, dtype=torch.int32)
    r = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
    pos = s["lens"][r] - s["cu"][1:][r] + at
    return pos, s["table"][r, (pos // s["case"]["page"]).long()].long(), (pos % s["case"]["page"]).long()


def _plain_write(s):
    case, n = s["case"], s["k"].shape[0]
    pos, page, slot = _places(s, n)
    turn = (pos, s["inv_freq"], s["factor"], case["rot"], case["layout"])
    q, k = _rotate(s["q"], *turn), _rotate(s["k"], *turn)
    if s["k_scales"] is None:
        s["k_pages"][page, :, slot], s["v_pages"][page, :, slot] = k, s["v"]
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    (kc, ks), (vc, vs) = _quantise(k), _quantise(s["v"])
    s["k_pages"].view(torch.uint8)[page, :, slot], s["v_pages"].view(torch.uint8)[page, :, slot] = kc.view(torch.uint8), vc.view(torch.uint8)
    s["k_scales"][page, :, slot], s["v_scales"][page, :, slot] = ks, vs
    return _written(s, q)


def _written(s, q):
    """The pages and the scales as the values they stand for."""
    out = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_scales"] is not None:
        out["k_scales"], out["v_scales"] = s["k_scales"].view(torch.float8_e8m0fnu), s["v_scales"].view(torch.float8_e8m0fnu)
    return out


def _plain_read(s):
    io = s["k_out"].dtype
    _, page, slot = _places(s, s["k_out"].shape[0])
    if s["k_scales"] is None:
        return s["k_pages"][page, :, slot], s["v_pages"][page, :, slot]
    k = _values(s["k_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn), s["k_scales"][page, :, slot])
    v = _values(s["v_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn), s["v_scales"][page, :, slot])
    return k.to(io), v.to(io)


def _gather(pages, scales, table):
    """Every request's cached tokens side by side: [R, Hk, M * page, D] in float32."""
    at = table.clamp(min=0).long()
    if scales is None:
        x = pages[at].float()
    else:
        x = _values(pages.view(torch.uint8)[at].view(torch.float8_e4m3fn), scales[at])
    r, m, h, p, d = x.shape
    return x.transpose(1, 2).reshape(r, h, m * p, d)


def _plain_attention(s):
    case = s["case"]
    n, hq, d = s["q"].shape
    hk, r, t = case["hk"], case["reqs"], case["new"]
    k, v = _gather(s["k_pages"], s["k_scales"], s["table"]), _gather(s["v_pages"], s["v_scales"], s["table"])
    new = s["cu"][1:] - s["cu"][:-1]
    j, at = torch.arange(t, device=k.device), torch.arange(k.shape[2], device=k.device)
    token = (s["cu"][:-1, None] + j).clamp(max=n - 1).long()                   # [R, T], past a request's own tokens: any
    q = s["q"][token].float().reshape(r, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(r, hk, t * (hq // hk), d)
    last = (s["lens"] - new)[:, None] + j                                      # the newest position that token j attends
    sees = (at <= last[..., None]) & (at < s["lens"][:, None, None])
    if case["window"]:
        sees &= at > last[..., None] - case["window"]
    held = (at < s["lens"][:, None])[:, None, :, None]
    k, v = torch.where(held, k, 0.0), torch.where(held, v, 0.0)
    x = torch.matmul(q, k.transpose(-1, -2)).view(r, hk, t, hq // hk, -1) * d ** -0.5
    x = x.masked_fill(~sees[:, None, :, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(r, hk, t * (hq // hk), -1), v).view(r, hk, t, hq // hk, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(r, t, hq, d)
    mine = torch.arange(n, device=k.device, dtype=torch.int32)
    req = torch.searchsorted(s["cu"][1:].contiguous(), mine, right=True)
    return o[req, (mine - s["cu"][req]).long()].to(s["q"].dtype)


# ---------------------------------------------------------------------------------------------------- run
def _handles(s):
    """The cache's description and the workspace, which a program makes once."""
    import gateddeltanet_recurrence_amd as gdn
    if "cache" not in s:
        s["cache"] = gdn.KVCache(s["k_pages"], s["v_pages"], s["table"], k_scales=s["k_scales"], v_scales=s["v_scales"])
        if s["case"]["op"] == "attn":
            need = gdn.gdn_attn_workspace_bytes(s["q"].shape[0], s["case"]["reqs"], s["q"].shape[1], s["cache"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["q"].device)
    return gdn, s["cache"]


def run(s):
    case = s["case"]
    if case["op"] == "rope":
        if own:
            import gateddeltanet_recurrence_amd as gdn
            gdn.gdn_rope_forward(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"],
                                 rope_layout=gdn.ROPE_INTERLEAVED if case["layout"] == "interleaved" else gdn.ROPE_HALF, rope_factor=s["factor"])
            return s["q_out"], s["k_out"]
        turn = (s["positions"], s["inv_freq"], s["factor"], case["rot"], case["layout"])
        return _rotate(s["q"], *turn), _rotate(s["k"], *turn)
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attn": _plain_attention}[case["op"]](s)
    gdn, cache = _handles(s)
    cu = None if s["same"] else s["cu"]
    rows = dict(num_reqs=case["reqs"], seq_lens_host=s["lens_host"], cu_seqlens_host=None if s["same"] else s["cu_host"])
    if case["op"] == "write":
        gdn.gdn_kv_write(s["k"], s["v"], cache, s["lens"], cu, q=s["q"], q_out=s["q_out"], inv_freq=s["inv_freq"], rope_factor=s["factor"],
                         rope_layout=gdn.ROPE_INTERLEAVED if case["layout"] == "interleaved" else gdn.ROPE_HALF, **rows)
        return _written(s, s["q_out"])
    if case["op"] == "read":
        gdn.gdn_kv_read(s["k_out"], s["v_out"], cache, s["lens"], cu, **rows)
        return s["k_out"], s["v_out"]
    gdn.gdn_attn_forward(s["q"], cache, s["lens"], cu, s["out"], window=case["window"], workspace=s["workspace"], **rows)
    return s["out"]


# ---------------------------------------------------------------------------------------------------- 64 bits
def _turn_exact(x, pos, case, s):
    """x [H, D] or [N, H, D] as complex numbers, each pair times factor * e^(i pos f)."""
    x = x.double()
    half = case["rot"] // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + half)
    w = torch.polar(torch.full((len(pos), half), float(s["factor"]), dtype=torch.float64, device=x.device),
                    torch.outer(pos.double(), s["inv_freq"]))[:, None]
    z = torch.complex(x[..., first], x[..., second]) * w
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _codes_exact(x):
    """e4m3 values of x [..., D] over its row's scale, and the scale, rounded by the format's definition: steps of 2^(e-3), 2^-9 at the least."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    k = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX)), torch.full_like(amax, -127.0))
    k = torch.where(amax > E4M3_MAX * torch.exp2(k), k + 1, k)                  # log2 may be off by its last bit
    k = torch.where((amax > 0) & (amax <= E4M3_MAX * torch.exp2(k - 1)), k - 1, k)
    y = x / torch.exp2(k)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(k).squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    io = IO[case["dtype"]]
    if case["op"] == "rope":
        return _turn_exact(s["q"], s["positions"], case, s), _turn_exact(s["k"], s["positions"], case, s)
    cu, lens, ps = s["cu_host"], s["lens_host"], case["page"]
    eight = case["format"] == "e4m3"
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    if eight:
        ks, vs = torch.exp2(s["k_scales"].double() - 127), torch.exp2(s["v_scales"].double() - 127)

    def cells(r, lo, hi):
        at = torch.arange(lo, hi, device=kp.device)
        return s["table"][r].long()[at // ps], at % ps

    if case["op"] == "write":
        q = torch.empty(s["q"].shape, dtype=torch.float64, device=kp.device)
        for r in range(case["reqs"]):
            a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
            if a == b:
                continue
            pos = torch.arange(m - (b - a), m, device=kp.device)
            q[a:b] = _turn_exact(s["q"][a:b], pos, case, s)
            k, v = _turn_exact(s["k"][a:b], pos, case, s), s["v"][a:b].double()
            page, slot = cells(r, m - (b - a), m)
            if eight:                                          # what is quantised is the key in the type it is given in
                (k, k_scale), (v, v_scale) = _codes_exact(k.to(io)), _codes_exact(v)
                ks[page, :, slot], vs[page, :, slot] = k_scale, v_scale
            kp[page, :, slot], vp[page, :, slot] = k, v
        out = {"q": q, "k_pages": kp, "v_pages": vp}
        return {**out, "k_scales": ks, "v_scales": vs} if eight else out
    if eight:
        kp, vp = kp * ks[..., None], vp * vs[..., None]
    if case["op"] == "read":
        both = [cells(r, 0, int(lens[r])) for r in range(case["reqs"])]
        page, slot = torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])
        return kp[page, :, slot], vp[page, :, slot]
    hq, hk, d = case["hq"], case["hk"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=kp.device)
    for r in range(case["reqs"]):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        lowest = max(0, m - (b - a) + 1 - case["window"]) if case["window"] else 0
        page, slot = cells(r, lowest, m)
        k, v = kp[page, :, slot].transpose(0, 1).contiguous(), vp[page, :, slot].transpose(0, 1).contiguous()   # [Hk, L, D]
        for j in range(b - a):
            hi = m - (b - a) + j + 1
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= lo:
                continue
            q = s["q"][a + j].double().view(hk, hq // hk, d)
            x = torch.bmm(q, k[:, lo - lowest:hi - lowest].transpose(1, 2).contiguous()) / math.sqrt(d)
            out[a + j] = torch.bmm(torch.softmax(x, -1), v[:, lo - lowest:hi - lowest]).view(hq, d)
    return out
