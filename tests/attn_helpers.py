"""Inputs and calls shared by the GPU tests of the attention layer."""
from __future__ import annotations

import numpy as np

from gpu_helpers import dev
from oracle import attn_oracle as AO

FORMATS = ("f16", "f32", "e4m3")


def page_table(lens, page, rng, spare=2, extra=2):
    """(table [R, M], pages in the pool): every request's pages scattered, -1 behind them."""
    each = [-(-m // page) for m in lens]
    P = sum(each) + spare
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((len(lens), max(each, default=0) + extra), -1, np.int32)
    at = 0
    for r, n in enumerate(each):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, P


def make_cache(lens, *, Hk, D, fmt, page, seed, fill="nan", scale=1.0, wide=True):
    """The cache of requests with `lens` tokens; unused slots hold `fill` (0x7f, NaN, in 8-bit pages)."""
    rng = np.random.default_rng(seed)
    table, P = page_table(lens, page, rng)
    io = np.float32 if fmt == "f32" else np.float16
    full = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    c = {"fmt": fmt, "table": table, "P": P, "page": page, "Hk": Hk, "D": D, "lens": np.asarray(lens, np.int32)}
    for name in ("k", "v"):
        rows = rng.standard_normal((full[-1], Hk, D)) * scale
        if wide and name == "k":
            rows[..., 5::37] *= 4.0                     # a few channels above the others
        rows = rows.astype(io)
        pool = np.full((P, Hk, page, D), fill if fill != "nan" else np.nan, io)
        if fmt == "e4m3":
            codes, s = AO.quantise(rows)
            c[name + "_codes"] = AO.cache_write(codes, np.full(pool.shape, 0x7f, np.uint8), table, full, lens)
            c[name + "_scales"] = AO.cache_write(s, np.full(pool.shape[:3], 130, np.uint8), table, full, lens)
            c[name] = AO.dequantise(c[name + "_codes"], c[name + "_scales"])
        else:
            c[name] = AO.cache_write(rows, pool, table, full, lens)
    return c


def device_cache(c, torch, gdn, **kw):
    if c["fmt"] == "e4m3":
        return gdn.KVCache(dev(c["k_codes"], torch), dev(c["v_codes"], torch), dev(c["table"], torch),
                           k_scales=dev(c["k_scales"], torch), v_scales=dev(c["v_scales"], torch), **kw)
    return gdn.KVCache(dev(c["k"], torch), dev(c["v"], torch), dev(c["table"], torch), **kw)


def io_np(fmt):
    return np.float32 if fmt == "f32" else np.float16


def half_step(fmt, x):
    """Half a step of the I/O type at x."""
    x = np.abs(np.asarray(x, np.float64))
    return x * 2.0 ** -24 + 2.0 ** -149 if fmt == "f32" else np.maximum(x * 2.0 ** -11, 2.0 ** -25)


def oracle_attention(c, q, cu, *, scale=None, window=0, table=None):
    """(out, tolerance) of one call; the tolerance counts the output's own rounding."""
    eight = c["fmt"] == "e4m3"
    k, v = c["k"], c["v"]
    out, bound = AO.attention(q, k, v, c["table"] if table is None else table, cu, c["lens"], scale=scale,
                              window=window, rounded_weights=c["fmt"] != "f32",
                              v_codes=c["v_codes"] if eight else None, v_scales=c["v_scales"] if eight else None)
    return out, bound + half_step(c["fmt"], np.abs(out) + bound)


def run_attention(c, q, cu, torch, gdn, *, dense=False, mirrors=True, cache=None, out=None, **kw):
    """One gdn_attn_forward on fresh device copies; the output as float64 numpy, poisoned first."""
    N, Hq, _ = q.shape
    R = len(c["lens"])
    cache = device_cache(c, torch, gdn) if cache is None else cache
    dq = dev(q, torch)
    if out is None:
        out = torch.full_like(dq, -7.75)
    need = gdn.gdn_attn_workspace_bytes(N, R, Hq, cache)
    ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")     # NaN everywhere
    cu32 = np.asarray(cu, np.int32)
    gdn.gdn_attn_forward(dq, cache, dev(c["lens"], torch), None if dense else dev(cu32, torch), out, num_reqs=R,
                         cu_seqlens_host=cu32 if mirrors and not dense else None,
                         seq_lens_host=c["lens"] if mirrors else None, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def assert_within(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0)), got.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: got {got[i]}, want {want[i]}, "
                             f"tolerance {tol[i]:.3g}")
