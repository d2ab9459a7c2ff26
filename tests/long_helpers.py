"""Inputs and calls shared by the tests of the 4-bit cache and of sparse attention."""
from __future__ import annotations

import numpy as np

from attn_helpers import io_np, make_cache, page_table
from gpu_helpers import dev
from oracle import attn_oracle as AO
from oracle import sparse_oracle as SO

FORMATS = ("f16", "f32", "e4m3", "e2m1")


def transposed(scales):
    """Exponent bytes [P, Hk, page, D / 32] as the cache keeps them: [P, Hk, D / 32, page]."""
    return np.ascontiguousarray(np.swapaxes(scales, -1, -2))


def make_cache4(lens, *, Hk, D, page, seed, scale=1.0, fill=0xff):
    """A 4-bit cache of requests with `lens` tokens; unused slots hold the bytes `fill`, scales among them."""
    rng = np.random.default_rng(seed)
    table, P = page_table(lens, page, rng)
    full = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    c = {"fmt": "e2m1", "table": table, "P": P, "page": page, "Hk": Hk, "D": D, "lens": np.asarray(lens, np.int32)}
    for name in ("k", "v"):
        rows = rng.standard_normal((full[-1], Hk, D)) * scale
        if name == "k":
            rows[..., 5::37] *= 4.0
        codes, s = SO.quantise(rows.astype(np.float16))
        pool = AO.cache_write(SO.pack(codes), np.full((P, Hk, page, D // 2), fill, np.uint8), table, full, lens)
        scales = AO.cache_write(s, np.full((P, Hk, page, D // 32), fill, np.uint8), table, full, lens)
        c[name + "_codes"], c[name + "_scales"] = pool, transposed(scales)
        c[name] = SO.dequantise(SO.unpack(pool), scales)
    return c


def any_cache(lens, *, fmt, **kw):
    return make_cache4(lens, **kw) if fmt == "e2m1" else make_cache(lens, fmt=fmt, **kw)


def any_device_cache(c, torch, gdn, **kw):
    if "k_codes" in c:
        return gdn.KVCache(dev(c["k_codes"], torch), dev(c["v_codes"], torch), dev(c["table"], torch),
                           k_scales=dev(c["k_scales"], torch), v_scales=dev(c["v_scales"], torch), **kw)
    return gdn.KVCache(dev(c["k"], torch), dev(c["v"], torch), dev(c["table"], torch), **kw)


def queries(N, Hq, D, fmt, seed, scale=1.5):
    return (np.random.default_rng(seed).standard_normal((N, Hq, D)) * scale).astype(io_np(fmt))


def cu_of(T):
    return np.concatenate([[0], np.cumsum(T)]).astype(np.int32)


def run_select(c, q, bounds, cu, torch, gdn, *, K, first=1, newest=1, dense=False, mirrors=True, cache=None):
    """One gdn_attn_select on fresh device copies: (lists, counts), poisoned first."""
    N, Hq, _ = q.shape
    R = len(c["lens"])
    cache = any_device_cache(c, torch, gdn) if cache is None else cache
    lists = torch.full((N, c["Hk"], K), -77, dtype=torch.int32, device="cuda")
    counts = torch.full((N,), -77, dtype=torch.int32, device="cuda")
    ws = torch.full((max(gdn.gdn_attn_select_workspace_bytes(N, R, Hq, K, cache), 16),), 0xff, dtype=torch.uint8, device="cuda")
    cu32 = np.asarray(cu, np.int32)
    gdn.gdn_attn_select(dev(q, torch), dev(bounds, torch), cache, dev(c["lens"], torch), None if dense else dev(cu32, torch), lists,
                        counts, first_pages=first, newest_pages=newest, num_reqs=R,
                        cu_seqlens_host=cu32 if mirrors and not dense else None, seq_lens_host=c["lens"] if mirrors else None,
                        workspace=ws)
    torch.cuda.synchronize()
    return lists.cpu().numpy(), counts.cpu().numpy()


def run_sparse(c, q, cu, lists, counts, torch, gdn, *, dense=False, mirrors=True, cache=None, **kw):
    """One gdn_attn_sparse_forward on fresh device copies; the output as float64 numpy, poisoned first."""
    N, Hq, _ = q.shape
    R, K = len(c["lens"]), lists.shape[2]
    cache = any_device_cache(c, torch, gdn) if cache is None else cache
    dq = dev(q, torch)
    out = torch.full_like(dq, -7.75)
    ws = torch.full((max(gdn.gdn_attn_sparse_workspace_bytes(N, R, Hq, K, cache), 16),), 0xff, dtype=torch.uint8, device="cuda")
    cu32 = np.asarray(cu, np.int32)
    gdn.gdn_attn_sparse_forward(dq, cache, dev(c["lens"], torch), None if dense else dev(cu32, torch),
                                dev(np.ascontiguousarray(lists, np.int32), torch),
                                None if counts is None else dev(np.asarray(counts, np.int32), torch), out, num_reqs=R,
                                cu_seqlens_host=cu32 if mirrors and not dense else None,
                                seq_lens_host=c["lens"] if mirrors else None, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()
