"""Plain float64 reference of the 4-bit cache format and of sparse attention: the bounds of a page's
keys, the selection of pages by them, attention over listed pages.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the operator library.
"""
from __future__ import annotations

import numpy as np

from oracle import attn_oracle as AO

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_nearest(y):
    """Codes of y: the nearest value, ties to the even code, magnitudes past 6 as 6."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 1, 7)
    lo = hi - 1
    below, above = a - E2M1[lo], E2M1[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def quantise(x):
    """(codes [..., D] one a byte, exponent bytes [..., D / 32]) of rows x: for each 32 neighbours the smallest
    power of two, up to 2^13, that keeps the largest magnitude within 6; 255 and codes 0 where one is not finite."""
    x = np.asarray(x, np.float64)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    fine = np.isfinite(y).all(-1)
    y = np.where(fine[..., None], y, 0.0)
    amax = np.abs(y).max(-1)
    k = np.full(amax.shape, -60, np.int64)
    for _ in range(73):                             # from 2^-60 up to 2^13
        k = np.where((amax > 6 * 2.0 ** k) & (k < 13), k + 1, k)
    s = np.where(amax > 0, k + 127, 0)
    codes = e2m1_nearest(y * 2.0 ** -k.astype(np.float64)[..., None])
    codes = np.where(fine[..., None], codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), np.where(fine, s, 255).astype(np.uint8)


def values(codes):
    return np.where(codes >= 8, -E2M1[codes & 7], E2M1[codes & 7])


def dequantise(codes, s):
    v = values(codes).reshape(codes.shape[:-1] + (codes.shape[-1] // 32, 32))
    with np.errstate(invalid="ignore"):
        v = np.where(s[..., None] == 255, np.nan, v * 2.0 ** (s.astype(np.float64) - 127)[..., None])
    return v.reshape(codes.shape)


def pack(codes):
    """Two codes a byte, the even element in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (2 * packed.shape[-1],))


def bounds(k_pages, page_table, cu_seqlens, seq_lens, old):
    """old [P, Hk, 2, D] with the lowest and highest key of every page that holds a new token."""
    out = np.array(old, np.float64)
    P, _, ps, _ = k_pages.shape
    for r in range(len(seq_lens)):
        at = AO.token_positions(cu_seqlens, seq_lens, r)
        for i in sorted({int(p) // ps for p in at if p >= 0}):
            page, _ = AO.places(page_table, ps, P, r, [i * ps])
            if page[0] < 0:
                continue
            k = np.asarray(k_pages[page[0], :, :min(ps, int(seq_lens[r]) - i * ps)], np.float64)
            out[page[0], :, 0], out[page[0], :, 1] = k.min(1), k.max(1)     # a NaN goes through both
    return out


def select(q, page_bounds, page_table, page_size, cu_seqlens, seq_lens, K, first, newest):
    """(lists [N, Hk, K], counts [N], gaps [N, Hk]): gap is how far apart, relative to their size, the last score
    that is in and the first that is out are (inf where nothing is out)."""
    q = np.asarray(q, np.float64)
    b = np.asarray(page_bounds, np.float64)
    N, Hq, D = q.shape
    P, Hk = b.shape[:2]
    lists, counts, gaps = np.full((N, Hk, K), -1, np.int32), np.zeros(N, np.int32), np.full((N, Hk), np.inf)
    for r in range(len(seq_lens)):
        for j, pos in enumerate(AO.token_positions(cu_seqlens, seq_lens, r)):
            n = int(cu_seqlens[r]) + j
            held = min(int(pos) // page_size + 1, page_table.shape[1]) if pos >= 0 else 0
            page, _ = AO.places(page_table, page_size, P, r, np.arange(held) * page_size)
            there = np.flatnonzero(page >= 0)
            counts[n] = min(K, len(there))
            for h in range(Hk):
                g = q[n, h * (Hq // Hk):(h + 1) * (Hq // Hk)]
                plus, minus = np.where(g < 0, 0, g).sum(0), np.where(g > 0, 0, g).sum(0)
                with np.errstate(invalid="ignore"):
                    s = (plus * b[page[there], h, 1] + minus * b[page[there], h, 0]).sum(-1)
                always = (there < first) | (there >= held - newest)
                rank = np.where(np.isnan(s), np.inf, s)
                order = sorted(range(len(there)), key=lambda i: (not always[i], not np.isnan(s[i]), -rank[i], there[i]))
                lists[n, h, :counts[n]] = np.sort(there[order[:K]])
                if len(order) > K > 0 and not always[order[K - 1]]:
                    a, c = s[order[K - 1]], s[order[K]]
                    gaps[n, h] = abs(a - c) / max(abs(a), abs(c), 1e-300) if np.isfinite(a) and np.isfinite(c) and a != c else np.inf
    return lists, counts, gaps


def sparse_attention(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, lists, counts=None, scale=None, rounded_weights=True):
    """(out, bound): attention of every token over the positions up to its own of the listed entries of its
    request's page table; an entry listed twice counts twice. bound as AO.attention's, with weights taken at 2^-11 of
    each and 2^-25 of the largest where they are rounded to FP16 (rounded_weights)."""
    q = np.asarray(q, np.float64)
    N, Hq, D = q.shape
    P, Hk, ps, _ = k_pages.shape
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    u = 2.0 ** -24
    for r in range(len(seq_lens)):
        for j, last in enumerate(AO.token_positions(cu_seqlens, seq_lens, r)):
            n = int(cu_seqlens[r]) + j
            for h in range(Hk):
                mine = lists[n, h, :lists.shape[2] if counts is None else int(np.clip(counts[n], 0, lists.shape[2]))]
                at = np.concatenate([i * ps + np.arange(ps) for i in mine if 0 <= i < page_table.shape[1]] or [np.zeros(0, np.int64)])
                page, slot = AO.places(page_table, ps, P, r, at[at <= last].astype(np.int64))
                page, slot = page[page >= 0], slot[page >= 0]
                L = len(page)
                if L == 0:
                    continue
                k, v = np.asarray(k_pages[page, h, slot], np.float64), np.asarray(v_pages[page, h, slot], np.float64)
                qr = q[n, h * G:(h + 1) * G]
                s = scale * qr @ k.T
                w = np.exp(s - s.max(-1, keepdims=True))
                p = w / w.sum(-1, keepdims=True)
                A = p @ np.abs(v)
                size = scale * (np.abs(qr) @ np.abs(k).T).max(-1, keepdims=True)
                rel = 2 * (D + 2) * u * size + 4 * u * np.abs(s).max(-1, keepdims=True) + 2 * (L + 8) * u + 2.0 ** -22
                out[n, h * G:(h + 1) * G] = p @ v
                bound[n, h * G:(h + 1) * G] = A * rel
                if rounded_weights:
                    bound[n, h * G:(h + 1) * G] += A * 2.0 ** -11 + 2.0 ** -25 * np.abs(v).sum(0) / w.sum(-1, keepdims=True)
    return out, bound
