"""Plain float64 reference of the attention layer's serving step: rotary
positions, the paged key-value cache and attention over it.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the operator library.

Everything is written from the definitions: angles, sums and softmax in float64,
the 8-bit format from its table of values. Positions, page numbers and lengths
follow the paged contract: a page number outside the pool, or a position outside
the table, holds nothing.
"""
from __future__ import annotations

import numpy as np

HALF, INTERLEAVED = 0, 1


def frequencies(rotary_dim, base=10000.0):
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    return float(base) ** (-2.0 * i / rotary_dim)


def rope(x, positions, inv_freq, layout=HALF, factor=1.0):
    """x [N, H, D] with the leading 2 len(inv_freq) elements of every head rotated."""
    x = np.asarray(x, np.float64)
    inv_freq = np.asarray(inv_freq, np.float64)
    half = len(inv_freq)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if layout == INTERLEAVED else (i, i + half)
    angle = np.asarray(positions, np.float64)[:, None, None] * inv_freq
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    out = x.copy()
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., second] * c + x[..., first] * s
    return out


def e4m3_values():
    """The value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code >= 128, -v, v)


def e4m3_nearest(y):
    """Codes of y (|y| <= 448, or non-finite for NaN): the nearest value, ties to the even code."""
    y = np.asarray(y, np.float64)
    pos = e4m3_values()[:127]                       # 0 .. 448, increasing with the code
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    below, above = a - pos[lo], pos[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(y), code, 127)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x):
    """(codes [..., D], exponent bytes [...]) of rows x: the smallest power of two that keeps the
    largest finite magnitude within 448."""
    x = np.asarray(x, np.float64)
    amax = np.max(np.abs(np.where(np.isfinite(x), x, 0.0)), axis=-1)
    s = np.zeros(amax.shape, np.int64)
    some = amax > 0
    m, e = np.frexp(amax[some])                     # m in [0.5, 1); 448 = 0.875 * 2^9
    s[some] = e - 9 + (m > 0.875) + 127
    y = x * 2.0 ** (127.0 - np.where(some, s, 127))[..., None]
    return e4m3_nearest(y), s.astype(np.uint8)


def dequantise(codes, s):
    return e4m3_values()[codes] * 2.0 ** (s.astype(np.float64) - 127)[..., None]


def places(page_table, page_size, num_pages, r, positions):
    """(page, slot) of a request's positions; page -1 where nothing holds them."""
    positions = np.asarray(positions, np.int64)
    entry = positions // page_size
    ok = (positions >= 0) & (entry < page_table.shape[1])
    page = np.where(ok, page_table[r, np.clip(entry, 0, page_table.shape[1] - 1)], -1)
    return np.where((page >= 0) & (page < num_pages), page, -1), positions % page_size


def token_positions(cu_seqlens, seq_lens, r):
    T = int(cu_seqlens[r + 1] - cu_seqlens[r])
    return int(seq_lens[r]) - T + np.arange(T)


def cache_write(rows, pages, page_table, cu_seqlens, seq_lens):
    """rows [N, Hk, ...] to pages [P, Hk, page, ...] (a copy is returned)."""
    pages = pages.copy()
    for r in range(len(seq_lens)):
        page, slot = places(page_table, pages.shape[2], pages.shape[0], r, token_positions(cu_seqlens, seq_lens, r))
        for j, (pg, sl) in enumerate(zip(page, slot)):
            if pg >= 0:
                pages[pg, :, sl] = rows[cu_seqlens[r] + j]
    return pages


def cache_read(pages, page_table, cu_seqlens, seq_lens):
    """[N, Hk, ...] of every request's newest tokens, zeros where nothing holds them."""
    out = np.zeros((int(cu_seqlens[-1]), pages.shape[1]) + pages.shape[3:], pages.dtype)
    for r in range(len(seq_lens)):
        page, slot = places(page_table, pages.shape[2], pages.shape[0], r, token_positions(cu_seqlens, seq_lens, r))
        for j, (pg, sl) in enumerate(zip(page, slot)):
            if pg >= 0:
                out[cu_seqlens[r] + j] = pages[pg, :, sl]
    return out


def attended(page_table, page_size, num_pages, cu_seqlens, seq_lens, r, j, window=0):
    """(pages, slots) of the positions that token j of request r attends."""
    last = int(token_positions(cu_seqlens, seq_lens, r)[j])
    lo = max(0, last - window + 1) if window > 0 else 0
    page, slot = places(page_table, page_size, num_pages, r, np.arange(lo, max(last + 1, lo)))
    return page[page >= 0], slot[page >= 0]


def attention(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, scale=None, window=0, rounded_weights=True,
              v_codes=None, v_scales=None):
    """(out, bound): out [N, Hq, D] in float64, and for each element how far an FP32 kernel's
    result may be from it before its own rounding to the I/O type.

    With s the scores, p the softmax and A = sum p |v|, the terms are
      scores     a product over D in FP32 is off by at most (D + 2) 2^-24 scale sum |q k|, the exponent's
                 argument by two more roundings of its size: a weight by twice the largest of these, relative
      sums       the weights' sum and the product with v over L positions: 2 (L + 8) 2^-24 A
      exp2       2 ulp each: 2^-22 A
      weights    rounded to FP16 (rounded_weights): 2^-11 A, and 2^-25 of the largest weight for those below
                 FP16's normal range. With 8-bit values the weights carry the value's scale (v_codes, v_scales).
    """
    q = np.asarray(q, np.float64)
    N, Hq, D = q.shape
    P, Hk, page_size, _ = k_pages.shape
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    u = 2.0 ** -24
    for r in range(len(seq_lens)):
        for j in range(int(cu_seqlens[r + 1] - cu_seqlens[r])):
            page, slot = attended(page_table, page_size, P, cu_seqlens, seq_lens, r, j, window)
            n = int(cu_seqlens[r]) + j
            L = len(page)
            if L == 0:
                continue
            k = np.asarray(k_pages[page, :, slot], np.float64).transpose(1, 0, 2)      # [Hk, L, D]
            v = np.asarray(v_pages[page, :, slot], np.float64).transpose(1, 0, 2)
            qr = q[n].reshape(Hk, G, D)
            s = scale * np.matmul(qr, k.transpose(0, 2, 1))                             # [Hk, G, L]
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            p = w / w.sum(-1, keepdims=True)
            out[n] = np.matmul(p, v).reshape(Hq, D)
            A = np.matmul(p, np.abs(v)).reshape(Hq, D)
            size = scale * np.matmul(np.abs(qr), np.abs(k).transpose(0, 2, 1)).max(-1)  # [Hk, G]
            rel = (2 * (D + 2) * u * size + 4 * u * np.abs(s).max(-1)).reshape(Hq, 1) + 2 * (L + 8) * u + 2.0 ** -22
            if rounded_weights:
                rel = rel + 2.0 ** -11
                if v_codes is None:
                    low = np.abs(v).sum(1)[:, None] / w.sum(-1, keepdims=True)
                else:
                    sv = np.maximum(2.0 ** (np.asarray(v_scales[page, :, slot], np.float64).T - 127), 2.0 ** -33)
                    sm = s + np.log(sv)[:, None]                                        # weights times the value's scale
                    codes = np.abs(e4m3_values()[v_codes[page, :, slot]]).transpose(1, 0, 2).sum(1)
                    low = codes[:, None] / np.exp(s - sm.max(-1, keepdims=True)).sum(-1, keepdims=True)
                bound[n] = 2.0 ** -25 * low.reshape(Hq, D)
            bound[n] += A * rel
    return out, bound
