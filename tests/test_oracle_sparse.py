"""The float64 reference of the 4-bit format and of sparse attention against values worked out by hand."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attn_oracle as AO
from oracle import sparse_oracle as SO


def test_codes_are_the_formats():
    # sign, two exponent bits (bias 1), one bit of mantissa
    for code in range(16):
        e, m = (code >> 1) & 3, code & 1
        v = 0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
        assert SO.values(np.array([code]))[0] == (-v if code & 8 else v)


@pytest.mark.parametrize("x,code", [(0.0, 0), (0.25, 0), (0.2501, 1), (0.75, 2), (0.7499, 1), (1.25, 2), (1.26, 3), (1.75, 4), (2.5, 4),
                                    (2.51, 5), (3.5, 6), (3.49, 5), (5.0, 6), (5.01, 7), (6.0, 7), (7.9, 7), (-0.75, 10), (-6.5, 15)])
def test_nearest_with_ties_to_even(x, code):
    assert SO.e2m1_nearest(x) == code


@pytest.mark.parametrize("amax,s", [(6.0, 127), (6.01, 128), (3.0, 126), (3.001, 127), (2.0 ** -24, 101), (49152.0, 140), (65504.0, 140),
                                    (0.0, 0)])
def test_scales(amax, s):
    x = np.zeros((2, 64))
    x[1, 40] = -amax
    codes, got = SO.quantise(x)
    assert got.tolist() == [[0, 0], [0, s]]
    back = SO.dequantise(codes, got)
    assert back[1, 40] == -min(amax, 49152.0) or 0 < amax < 49152 and abs(back[1, 40] + amax) <= amax / 5


def test_blocks_with_something_not_finite_read_as_nan():
    x = np.ones((1, 96))
    x[0, 3], x[0, 70] = np.inf, np.nan
    codes, s = SO.quantise(x)
    assert s[0, 0] == s[0, 2] == 255 and s[0, 1] != 255 and not codes[0, :32].any()
    back = SO.dequantise(codes, s)
    assert np.isnan(back[0, :32]).all() and (back[0, 32:64] == 1).all() and np.isnan(back[0, 64:]).all()


def test_every_stored_value_is_an_fp16_value():
    x = np.arange(1 << 15, dtype=np.uint16).view(np.float16)
    x = np.sort(x[np.isfinite(x)].astype(np.float64))
    x = np.concatenate([x, np.full(-len(x) % 32, x[-1])]).reshape(-1, 32)
    codes, s = SO.quantise(x)
    back = SO.dequantise(codes, s)
    assert (back == back.astype(np.float16)).all() and set(np.unique(s)) <= {0, *range(101, 141)}


def test_packing():
    c = np.arange(32, dtype=np.uint8).reshape(1, 32) & 15
    assert SO.pack(c)[0, :3].tolist() == [0x10, 0x32, 0x54]
    assert (SO.unpack(SO.pack(c)) == c).all()


def test_selection_is_the_bounds_and_the_always_selected_pages():
    rng = np.random.default_rng(0)
    Hk, G, D, ps, M = 2, 3, 64, 16, 9
    table = rng.permutation(M).astype(np.int32)[None]
    k = rng.standard_normal((M, Hk, ps, D))
    b = SO.bounds(k, table, [0, M * ps], [M * ps], np.zeros((M, Hk, 2, D)))
    assert np.allclose(b[:, :, 0], k.min(2)) and np.allclose(b[:, :, 1], k.max(2))
    q = rng.standard_normal((1, Hk * G, D))
    lists, counts, _ = SO.select(q, b, table, ps, [0, 1], [M * ps - 3], 4, 1, 1)
    assert counts.tolist() == [4] and (lists[0, :, 0] == 0).all() and (lists[0, :, 3] == M - 1).all()
    for h in range(Hk):
        s = sum(np.maximum(q[0, h * G + g] * b[table[0], h, 0], q[0, h * G + g] * b[table[0], h, 1]).sum(-1) for g in range(G))
        best = sorted(range(1, M - 1), key=lambda i: -s[i])[:2]
        assert lists[0, h, 1:3].tolist() == sorted(best)
        # the bound holds for every key of the page
        for i in range(M):
            assert (q[0, h * G:(h + 1) * G] @ k[table[0, i], h].T).sum(0).max() <= s[i] + 1e-9


def test_attention_over_every_page_is_attention():
    rng = np.random.default_rng(1)
    Hk, D, ps, lens = 2, 64, 16, [37, 5]
    table = np.array([[3, 0, 4], [1, -1, -1]], np.int32)
    k, v = rng.standard_normal((2, 5, Hk, ps, D))
    q, cu = rng.standard_normal((4, 4, D)), [0, 3, 4]
    lists = np.tile(np.array([2, 0, 1, -1], np.int32), (4, Hk, 1))
    out, _ = SO.sparse_attention(q, k, v, table, cu, lens, lists)
    ref, _ = AO.attention(q, k, v, table, cu, lens)
    assert np.allclose(out, ref, atol=1e-12)
    twice = np.tile(np.array([0, 0], np.int32), (4, Hk, 1))
    once = np.tile(np.array([0], np.int32), (4, Hk, 1))
    assert np.allclose(SO.sparse_attention(q, k, v, table, cu, lens, twice)[0], SO.sparse_attention(q, k, v, table, cu, lens, once)[0])
    assert not SO.sparse_attention(q, k, v, table, cu, lens, lists, np.zeros(4, np.int32))[0].any()
