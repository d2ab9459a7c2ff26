"""Pins of oracle/attn_oracle.py, each against something other than itself: the
rotation against complex numbers and its invariants, the 8-bit format against
torch's own conversion, the cache against a dictionary of tokens, and attention
against a dense softmax."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attn_oracle as AO


@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
def test_rope_is_a_complex_product(layout):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64))
    pos, f = np.array([0, 1, 7, 1000, -3]), AO.frequencies(32, 500.0)
    y = AO.rope(x, pos, f, layout, 1.5)
    pick = (lambda z: (z[..., 0:32:2], z[..., 1:32:2])) if layout == AO.INTERLEAVED else (lambda z: (z[..., :16], z[..., 16:32]))
    a, b = pick(x)
    z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    ya, yb = pick(y)
    np.testing.assert_allclose(ya, z.real, atol=1e-12)
    np.testing.assert_allclose(yb, z.imag, atol=1e-12)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(AO.rope(x, np.zeros(5), f, layout), x)


@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
def test_rope_products_depend_on_the_distance(layout):
    rng = np.random.default_rng(1)
    q, k, f = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32)), AO.frequencies(32)
    dots = [np.sum(AO.rope(q, [40 + d], f, layout) * AO.rope(k, [7 + d], f, layout)) for d in (0, 1, 5000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_e4m3_table_is_torch_s():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, AO.e4m3_values())


def test_e4m3_nearest_is_torch_s():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    v = AO.e4m3_values()
    v = np.sort(v[np.isfinite(v)])
    ties = (v[1:] + v[:-1]) / 2
    y = np.concatenate([v, ties, np.nextafter(ties.astype(np.float32), np.float32(1e9)), rng.uniform(-448, 448, 2000),
                        rng.standard_normal(2000) * 0.01]).astype(np.float32)
    got = AO.e4m3_nearest(y)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(AO.e4m3_values()[got], AO.e4m3_values()[want])


def test_quantise_scale_is_the_smallest_power_that_fits():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((200, 8)) * 2.0 ** rng.integers(-20, 12, (200, 1))).astype(np.float16)
    x[0, :] = 0
    x[1, 0], x[1, 1:] = 448.0, 1.0
    x[2, 0], x[2, 1:] = 448.5, 1.0
    x[3, 0] = np.inf
    codes, s = AO.quantise(x)
    amax = np.max(np.abs(np.where(np.isfinite(x), x, 0)).astype(np.float64), -1)
    assert s[0] == 0 and s[1] == 127 and s[2] == 128 and AO.e4m3_values()[codes[3, 0]] != AO.e4m3_values()[codes[3, 0]]
    scale = 2.0 ** (s.astype(np.float64) - 127)
    assert np.all(amax <= 448 * scale) and np.all(amax[1:] > 224 * scale[1:])
    back = AO.dequantise(codes, s)
    fine = np.isfinite(x.astype(np.float64))
    step = np.maximum(np.abs(x.astype(np.float64)) * 2.0 ** -4, 2.0 ** -10 * scale[:, None])   # half a step
    assert np.all(np.abs(back - x)[fine] <= step[fine])


def _layout(lens, page, P, seed):
    rng = np.random.default_rng(seed)
    table = np.full((len(lens), max(-(-max(lens) // page), 1) + 1), -1, np.int32)
    ids = iter(rng.permutation(P))
    for r, m in enumerate(lens):
        for i in range(-(-m // page)):
            table[r, i] = next(ids)
    return table


def test_cache_write_then_read():
    rng = np.random.default_rng(4)
    lens, new = [5, 40, 17], [2, 9, 17]
    cu = np.concatenate([[0], np.cumsum(new)])
    table = _layout(lens, 16, 9, 4)
    rows = rng.standard_normal((cu[-1], 2, 4))
    pool = rng.standard_normal((9, 2, 16, 4))
    got = AO.cache_write(rows, pool, table, cu, lens)
    np.testing.assert_array_equal(AO.cache_read(got, table, cu, lens), rows)
    held = {}
    for r in range(3):
        for j in range(new[r]):
            pos = lens[r] - new[r] + j
            held[(table[r, pos // 16], pos % 16)] = rows[cu[r] + j]
    for pg in range(9):
        for sl in range(16):
            np.testing.assert_array_equal(got[pg, :, sl], held.get((pg, sl), pool[pg, :, sl]))


@pytest.mark.parametrize("window", [0, 3])
def test_attention_is_a_dense_softmax(window):
    rng = np.random.default_rng(5)
    lens, new = [6, 33, 0, 20], [3, 1, 1, 20]
    cu = np.concatenate([[0], np.cumsum(new)])
    table = _layout(lens, 16, 8, 5)
    Hk, G, D = 2, 3, 8
    k = [rng.standard_normal((m, Hk, D)) for m in lens]
    v = [rng.standard_normal((m, Hk, D)) for m in lens]
    full = np.concatenate([[0], np.cumsum(lens)])
    pool = np.full((8, Hk, 16, D), np.nan)                   # what no request holds has no influence
    kp = AO.cache_write(np.concatenate(k), pool, table, full, lens)
    vp = AO.cache_write(np.concatenate(v), pool, table, full, lens)
    q = rng.standard_normal((cu[-1], Hk * G, D))
    out, bound = AO.attention(q, kp, vp, table, cu, lens, window=window)
    assert np.all(np.isfinite(bound))
    for r in range(4):
        for j in range(new[r]):
            last = lens[r] - new[r] + j
            lo = max(0, last - window + 1) if window else 0
            for h in range(Hk * G):
                if last < lo:
                    assert np.all(out[cu[r] + j, h] == 0)
                    continue
                s = k[r][lo:last + 1, h // G] @ q[cu[r] + j, h] / np.sqrt(D)
                p = np.exp(s) / np.exp(s).sum()
                np.testing.assert_allclose(out[cu[r] + j, h], p @ v[r][lo:last + 1, h // G], atol=1e-12)
