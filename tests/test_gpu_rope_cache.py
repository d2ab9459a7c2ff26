"""GPU parity of rotary positions (gdn_rope_forward) and of the paged cache's write
and read (gdn_kv_write, gdn_kv_read) against the float64 oracle, through the C ABI.

Rotation: cos and sin are within 6 * 2^-24 of theirs (the reduced angle 2^-26 turns, 1.6 of
those units; the function 2 ulp, 4 more at its largest), two products and a sum add 3 roundings
of 2^-24: the result is off by at most 9 * 2^-24 factor (|x| + |y|) before its own rounding to
the I/O type. What the cache holds is compared bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import FORMATS, assert_within, half_step, io_np, page_table
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
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def _rope_tol(x, want, rot, layout, factor, fmt):
    x = np.abs(x.astype(np.float64))
    pair = np.zeros(x.shape)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if layout == AO.INTERLEAVED else (i, i + rot // 2)
    pair[..., a] = pair[..., b] = x[..., a] + x[..., b]
    tol = 9 * 2.0 ** -24 * factor * pair
    out = tol + half_step(fmt, np.abs(want) + tol)
    out[..., rot:] = 0.0
    return out


@pytest.mark.parametrize("fmt", ["f16", "f32"])
@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 96), (128, 128), (256, 64), (256, 256)])
def test_rope(fmt, layout, D, rot):
    for N, Hq, Hk, far in ((1, 1, 1, 5), (7, 3, 2, 1 << 20), (1100, 2, 1, 40000)):
        _case(f"{fmt} layout={layout} D={D} rot={rot} N={N}")
        rng = np.random.default_rng(N + rot)
        q, k = (rng.standard_normal((N, h, D)).astype(io_np(fmt)) for h in (Hq, Hk))
        pos = rng.integers(-far, far + 1, N).astype(np.int32)
        f = AO.frequencies(rot, 1e6)
        outs = [torch.full(x.shape, float("nan"), dtype=dev(x, torch).dtype, device="cuda") for x in (q, k)]
        gdn.gdn_rope_forward(dev(q, torch), dev(k, torch), dev(pos, torch), dev(f, torch), outs[0], outs[1],
                             rope_layout=layout, rope_factor=1.25)
        torch.cuda.synchronize()
        for x, got, name in ((q, outs[0], "q"), (k, outs[1], "k")):
            want = AO.rope(x, pos, f, layout, 1.25)
            assert_within(got.double().cpu().numpy(), want, _rope_tol(x, want, rot, layout, 1.25, fmt), name)


def test_rope_far_positions():
    """Positions at the ends of int32: the angle is reduced in double precision."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1999999999], np.int32)
    rng = np.random.default_rng(1)
    q = rng.standard_normal((4, 2, 64)).astype(np.float32)
    f = AO.frequencies(64)
    # position * frequency is exact to half an ulp of a double up to 2^31: 2^-23 radians, once in the
    # oracle and once (in turns) in the kernel
    out = torch.empty((4, 2, 64), device="cuda")
    gdn.gdn_rope_forward(dev(q, torch), None, dev(pos, torch), dev(f, torch), out, None)
    torch.cuda.synchronize()
    want = AO.rope(q, pos, f)
    pair = np.abs(q[..., :32]) + np.abs(q[..., 32:])
    extra = 3 * 2.0 ** -23 * np.concatenate([pair, pair], -1)
    assert_within(out.double().cpu().numpy(), want, _rope_tol(q, want, 64, AO.HALF, 1.0, "f32") + extra, "far")


@pytest.mark.parametrize("fmt", ["f16", "f32"])
@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
def test_rope_in_place_and_strided(fmt, layout):
    """q and k as slices of one projection's output, in place: the same bytes as dense and out of place."""
    N, Hq, Hk, D, rot = 33, 4, 2, 128, 64
    rng = np.random.default_rng(2)
    wide = dev(rng.standard_normal((N, (Hq + 2 * Hk) * D)).astype(io_np(fmt)), torch)
    before = wide.clone()
    q, k = wide[:, :Hq * D].view(N, Hq, D), wide[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
    pos, f = dev(rng.integers(0, 9999, N).astype(np.int32), torch), dev(AO.frequencies(rot), torch)
    qd, kd = q.contiguous(), k.contiguous()
    qo, ko = torch.empty_like(qd), torch.empty_like(kd)
    gdn.gdn_rope_forward(qd, kd, pos, f, qo, ko, rope_layout=layout)
    gdn.gdn_rope_forward(q, k, pos, f, q, k, rope_layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(wide[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


def _pool(P, Hk, page, D, fmt, rng):
    """Device pages of junk, and their host copies: (codes or values, scales)."""
    if fmt == "e4m3":
        h = [rng.integers(0, 256, (P, Hk, page, D)).astype(np.uint8), rng.integers(0, 256, (P, Hk, page)).astype(np.uint8)]
    else:
        h = [rng.standard_normal((P, Hk, page, D)).astype(io_np(fmt)), None]
    return h, [None if x is None else dev(x, torch) for x in h]


def _expect(rows, host, table, cu, lens, fmt):
    if fmt != "e4m3":
        return AO.cache_write(rows, host[0], table, cu, lens), None
    codes, s = AO.quantise(rows)
    return AO.cache_write(codes, host[0], table, cu, lens), AO.cache_write(s, host[1], table, cu, lens)


def _same_codes(got, want):
    """Equal codes; any NaN code stands for NaN."""
    nan = (want & 127) == 127
    assert np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 127) == 127)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([5, 40, 17], [2, 9, 17]), ([130, 1, 64, 0, 33], [3, 1, 64, 0, 33]),
                                      ([2000, 30], [1500, 30])])
def test_write_and_read(fmt, D, page, lens, new):
    _case(f"{fmt} D={D} page={page} lens={lens} new={new}")
    rng = np.random.default_rng(D + page)
    Hk, cu = 3, _cu(new)
    table, P = page_table(lens, page, rng)
    k, v = (rng.standard_normal((cu[-1], Hk, D)).astype(io_np(fmt)) for _ in range(2))
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, fmt, rng), _pool(P, Hk, page, D, fmt, rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch), k_scales=dk[1], v_scales=dv[1], page_table_host=table)
    lens32 = np.asarray(lens, np.int32)
    args = (cache, dev(lens32, torch), dev(cu, torch))
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), *args, cu_seqlens_host=cu, seq_lens_host=lens32)
    ko, vo = (torch.full((cu[-1], Hk, D), float("nan"), dtype=dev(k, torch).dtype, device="cuda") for _ in range(2))
    gdn.gdn_kv_read(ko, vo, *args)
    torch.cuda.synchronize()
    for rows, host, d, out in ((k, hk, dk, ko), (v, hv, dv, vo)):
        pages, scales = _expect(rows, host, table, cu, lens, fmt)
        if fmt == "e4m3":
            _same_codes(d[0].cpu().numpy(), pages)
            assert np.array_equal(d[1].cpu().numpy(), scales)
            codes, s = AO.quantise(rows)
            assert np.array_equal(out.double().cpu().numpy(), AO.dequantise(codes, s))
        else:
            assert np.array_equal(d[0].cpu().numpy(), pages)
            assert np.array_equal(out.cpu().numpy(), rows)


def test_quantising_every_fp16_magnitude():
    """Rows led by every finite fp16 magnitude, with ties, subnormals, NaN and infinities among the rest."""
    bits = np.arange(1, 0x7c00, dtype=np.uint16)
    N, D, page = 1024, 64, 64
    rng = np.random.default_rng(3)
    lead = bits[rng.integers(0, len(bits), (N, 31))]
    lead[:, 0] = bits[np.linspace(0, len(bits) - 1, N).astype(int)]
    lead = lead.view(np.float16)
    rows = np.zeros((N, 31, D), np.float16)
    # fractions of the leading value on the format's ties and between them
    frac = np.concatenate([[1.0], (np.arange(1, 32) / 32.0), rng.uniform(-1, 1, 32)])
    rows[:] = (lead.astype(np.float64)[..., None] * frac).astype(np.float16)
    rows[5, :, 7], rows[6, :, 8], rows[7, :, 9], rows[8] = np.nan, np.inf, -np.inf, 0
    rows[9], rows[10, :, 1:] = np.nan, np.inf
    Hk = 31
    table, P = page_table([N], page, rng)
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, "e4m3", rng), _pool(P, Hk, page, D, "e4m3", rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch), k_scales=dk[1], v_scales=dv[1])
    lens = dev(np.array([N], np.int32), torch)
    gdn.gdn_kv_write(dev(rows, torch), dev(rows, torch), cache, lens)
    torch.cuda.synchronize()
    pages, scales = _expect(rows, hk, table, _cu([N]), [N], "e4m3")
    _same_codes(dk[0].cpu().numpy(), pages)
    assert np.array_equal(dk[1].cpu().numpy(), scales)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (64, 48)])
def test_fused_rotation_is_rotation_then_write(fmt, layout, positions, D, rot):
    rng = np.random.default_rng(rot)
    lens, new, page, Hq, Hk = [50, 9, 700], [4, 1, 130], 32, 6, 2
    cu = _cu(new)
    N = int(cu[-1])
    table, P = page_table(lens, page, rng)
    io = io_np(fmt)
    q, k, v = (dev(rng.standard_normal((N, h, D)).astype(io), torch) for h in (Hq, Hk, Hk))
    own = np.concatenate([np.arange(m - t, m) for m, t in zip(lens, new)]).astype(np.int32)
    pos = rng.integers(0, 1 << 20, N).astype(np.int32) if positions else own
    f = dev(AO.frequencies(rot, 1e6), torch)
    caches, junk = [], [_pool(P, Hk, page, D, fmt, np.random.default_rng(9))[0] for _ in range(2)]
    for _ in range(2):
        dk, dv = ([None if x is None else dev(x, torch) for x in h] for h in junk)
        caches.append((gdn.KVCache(dk[0], dv[0], dev(table, torch), k_scales=dk[1], v_scales=dv[1]), dk, dv))
    rows = (dev(np.asarray(lens, np.int32), torch), dev(cu, torch))
    qo, qf, ko = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    gdn.gdn_rope_forward(q, k, dev(pos, torch), f, qo, ko, rope_layout=layout, rope_factor=1.1)
    gdn.gdn_kv_write(ko, v, caches[0][0], *rows)
    gdn.gdn_kv_write(k, v, caches[1][0], *rows, q=q, q_out=qf, inv_freq=f, rope_layout=layout, rope_factor=1.1,
                     positions=dev(pos, torch) if positions else None)
    torch.cuda.synchronize()
    assert torch.equal(qo, qf)
    for a, b in zip(caches[0][1] + caches[0][2], caches[1][1] + caches[1][2]):
        assert a is None or torch.equal(a, b)
    # the rotated query in place
    qi = q.clone()
    gdn.gdn_kv_write(k, v, caches[1][0], *rows, q=qi, q_out=qi, inv_freq=f, rope_layout=layout, rope_factor=1.1,
                     positions=dev(pos, torch) if positions else None)
    torch.cuda.synchronize()
    assert torch.equal(qo, qi)


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_positions_without_a_page(fmt):
    """Pages -1 and past the pool, positions below zero and past the table: nothing is written, zeros are read."""
    rng = np.random.default_rng(4)
    page, Hk, D = 16, 2, 64
    lens, new = [40, 3, 70], [40, 6, 8]                 # the second request has 6 new of 3 cached tokens
    table, P = page_table([40, 3, 64], page, rng, extra=0)
    table[0, 1], table[1, 0] = -1, table[1, 0]
    table[2, 3] = P + 5
    cu = _cu(new)
    k, v = (rng.standard_normal((cu[-1], Hk, D)).astype(np.float16) for _ in range(2))
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, fmt, rng), _pool(P, Hk, page, D, fmt, rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch), k_scales=dk[1], v_scales=dv[1])
    rows = (dev(np.asarray(lens, np.int32), torch), dev(cu, torch))
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), cache, *rows)
    ko, vo = (torch.full((cu[-1], Hk, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    gdn.gdn_kv_read(ko, vo, cache, *rows)
    torch.cuda.synchronize()
    for x, host, d, out in ((k, hk, dk, ko), (v, hv, dv, vo)):
        pages, scales = _expect(x, host, table, cu, lens, fmt)
        if fmt == "e4m3":
            _same_codes(d[0].cpu().numpy(), pages)
            assert np.array_equal(d[1].cpu().numpy(), scales)
            x = AO.dequantise(*AO.quantise(x))
        else:
            assert np.array_equal(d[0].cpu().numpy(), pages)
        want = np.zeros(out.shape)
        for r in range(3):
            pg, _ = AO.places(table, page, P, r, AO.token_positions(cu, lens, r))
            want[cu[r]:cu[r + 1]][pg >= 0] = x[cu[r]:cu[r + 1]][pg >= 0]
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_padded_batch_leaves_rows_behind_the_last_request():
    rng = np.random.default_rng(5)
    page, Hk, Hq, D, lens, new = 16, 2, 4, 64, [20, 7], [3, 2]
    table, P = page_table(lens, page, rng)
    cu, N = _cu(new), 40
    q, k, v = (dev(rng.standard_normal((N, h, D)).astype(np.float16), torch) for h in (Hq, Hk, Hk))
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, "f16", rng), _pool(P, Hk, page, D, "f16", rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch))
    rows = (dev(np.asarray(lens, np.int32), torch), dev(cu, torch))
    f = dev(AO.frequencies(64), torch)
    qo = torch.full_like(q, -7.75)
    gdn.gdn_kv_write(k, v, cache, *rows, q=q, q_out=qo, inv_freq=f)
    ko, vo = torch.full_like(k, -7.75), torch.full_like(v, -7.75)
    gdn.gdn_kv_read(ko, vo, cache, *rows)
    torch.cuda.synchronize()
    for x in (qo, ko, vo):
        assert bool((x[5:] == -7.75).all()) and not bool((x[:5] == -7.75).any())
    assert np.array_equal(dv[0].cpu().numpy(), AO.cache_write(v.cpu().numpy()[:5], hv[0], table, cu, lens))


def test_dense_tokens_and_strided_rows():
    """cu_seqlens None; k, v slices of a projection's output."""
    rng = np.random.default_rng(6)
    page, Hk, D, lens = 16, 2, 128, [20, 7, 33, 4]
    table, P = page_table(lens, page, rng)
    wide = dev(rng.standard_normal((8, 3 * Hk * D)).astype(np.float16), torch)
    k, v = wide[:, Hk * D:2 * Hk * D].view(8, Hk, D), wide[:, 2 * Hk * D:].view(8, Hk, D)
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, "f16", rng), _pool(P, Hk, page, D, "f16", rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch))
    gdn.gdn_kv_write(k, v, cache, dev(np.asarray(lens, np.int32), torch))
    torch.cuda.synchronize()
    cu = _cu([2] * 4)
    assert np.array_equal(dk[0].cpu().numpy(), AO.cache_write(k.cpu().numpy(), hk[0], table, cu, lens))
    assert np.array_equal(dv[0].cpu().numpy(), AO.cache_write(v.cpu().numpy(), hv[0], table, cu, lens))


def test_many_requests_and_empty_ones():
    rng = np.random.default_rng(7)
    new = [int(x) for x in rng.integers(0, 3, 700)]
    lens = [int(x) + n for x, n in zip(rng.integers(0, 50, 700), new)]
    page, Hk, D = 16, 1, 64
    table, P = page_table(lens, page, rng)
    cu = _cu(new)
    k, v = (rng.standard_normal((cu[-1], Hk, D)).astype(np.float32) for _ in range(2))
    (hk, dk), (hv, dv) = _pool(P, Hk, page, D, "f32", rng), _pool(P, Hk, page, D, "f32", rng)
    cache = gdn.KVCache(dk[0], dv[0], dev(table, torch))
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), cache, dev(np.asarray(lens, np.int32), torch), dev(cu, torch))
    torch.cuda.synchronize()
    assert np.array_equal(dk[0].cpu().numpy(), AO.cache_write(k, hk[0], table, cu, lens))
    assert np.array_equal(dv[0].cpu().numpy(), AO.cache_write(v, hv[0], table, cu, lens))


def test_offsets_past_32_bits():
    D, Hk, page, P = 256, 8, 256, 4200
    assert P * Hk * page * D > 2 ** 31
    rng = np.random.default_rng(8)
    kp = torch.zeros((P, Hk, page, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    table = np.array([[P - 1, P - 2], [P - 3, 0]], np.int32)
    lens, cu = np.array([300, 10], np.int32), _cu([60, 10])
    k, v = (rng.standard_normal((70, Hk, D)).astype(np.float16) for _ in range(2))
    cache = gdn.KVCache(kp, vp, dev(table, torch))
    rows = (dev(lens, torch), dev(cu, torch))
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), cache, *rows)
    ko, vo = (torch.empty((70, Hk, D), dtype=torch.float16, device="cuda") for _ in range(2))
    gdn.gdn_kv_read(ko, vo, cache, *rows)
    torch.cuda.synchronize()
    assert np.array_equal(ko.cpu().numpy(), k) and np.array_equal(vo.cpu().numpy(), v)
    assert np.array_equal(kp[P - 1, :, 240:].cpu().numpy(), k[:16].transpose(1, 0, 2))
    assert not bool(kp[1:P - 3].any())
