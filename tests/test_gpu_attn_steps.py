"""GPU: the attention layer's entry points run together, as a serving loop uses them,
eagerly and captured in HIP graphs; and the places where the attention's work is split.

The values are held against the float64 oracle with its derived tolerances
(test_gpu_attn.py); replays, fused and separate calls are held against each other
bit for bit, since every sum's order is fixed by the lengths.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import FORMATS, assert_within, io_np, make_cache, oracle_attention, page_table, run_attention
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
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def _i32(x):
    return dev(np.asarray(x, np.int32), torch)


class Layer:
    """One attention layer's cache on the device, and what a step does with it."""

    def __init__(self, most, *, Hk, G, D, fmt, page, seed, rot=None, layout=0):
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.page, self.Hk, self.Hq, self.D, self.layout = rng, fmt, page, Hk, Hk * G, D, layout
        self.table, self.P = page_table(most, page, rng)
        shape = (self.P, Hk, page, D)
        self.io = torch.float32 if fmt == "f32" else torch.float16
        if fmt == "e4m3":
            pages = [torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.full(shape[:3], 130, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.pools = pages + scales
            self.cache = gdn.KVCache(*pages, _i32(self.table), k_scales=scales[0], v_scales=scales[1])
        else:
            self.pools = [torch.full(shape, float("nan"), dtype=self.io, device="cuda") for _ in range(2)]
            self.cache = gdn.KVCache(*self.pools, _i32(self.table))
        inv, self.factor = gdn.gdn_rope_frequencies(D if rot is None else rot, base=1e6)
        self.inv_np, self.inv = inv, dev(inv, torch)

    def tokens(self, N):
        """q, k, v [N, heads, D] on the host."""
        return [self.rng.standard_normal((N, h, self.D)).astype(io_np(self.fmt)) for h in (self.Hq, self.Hk, self.Hk)]

    def workspace(self, N, R):
        return torch.full((gdn.gdn_attn_workspace_bytes(N, R, self.Hq, self.cache) + 16,), 0xff, dtype=torch.uint8,
                          device="cuda")

    def step(self, q, k, v, q_rot, out, ws, lens, cu, *, R, window=0, lens_host=None, cu_host=None):
        gdn.gdn_kv_write(k, v, self.cache, lens, cu, q=q, q_out=q_rot, inv_freq=self.inv, rope_layout=self.layout,
                         rope_factor=self.factor, num_reqs=R, cu_seqlens_host=cu_host, seq_lens_host=lens_host)
        gdn.gdn_attn_forward(q_rot, self.cache, lens, cu, out, window=window, num_reqs=R, workspace=ws,
                             cu_seqlens_host=cu_host, seq_lens_host=lens_host)


def _oracle_step(layer, q, k, v, cu, lens, window):
    """Holds the pool's newest rows against the step's rotated keys and its values, and returns the
    (out, tolerance) of its attention over the pool, with q as rotated by the step."""
    pools = [x.cpu().numpy() for x in layer.pools]
    c = {"fmt": layer.fmt, "table": layer.table, "lens": np.asarray(lens, np.int32)}
    if layer.fmt == "e4m3":
        c.update(k_codes=pools[0], v_codes=pools[1], k_scales=pools[2], v_scales=pools[3],
                 k=AO.dequantise(pools[0], pools[2]), v=AO.dequantise(pools[1], pools[3]))
    else:
        c.update(k=pools[0], v=pools[1])
    # the pool's newest rows against the formula: half a step of the cache's type for v; the rotation's
    # FP32 operations (three roundings) before the rounding for k
    positions = np.concatenate([np.arange(m - t, m) for m, t in zip(lens, np.diff(cu))]).astype(np.int64)
    for name, rows in (("k", AO.rope(k, positions, layer.inv_np, layer.layout, layer.factor)), ("v", v.astype(np.float64))):
        got = AO.cache_read(c[name], layer.table, cu, lens)
        top = np.abs(rows).max(-1, keepdims=True)
        step = {"f16": 2.0 ** -11, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}[layer.fmt]
        # 8-bit: codes below the row's normal range are 2^-9 of its scale apart, the scale at most top / 224
        low = {"f16": 2.0 ** -25, "f32": 2.0 ** -149, "e4m3": 2.0 ** -10 / 224}[layer.fmt]
        tol = np.abs(rows) * step + low * np.maximum(top, 1.0) + (4 * 2.0 ** -24 * 2 * top if name == "k" else 0.0)
        if layer.fmt == "e4m3" and name == "k":
            tol = tol + step * 4 * 2.0 ** -24 * 2 * top + 2.0 ** -4 * 2.0 ** -8 * top    # a code's neighbour at a tie
        assert_within(got, rows, tol, f"{name} pool")
    return oracle_attention(c, q, cu, window=window)


@pytest.mark.parametrize("fmt,layout", [("f16", 0), ("f32", 1), ("e4m3", 0)])
@pytest.mark.parametrize("window", [0, 50])
def test_prompt_drafts_and_decode(fmt, layout, window):
    """Prompts, then speculative steps of which a part is accepted, then decode: every step's
    attention is that of the tokens kept so far, and the cache reads back what was kept."""
    R, G, D = 3, 3, 64
    layer = Layer([150, 80, 210], Hk=2, G=G, D=D, fmt=fmt, page=16, seed=40, rot=32, layout=layout)
    lens = np.zeros(R, np.int64)
    steps = [([100, 1, 130], [100, 1, 130]), ([4, 3, 4], [2, 0, 4]), ([4, 4, 2], [4, 1, 1]), ([1, 1, 1], [1, 1, 1]),
             ([1, 0, 1], [1, 0, 1]), ([30, 17, 9], [30, 17, 9]), ([1, 1, 1], [1, 1, 1])]
    for i, (new, kept) in enumerate(steps):
        _case(f"{fmt} window {window} step {i}: {new}")
        cu, total = _cu(new), lens + np.asarray(new)
        q, k, v = layer.tokens(cu[-1])
        N = int(cu[-1])
        dq, dk, dv = (dev(x, torch) for x in (q, k, v))
        q_rot, out = torch.empty_like(dq), torch.full_like(dq, -7.75)
        lens32, cu32 = total.astype(np.int32), cu.astype(np.int32)
        layer.step(dq, dk, dv, q_rot, out, layer.workspace(N, R), _i32(lens32), _i32(cu32), R=R, window=window,
                   lens_host=lens32, cu_host=cu32)
        torch.cuda.synchronize()
        want, tol = _oracle_step(layer, q_rot.cpu().numpy(), k, v, cu, total, window)
        assert_within(out.double().cpu().numpy(), want, tol, f"step {i}")
        lens = lens + np.asarray(kept)
    # everything kept, read back as one packed batch
    cu = _cu(lens)
    k_out = torch.empty((int(cu[-1]), 2, D), dtype=layer.io, device="cuda")
    v_out = torch.empty_like(k_out)
    gdn.gdn_kv_read(k_out, v_out, layer.cache, _i32(lens), _i32(cu), seq_lens_host=lens, cu_seqlens_host=cu)
    torch.cuda.synchronize()
    pools = [x.cpu().numpy() for x in layer.pools]
    for got, i in ((k_out, 0), (v_out, 1)):
        held = AO.dequantise(pools[i], pools[i + 2]) if fmt == "e4m3" else pools[i]
        want = AO.cache_read(held, layer.table, cu, lens).astype(io_np(fmt))
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_decode_over_growing_lengths(fmt):
    """One graph of a decode step, replayed while the program writes the next tokens and
    lengths into the graph's inputs; a second one, of another layer, between the replays.
    Given the lengths of the first step, or none."""
    R, G, D, start = 5, 6, 128, [700, 3, 64, 1, 2100]
    for mirrors in (True, False):
        layers = [Layer([m + 16 for m in start], Hk=2, G=G, D=D, fmt=fmt, page=32, seed=50 + i) for i in range(2)]
        prompts = [x.tokens(sum(start)) for x in layers]
        inputs = [x.tokens(R * 6) for x in layers]
        lens_first = np.asarray(start, np.int32) + 1
        both = []
        for x, (q, k, v) in zip(layers, prompts):
            gdn.gdn_kv_write(dev(k, torch), dev(v, torch), x.cache, _i32(start), _i32(_cu(start)), inv_freq=x.inv)
            b = {"q": torch.zeros((R, x.Hq, D), dtype=x.io, device="cuda"), "lens": _i32(lens_first),
                 "k": torch.zeros((R, 2, D), dtype=x.io, device="cuda"), "ws": x.workspace(R, R)}
            b["v"], b["q_rot"], b["out"] = torch.zeros_like(b["k"]), torch.empty_like(b["q"]), torch.empty_like(b["q"])
            both.append(b)
        torch.cuda.synchronize()
        before = [[p.clone() for p in x.pools] for x in layers]

        def call(i):
            x, b = layers[i], both[i]
            x.step(b["q"], b["k"], b["v"], b["q_rot"], b["out"], b["ws"], b["lens"], None, R=R,
                   lens_host=lens_first if mirrors else None)

        def feed(i, s):
            for name, src in zip(("q", "k", "v"), inputs[i]):
                both[i][name].copy_(dev(src[R * s:R * (s + 1)], torch))
            both[i]["lens"].copy_(_i32(lens_first + s))

        _case(f"{fmt}: eager steps")
        want = []
        for i in range(2):
            want.append([])
            for s in range(6):
                feed(i, s)
                call(i)
                torch.cuda.synchronize()
                want[i].append(both[i]["out"].clone())
        after = [[p.clone() for p in x.pools] for x in layers]
        for x, ps in zip(layers, before):
            for p, b in zip(x.pools, ps):
                p.copy_(b)
        _case(f"{fmt}: capture")
        graphs = []
        for i in range(2):
            feed(i, 0)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(i)
            graphs.append(g)
        for s in range(6):
            _case(f"{fmt}: replay {s}")
            for i in range(2):
                feed(i, s)
                both[i]["out"].fill_(float("nan"))
            for g in graphs:
                g.replay()
            noise = torch.randn(1000, device="cuda").sum()      # the program's own work
            for i in range(2):
                assert torch.equal(both[i]["out"], want[i][s]), (mirrors, i, s)
            assert bool(torch.isfinite(noise))
        bits = lambda p: p.view(torch.uint8)
        for x, ps in zip(layers, after):
            for p, b in zip(x.pools, ps):
                assert torch.equal(bits(p), bits(b))


def test_captured_verify_with_changing_drafts():
    """A captured speculative step without mirrors: draft counts, lengths and the page table change
    between the replays, down to no draft at all; tokens behind the last request are padding."""
    R, G, D, N = 4, 4, 128, 16
    layer = Layer([900, 300, 64, 20], Hk=2, G=G, D=D, fmt="f16", page=16, seed=60)
    start = [850, 250, 20, 0]
    q, k, v = layer.tokens(sum(start))
    gdn.gdn_kv_write(dev(k, torch), dev(v, torch), layer.cache, _i32(start), _i32(_cu(start)), inv_freq=layer.inv)
    b = {n: torch.zeros((N, h, D), dtype=layer.io, device="cuda") for n, h in
         (("q", layer.Hq), ("k", 2), ("v", 2), ("q_rot", layer.Hq), ("out", layer.Hq))}
    lens, cu, ws = _i32(np.asarray(start) + 4), _i32(_cu([4] * 4)), layer.workspace(N, R)
    table = layer.cache._keep[4]

    def call():
        layer.step(b["q"], b["k"], b["v"], b["q_rot"], b["out"], ws, lens, cu, R=R)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    torch.cuda.synchronize()
    first = layer.table.copy()
    for s, new in enumerate([[4, 4, 4, 4], [1, 0, 3, 2], [0, 0, 0, 0], [4, 4, 1, 4], [13, 1, 1, 1]]):
        _case(f"replay {s}: {new}")
        fresh = layer.tokens(N)
        for name, x in zip(("q", "k", "v"), fresh):
            b[name].copy_(dev(x, torch))
        if s == 3:                                              # request 1's pages are taken away
            layer.table = first.copy()
            layer.table[1, 3:] = -1
        table.copy_(_i32(layer.table))
        total = np.asarray(start) + np.asarray(new)
        lens.copy_(_i32(total))
        cu.copy_(_i32(_cu(new)))
        saved = [p.clone() for p in layer.pools]
        b["q_rot"].fill_(-3.0)
        b["out"].fill_(-7.75)
        call()
        torch.cuda.synchronize()
        want, want_q, pools = b["out"].clone(), b["q_rot"].clone(), [p.clone() for p in layer.pools]
        for p, x in zip(layer.pools, saved):
            p.copy_(x)
        b["q_rot"].fill_(-3.0)
        b["out"].fill_(-7.75)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want) and torch.equal(b["q_rot"], want_q)
        for p, x in zip(layer.pools, pools):
            assert torch.equal(p.view(torch.uint8), x.view(torch.uint8))
        used = sum(new)
        assert torch.all(b["out"][used:] == -7.75) and torch.all(b["q_rot"][used:] == -3.0)
        c = {"fmt": "f16", "table": layer.table, "lens": total, "k": pools[0].cpu().numpy(), "v": pools[1].cpu().numpy()}
        ref, tol = oracle_attention(c, want_q.cpu().numpy()[:used], _cu(new))
        assert_within(want.double().cpu().numpy()[:used], ref, tol, f"replay {s}")


def _check(lens, new, *, Hk, G, D, fmt, page, seed=0, **kw):
    what = f"lens={lens if len(lens) < 9 else len(lens)} new={new if len(new) < 9 else ''} Hk={Hk} G={G} D={D} {fmt} {kw}"
    _case(what)
    run = {n: kw.pop(n) for n in ("dense", "mirrors") if n in kw}
    c = make_cache(lens, Hk=Hk, D=D, fmt=fmt, page=page, seed=seed)
    q = (np.random.default_rng(seed + 1).standard_normal((sum(new), Hk * G, D)) * 1.5).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu(new), **kw)
    assert_within(run_attention(c, q, _cu(new), torch, gdn, **run, **kw), want, tol, what)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_past_a_segment(fmt, D):
    """Prompts of more than 64 rows, the last segment full or of one or two rows; rows of one token in two segments."""
    _check([300, 130], [33, 65], Hk=1, G=2, D=D, fmt=fmt, page=16, seed=70)
    _check([200, 77], [7, 1], Hk=1, G=24, D=D, fmt=fmt, page=32, seed=71)
    _check([2000], [40], Hk=1, G=3, D=D, fmt=fmt, page=64, seed=72, mirrors=False)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,new,G", [([3000, 2000], [8, 8], 8), ([2500, 999, 4000], [24, 23, 25], 4), ([1500], [100], 2),
                                        ([5000, 700], [40, 41], 6), ([1500], [70], 5), ([4000, 130, 2], [16, 16, 2], 4),
                                        ([3000, 2500, 60, 500], [9, 0, 9, 10], 4)])
def test_segments_side_by_side(fmt, D, lens, new, G):
    """Requests of 2, 3, 7, 8 and more segments over long caches, equally many or not, one without tokens."""
    _check(lens, new, Hk=2, G=G, D=D, fmt=fmt, page=64, seed=80)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 40, 1500])
@pytest.mark.parametrize("mirrors", [True, False])
def test_many_requests_side_by_side(fmt, window, mirrors):
    """Two segments each: notes by segment with few requests, by workgroup with many."""
    rng = np.random.default_rng(81)
    for R in (5, 90):
        lens = [int(x) for x in rng.integers(40, 900, R)]
        lens[1] = 5000
        _check(lens, [10] * R, Hk=2, G=5, D=64, fmt=fmt, page=32, seed=82, window=window, mirrors=mirrors, dense=not mirrors)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("mirrors", [True, False])
@pytest.mark.parametrize("R", [1, 20, 129, 400])
def test_segments_and_workgroups(fmt, mirrors, R):
    """Fewer and more segments than workgroups, decode and drafts, one long request among short ones:
    notes by segment and by workgroup, segments in one workgroup and in many."""
    rng = np.random.default_rng(R)
    lens = [int(x) for x in rng.integers(1, 300, R)]
    lens[R // 2] = 6000
    _check(lens, [1] * R, Hk=2, G=2, D=64, fmt=fmt, page=64, seed=73, dense=True, mirrors=mirrors)
    new = [int(min(x, n)) for x, n in zip(rng.integers(1, 5, R), lens)]
    _check(lens, new, Hk=2, G=6, D=64, fmt=fmt, page=64, seed=74, mirrors=mirrors)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G", [2, 20])
def test_many_short_requests(fmt, G):
    """More unsplit segments than get a workgroup each: shared out by length, some requests without tokens,
    some without a cached position, one far longer than the rest."""
    rng = np.random.default_rng(83)
    R = 700
    lens = [int(x) for x in rng.integers(0, 60, R)]
    new = [int(min(x, n)) for x, n in zip(rng.integers(0, 3, R), lens)]
    lens[130] = 700
    lens[131:200] = [5] * 69
    new[131:200] = [0] * 69                                # a run of requests with nothing to do
    lens[R - 1], new[R - 1] = 33, 1
    c = make_cache(lens, Hk=2, D=64, fmt=fmt, page=16, seed=84)
    q = (np.random.default_rng(85).standard_normal((sum(new), 2 * G, 64))).astype(io_np(fmt))
    want, tol = oracle_attention(c, q, _cu(new))
    assert_within(run_attention(c, q, _cu(new), torch, gdn), want, tol, f"{fmt} {G}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 100, 128, 1000])
def test_windows_of_long_caches(fmt, window):
    _check([5000, 4097, 127], [1, 1, 1], Hk=2, G=4, D=128, fmt=fmt, page=128, window=window, seed=75)
    _check([5000, 4097, 127], [5, 20, 3], Hk=2, G=4, D=128, fmt=fmt, page=128, window=window, seed=76)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("mirrors", [True, False])
@pytest.mark.parametrize("new", [1, 5])
def test_nan_scores_show(fmt, mirrors, new):
    """A row whose q is NaN gives NaN, however its positions are split; so does one key that is NaN, alone or
    among others, at the first position or the last."""
    G, D = 4, 64
    for length in (new, 40, 5000):
        c = make_cache([length, 30], Hk=2, D=D, fmt=fmt, page=64, seed=77)
        q = (np.random.default_rng(78).standard_normal((2 * new, 2 * G, D))).astype(io_np(fmt))
        cu = _cu([new, new])
        clean, tol = oracle_attention(c, q, cu)
        q[new - 1, 3, 5] = np.nan
        got = run_attention(c, q, cu, torch, gdn, mirrors=mirrors)
        assert np.all(np.isnan(got[new - 1, 3]))
        ok = np.ones(got.shape[:2], bool)
        ok[new - 1, 3] = False
        assert_within(got[ok], clean[ok], tol[ok], f"{fmt} {length}: rows beside a NaN row")
        q[new - 1, 3, 5] = 0
        for pos in {0, length - 1, length // 2}:
            for value in (np.nan,) if fmt == "e4m3" else (np.nan, np.inf):
                d = {**c, "k": c["k"].copy()}
                if fmt == "e4m3":
                    d["k_codes"] = c["k_codes"].copy()
                    d["k_codes"][c["table"][0, pos // 64], 1, pos % 64, 9] = 0x7f
                else:
                    d["k"][c["table"][0, pos // 64], 1, pos % 64, 9] = value
                q[:, :, 9] = np.abs(q[:, :, 9]) + 0.25                # inf times it: +inf, no softmax
                got = run_attention(d, q, cu, torch, gdn, mirrors=mirrors)
                want, tol2 = oracle_attention(c, q, cu)
                sees = np.arange(new) >= new - (length - pos)
                assert np.all(np.isnan(got[:new, G:][sees])), (fmt, length, pos, value)
                assert_within(got[:, :G], want[:, :G], tol2[:, :G], "the other key head")
                assert_within(got[new:], want[new:], tol2[new:], "the other request")
                assert_within(got[:new, G:][~sees], want[:new, G:][~sees], tol2[:new, G:][~sees], "rows before it")


def test_minus_infinity_everywhere_is_an_empty_row():
    """Scores that are all -inf leave nothing to attend."""
    c = make_cache([50], Hk=1, D=64, fmt="f32", page=16, seed=79)
    c["k"][..., 3] = np.where(np.isnan(c["k"][..., 3]), np.nan, -np.inf)
    q = np.zeros((1, 2, 64), np.float32)
    q[..., 3] = 1.0
    c["k"][..., 4:], c["k"][..., :3] = np.nan_to_num(c["k"][..., 4:]), np.nan_to_num(c["k"][..., :3])
    assert np.all(run_attention(c, q, _cu([1]), torch, gdn) == 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G", [2, 20])
def test_lengths_and_windows_at_the_ends_of_int32(fmt, G):
    """Any int32 in seq_lens (no host mirror), and the largest window: positions past the table count as far as
    the table goes, those before 0 not at all."""
    D, page = 64, 16
    c = make_cache([64, 64, 64, 64], Hk=2, D=D, fmt=fmt, page=page, seed=90)
    c["table"] = np.ascontiguousarray(c["table"][:, :4])       # 64 positions are all there is
    new = [2, 1, 2, 1]
    q = np.random.default_rng(91).standard_normal((6, 2 * G, D)).astype(io_np(fmt))
    rows = [q[0:1], q[1:2], q[2:3], q[3:4], q[4:5], q[5:6]]
    of = [0, 0, 1, 2, 2, 3]                                    # request of each row
    odd = {**c, "lens": np.asarray([2 ** 31 - 1, -2 ** 31, -1, 2 ** 31 - 1], np.int32)}
    for window in (0, 2 ** 31 - 1, 1000):
        got = run_attention(odd, q, _cu(new), torch, gdn, mirrors=False, window=window)
        for i, (row, r) in enumerate(zip(rows, of)):
            if r in (1, 2) or window == 1000:
                assert np.all(got[i] == 0), (window, i)
                continue
            one = {**c, "table": c["table"][r:r + 1], "lens": np.asarray([64], np.int32)}
            want, tol = oracle_attention(one, row, _cu([1]))
            assert_within(got[i:i + 1], want, tol, f"{fmt} {i}")
    # the largest window on ordinary lengths is no window
    plain = run_attention(c, q, _cu(new), torch, gdn)
    assert np.array_equal(run_attention(c, q, _cu(new), torch, gdn, window=2 ** 31 - 1), plain)
