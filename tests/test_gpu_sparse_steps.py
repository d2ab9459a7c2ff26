"""The operators for long contexts as a program uses them, one after the other: prompts and decode steps
into a cache (16, 8 and 4 bits), the bounds of the pages that got new keys, the selection, attention over
the selected pages; eagerly, on a stream of its own, and captured in a HIP graph that is replayed while
the requests grow.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, half_step
from gpu_helpers import dev
from long_helpers import cu_of, queries
from oracle import attn_oracle as AO
from oracle import sparse_oracle as SO

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402

HK, HQ, D, PAGE, K, FIRST, NEWEST, ROT = 2, 8, 64, 16, 4, 1, 1, 32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


class Server:
    """A cache with its bounds, and the buffers of a step of one token a request."""

    def __init__(self, fmt, reqs, most, seed=0, dim=D, page=PAGE):
        rng = np.random.default_rng(seed)
        self.fmt, self.reqs, self.dim, self.page = fmt, reqs, dim, page
        M = -(-most // page)
        P = reqs * M + 2
        self.table = rng.permutation(P)[:reqs * M].reshape(reqs, M).astype(np.int32)
        codes = {"f16": (dim, torch.float16), "e4m3": (dim, torch.uint8), "e2m1": (dim // 2, torch.uint8)}[fmt]
        scales = {"f16": None, "e4m3": (P, HK, page), "e2m1": (P, HK, dim // 32, page)}[fmt]
        pool = lambda: torch.zeros((P, HK, page, codes[0]), dtype=codes[1], device="cuda")  # noqa: E731
        scale = lambda: None if scales is None else torch.zeros(scales, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k, self.v, self.ks, self.vs = pool(), pool(), scale(), scale()
        self.cache = gdn.KVCache(self.k, self.v, dev(self.table, torch), k_scales=self.ks, v_scales=self.vs)
        self.bounds = torch.zeros((P, HK, 2, dim), dtype=torch.float16, device="cuda")
        self.freq = dev(AO.frequencies(ROT), torch)
        self.lens = torch.zeros(reqs, dtype=torch.int32, device="cuda")
        self.new = {n: torch.zeros((reqs, h, dim), dtype=torch.float16, device="cuda") for n, h in (("q", HQ), ("k", HK), ("v", HK))}
        self.q, self.out = (torch.zeros((reqs, HQ, dim), dtype=torch.float16, device="cuda") for _ in range(2))
        self.lists = torch.zeros((reqs, HK, K), dtype=torch.int32, device="cuda")
        self.counts = torch.zeros(reqs, dtype=torch.int32, device="cuda")
        self.ws = [torch.empty(max(f(reqs, reqs, HQ, K, self.cache), 16), dtype=torch.uint8, device="cuda")
                   for f in (gdn.gdn_attn_select_workspace_bytes, gdn.gdn_attn_sparse_workspace_bytes)]

    def write(self, k, v, lens, T=None, **kw):
        """New tokens and their pages' bounds."""
        cu = None if T is None else dev(cu_of(T), torch)
        gdn.gdn_kv_write(k, v, self.cache, lens, cu, inv_freq=self.freq, num_reqs=self.reqs, **kw)
        gdn.gdn_kv_bounds(self.bounds, self.cache, lens, cu, num_tokens=k.shape[0], num_reqs=self.reqs)

    def step(self, **kw):
        """One decode step of every request."""
        n = self.new
        self.write(n["k"], n["v"], self.lens, q=n["q"], q_out=self.q, **kw)
        gdn.gdn_attn_select(self.q, self.bounds, self.cache, self.lens, None, self.lists, self.counts, first_pages=FIRST,
                            newest_pages=NEWEST, workspace=self.ws[0])
        gdn.gdn_attn_sparse_forward(self.q, self.cache, self.lens, None, self.lists, self.counts, self.out, workspace=self.ws[1])

    def values(self, name):
        pages, scales = {"k": (self.k, self.ks), "v": (self.v, self.vs)}[name]
        pages = pages.cpu().numpy()
        if self.fmt == "f16":
            return pages.astype(np.float64)
        s = scales.cpu().numpy()
        return AO.dequantise(pages, s) if self.fmt == "e4m3" else SO.dequantise(SO.unpack(pages), np.swapaxes(s, -1, -2))

    def check(self, what):
        """The step's lists and output against the oracle, from what the cache holds and the rotated q."""
        torch.cuda.synchronize()
        lens, cu, q = self.lens.cpu().numpy(), np.arange(self.reqs + 1), self.q.cpu().numpy()
        k, v = self.values("k"), self.values("v")
        b = self.bounds.cpu().numpy().astype(np.float64)
        # bounds of every page that is in use, whoever wrote them and when
        for r in range(self.reqs):
            for i in range(-(-int(lens[r]) // self.page)):
                page = k[self.table[r, i], :, :min(self.page, int(lens[r]) - i * self.page)]
                assert np.array_equal(b[self.table[r, i], :, 0], page.min(1)) and np.array_equal(b[self.table[r, i], :, 1], page.max(1)), what
        lists, counts, gaps = SO.select(q, b, self.table, self.page, cu, lens, K, FIRST, NEWEST)
        assert gaps.min() > 1e-12
        assert np.array_equal(self.lists.cpu().numpy(), lists) and np.array_equal(self.counts.cpu().numpy(), counts), what
        want, tol = SO.sparse_attention(q, k, v, self.table, cu, lens, lists, counts)
        assert_within(self.out.double().cpu().numpy(), want, tol + half_step("f16", np.abs(want) + tol), what)

    def feed(self, seed):
        for i, (n, x) in enumerate(self.new.items()):
            x.copy_(dev(queries(*x.shape, "f16", 10 * seed + i), torch))


def _prompts(s, T, seed):
    N = sum(T)
    k, v = (dev(queries(N, HK, s.dim, "f16", seed + i), torch) for i in range(2))
    s.lens.copy_(dev(np.asarray(T, np.int32), torch))
    s.write(k, v, s.lens, T)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "e2m1"])
def test_prompts_and_decode_steps(fmt):
    _case(f"prompts and decode steps {fmt}")
    s = Server(fmt, 3, 300)
    _prompts(s, [100, 5, 260], 1)
    for i in range(20):
        s.feed(i)
        s.lens += 1
        s.step()
        if i % 3 == 0:
            s.check(f"{fmt} step {i}")


@pytest.mark.parametrize("fmt", ["f16", "e2m1"])
def test_steps_on_another_stream(fmt):
    _case(f"another stream {fmt}")
    s, t = Server(fmt, 2, 200), Server(fmt, 2, 200)
    side = torch.cuda.Stream()
    for x in (s, t):
        _prompts(x, [64, 33], 1)
        x.lens += 1
        x.feed(3)
    torch.cuda.synchronize()
    s.step()
    with torch.cuda.stream(side):
        t.step()
    torch.cuda.synchronize()
    s.check("current stream")
    t.check("side stream")
    assert torch.equal(s.out, t.out) and torch.equal(s.lists, t.lists)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "e2m1"])
def test_captured_step(fmt):
    """One graph for all steps: lengths, keys and lists change between replays, with eager work beside them."""
    _case(f"captured {fmt}")
    s, eager = Server(fmt, 3, 400), Server(fmt, 3, 400)
    for x in (s, eager):
        _prompts(x, [200, 3, 15], 1)
        x.feed(0)
        x.lens += 1
        x.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for i in range(1, 24):
        for x in (s, eager):
            x.feed(i)
            x.lens += 1
        g.replay()
        eager.step()
        torch.cuda.synchronize()
        assert torch.equal(s.lists, eager.lists) and torch.equal(s.counts, eager.counts), i
        assert torch.equal(s.out, eager.out) and torch.equal(s.bounds, eager.bounds), i
        if i % 8 == 0:
            s.check(f"{fmt} replay {i}")


def test_captured_with_short_lengths_and_replayed_over_long_ones():
    """Mirrors at capture guide the split only: lists and outputs are those of a call without them."""
    _case("captured short, replayed long")
    reqs, most = 2, 9000
    s = Server("e2m1", reqs, most)
    _prompts(s, [9000, 5000], 1)
    s.feed(1)
    cu = None
    short = np.array([40, 20], np.int32)
    rows = dict(num_reqs=reqs, seq_lens_host=short)

    def calls():
        gdn.gdn_attn_select(s.new["q"], s.bounds, s.cache, s.lens, cu, s.lists, s.counts, first_pages=FIRST, newest_pages=NEWEST,
                            workspace=s.ws[0], **rows)
        gdn.gdn_attn_sparse_forward(s.new["q"], s.cache, s.lens, cu, s.lists, s.counts, s.out, workspace=s.ws[1], **rows)

    s.lens.copy_(dev(short, torch))
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for lens in ([9000, 5000], [40, 20], [17, 8999]):
        s.lens.copy_(dev(np.asarray(lens, np.int32), torch))
        s.q.copy_(s.new["q"])
        g.replay()
        torch.cuda.synchronize()
        q, k, v, b = s.q.cpu().numpy(), s.values("k"), s.values("v"), s.bounds.cpu().numpy()
        lists, counts, gaps = SO.select(q, b, s.table, PAGE, np.arange(3), lens, K, FIRST, NEWEST)
        assert gaps.min() > 1e-12
        assert np.array_equal(s.lists.cpu().numpy(), lists) and np.array_equal(s.counts.cpu().numpy(), counts)
        want, tol = SO.sparse_attention(q, k, v, s.table, np.arange(3), lens, lists, counts)
        assert_within(s.out.double().cpu().numpy(), want, tol + half_step("f16", np.abs(want) + tol), f"replayed over {lens}")


def test_the_same_call_twice_gives_the_same_bits():
    _case("repeatable")
    s = Server("e2m1", 4, 6000, page=64)
    _prompts(s, [6000, 4000, 77, 1], 1)
    s.feed(2)
    outs = []
    for _ in range(3):
        s.step()
        torch.cuda.synchronize()
        outs.append((s.out.clone(), s.lists.clone(), s.bounds.clone()))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
