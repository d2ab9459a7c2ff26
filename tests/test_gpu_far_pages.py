"""GPU: a step over pages that lie past 4 GiB in their pools, and in the array of bounds, gives what it gives over near ones.

Write with the rotation, bounds, selection, attention over the selected pages and over all, read back, with the
pages' numbers as the only difference: every output is the same bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest

from gpu_helpers import dev
from long_helpers import cu_of, queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import attn_oracle as AO                 # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


D, HK, HQ, PAGE = 64, 1, 4, 16
LENS, NEW = [70, 300, 33], [70, 300, 33]
WIDTH = {"f16": D, "e4m3": D, "e2m1": D // 2}


def _pool(fmt, P):
    """k_pages, v_pages and the scales of P pages, unwritten."""
    t = torch.float16 if fmt == "f16" else torch.uint8
    pages = [torch.empty((P, HK, PAGE, WIDTH[fmt]), dtype=t, device="cuda") for _ in range(2)]
    shape = {"f16": None, "e4m3": (P, HK, PAGE), "e2m1": (P, HK, D // 32, PAGE)}[fmt]
    scales = {} if shape is None else {n: torch.empty(shape, dtype=torch.uint8, device="cuda") for n in ("k_scales", "v_scales")}
    return pages, scales


def _step(fmt, P, ids):
    """All calls with request r's pages ids[r]; the outputs."""
    pages, scales = _pool(fmt, P)
    table = np.full((len(LENS), max(len(i) for i in ids) + 1), -1, np.int32)
    for r, i in enumerate(ids):
        table[r, :len(i)] = i
    cache = gdn.KVCache(*pages, dev(table, torch), **scales, page_table_host=table)
    lens, cu = np.asarray(LENS, np.int32), cu_of(NEW)
    N, R, K = int(cu[-1]), len(LENS), 5
    q, k, v = (dev(queries(N, h, D, "f16", s), torch) for h, s in ((HQ, 1), (HK, 2), (HK, 3)))
    q_out = torch.empty_like(q)
    mirrors = dict(cu_seqlens_host=cu, seq_lens_host=lens)
    dcu, dlens = dev(cu, torch), dev(lens, torch)
    gdn.gdn_kv_write(k, v, cache, dlens, dcu, q=q, q_out=q_out, inv_freq=dev(AO.frequencies(D), torch), **mirrors)
    bounds = torch.empty((P, HK, 2, D), dtype=torch.float16, device="cuda")
    gdn.gdn_kv_bounds(bounds, cache, dlens, dcu, num_tokens=N, num_reqs=R, **mirrors)
    lists = torch.full((N, HK, K), -77, dtype=torch.int32, device="cuda")
    counts = torch.full((N,), -77, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(gdn.gdn_attn_select_workspace_bytes(N, R, HQ, K, cache), gdn.gdn_attn_workspace_bytes(N, R, HQ, cache),
                         gdn.gdn_attn_sparse_workspace_bytes(N, R, HQ, K, cache)), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_select(q_out, bounds, cache, dlens, dcu, lists, counts, workspace=ws, **mirrors)
    sparse, full = torch.empty_like(q), torch.empty_like(q)
    gdn.gdn_attn_sparse_forward(q_out, cache, dlens, dcu, lists, counts, sparse, workspace=ws, **mirrors)
    gdn.gdn_attn_forward(q_out, cache, dlens, dcu, full, workspace=ws, **mirrors)
    back_k, back_v = torch.empty_like(k), torch.empty_like(v)
    gdn.gdn_kv_read(back_k, back_v, cache, dlens, dcu, **mirrors)
    torch.cuda.synchronize()
    at = dev(np.concatenate(ids).astype(np.int64), torch)
    return [x.cpu() for x in (q_out, bounds[at], lists, counts, sparse, full, back_k, back_v)]


@pytest.mark.parametrize("fmt,P", [("f16", (1 << 22) + 9), ("e4m3", (1 << 23) + 9), ("e2m1", (1 << 24) + 9)])
def test_pages_past_4_gib(fmt, P):
    print(f"[gpu case] far pages {fmt} P={P}", flush=True)
    assert P * HK * PAGE * D * {"f16": 16, "e4m3": 8, "e2m1": 4}[fmt] // 8 > 1 << 33
    need = [-(-m // PAGE) for m in LENS]
    rng = np.random.default_rng(0)
    near = np.split(rng.permutation(sum(need)), np.cumsum(need)[:-1])
    # from both ends of the pool and around the places where a byte offset passes 2^31, 2^32 and 2^33
    row = PAGE * D * {"f16": 16, "e4m3": 8, "e2m1": 4}[fmt] // 8
    places = np.unique(np.concatenate([[(1 << b) // row + d for d in (-2, -1, 0, 1)] for b in (31, 32, 33)] + [P - 1 - np.arange(20), np.arange(20)]))
    some = rng.permutation(places[places < P])
    assert len(some) >= sum(need)
    far = np.split(some[:sum(need)], np.cumsum(need)[:-1])
    want, got = _step(fmt, sum(need), near), _step(fmt, P, far)
    torch.cuda.empty_cache()
    names = ("q", "bounds", "lists", "counts", "sparse attention", "attention", "keys", "values")
    for name, a, b in zip(names, want, got):
        assert torch.equal(a, b), name
        assert not torch.isnan(a.float()).any(), name
