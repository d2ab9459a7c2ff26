"""GPU: gdn_attn_select among NaN, infinite and finite scores, by each of the ways that it finds a list's last
score, and that nothing but the lists and their lengths is written.

Pages are shared by many entries, so that scores are equal, too; the selections are compared exactly, as in
test_gpu_sparse.py.
"""
from __future__ import annotations

import numpy as np
import pytest

from gpu_helpers import dev
from long_helpers import cu_of, queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import sparse_oracle as SO               # noqa: E402

GUARD = 4096
PAGE, PAGES = 16, 257


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _guarded(n):
    x = torch.full((n + 2 * GUARD,), -77, dtype=torch.int32, device="cuda")
    return x, x[GUARD:GUARD + n]


def _check(what, held, T, *, Hk, G, D, fmt, K, first, newest, broken, said=None, seed=0):
    """Requests of `held` entries and T new tokens each; `said` entries by the host's mirror. `broken`: of the pages,
    which share has NaN bounds, or "infinite" for one infinite channel in a third of them."""
    what = f"{what}: held={held[:4]} T={T[:4]} Hk={Hk} G={G} D={D} {fmt} K={K} first={first} newest={newest} broken={broken} said={said}"
    _case(what)
    rng = np.random.default_rng(seed)
    io = np.float32 if fmt == "f32" else np.float16
    R, N = len(held), sum(T)
    table = rng.integers(0, PAGES, (R, max(held))).astype(np.int32)
    b = (rng.standard_normal((PAGES, Hk, 1, D)) * 0.5 + np.array([-1.0, 1.0])[:, None] * (2 + rng.random((PAGES, Hk, 1, D)))).astype(io)
    if broken == "infinite":
        some = rng.permutation(PAGES)[:PAGES // 3]
        b[some, :, 1, 3], b[some, :, 0, 5] = np.inf, -np.inf
    else:
        b[rng.permutation(PAGES)[:int(broken * PAGES)], :, :, 7] = np.nan
    lens = np.asarray([PAGE * (h - 1) + 1 + int(rng.integers(0, PAGE)) for h in held], np.int32)
    lens = np.maximum(lens, np.asarray(T, np.int32))
    cu, q = cu_of(T), queries(N, Hk * G, D, fmt, seed + 1)
    with np.errstate(invalid="ignore"):
        lists, counts, gaps = SO.select(q, b, table, PAGE, cu, lens, K, first, newest)
    assert gaps.min(initial=1.0) > 1e-12, what
    pool = torch.zeros((PAGES, Hk, PAGE, D), dtype=torch.float32 if fmt == "f32" else torch.float16, device="cuda")
    cache = gdn.KVCache(pool, torch.zeros_like(pool), dev(table, torch))
    all_lists, got = _guarded(N * Hk * K)
    all_counts, n = _guarded(N)
    ws = torch.full((gdn.gdn_attn_select_workspace_bytes(N, R, Hk * G, K, cache),), 0xff, dtype=torch.uint8, device="cuda")
    mirror = lens if said is None else np.minimum(lens, said * PAGE).astype(np.int32)
    gdn.gdn_attn_select(dev(q, torch), dev(b, torch), cache, dev(lens, torch), dev(cu, torch), got.view(N, Hk, K), n, first_pages=first,
                        newest_pages=newest, cu_seqlens_host=cu, seq_lens_host=mirror, workspace=ws)
    torch.cuda.synchronize()
    for x in (all_lists, all_counts):
        assert (x[:GUARD] == -77).all().item() and (x[-GUARD:] == -77).all().item(), f"{what}: written outside the lists"
    assert np.array_equal(n.cpu().numpy(), counts), what
    assert np.array_equal(got.view(N, Hk, K).cpu().numpy(), lists), what


# (what, held, T, said): one launch, its keys in LDS, or read again by four waves where the mirror says less than there
# is; two launches, the list by one, four and sixteen waves with the keys in registers, or read again by each
WAYS = {
    "one launch": ([200, 37, 256], [1, 2, 1], None),
    "one launch, keys read again": ([200, 256], [1, 3], 4),
    "one wave": ([500, 257, 512], [1, 3, 5], None),
    "one wave, keys read again": ([700] * 130, [1] * 130, 2),
    "four waves": ([1250, 513], [3, 1], None),
    "four waves, keys read again": ([2500, 900], [2, 1], 600),
    "sixteen waves": ([4100, 2060], [3, 2], None),
    "sixteen waves, keys read again": ([8800, 8200], [1, 3], None),
}


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("broken", [0.02, 0.3, 0.9, "infinite"])
@pytest.mark.parametrize("K,first,newest", [(8, 1, 2), (8, 0, 0), (33, 1, 1)])
def test_nan_scores_beside_finite_ones(way, broken, K, first, newest):
    held, T, said = WAYS[way]
    Hk = 8 if len(held) > 100 else 2
    _check(way, held, T, Hk=Hk, G=1, D=64, fmt="f16", K=K, first=first, newest=newest, broken=broken, said=said)


@pytest.mark.parametrize("way", ["one launch", "one wave", "sixteen waves"])
@pytest.mark.parametrize("fmt,D,G", [("f32", 64, 4), ("f32", 256, 2), ("f16", 128, 6)])
def test_nan_scores_of_every_type(way, fmt, D, G):
    held, T, said = WAYS[way]
    for K in (1, 7, 120):
        _check(way, held, T, Hk=2, G=G, D=D, fmt=fmt, K=K, first=min(1, K - 1), newest=1, broken=0.4, said=said, seed=K)
