"""GPU: how exactly attention over listed pages is computed (gdn_attn_sparse_forward).

FP32: scores, weights, sums and output in FP32 throughout, so the tolerance is that of
oracle.sparse_oracle.sparse_attention without rounded weights, and half a step of FP32. FP16 I/O: a
weight counts to 2^-19 of it, or to 2^-38 of the row's largest, and 2^-18 stands for the exponent's
arithmetic, as in test_gpu_attn_weights.py; then half a step of fp16. Weights rounded once to fp16
fail the first at every D, the second at 64 and 128 (at 256 the scores' own term hides them).
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, half_step
from long_helpers import any_cache, cu_of, queries, run_sparse

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import attn_oracle as AO                 # noqa: E402
from oracle import sparse_oracle as SO               # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _lists(c, T, K, seed):
    """Random entries that the token holds, in random order, as many as there are up to K."""
    rng = np.random.default_rng(seed)
    lists, counts, n = np.full((sum(T), c["Hk"], K), -1, np.int32), np.zeros(sum(T), np.int32), 0
    for t, m in zip(T, c["lens"]):
        for j in range(t):
            held = (int(m) - t + j) // c["page"] + 1
            counts[n] = min(K, held)
            for h in range(c["Hk"]):
                lists[n, h, :counts[n]] = rng.permutation(held)[:counts[n]]
            n += 1
    return lists, counts


def _scale_floor(c, q, cu, lists, counts):
    """8-bit values: 2^-38 of a row's largest product of weight and scale, for every code, as AO.attention's 2^-25."""
    v_scale = np.maximum(2.0 ** (c["v_scales"].astype(np.float64) - 127), 2.0 ** -33)[..., None]
    codes = np.abs(AO.e4m3_values()[c["v_codes"]])
    top = np.max(np.where(np.isfinite(codes * v_scale), v_scale, 0))
    # codes times the largest scale in place of the values' magnitudes: at least what the kernel's weights stand for
    big = np.where(np.isfinite(codes), codes, 0) * top
    _, rounded = SO.sparse_attention(q, c["k"], big, c["table"], cu, c["lens"], lists, counts)
    A, plain = SO.sparse_attention(q, c["k"], big, c["table"], cu, c["lens"], lists, counts, rounded_weights=False)
    return np.maximum(rounded - plain - 2.0 ** -11 * A, 0) * 2.0 ** -13


def _check(lens, T, *, Hk, G, D, fmt, page, K, seed=0, **kw):
    what = f"digits lens={lens[:6]} T={T[:6]} Hk={Hk} G={G} D={D} {fmt} page={page} K={K} {kw}"
    print(f"[gpu case] {what}", flush=True)
    c = any_cache(lens, fmt=fmt, Hk=Hk, D=D, page=page, seed=seed)
    cu, q = cu_of(T), queries(sum(T), Hk * G, D, fmt, seed + 7, scale=0.7)
    lists, counts = _lists(c, T, K, seed)
    args = (c["table"], cu, c["lens"], lists, counts)
    want, tol = SO.sparse_attention(q, c["k"], c["v"], *args, rounded_weights=False)
    if fmt != "f32":
        A, _ = SO.sparse_attention(q, c["k"], np.abs(c["v"]), *args, rounded_weights=False)
        if fmt == "e4m3":
            floor = _scale_floor(c, q, cu, lists, counts)
        else:
            floor = np.maximum(SO.sparse_attention(q, c["k"], c["v"], *args)[1] - tol - 2.0 ** -11 * A, 0) * 2.0 ** -13
        tol = tol + (2.0 ** -19 + 2.0 ** -18) * A + floor
    got = run_sparse(c, q, cu, lists, counts, torch, gdn, **kw)
    assert_within(got, want, tol + half_step(fmt, np.abs(want) + tol), what)


FORMATS = ("f32", "f16", "e4m3", "e2m1")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 6, 20])
def test_heads(fmt, D, G):
    _check([1, 16, 17, 100, 700], [1] * 5, Hk=2, G=G, D=D, fmt=fmt, page=16, K=5, dense=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,K", [(16, 3), (32, 4), (64, 9), (1024, 1)])
def test_pages_and_drafts(fmt, page, K):
    _check([1500, 64, 33, 5], [3, 1, 2, 0], Hk=2, G=4, D=128, fmt=fmt, page=page, K=K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mirrors", [True, False])
def test_lists_that_workgroups_share(fmt, D, mirrors):
    """Split over workgroups and joined from their parts."""
    _check([20000, 9000], [1, 3], Hk=2, G=6, D=D, fmt=fmt, page=64, K=100, mirrors=mirrors)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_lists(fmt):
    _check([200] * 150, [1] * 150, Hk=8, G=1, D=128, fmt=fmt, page=16, K=6, dense=True)
