"""GPU: how exactly softmax weights enter the output over 4-bit pages (gdn_attn_forward and
gdn_attn_sparse_forward), as test_gpu_attn_weights.py does for the other formats.

A weight takes part to 2^-19 of it, or to 2^-38 of the row's largest, whatever the size of the
scores. Tolerances: this, the FP32 terms of oracle.attn_oracle.attention (no rounded weights) and
2^-18 for the exponent's own arithmetic, then half a step of fp16.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, half_step, run_attention
from long_helpers import any_device_cache, cu_of, make_cache4, queries, run_sparse

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


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _run(c, q, cu, lists, **kw):
    """Over all positions, or over all pages as lists."""
    cache = any_device_cache(c, torch, gdn)
    if not lists:
        return run_attention(c, q, cu, torch, gdn, cache=cache, **kw)
    K = c["table"].shape[1]
    every = np.broadcast_to(np.arange(K, dtype=np.int32), (len(q), c["Hk"], K)).copy()
    return run_sparse(c, q, cu, every, None, torch, gdn, cache=cache, **kw)


def _oracle(c, q, cu, scale=None):
    """(out, tolerance) as the module's text has it."""
    def attention(v, **kw):
        return AO.attention(q, c["k"], v, c["table"], cu, c["lens"], scale=scale, **kw)
    out, bound = attention(c["v"], rounded_weights=False)
    A = attention(np.abs(c["v"]), rounded_weights=False)[0]
    # the rounded bound's terms beyond `bound` are 2^-11 A and 2^-25 of the largest weight for every |v|
    floor = np.maximum(attention(c["v"])[1] - bound - 2.0 ** -11 * A, 0.0) * 2.0 ** -13
    tol = bound + (2.0 ** -19 + 2.0 ** -18) * A + floor
    return out, tol + half_step("e2m1", np.abs(out) + tol)


def _set_key(c, pos, code):
    """The key of request 0's position pos: `code` in every channel, times 1."""
    page, slot = c["table"][0, pos // c["page"]], pos % c["page"]
    c["k_codes"][page, :, slot], c["k_scales"][page, :, :, slot] = code * 17, 127
    c["k"][page, :, slot] = SO.values(np.array([code]))[0]


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,new,G", [([2, 3, 5], [1, 1, 1], 4), ([40, 300], [4, 5], 4), ([700, 90], [2, 1], 24), ([3000], [8], 8)])
def test_weights_keep_their_digits(lists, D, lens, new, G):
    _case(f"lists={lists} D={D} lens={lens} new={new} G={G}")
    c = make_cache4(lens, Hk=2, D=D, page=16, seed=100 + D)
    cu, q = cu_of(new), queries(sum(new), 2 * G, D, "f16", 101, scale=0.7)
    want, tol = _oracle(c, q, cu)
    assert_within(_run(c, q, cu, lists), want, tol, f"D={D} {lens}")


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 12, 2.0 ** 23, 2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27, 2.0 ** 28, 2.0 ** 33])
@pytest.mark.parametrize("length,D,G", [(37, 64, 2), (700, 128, 20), (3000, 256, 6)])
def test_equal_scores_of_any_size(lists, size, length, D, G):
    """Equal keys weigh equally, however large their score is: the output is the values' mean. A score's float may have
    steps of 16 and more, so that a reference 15 below it is not a float."""
    _case(f"equal scores lists={lists} size={size} length={length} D={D} G={G}")
    for factor in (1.0, 1.37, 1.9, -1.37):
        c = make_cache4([length], Hk=1, D=D, page=16, seed=120)
        for pos in range(length):
            _set_key(c, pos, 2)                              # 1.0
        q = np.full((1, G, D), factor, np.float16)
        got = _run(c, q, cu_of([1]), lists, scale=size / D)
        pos = np.arange(length)
        v = c["v"][c["table"][0, pos // 16], 0, pos % 16]
        want, A = (np.broadcast_to(x.mean(0), (1, G, D)) for x in (v, np.abs(v)))
        tol = A * (2.0 ** -18 + 2 * (length + 8) * 2.0 ** -24)
        assert_within(got, want, tol + half_step("e2m1", np.abs(want) + tol), f"size={size} factor={factor}")


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 22, 2.0 ** 26, 2.0 ** 29, 2.0 ** 33])
@pytest.mark.parametrize("length,D,G", [(90, 64, 4), (2000, 128, 20)])
def test_the_largest_of_far_scores(lists, size, length, D, G):
    """Keys of 1, 1.5 and 2 in turn, scores thousands apart: the mean over the positions of the largest, for each row."""
    _case(f"far scores lists={lists} size={size} length={length} D={D} G={G}")
    c = make_cache4([length], Hk=1, D=D, page=32, seed=121)
    code = np.random.default_rng(5).integers(2, 5, length)
    for pos in range(length):
        _set_key(c, pos, code[pos])
    q = np.ones((1, G, D), np.float16) * np.linspace(1.0, 1.9, G)[None, :, None].astype(np.float16)
    q[0, 1::2] *= -1
    got = _run(c, q, cu_of([1]), lists, scale=size / D)
    pos = np.arange(length)
    v = c["v"][c["table"][0, pos // 32], 0, pos % 32]
    for g in range(G):
        top = v[code == (2 if g % 2 else 4)]
        want, A = top.mean(0), np.abs(top).mean(0)
        tol = A * (2.0 ** -18 + 2 * (length + 8) * 2.0 ** -24)
        assert_within(got[0, g], want, tol + half_step("e2m1", np.abs(want) + tol), f"size={size} row {g}")


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("length,new", [(1, 1), (50, 1), (50, 4), (700, 3), (6000, 2)])
def test_a_row_without_a_finite_score_is_zero_and_alone(lists, length, new):
    """Scores that are all -inf give zeros, whatever the values; other rows of the same tile are as without it, and a NaN
    in q is its row's."""
    _case(f"scores of -inf lists={lists} length={length} new={new}")
    D, G = 64, 4
    c = make_cache4([length], Hk=1, D=D, page=16, seed=140)
    pos = np.arange(length)
    page, slot = c["table"][0, pos // 16], pos % 16
    byte = c["k_codes"][page, 0, slot, 1]
    c["k_codes"][page, 0, slot, 1] = (byte & 15) | 0xf0      # channel 3 below zero, at its block's scale
    c["k_scales"][page, 0, 0, slot] = np.maximum(c["k_scales"][page, 0, 0, slot], 110)
    cu, q = cu_of([new]), queries(new, G, D, "f16", 141)
    clean = _run(c, q, cu, lists)
    q[:, 1, 3], q[:, 2, 7] = np.inf, np.nan
    got = _run(c, q, cu, lists)
    assert (got[:, 1] == 0).all() and np.isnan(got[:, 2]).all()
    assert np.array_equal(got[:, [0, 3]], clean[:, [0, 3]])
    c["v_scales"][page[0], 0, 1, slot[0]] = 255
    assert (_run(c, q, cu, lists)[:, 1] == 0).all()
