"""GPU: infinite and NaN values that the attention (gdn_attn_forward) reads at attended positions."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import make_cache, run_attention

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _case(msg):
    print(f"[gpu case] {msg}", flush=True)


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def _place(c, r, pos):
    return c["table"][r, pos // c["page"]], pos % c["page"]


@pytest.mark.parametrize("fmt", ["f16", "f32"])
@pytest.mark.parametrize("length,new", [(1, 1), (2, 1), (33, 3), (700, 4), (5000, 1), (40000, 1), (9000, 12)])
def test_an_infinite_value_that_is_attended_is_infinite(fmt, length, new):
    """Whatever the weight's digits are (alone: weight 1; beside equal ones), in a draft's own position, and
    however many workgroups share the length."""
    D, G = 64, 4
    for sign in (1.0, -1.0):
        c = make_cache([length], Hk=1, D=D, fmt=fmt, page=16, seed=130, wide=False)
        for pos in {0, length - 1, length // 2}:
            _case(f"{fmt} length={length} new={new} pos={pos} {sign}")
            d = {**c, "v": c["v"].copy()}
            p, s = _place(c, 0, pos)
            d["v"][p, 0, s, 9] = sign * np.inf
            for q in (np.zeros((new, G, D)), np.random.default_rng(131).standard_normal((new, G, D))):
                q = q.astype(c["k"].dtype)
                got = run_attention(d, q, _cu([new]), torch, gdn)
                sees = np.arange(new) >= new - (length - pos)
                assert np.all(got[sees][..., 9] == sign * np.inf), (pos, got[..., 9])
                assert np.all(np.isfinite(got[~sees])) and np.all(np.isfinite(np.delete(got, 9, -1)))


@pytest.mark.parametrize("fmt", ["f16", "f32"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("length,new", [(1, 1), (50, 1), (50, 4), (700, 3), (6000, 2)])
def test_a_row_without_a_finite_score_is_zero_whatever_its_values(fmt, value, length, new):
    """Scores that are all -inf give zeros."""
    D, G = 64, 4
    c = make_cache([length], Hk=1, D=D, fmt=fmt, page=16, seed=140, wide=False)
    for p, s in (_place(c, 0, pos) for pos in range(length)):
        c["k"][p, 0, s, 3] = -np.inf
    p, s = _place(c, 0, 0)
    c["v"][p, 0, s, 9] = value
    q = np.random.default_rng(141).standard_normal((new, G, D)).astype(c["k"].dtype)
    q[:, :, 3] = 1.0
    for mirrors in (True, False):
        _case(f"{fmt} {value} length={length} new={new} mirrors={mirrors}")
        got = run_attention(c, q, _cu([new]), torch, gdn, mirrors=mirrors)
        assert np.all(got == 0)
