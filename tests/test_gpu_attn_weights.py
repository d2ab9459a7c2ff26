"""GPU: how exactly the attention's softmax weights enter the output (gdn_attn_forward).

With FP16 I/O a weight w takes part in the product with v as two fp16 values whose sum is
(1 + 2^-11) w to 2^-19 of it, or to 2^-38 of the row's largest: hi is rounded toward zero (off
by less than 2^-10 w), lo holds what hi lost and 2^-11 hi, at most 1.5 * 2^-10 w, rounded toward
zero to 2^-10 of that, and 2^-11 of what hi lost is missing (2^-21 w); below fp16's range steps
are 2^-24, twice, of weights up to 2^15. The tolerances are this, the FP32 terms of
oracle.attn_oracle.attention (no rounded weights) and 2^-18 for the FP32 exponent's own
arithmetic; then half a step of the I/O type, taken at the value itself. A weight rounded once
to fp16 fails them.
"""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within, make_cache, run_attention

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


def _half_step(x):
    """Half a step of fp16 at |x|."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -14)))
    return 2.0 ** (e - 11)


def _oracle(c, q, cu, scale=None):
    """(out, tolerance) as the module's text has it, for FP16 I/O."""
    out, bound = AO.attention(q, c["k"], c["v"], c["table"], cu, c["lens"], scale=scale, rounded_weights=False)
    _, low = AO.attention(q, c["k"], c["v"], c["table"], cu, c["lens"], scale=scale,
                          v_codes=c.get("v_codes"), v_scales=c.get("v_scales"))
    # that bound's terms beyond `bound` are 2^-11 sum p |v| and 2^-25 of the largest weight for every |v|
    _, mass = AO.attention(q, c["k"], np.abs(np.asarray(c["v"], np.float64)), c["table"], cu, c["lens"], scale=scale,
                           rounded_weights=False)
    A = AO.attention(q, c["k"], np.abs(np.asarray(c["v"], np.float64)), c["table"], cu, c["lens"], scale=scale,
                     rounded_weights=False)[0]
    assert np.array_equal(mass, bound)
    floor = np.maximum(low - bound - 2.0 ** -11 * A, 0.0) * 2.0 ** -13
    tol = bound + (2.0 ** -19 + 2.0 ** -18) * A + floor
    return out, tol + _half_step(np.abs(out) + tol)


def _place(c, r, pos):
    return c["table"][r, pos // c["page"]], pos % c["page"]


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,new,G", [([2, 3, 5], [1, 1, 1], 4), ([40, 300], [4, 5], 4), ([700, 90], [2, 1], 24), ([3000], [8], 8)])
def test_weights_keep_their_digits(fmt, D, lens, new, G):
    _case(f"{fmt} D={D} lens={lens} new={new} G={G}")
    c = make_cache(lens, Hk=2, D=D, fmt=fmt, page=16, seed=100 + D, wide=False)
    cu = _cu(new)
    q = np.random.default_rng(101).standard_normal((cu[-1], 2 * G, D)).astype(np.float16)
    want, tol = _oracle(c, q, cu)
    assert_within(run_attention(c, q, cu, torch, gdn), want, tol, fmt)


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("length", [600, 16384])
@pytest.mark.parametrize("gap", [8.0, 12.0, 17.5, 21.0])
def test_a_dominating_key_leaves_the_rest_its_digits(fmt, length, gap):
    """One key `gap` above the others whose value is small or zero: what the row gives comes from a long flat
    tail of weights e^-gap of the largest."""
    D = 64
    for place in (0, length // 2, length - 1):
        _case(f"{fmt} length={length} gap={gap} place={place}")
        c = make_cache([length], Hk=1, D=D, fmt=fmt, page=64, seed=110, wide=False)
        rng = np.random.default_rng(111)
        rows = np.zeros((1, length, 1, D))
        rows[..., 1:] = rng.standard_normal((1, length, 1, D - 1)) * 0.125
        rows[0, place, 0] = 0
        rows[0, place, 0, 0] = gap
        values = rng.standard_normal((length, 1, D)) + 1.0
        values[place, 0] = 0
        values[place, 0, 5] = 1.0                        # an 8-bit row has the others' scale
        full = np.array([0, length])
        for name, x in (("k", rows[0]), ("v", values)):
            x = x.astype(np.float16)
            if fmt == "e4m3":
                codes, s = AO.quantise(x)
                c[name + "_codes"] = AO.cache_write(codes, c[name + "_codes"], c["table"], full, [length])
                c[name + "_scales"] = AO.cache_write(s, c[name + "_scales"], c["table"], full, [length])
                c[name] = AO.dequantise(c[name + "_codes"], c[name + "_scales"])
            else:
                c[name] = AO.cache_write(x, c[name], c["table"], full, [length])
        q = np.zeros((1, 2, D), np.float16)
        q[..., 0], q[..., 1:] = 1.0, rng.standard_normal((1, 2, D - 1)) * 0.125
        want, tol = _oracle(c, q, _cu([1]), scale=1.0)
        got = run_attention(c, q, _cu([1]), torch, gdn, scale=1.0)
        assert_within(got, want, tol, f"{fmt} {place}")


@pytest.mark.parametrize("fmt", ["f16", "f32", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 12, 2.0 ** 23, 2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27, 2.0 ** 28, 2.0 ** 33])
def test_equal_scores_of_any_size(fmt, size):
    """Equal keys weigh equally, however large their score is: the output is the values' mean. A score's float
    may have steps of 16 and more, so that a reference 15 below it is not a float."""
    D, length = 64, 37
    for factor in (1.0, 1.37, 1.9, -1.37):
        c = make_cache([length], Hk=1, D=D, fmt=fmt, page=16, seed=120, wide=False)
        pg = [_place(c, 0, pos) for pos in range(length)]
        for p, s in pg:
            if fmt == "e4m3":
                c["k_codes"][p, :, s], c["k_scales"][p, :, s] = 0x38, 127                     # 1.0
            c["k"][p, :, s] = 1.0
        q = np.full((1, 2, D), factor, np.float16 if fmt != "f32" else np.float32)
        got = run_attention(c, q, _cu([1]), torch, gdn, scale=size / D)
        v = np.stack([c["v"][p, 0, s] for p, s in pg]).astype(np.float64)
        want = np.broadcast_to(v.mean(0), (1, 2, D))
        A = np.broadcast_to(np.abs(v).mean(0), (1, 2, D))
        tol = A * (2.0 ** -18 + 2 * (length + 8) * 2.0 ** -24)
        if fmt == "e4m3":
            # the exponent is the score times log2(e) plus the value's scale's, rounded to a float: off by
            # |x| 2^-24 in each weight, a factor e^d with d = ln 2 |x| 2^-24, and as much in their sum. Far
            # scores leave their weights no digits.
            x = size * abs(factor) * 1.4427 + 40
            tol = tol + A * np.expm1(min(2 * np.log(2) * x * 2.0 ** -24, 700.0))
        tol = tol + (_half_step(np.abs(want) + tol) if fmt != "f32" else np.abs(want) * 2.0 ** -24)
        assert_within(got, want, tol, f"{fmt} {size} {factor}")
