"""The selection's threshold search on the host: csrc/gdn_pick.h, which the kernels of gdn_attn_select run, compiled
here with the counting that a list's waves do, against a sort of the same scores.

Two ways a cut is what one wave does, four ways what several do. Whatever the scores, K entries are
taken: those always in, then NaN, then the highest, equal ones from the lowest entry on.
"""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gateddeltanet_recurrence_amd", "csrc")
COMPILER = shutil.which("g++") or shutil.which("clang++")

pytestmark = pytest.mark.skipif(COMPILER is None, reason="no C++ compiler")

DRIVER = r"""
#include <stddef.h>
#include <vector>
#include "gdn_pick.h"
using namespace gdn;

// The entries that a list takes, ascending, up to `room` of them, and how many there would be.
template <int WAYS> static int pick(const std::vector<uint64_t>& keys, int K, int32_t* list, int room) {
  uint64_t lo = kAlways, hi = 0;
  int there = 0, always = 0;
  for (uint64_t key : keys) {
    there += key != 0;
    always += key == kAlways;
    if (key != kAlways && key > hi) hi = key;
    if (key != 0 && key < lo) lo = key;
  }
  Cut cut{1, 0};
  if (there > K && always == K) {
    cut.least = kAlways;
  } else if (there > K) {
    ShortKeys shorts{0, 0};
    const auto from = [&](auto of, auto x) {
      int n = 0;
      for (uint64_t key : keys) n += of(key) >= x;
      return n;
    };
    const auto prepare = [&](ShortKeys x) { shorts = x; };
    const auto shorter = [&](uint32_t x, uint32_t y, uint32_t z) {
      const auto of = [&](uint64_t key) { return shorts.of(key); };
      return Three{from(of, x), from(of, y), from(of, z)};
    };
    const auto whole = [&](uint64_t x, uint64_t y, uint64_t z) {
      const auto of = [](uint64_t key) { return key; };
      return Three{from(of, x), from(of, y), from(of, z)};
    };
    cut = find_cut<WAYS>(K, there, lo, hi, prepare, shorter, whole);
  }
  int kept = 0, n = 0;                                     // ties: all but the last `surplus` of them
  for (uint64_t key : keys) kept += key == cut.least;
  kept -= cut.surplus;
  for (size_t i = 0; i < keys.size(); ++i) {
    bool in = keys[i] >= cut.least;
    if (cut.surplus > 0 && keys[i] == cut.least) in = kept-- > 0;
    if (!in) continue;
    if (n < room) list[n] = (int32_t)i;
    ++n;
  }
  return n;
}

extern "C" int pick_scores(const double* scores, const int32_t* kind, int n, int K, int ways, int32_t* list, int room) {
  std::vector<uint64_t> keys(n);
  for (int i = 0; i < n; ++i) keys[i] = kind[i] < 0 ? 0 : kind[i] > 0 ? kAlways : key_of(scores[i]);
  return ways == 2 ? pick<2>(keys, K, list, room) : pick<4>(keys, K, list, room);
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    at = tmp_path_factory.mktemp("pick")
    (at / "pick.cpp").write_text(DRIVER)
    out = at / "pick.so"
    subprocess.run([COMPILER, "-std=c++17", "-O2", "-Wall", "-shared", "-fPIC", "-I", CSRC, str(at / "pick.cpp"), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def _check(library, scores, kind, K, what):
    scores, kind = np.ascontiguousarray(scores, np.float64), np.ascontiguousarray(kind, np.int32)
    there = np.flatnonzero(kind >= 0)
    s = scores[there]
    rank = np.where(np.isnan(s), 0.0, s)
    order = np.lexsort((there, -rank, ~np.isnan(s) & (kind[there] == 0), kind[there] == 0))
    want = np.sort(there[order[:K]])
    for ways in (2, 4):
        got = np.full(len(scores) + 1, -77, np.int32)
        n = library.pick_scores(scores.ctypes.data_as(ctypes.c_void_p), kind.ctypes.data_as(ctypes.c_void_p), len(scores), K, ways,
                                got.ctypes.data_as(ctypes.c_void_p), len(got))
        assert n == len(want), f"{what}, {ways} ways: {n} entries instead of {len(want)}"
        assert (got[:n] == want).all(), f"{what}, {ways} ways"


def _scores(rng, n, how):
    x = rng.standard_normal(n)
    return {"both signs": x * 7.3, "positive": np.abs(x) + 12.3, "negative": -np.abs(x) - 7.77, "round": np.round(x * 4) / 4,
            "wide": x * 10.0 ** rng.integers(-300, 300, n), "equal": np.full(n, 1.0 / 3)}[how]


HOW = ["both signs", "positive", "negative", "round", "wide", "equal"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("n,K", [(40, 8), (256, 8), (1024, 8), (700, 33), (9, 1)])
@pytest.mark.parametrize("first,newest", [(0, 0), (1, 0), (0, 1), (1, 2), (3, 5)])
def test_any_number_of_nan_scores_beside_finite_ones(library, how, n, K, first, newest):
    if first + newest > K:
        first, newest = 1, 0
    rng = np.random.default_rng(n + K)
    for broken in {0, 1, K - 1, K, K + 1, 2 * K, n // 2, n - 9, n - 1, n}:
        if not 0 <= broken <= n:
            continue
        for where in ("anywhere", "late"):
            scores, kind = _scores(rng, n, how), np.zeros(n, np.int32)
            scores[rng.permutation(n)[:broken] if where == "anywhere" else np.arange(n - broken, n)] = np.nan
            kind[:first], kind[n - newest:] = 1, 1
            _check(library, scores, kind, K, f"{how} n={n} K={K} {broken} NaN {where}, {first} first, {newest} newest")


@pytest.mark.parametrize("how", HOW)
def test_infinities_and_entries_without_a_page(library, how):
    rng = np.random.default_rng(7)
    for n, K in ((30, 4), (300, 20), (1500, 130)):
        for step in range(40):
            scores = _scores(rng, n, how)
            for value in (np.inf, -np.inf, np.nan, 0.0, np.finfo(np.float64).max, 5e-324):
                scores[rng.permutation(n)[:rng.integers(0, 2 * K)]] = value
            kind = np.where(rng.random(n) < 0.2, -1, 0)
            kind[rng.permutation(n)[:rng.integers(0, K + 1)]] = 1
            _check(library, scores, kind, K, f"{how} n={n} K={K} step {step}")


def test_keys_that_differ_in_their_last_bits(library):
    """The short keys do not tell them apart."""
    rng = np.random.default_rng(3)
    for n, K in ((64, 5), (600, 40)):
        near = (np.float64(1.0).view(np.uint64) + rng.integers(0, n // 2, n).astype(np.uint64)).view(np.float64)
        for far in (-1e9, 1e9, np.inf, np.nan):
            for some in (0, 1, K - 1, K, K + 1):
                scores = near.copy()
                scores[rng.permutation(n)[:some]] = far
                _check(library, scores, np.zeros(n, np.int32), K, f"near n={n} K={K} {some} of {far}")
