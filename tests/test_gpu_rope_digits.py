"""GPU: how exactly gdn_rope_forward rotates, at any int32 position.

cos and sin times the factor are off by half a float's step at most (2^-25 up to 1) and by
2^-40 of themselves, the angle being reduced without rounding; the rotation of FP32 rows adds
two products and a sum: (2^-25 + 2^-24 + 2^-24) (|x| + |y|) factor.
"""
from __future__ import annotations

import math
from decimal import Decimal, localcontext

import numpy as np
import pytest

from attn_helpers import assert_within
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gateddeltanet_recurrence_amd as gdn          # noqa: E402
from oracle import attn_oracle as AO                 # noqa: E402

PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def _exact_turns(positions, inv_freq):
    """cos and sin [N, r / 2] of position * frequency, the angle reduced to an eighth of a turn with 80 digits."""
    c, s = (np.empty((len(positions), len(inv_freq))) for _ in range(2))
    with localcontext() as ctx:
        ctx.prec = 80
        quarter = Decimal(PI) / 2
        for i, p in enumerate(positions):
            for j, f in enumerate(inv_freq):
                t = Decimal(int(p)) * Decimal(float(f))
                n = (t / quarter).to_integral_value()
                y = float(t - n * quarter)
                a, b = math.cos(y), math.sin(y)
                c[i, j], s[i, j] = ((a, b), (-b, a), (-a, -b), (b, -a))[int(n) % 4]
    return c, s


def _positions():
    rng = np.random.default_rng(150)
    ends = [2 ** 31 - 1, -2 ** 31, 0, 1, -1, 2 ** 24 + 1, 355, 103993, 1146408 // 2]
    return np.array(ends + [int(x) for e in (8, 16, 20, 24, 28, 31) for x in rng.integers(-2 ** e, 2 ** e, 6)], np.int64).astype(np.int32)


@pytest.mark.parametrize("factor", [1.0, 1.25])
@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
def test_turns_are_rounded_once_at_any_position(factor, layout):
    """Unit vectors come back as cos and sin themselves."""
    pos, rot = _positions(), 64
    f = gdn.gdn_rope_frequencies(rot, base=1e6)[0].copy()
    f[1], f[2], f[3] = 1.0, 0.5, math.pi                  # whole radians, and close to half turns
    c, s = _exact_turns(pos, f)
    x = np.zeros((len(pos), 1, 64), np.float32)
    first, second = (np.arange(0, 64, 2), np.arange(1, 64, 2)) if layout == AO.INTERLEAVED else (np.arange(32), np.arange(32, 64))
    x[..., first] = 1.0
    out = torch.empty(x.shape, device="cuda")
    gdn.gdn_rope_forward(dev(x, torch), None, dev(pos, torch), dev(f, torch), out, None, rope_layout=layout,
                         rope_factor=factor)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()[:, 0]
    for name, g, want in (("cos", got[:, first], factor * c), ("sin", got[:, second], factor * s)):
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 24)
        assert_within(g, want, step + np.abs(want) * 2.0 ** -40 + 2.0 ** -75, name)


@pytest.mark.parametrize("layout", [AO.HALF, AO.INTERLEAVED])
@pytest.mark.parametrize("D,rot", [(64, 48), (128, 128), (256, 64)])
def test_rotation_of_fp32_rows(layout, D, rot):
    rng = np.random.default_rng(151)
    N, H = 300, 2
    q = rng.standard_normal((N, H, D)).astype(np.float32)
    pos = rng.integers(-2 ** 17, 2 ** 17, N).astype(np.int32)     # the oracle's angles are then good to 2^-35
    f = AO.frequencies(rot, 1e6)
    out = torch.empty((N, H, D), device="cuda")
    gdn.gdn_rope_forward(dev(q, torch), None, dev(pos, torch), dev(f, torch), out, None, rope_layout=layout,
                         rope_factor=1.25)
    torch.cuda.synchronize()
    want = AO.rope(q, pos, f, layout, 1.25)
    pair = np.zeros(q.shape)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if layout == AO.INTERLEAVED else (i, i + rot // 2)
    pair[..., a] = pair[..., b] = np.abs(q[..., a].astype(np.float64)) + np.abs(q[..., b])
    # half a step of the factor's own float range: 1.25 cos t may lie above 1
    assert_within(out.double().cpu().numpy(), want, (2.0 ** -24 * 2.5 * 1.25 + 2.0 ** -34) * pair, "rows")
