"""GPU: more tokens than a launch has work-items in one dimension for (2^24 workgroups of 256)."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import assert_within
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


def test_rotation_of_2_to_the_28_tokens():
    """One head of 64, in place: 34 GB. A few tokens hold values, the rest zeros, which any angle leaves."""
    N, D, rot = (1 << 28) + 5, 64, 64
    at = [0, 1, 15, 16, (1 << 27) - 1, (1 << 28) - 1, 1 << 28, N - 2, N - 1]
    x = np.random.default_rng(180).standard_normal((len(at), 1, D)).astype(np.float16)
    q = torch.zeros((N, 1, D), dtype=torch.float16, device="cuda")
    q[torch.tensor(at, device="cuda")] = dev(x, torch)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    f = AO.frequencies(rot, 1e6)
    print("[gpu case] in place", flush=True)
    gdn.gdn_rope_forward(q, None, pos, dev(f, torch), q, None)
    torch.cuda.synchronize()
    got = q[torch.tensor(at, device="cuda")].double().cpu().numpy()
    want = AO.rope(x, np.array(at), f)
    pair = np.abs(x[..., :32].astype(np.float64)) + np.abs(x[..., 32:])
    tol = np.concatenate([pair, pair], -1) * (2.5 * 2.0 ** -24 + 2.0 ** -23)     # the oracle's angle: 2^28 2^-52
    assert_within(got, want, tol + np.maximum(np.abs(want) * 2.0 ** -11, 2.0 ** -25), "rows")
    others = torch.ones(N, dtype=torch.bool, device="cuda")
    others[torch.tensor(at, device="cuda")] = False
    for i in range(0, N, 1 << 25):
        assert not bool((q[i:i + (1 << 25)].view(-1, D).any(1) & others[i:i + (1 << 25)]).any())
