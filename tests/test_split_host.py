"""Host: very many requests in a call: the attention's split of their lengths into units of work, and what
gdn_kv_bounds takes.

No call here launches a kernel (there is no GPU to launch it on), and the module runs only where none is visible.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest

import gateddeltanet_recurrence_amd as gdn


def _gpu_visible() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:
        return False


pytestmark = [
    pytest.mark.skipif(not os.path.exists(gdn.library_path()), reason="libgdn.so not built (run the build first)"),
    pytest.mark.skipif(_gpu_visible(), reason="fake-pointer host checks run only without a GPU"),
]

CALL = """
import ctypes, sys
import numpy as np
import gateddeltanet_recurrence_amd as gdn
R, pages = (1 << 29) + 1, 100
lens = np.zeros(R, np.int32)                     # three long requests, the others without a position
lens[:3] = pages * 1024
at = [(i + 1) << 42 for i in range(10)]          # disjoint, never dereferenced
cache = gdn.GdnKvCache(at[0], at[1], at[2], at[3], at[4], None, 1000, 1024, pages, 1, 64, gdn.GDN_F16, gdn.CACHE_E2M1)
params = gdn.GdnAttnParams(1, R, 1, 0.0, 0, 0)
tensors = gdn.GdnAttnTensors(at[5], at[6], None, at[7], lens.ctypes.data, at[8])
print(gdn.lib().gdn_attn_forward(ctypes.byref(params), ctypes.byref(tensors), ctypes.byref(cache), at[9], 1 << 40, None))
"""


def test_more_segments_than_units_can_count_twice():
    """(N + R) Hq D / 64 is within 2^30, but a segment's fixed part would not fit beside its own unit: the call ends, here
    for want of a device."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CALL], cwd=root, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout.split()[-1]) == gdn.GDN_ERR_HIP


@pytest.mark.parametrize("R,status", [((1 << 31) - 1, gdn.GDN_ERR_SHAPE), ((1 << 31) - 63, gdn.GDN_ERR_SHAPE), ((1 << 31) - 64, gdn.GDN_ERR_HIP)])
def test_as_many_requests_as_bounds_can_count(R, status):
    """Past 2^31 - 64 the requests of a lane would pass 32 bits (and no page's bounds be written); below, the call ends here
    for want of a device."""
    at = [(i + 1) << 42 for i in range(7)]
    cache = gdn.GdnKvCache(at[0], at[1], None, None, at[2], None, 1000, 16, 1, 1, 64, gdn.GDN_F16, gdn.CACHE_IO)
    params = gdn.GdnKvParams(1, R, 0, 0, 0, 0.0, 0, 0, 0)
    tensors = gdn.GdnKvTensors(None, None, at[3], None, at[4], None, None, None, None, None)
    assert gdn.lib().gdn_kv_bounds(ctypes.byref(params), ctypes.byref(tensors), ctypes.byref(cache), at[5], None) == status
