"""Host-side checks that the Python binding makes before the attention layer's C calls: no GPU, no
library call."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")
from gateddeltanet_recurrence_amd import binding          # noqa: E402


def _strided(N=6, H=2, D=64, gap=128):
    """q as a slice of a projection's output, and dense rows that begin at the same address."""
    wide = torch.zeros(N, H * D + gap)
    return wide[:, :H * D].view(N, H, D), wide.flatten()[:N * H * D].view(N, H, D)


def test_an_output_at_its_inputs_address_has_its_strides():
    """Equal addresses mean in place, with the input's stride: dense rows there would not be what is written."""
    q, dense = _strided()
    assert q.data_ptr() == dense.data_ptr() and not q.is_contiguous() and dense.is_contiguous()
    with pytest.raises(ValueError, match="q_out"):
        binding._out_rows(dense, q, "q_out")
    with pytest.raises(ValueError, match="q_out"):
        binding._out_rows(q, dense, "q_out")
    square = torch.zeros(3, 64, 64)
    with pytest.raises(ValueError, match="q_out"):
        binding._out_rows(square.transpose(1, 2), square, "q_out")


def test_outputs_that_are_taken():
    q, dense = _strided()
    binding._out_rows(q, q, "q_out")
    binding._out_rows(q.view(q.shape), q, "q_out")              # the same rows as another tensor
    binding._out_rows(dense.view(dense.shape), dense, "q_out")
    binding._out_rows(torch.zeros(q.shape), q, "q_out")
    one, dense_one = _strided(N=1)
    binding._out_rows(dense_one, one, "q_out")                  # one token has no stride
    q0, _ = _strided(N=0)
    binding._out_rows(torch.zeros(q0.shape), q0, "q_out")


@pytest.mark.parametrize("bad", [lambda q: None, lambda q: torch.zeros(q.shape[0] + 1, *q.shape[1:]),
                                 lambda q: torch.zeros(q.shape, dtype=torch.float16), lambda q: _strided()[0]])
def test_outputs_that_are_refused(bad):
    q = torch.zeros(6, 2, 64)
    with pytest.raises(ValueError):
        binding._out_rows(bad(q), q, "q_out")


class _Function:
    def __init__(self, value):
        self.value = value

    def __call__(self):
        return self.value


class _Older:
    """A library with the version's number and a few of its functions."""

    def __init__(self, version, names):
        self.gdn_abi_version = _Function(version)
        for n in names:
            setattr(self, n, _Function(0))


@pytest.mark.parametrize("version,names", [
    (binding.ABI_VERSION, ["gdn_forward"]),                     # this number, without the newer functions
    (binding.ABI_VERSION - 1, []), (binding.ABI_VERSION + 1, []),
])
def test_a_library_of_another_build_says_rebuild(monkeypatch, tmp_path, version, names):
    path = tmp_path / "libgdn.so"
    path.write_bytes(b"")
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(binding, "library_path", lambda: str(path))
    monkeypatch.setattr(ctypes, "CDLL", lambda p: _Older(version, names))
    for call in (binding.lib, binding.gdn_abi_version, lambda: binding._call("gdn_kv_write")):
        with pytest.raises(binding.LibraryNotBuilt, match="rebuild it"):
            call()
    assert binding._lib is None and binding._calls is None


def test_a_library_without_a_version_says_rebuild(monkeypatch, tmp_path):
    path = tmp_path / "libgdn.so"
    path.write_bytes(b"")
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "library_path", lambda: str(path))
    monkeypatch.setattr(ctypes, "CDLL", lambda p: object())
    with pytest.raises(binding.LibraryNotBuilt, match="rebuild it"):
        binding.lib()


def test_int32_mirrors_are_read_in_place():
    """A mirror that the program changes later is the one that the next call's checks see."""
    import numpy as np
    a = np.arange(12, dtype=np.int32).reshape(3, 4)
    kept, at = binding._host_i32(a)
    assert at == a.ctypes.data and np.shares_memory(kept, a)
    t = torch.arange(12, dtype=torch.int32).view(3, 4)
    kept, at = binding._host_i32(t)
    assert at == t.data_ptr()
    t[1, 2] = 77
    assert kept[1, 2] == 77
    for copied in (a.astype(np.int64), a[:, :2], [[1, 2], [3, 4]]):
        kept, at = binding._host_i32(copied)
        assert kept.dtype == np.int32 and at == kept.ctypes.data and np.array_equal(kept, copied)
