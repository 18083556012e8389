"""CPU test of the Muon step's workspace: the sizes that the documents state."""

import ctypes

import pytest

pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import _lib  # noqa: E402


@pytest.mark.parametrize("shapes,gigabytes", [
    ([(4096, 11008)], 1.01), ([(32000, 4096)], 2.04), ([(2048, 2048)] * 4 + [(8192, 2048), (2048, 8192)], 1.24),
    (([(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]) * 32, 3.17)])
def test_stated_sizes(shapes, gigabytes):
    arr = (_lib.qopt_muon_tensor * len(shapes))(*[(0, 0, 0, 0, *s) for s in shapes])
    need = ctypes.c_size_t(0)
    assert _lib.LIB.qopt_muon_workspace(arr, len(arr), ctypes.byref(need)) == 0
    assert round(need.value / 1e9, 2) == gigabytes
    # 12 bytes per element, 20 per value of m x m, and at most 2 x 256 tiles of 256 x 256 partial sums
    own = [12 * r * c + 20 * min(r, c) ** 2 for r, c in shapes]
    assert min(own) <= need.value <= sum(sorted(own)[-16:]) * 1.01 + (1 << 27)
