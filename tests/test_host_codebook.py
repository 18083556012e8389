"""CPU test of the codebook cache's argument checks."""

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import functional  # noqa: E402


def test_a_cached_codebook_is_only_given_for_its_gpu(monkeypatch):
    """Another device of the same index is refused as it is while nothing is cached."""
    kept = torch.zeros(1)  # stands for the copy on GPU 0
    for cache in ({}, {(functional.SIGNED, 0): kept}):
        monkeypatch.setattr(functional, "_cb_cache", cache)
        for device in (torch.device("cpu", 0), torch.device("cpu"), "cpu", torch.device("meta", 0)):
            with pytest.raises(ValueError):
                functional.codebook(functional.SIGNED, device)
    assert functional.codebook(functional.SIGNED, torch.device("cuda", 0)) is kept
