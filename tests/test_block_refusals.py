"""Arguments of the binding's block operators that are refused before the library or a device is reached (CPU only)."""

import pytest
import torch

import packed_variable_length_gb300 as pvl


@pytest.fixture
def closed(monkeypatch):
    """No call of the library gets through."""
    def load():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(pvl.api._lib, "load", load)


def test_devices_that_are_not_cuda_are_refused(closed):
    for kw in (dict(device="cpu"), dict(device=torch.device("cpu")), dict(device="meta"),
               dict(out=torch.zeros(1, 4, 1, dtype=torch.int32)), dict(device="cpu", stream=0)):
        with pytest.raises(ValueError):
            pvl.pack_build_positions([[1]], 4, 4, **kw)
