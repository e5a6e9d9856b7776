"""Arguments of the binding's block operators that are refused before the library or a device is reached (CPU only)."""

import dataclasses

import numpy as np
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


def test_three_axes_need_a_row_width(closed):
    """Refused for the row width, not for the device that comes after it; two axes do without."""
    for width in (None, 0, -1):
        with pytest.raises(ValueError, match="row_width"):
            pvl.pack_build_positions([[1]], 4, 4, axes=3, row_width=width, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        pvl.pack_build_positions([[1]], 4, 4, axes=2, row_width=0, device="cpu")


@pytest.mark.parametrize("kind", [int, float, np.int64, np.float32, np.float64])
def test_plan_arguments_of_any_kind_of_number(kind):
    ref = pvl.rotary_plan(64, base=10000.0, scaling="parts", factor=4.0, length=4096, slow=1.0, fast=32.0, device="cpu")
    got = pvl.rotary_plan(64, base=kind(10000), scaling="parts", factor=kind(4), length=kind(4096), slow=kind(1),
                          fast=kind(32), device="cpu")
    assert torch.equal(got.turns, ref.turns) and got.gain == ref.gain


def test_plan_numbers_that_are_not_finite():
    for kw in (dict(length=float("inf")), dict(length=float("nan")), dict(length=0.5), dict(fast=float("inf")),
               dict(slow=float("nan")), dict(factor=float("nan")), dict(base=float("nan"))):
        with pytest.raises(ValueError):
            pvl.rotary_plan(64, **{**dict(scaling="parts", factor=4.0, length=4096, device="cpu"), **kw})


def test_plans_that_do_not_hold_what_they_say(closed):
    """A plan made by hand whose table is shorter than its rotary_dim, of another type or not contiguous, or whose
    layout is unknown: the kernel would read past it or take another layout."""
    q, pos = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32)
    plan = pvl.rotary_plan(64, device="cpu")
    for change in (dict(turns=plan.turns[:16]), dict(turns=plan.turns.int()), dict(turns=plan.turns.double()),
                   dict(turns=plan.turns.repeat_interleave(2)[::2]), dict(turns=plan.turns[None]), dict(rotary_dim=128)):
        bad = dataclasses.replace(plan, **change)
        for call in (pvl.pack_rotary_fwd, pvl.pack_rotary_bwd):
            with pytest.raises(ValueError, match="turns"):
                call(q, q, pos, bad)
    with pytest.raises(ValueError, match="layout"):
        pvl.pack_rotary_fwd(q, q, pos, dataclasses.replace(plan, layout="other"))
    with pytest.raises(ValueError, match="CUDA"):
        pvl.pack_rotary_fwd(q, q, pos, plan)
