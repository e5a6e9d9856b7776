"""Rotary positions of values that are not finite, against the fp64 oracle (GPU)."""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_rotary import f64, freqs_of, make, pvl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [20, 700])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(128, 96), (128, 90), (128, 2), (72, 40), (20, 6), (54, 30), (256, 250)])
def test_features_past_the_rotated_part_keep_their_bits(pvl, D, R, layout, L):  # noqa: F811
    """Without a norm they pass through, an infinity, a NaN and a zero's sign among them, and touch no neighbour:
    forward, and the gradient's backward.  A NaN stays one, of whatever bits: the conversion to bf16 has one NaN."""
    q, k, *_, pos, sections = make(1, L, 3, 2, D, R, 1, layout, None, D + R)
    plan = pvl.rotary_plan(R, layout=layout, gain=1.25)
    clean = pvl.pack_rotary_fwd(q, k, pos, plan)
    rng = np.random.default_rng(R)
    for n, v in enumerate((float("inf"), -float("inf"), float("nan"), -0.0)):
        for x in (q, k):
            for _ in range(3):
                x[0, int(rng.integers(L)), int(rng.integers(x.shape[2])), int(rng.integers(R, D))] = v
    for call in (pvl.pack_rotary_fwd, pvl.pack_rotary_bwd):
        for x, got in zip((q, k), call(q, k, pos, plan)[:2]):
            a, b = got[..., R:], x[..., R:]
            assert torch.equal(a.isnan(), b.isnan())
            bits = [torch.where(t.isnan(), 0.0, t).view(torch.int16) for t in (a, b)]
            assert torch.equal(*bits)
            assert bool(got[..., :R].isfinite().all())
    for a, b in zip(clean, pvl.pack_rotary_fwd(q, k, pos, plan)):
        assert torch.equal(a[..., :R], b[..., :R])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", ["head", "token"])
@pytest.mark.parametrize("D,R", [(128, 96), (72, 40), (54, 30)])
def test_an_infinity_under_a_norm(pvl, D, R, norm, layout):  # noqa: F811
    """1 / rms is then 0: NaN for the infinity itself and, where it is turned, its pair; zeros for what it is normed
    with; forward as the oracle has it."""
    q, k, _, _, wq, wk, pos, sections = make(1, 30, 3, 2, D, R, 1, layout, norm, D)
    plan = pvl.rotary_plan(R, layout=layout)
    for f in (D - 1, R, 1):
        x = q.clone()
        x[0, 11, 1, f] = float("inf")
        got, _ = pvl.pack_rotary_fwd(x, k, pos, plan, norm, wq, wk)
        with np.errstate(invalid="ignore"):
            ref = oracle.rotary_fwd(x, pos.cpu().numpy(), freqs_of((R // 2,)), (R // 2,), layout, 1.0, norm, wq)
        got = f64(got)
        assert np.array_equal(np.isnan(got), np.isnan(ref)), f
        assert np.array_equal(got[0, 11, 1] == 0, ref[0, 11, 1] == 0)
