"""AdamW where a gradient is not finite or its square leaves fp32: with 8-bit moments what is wrong with one element
stays with it; with 32-bit ones squares below the normal numbers count (GPU)."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = 600       # three blocks, the last one not whole


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def gradients(spread):
    """Of one size, so that no code is below 2^-6, or of many."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = 1.0 + torch.rand(FAR, generator=g, device="cuda")
    return x * torch.exp(-spread * torch.rand(FAR, generator=g, device="cuda") * math.log(1e6))


def two_steps(pvl, dtype, bad, at, spread, seed=1):
    p = torch.ones(FAR, dtype=dtype, device="cuda")
    state = pvl.adamw_state([p], bits=8, seed=seed)
    g = gradients(spread)
    first = g.clone()
    first[at] = bad
    pvl.adamw_step([p], [first], state, 1e-3)
    mid = [t.clone() for t in state.moments(0)]
    pvl.adamw_step([p], [g], state, 1e-3)
    torch.cuda.synchronize()
    return p, mid, [t.clone() for t in state.moments(0)], state


@pytest.mark.parametrize("bad", [math.nan, -math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("at", [[3], [300], [599], [0, 7, 255], [512, 590]])
def test_what_is_not_finite_stays_with_its_element(pvl, bad, dtype, spread, at):
    """The others: bit by bit as if that gradient were 0, whose moments of 0 no other element sees."""
    p, mid, end, state = two_steps(pvl, dtype, bad, at, spread)
    q, other, last, _ = two_steps(pvl, dtype, 0.0, at, spread)
    keep = torch.ones(FAR, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(p[keep], q[keep]) and torch.isfinite(p[keep]).all()
    for a, b in zip(mid + end, other + last):
        assert torch.equal(a[keep], b[keep])
        assert torch.isnan(a[~keep]).all()
    assert torch.isnan(p[~keep]).all()
    for t in (state.m, state.v) + ((state.master,) if state.master is not None else ()):
        assert not t[FAR:].float().any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("big", [1e21, -1e21, 3e38])
@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("at", [[300], [0, 256, 599]])
def test_a_square_past_fp32_stops_its_element(pvl, dtype, big, spread, at):
    """As with 32-bit moments its v is infinite and the element only decays; the others bit by bit as if that gradient
    were 0."""
    p, mid, end, state = two_steps(pvl, dtype, big, at, spread)
    q, other, last, _ = two_steps(pvl, dtype, 0.0, at, spread)
    own = torch.zeros(FAR, dtype=torch.bool, device="cuda")
    own[at] = True
    assert torch.isfinite(p).all() and torch.equal(p[~own], q[~own])
    for a, b in zip(mid + end, other + last):
        assert torch.equal(a[~own], b[~own])
    for m, v in (mid, end):
        assert not m[own].any() and (v[own] == math.inf).all()
    # the decay of two steps alone; one rounding a step, and bf16's
    want = (1.0 - 1e-5) ** 2
    assert ((p[own].double() - want).abs() <= 2.0 ** -23 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)).all()
    # as 32-bit moments have it
    r = torch.ones(FAR, dtype=dtype, device="cuda")
    wide = pvl.adamw_state([r])
    for g in (gradients(spread).index_fill_(0, torch.tensor(at, device="cuda"), big), gradients(spread)):
        pvl.adamw_step([r], [g], wide, 1e-3)
    assert torch.equal(r[own], p[own]) and (wide.moments(0)[1][own] == math.inf).all()


@pytest.mark.parametrize("g", [1e-18, 3e-19, 1e-20])
def test_a_small_denominator(pvl, g):
    """32-bit moments whose v lies below the normal numbers, and an eps that does not cover it: the first step moves by
    lr, as the formula has it.  v is a multiple of 2^-149: its root is off by 2^-150 / v of itself, twice (b2 v, c2 g^2)
    and 2^-19 for the rest."""
    from oracle import adamw as oa
    p = torch.zeros(1000, device="cuda")
    grads = torch.full((1000,), g, device="cuda")
    state = pvl.adamw_state([p])
    for t in (1, 2):
        before, was = p.double().cpu().numpy(), [x.double().cpu().numpy() for x in state.moments(0)]
        pvl.adamw_step([p], [grads], state, 1e-2, eps=1e-30, weight_decay=0.0)
        want, _, v, change = oa.step(before, grads.double().cpu().numpy(), *was, t, 1e-2, eps=1e-30, decay=0.0)
        tol = (2.0 ** -19 + 2 * 2.0 ** -149 / v) * np.abs(change) + 2.0 ** -23 * np.abs(want)
        assert (np.abs(p.double().cpu().numpy() - want) <= tol).all(), (p[0].item(), want[0])
