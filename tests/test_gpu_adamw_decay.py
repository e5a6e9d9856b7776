"""AdamW at the small rates of post-training: the decay of a step, lr * decay, is far below the spacing of fp32 (GPU).

Two runs from the same parameters with gradients of opposite signs: their updates are opposite, so the mean of both is
the decay alone, (1 - lr decay)^T, but for roundings.  A step rounds a parameter by at most 2^-24 of it, either way:
deviation 2^-24 / sqrt 3 at most, and of the mean over n elements, two runs and T steps that times sqrt(T / 2 n); six of
these, and 2^-22 of the decay for the roundings of its factor."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lr,decay", [(1e-5, 0.01), (1e-6, 0.01), (1e-7, 0.1), (1e-7, 0.01)])
def test_small_decay_adds_up(pvl, bits, dtype, lr, decay):
    n, T = 1 << 18, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    sign = torch.randint(0, 2, (n,), generator=g, device="cuda") * 2 - 1
    start = ((0.5 + 1.5 * torch.rand(n, generator=g, device="cuda")).clamp_(max=1.999) * sign).to(dtype)
    ends = []
    for up in (1.0, -1.0):
        p = start.clone()
        state = pvl.adamw_state([p], bits=bits, seed=3)
        # in the middle of training: v = 1, so that an update is lr times the gradient
        if bits == 32:
            state.v.fill_(1.0)
        else:
            state.v.copy_(torch.full_like(state.m_scale, 448.0).repeat_interleave(256))
            state.v_scale.fill_(1 / 448)
        state.steps.fill_(100000)
        draws = torch.Generator(device="cuda").manual_seed(2)
        for _ in range(T):
            pvl.adamw_step([p], [torch.randn(n, generator=draws, device="cuda") * up], state, lr, betas=(0.0, 0.999),
                           weight_decay=decay)
        ends.append((state.masters(0) if dtype == torch.bfloat16 else p).double())
    kept = ((ends[0] + ends[1]) / (2 * start.double())).mean().item()
    gone = -math.expm1(T * math.log1p(-lr * decay))
    tol = 6 * 2.0 ** -24 / math.sqrt(3) * math.sqrt(T / (2 * n)) + 2.0 ** -22 * gone
    assert tol < 0.25 * gone        # the test can see a decay
    assert abs((1 - kept) - gone) <= tol, (1 - kept, gone, tol)


def test_decay_alone_and_large(pvl):
    """No gradient: p (1 - lr decay), two roundings; also where the decay is most of the step."""
    p = torch.randn(5000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    for rate in (1e-3, 0.5, 1.0, 1.5):
        q = p.clone()
        state = pvl.adamw_state([q])
        pvl.adamw_step([q], [torch.zeros_like(q)], state, rate, weight_decay=1.0)
        want = p.double() * (1 - rate)
        assert ((q.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -23 * rate * p.double().abs()).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_a_step_of_nothing_leaves(pvl, bits, dtype):
    """Infinite parameters (as masks hold them) stay infinite under any decay below 1; with no rate or no decay every
    value stays what it is, to the last bit."""
    p = torch.tensor([math.inf, -math.inf, 1.0, -3.14, 0.0, -0.0, 1e-38, 1e-44, 3.38e38, 2.0 ** -126, 2.0 ** -110]).to(dtype).cuda()
    for lr, decay in ((1e-3, 0.1), (1e-8, 0.01), (0.5, 1.0), (1e-3, 0.0), (0.0, 0.1)):
        q = p.clone()
        state = pvl.adamw_state([q], bits=bits)
        pvl.adamw_step([q], [torch.zeros_like(q)], state, lr, weight_decay=decay)
        assert q[:2].tolist() == [math.inf, -math.inf] and torch.isfinite(q[2:]).all(), (lr, decay, q)
        if lr * decay == 0.0:
            bits_of = torch.int32 if dtype == torch.float32 else torch.int16
            assert torch.equal(q.view(bits_of), p.view(bits_of)), (q, p)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_decay_of_all_leaves_nothing(pvl, bits, dtype):
    p = torch.randn(1000, device="cuda").to(dtype)
    state = pvl.adamw_state([p], bits=bits)
    pvl.adamw_step([p], [torch.zeros_like(p)], state, 0.5, weight_decay=2.0)
    assert not p.any()
