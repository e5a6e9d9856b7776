"""Gradients of log-probabilities: large gradients of the entropy beside banned logits (GPU)."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def case(B=1, L=4, V=300, seed=1, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(B, L, V, generator=g, device="cuda") * 2).to(dtype)
    return x, torch.randint(0, V // 2, (B, L), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 300, 9000])
@pytest.mark.parametrize("scale", [1e8, 1e10, 1e20, 1e30])
def test_large_gradients_of_the_entropy_beside_banned_logits(pvl, dtype, V, scale):
    """As in a loss scaled for narrow gradients: 0 for what is banned, the others in proportion."""
    x, t = case(V=V, dtype=dtype)
    x[..., V // 2:V // 2 + 7] = -math.inf
    x[..., -5:] = torch.finfo(dtype).min
    x[..., -9] = -400.0
    logp, lse, ent = pvl.pack_logprob_fwd(x, t, entropy=True)
    up = torch.ones_like(logp)
    one = pvl.pack_logprob_bwd(None, x, t, lse, ent=ent, dent=up)
    many = pvl.pack_logprob_bwd(None, x, t, lse, ent=ent, dent=scale * up)
    assert torch.isfinite(many).all()
    assert not many[..., V // 2:V // 2 + 7].any() and not many[..., -5:].any() and not many[..., -9].any()
    # both round once to their type, and the products in fp32
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    want = one.double() * scale
    assert ((many.double() - want).abs() <= 2 * unit * want.abs() + scale * 2.0 ** -125).all()
