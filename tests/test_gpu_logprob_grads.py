"""Gradients of log-probabilities: large gradients of the entropy beside banned logits, and outputs over tensors that an
older graph still needs (GPU)."""

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


def test_a_gradient_over_the_logits_counts_as_a_change_in_place(pvl):
    """A graph that still needs those logits refuses instead of going on with the gradient in their place."""
    x, t = case()
    leaf = x.clone().requires_grad_()
    y = leaf * 1.0
    loss = (y * y).sum()                    # needs y
    logp, lse, _ = pvl.pack_logprob_fwd(y.detach(), t)
    was = y._version
    pvl.pack_logprob_bwd(torch.ones_like(logp), y.detach(), t, lse, dlogits=y.detach())
    assert y._version > was
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_that_are_given_count_as_changed(pvl):
    x, t = case()
    ids = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[0, 0]], dtype=torch.int32, device="cuda")
    out = {name: torch.zeros(1, 4, device="cuda") for name in ("logp", "lse", "ent", "pref", "pol")}
    versions = {name: o._version for name, o in out.items()}
    pvl.pack_logprob_fwd(x, t, entropy=True, logp=out["logp"], lse=out["lse"], ent=out["ent"])
    pref = pvl.pack_preference_fwd(out["logp"], None, ids, pairs, 1)
    pvl.pack_preference_bwd(None, pref.coef, ids, dlogp=out["pref"])
    adv = torch.ones(1, device="cuda")
    pol = pvl.pack_policy_fwd(out["logp"], None, adv, ids, 1)
    pvl.pack_policy_bwd(None, out["logp"], None, adv, ids, pol.coef, dlogp=out["pol"])
    norm = torch.zeros(1, device="cuda")
    pvl.grad_norm([x], out=norm)
    assert all(o._version > versions[name] for name, o in out.items()) and norm._version > 0
    # tensors of inference mode have no version and are written as before
    with torch.inference_mode():
        free = torch.zeros_like(x)
    lse = out["lse"]
    pvl.pack_logprob_bwd(out["logp"], x, t, lse, dlogits=free)
    assert torch.equal(free, pvl.pack_logprob_bwd(out["logp"], x, t, lse))
