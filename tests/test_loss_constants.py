"""What the losses over episodes take as given: a gradient to it is refused, not dropped (CPU only)."""

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """The autograd ops, with the library's calls counted and answered on the host."""
    import packed_variable_length_gb300 as pvl
    seen = []

    def preference(logp, *args, **how):
        seen.append("preference")
        return pvl.PreferenceLoss(torch.zeros(1), torch.zeros(1, 2), torch.zeros(2))

    def policy(logp, *args, **how):
        seen.append("policy")
        return pvl.PolicyLoss(torch.zeros(1), torch.zeros(2), torch.zeros(2, 2))
    monkeypatch.setattr(pvl.autograd.objectives, "pack_preference_fwd", preference)
    monkeypatch.setattr(pvl.autograd.objectives, "pack_policy_fwd", policy)
    return pvl, seen


def inputs():
    return [torch.zeros(1, 4) for _ in range(4)], torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)


def test_constants_that_require_a_gradient_are_refused(calls):
    pvl, seen = calls
    (lp, old, ref, adv), ids, pairs = inputs()
    lp.requires_grad_()
    on = torch.zeros(1, 4, requires_grad=True)
    for call, name in ((lambda: pvl.preference_loss(lp, on, ids, pairs, 2), "ref_logp"),
                       (lambda: pvl.policy_loss(lp, on, adv, ids, 2), "old_logp"),
                       (lambda: pvl.policy_loss(lp, lp, adv, ids, 2), "old_logp"),
                       (lambda: pvl.policy_loss(lp, old, on, ids, 2), "advantages"),
                       (lambda: pvl.policy_loss(lp, old, adv, ids, 2, ref_logp=on * 2.0), "ref_logp")):
        with pytest.raises(ValueError, match=name + ".*detach"):
            call()
    assert not seen


def test_constants_without_one_are_taken(calls):
    pvl, seen = calls
    (lp, old, ref, adv), ids, pairs = inputs()
    lp.requires_grad_()
    on = torch.zeros(1, 4, requires_grad=True)
    loss, _ = pvl.preference_loss(lp, None, ids, pairs, 2)
    assert loss.requires_grad
    pvl.preference_loss(lp, on.detach(), ids, pairs, 2)
    loss, _ = pvl.policy_loss(lp, None, adv, ids, 2, ref_logp=ref)
    assert loss.requires_grad
    pvl.policy_loss(lp, lp.detach(), on.detach(), ids, 2, ref_logp=on.detach())
    with torch.no_grad():       # nothing is differentiated here
        pvl.preference_loss(lp, on, ids, pairs, 2)
        pvl.policy_loss(lp, on, on, ids, 2, ref_logp=on)
    assert sorted(seen) == ["policy"] * 3 + ["preference"] * 3
