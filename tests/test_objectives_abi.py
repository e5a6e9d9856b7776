"""The C entry points of the log-probabilities, the losses over packed episodes and the update without a GPU:
descriptions laid out as the header's structures, refusals before any device work, workspace sizes; and what the
binding refuses (CPU only)."""

import os
import re
import struct

import numpy as np
import pytest
import torch

from test_abi import ROOT, lib  # noqa: F401

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096          # an aligned address that nothing reads: every call here is refused first
NAN, INF = float("nan"), float("inf")


def fields(name):
    """Format characters of a structure of the header, in order."""
    src = open(os.path.join(ROOT, "include", "pvl.h")).read()
    body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name + ";", src, re.S).group(1)
    out = ""
    for line in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";"):
        m = re.match(r"\s*(?:const )?(\w+)(\*?)\s*(.*)", line.strip(), re.S)
        if m:
            kind = "P" if m.group(2) else {"int32_t": "i", "uint32_t": "I", "float": "f", "double": "d", "int64_t": "q"}[m.group(1)]
            out += kind * len(m.group(3).split(","))
    return out


def test_descriptions_match_the_header():
    from packed_variable_length_gb300 import _lib, optim
    for pack, name in ((_lib.PACK_LOGPROB, "pvl_logprob"), (_lib.PACK_PREFERENCE, "pvl_preference"),
                       (_lib.PACK_POLICY, "pvl_policy"), (_lib.PACK_ADAMW, "pvl_adamw")):
        s = pack.__self__
        assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([iIfdPq])", s.format)) == fields(name), name
    assert fields("pvl_adamw_tensor") == "PPqqif"
    assert optim._TENSOR.itemsize == struct.calcsize("@PPqqif")
    kinds = {"P": np.uint64, "q": np.int64, "i": np.int32, "f": np.float32}
    assert [optim._TENSOR[n] for n in optim._TENSOR.names] == [np.dtype(kinds[c]) for c in "PPqqif"]


def logprob(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(B=2, L=3, V=10, dtype=0, wide=0, T=1.0, logits=P, targets=P, ids=0, sb=30, sl=10)
    d.update(kw)
    return _lib.PACK_LOGPROB(*d.values())


@pytest.mark.parametrize("change,status", [
    (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(V=0), INVALID), (dict(dtype=2), INVALID), (dict(wide=2), INVALID),
    (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID), (dict(T=NAN), INVALID), (dict(T=INF), INVALID), (dict(logits=0), INVALID),
    (dict(targets=0), INVALID), (dict(sb=-1), INVALID), (dict(sl=-1), INVALID), (dict(logits=P + 1), UNSUPPORTED),
    (dict(dtype=1, logits=P + 2), UNSUPPORTED), (dict(targets=P + 2), UNSUPPORTED), (dict(wide=1, targets=P + 4), UNSUPPORTED),
    (dict(ids=P + 2), UNSUPPORTED), (dict(V=(1 << 28) + 1), UNSUPPORTED), (dict(B=1 << 14, L=1 << 13), UNSUPPORTED),
    (dict(L=1 << 20, V=1 << 22), UNSUPPORTED)])
def test_logprob_refusals(lib, change, status):  # noqa: F811
    how = logprob(**change)
    assert lib.pack_logprob_fwd(how, P, P, None, None) == status
    assert lib.pack_logprob_bwd(how, P, None, P, None, P, 30, 10, None) == status


def test_logprob_outputs(lib):  # noqa: F811
    how = logprob()
    for args in ((None, P, P, None), (how, None, P, None), (how, P, None, None)):
        assert lib.pack_logprob_fwd(*args, None) == INVALID
    for args in ((how, P + 2, P, None), (how, P, P + 1, None), (how, P, P, P + 2)):
        assert lib.pack_logprob_fwd(*args, None) == UNSUPPORTED
    for args in ((how, None, None, P, None, P), (how, P, None, None, None, P), (how, P, None, P, None, None),
                 (how, P, None, P, P, P), (how, P, None, None, P, P)):
        assert lib.pack_logprob_bwd(*args, 30, 10, None) == INVALID
    for sb, sl in ((30, 9), (29, 10), (0, 10), (30, 0), (9, 20), (10, 19), (-30, 10), (30, -10)):
        assert lib.pack_logprob_bwd(how, P, None, P, None, P, sb, sl, None) == INVALID, (sb, sl)
        assert b"overlap" in lib.pvl_last_error_message()
    assert lib.pack_logprob_bwd(how, P, None, P, None, P + 1, 30, 10, None) == UNSUPPORTED
    # 60 logits of 2 bytes from P on: anything within them but the logits themselves
    for at, sb, sl in ((P + 2, 30, 10), (P - 2, 30, 10), (P + 118, 30, 10), (P - 118, 30, 10), (P, 30, 20), (P, 60, 10)):
        assert lib.pack_logprob_bwd(how, P, None, P, None, at, sb, sl, None) == INVALID, (at, sb, sl)
    assert lib.pack_logprob_bwd(how, P, None, P, None, P, 60, 10, None) == INVALID
    assert b"reaches into" in lib.pvl_last_error_message()


def preference(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(tokens=100, E=4, n=2, kind=0, mean=0, beta=0.1, smoothing=0.0, margin=0.0, logp=P, ref=0, ids=P, pairs=P)
    d.update(kw)
    return _lib.PACK_PREFERENCE(*d.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), INVALID), (dict(E=0), INVALID), (dict(n=0), INVALID), (dict(kind=3), INVALID), (dict(kind=-1), INVALID),
    (dict(mean=2), INVALID), (dict(beta=0.0), INVALID), (dict(beta=-1.0), INVALID), (dict(beta=NAN), INVALID),
    (dict(beta=INF), INVALID), (dict(margin=NAN), INVALID), (dict(margin=INF), INVALID), (dict(smoothing=-0.1), INVALID),
    (dict(smoothing=0.6), INVALID), (dict(smoothing=NAN), INVALID), (dict(kind=1, smoothing=0.1), INVALID), (dict(logp=0), INVALID),
    (dict(ids=0), INVALID), (dict(pairs=0), INVALID), (dict(tokens=(1 << 23) + 1), UNSUPPORTED),
    (dict(E=(1 << 16) + 1), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(logp=P + 2), UNSUPPORTED),
    (dict(ref=P + 1), UNSUPPORTED), (dict(ids=P + 2), UNSUPPORTED), (dict(pairs=P + 2), UNSUPPORTED)])
def test_preference_refusals(lib, change, status):  # noqa: F811
    assert lib.pack_preference_fwd(preference(**change), P, P, P, P, 1 << 30, None) == status


def policy(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(tokens=100, E=4, ratio=0, mean=0, tok=1, low=0.2, high=0.2, kl=0.0, logp=P, old=0, ref=0, adv=P, ids=P)
    d.update(kw)
    return _lib.PACK_POLICY(*d.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), INVALID), (dict(E=0), INVALID), (dict(ratio=2), INVALID), (dict(mean=2), INVALID), (dict(tok=2), INVALID),
    (dict(ratio=1), INVALID), (dict(low=-0.1), INVALID), (dict(low=1.0), INVALID), (dict(low=NAN), INVALID),
    (dict(high=-0.1), INVALID), (dict(high=INF), INVALID), (dict(high=NAN), INVALID), (dict(kl=0.1), INVALID),
    (dict(kl=-0.1, ref=P), INVALID), (dict(kl=NAN, ref=P), INVALID), (dict(kl=INF, ref=P), INVALID), (dict(logp=0), INVALID),
    (dict(adv=0), INVALID), (dict(ids=0), INVALID), (dict(tokens=(1 << 23) + 1), UNSUPPORTED),
    (dict(E=(1 << 16) + 1), UNSUPPORTED), (dict(old=P + 2), UNSUPPORTED), (dict(adv=P + 1), UNSUPPORTED)])
def test_policy_refusals(lib, change, status):  # noqa: F811
    how = policy(**change)
    assert lib.pack_policy_fwd(how, P, P, P, P, 1 << 30, None) == status
    assert lib.pack_policy_bwd(how, P, P, P, None) == status


def test_loss_outputs_and_workspaces(lib):  # noqa: F811
    for size in (lib.pack_preference_ws_bytes, lib.pack_policy_ws_bytes):
        assert size(0) == size(-1) == size((1 << 16) + 1) == 0 and size(1) > 0 and size(1 << 16) < 1 << 25
    need = lib.pack_preference_ws_bytes(4)
    ok = [preference(), P, P, P, P, need]
    for i in range(5):
        assert lib.pack_preference_fwd(*[None if j == i else a for j, a in enumerate(ok)], None) == INVALID, i
    assert lib.pack_preference_fwd(*ok[:5], need - 1, None) == INVALID
    assert lib.pack_preference_fwd(*ok[:4], P + 8, need, None) == UNSUPPORTED
    assert lib.pack_preference_fwd(*ok[:1], P + 2, *ok[2:], None) == UNSUPPORTED
    need = lib.pack_policy_ws_bytes(4)
    ok = [policy(), P, P, P, P, need]
    for i in range(5):
        assert lib.pack_policy_fwd(*[None if j == i else a for j, a in enumerate(ok)], None) == INVALID, i
    assert lib.pack_policy_fwd(*ok[:5], need - 1, None) == INVALID
    assert lib.pack_policy_fwd(*ok[:3], P + 4, P, need, None) == UNSUPPORTED          # pairs of floats
    for args in ((None, None, P, 10, 4, P), (None, P, None, 10, 4, P), (None, P, P, 10, 4, None), (None, P, P, 0, 4, P),
                 (None, P, P, 10, 0, P)):
        assert lib.pack_preference_bwd(*args, None) == INVALID
    assert lib.pack_preference_bwd(P + 2, P, P, 10, 4, P, None) == UNSUPPORTED
    assert lib.pack_policy_bwd(None, P, P, P, None) == lib.pack_policy_bwd(policy(), P, None, P, None) == INVALID
    assert lib.pack_policy_bwd(policy(), P, P, None, None) == INVALID
    assert lib.pack_policy_bwd(policy(), P, P + 4, P, None) == UNSUPPORTED


def adamw(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(pt=1, gt=1, bits=32, seed=0, b1=0.9, b2=0.999, lr=1e-3, eps=1e-8, most=1.0, lr_dev=0, norm=0, m=P, v=P, ms=0, vs=0,
             master=0, steps=P, done=P)
    d.update(kw)
    return _lib.PACK_ADAMW(*d.values())


def entry(**kw):
    d = dict(p=P, g=P, size=10, block=0, slot=0, decay=0.0)
    d.update(kw)
    return struct.pack("@PPqqif", *d.values())


@pytest.mark.parametrize("change,status", [
    (dict(pt=2), INVALID), (dict(gt=-1), INVALID), (dict(bits=16), INVALID), (dict(bits=8), INVALID), (dict(bits=8, ms=P), INVALID),
    (dict(pt=0), INVALID), (dict(master=P), INVALID), (dict(lr=NAN), INVALID), (dict(lr=INF), INVALID), (dict(b1=1.0), INVALID),
    (dict(b1=-0.1), INVALID), (dict(b2=1.0), INVALID), (dict(b2=NAN), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(norm=P, most=0.0), INVALID), (dict(norm=P, most=NAN), INVALID), (dict(m=0), INVALID),
    (dict(v=0), INVALID), (dict(steps=0), INVALID), (dict(done=0), INVALID), (dict(m=P + 16), UNSUPPORTED),
    (dict(v=P + 16), UNSUPPORTED), (dict(pt=0, master=P + 16), UNSUPPORTED), (dict(steps=P + 2), UNSUPPORTED),
    (dict(norm=P + 2), UNSUPPORTED), (dict(lr_dev=P + 1), UNSUPPORTED)])
def test_adamw_refusals(lib, change, status):  # noqa: F811
    assert lib.pvl_adamw_step(adamw(**change), entry(), 1, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(p=0), INVALID), (dict(g=0), INVALID), (dict(size=0), INVALID), (dict(block=-1), INVALID), (dict(slot=-1), INVALID),
    (dict(decay=NAN), INVALID), (dict(decay=INF), INVALID), (dict(size=1 << 38), UNSUPPORTED), (dict(block=1 << 40), UNSUPPORTED),
    (dict(p=P + 2), UNSUPPORTED), (dict(g=P + 1), UNSUPPORTED)])
def test_adamw_tensor_refusals(lib, change, status):  # noqa: F811
    assert lib.pvl_adamw_step(adamw(), entry() + entry(**change), 2, None) == status
    assert lib.pvl_adamw_step(adamw(), None, 1, None) == lib.pvl_adamw_step(adamw(), entry(), 0, None) == INVALID


def test_norm_refusals(lib):  # noqa: F811
    need = lib.pvl_grad_norm_ws_bytes()
    ptrs, sizes = struct.pack("@2P", P, P), struct.pack("@2q", 5, 5)
    ok = [ptrs, sizes, 2, 0, P, P, need]
    for i in (0, 1, 4, 5):
        assert lib.pvl_grad_norm(*[None if j == i else a for j, a in enumerate(ok)], None) == INVALID, i
    for i, bad in ((2, 0), (3, 2), (6, need - 1), (0, struct.pack("@2P", P, 0)), (1, struct.pack("@2q", 5, 0))):
        assert lib.pvl_grad_norm(*[bad if j == i else a for j, a in enumerate(ok)], None) == INVALID, i
    for i, bad in ((4, P + 2), (5, P + 8), (0, struct.pack("@2P", P, P + 1)), (1, struct.pack("@2q", 5, 1 << 41)),
                   (2, (1 << 17) + 1)):
        assert lib.pvl_grad_norm(*[bad if j == i else a for j, a in enumerate(ok)], None) == UNSUPPORTED, i
    many = struct.pack("@2q", 1 << 40, 1 << 40)
    assert lib.pvl_grad_norm(ptrs, many, 2, 0, P, P, need, None) == UNSUPPORTED


@pytest.fixture
def closed(monkeypatch):
    """No call of the library gets through."""
    import packed_variable_length_gb300 as pvl

    def load():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(pvl.api._lib, "load", load)
    return pvl


def test_binding_refuses_tensors_of_the_host(closed):
    pvl = closed
    x, t = torch.zeros(1, 4, 9), torch.zeros(1, 4, dtype=torch.int32)
    lp, pairs = torch.zeros(1, 4), torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: pvl.pack_logprob_fwd(x, t), lambda: pvl.pack_logprob_bwd(lp, x, t, lp),
                 lambda: pvl.pack_preference_fwd(lp, None, t, pairs, 2), lambda: pvl.pack_preference_bwd(None, lp[0], t),
                 lambda: pvl.pack_policy_fwd(lp, None, lp, t, 2), lambda: pvl.pack_policy_bwd(None, lp, None, lp, t, torch.zeros(2, 2)),
                 lambda: pvl.grad_norm([lp]), lambda: pvl.adamw_state([lp])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_types_and_shapes(closed):
    """Before the device is looked at."""
    pvl = closed
    x, t = torch.zeros(1, 4, 9), torch.zeros(1, 4, dtype=torch.int32)
    for args in ((x.half(), t), (x.double(), t), (x[0], t), (None, t), (x, t.short()), (x, None)):
        with pytest.raises(ValueError):
            pvl.pack_logprob_fwd(*args)
    for kw in (dict(dlogp=None), dict(dlogp=torch.zeros(1, 4), dent=torch.zeros(1, 4))):
        with pytest.raises(ValueError):
            pvl.pack_logprob_bwd(kw.pop("dlogp"), x, t, torch.zeros(1, 4), **kw)
    for bits in (16, 0, "8"):
        with pytest.raises(ValueError):
            pvl.adamw_state([x], bits=bits)
    for seed in (-1, 1 << 32):
        with pytest.raises(ValueError):
            pvl.adamw_state([x], seed=seed)
    for params in ([], [x.half()], [x, None]):
        with pytest.raises(ValueError):
            pvl.adamw_state(params)
    with pytest.raises(ValueError):
        pvl.grad_norm([])
    with pytest.raises(ValueError):
        pvl.grad_norm([None, None])
