"""The C entry points of positions, rotary positions and the gated residual without a GPU: descriptions laid out as
the header's structures, refusals before any device work, workspace sizes, and the plan's arguments (CPU only)."""

import os
import re
import struct

import pytest

from test_abi import ROOT, lib  # noqa: F401

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096          # an aligned address that nothing reads: every call here is refused first


def fields(name):
    src = open(os.path.join(ROOT, "include", "pvl.h")).read()
    body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name, src, re.S).group(1)
    out = ""
    for line in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";"):
        m = re.match(r"\s*(const )?(\w+)\s*(.*)", line.strip(), re.S)
        if not m:
            continue
        kind, names = m.group(2), m.group(3)
        for n in names.split(","):
            out += "P" if "*" in n or "*" in names.split(",")[0] else {"int32_t": "i", "float": "f", "int64_t": "q"}[kind]
    return out


def test_descriptions_match_the_header():
    from packed_variable_length_gb300 import _lib
    for pack, name in ((_lib.PACK_ROTARY, "pvl_rotary"), (_lib.PACK_HEADS, "pvl_heads"),
                       (_lib.PACK_RESIDUAL, "pvl_residual"), (_lib.PACK_RESIDUAL_GRADS, "pvl_residual_grads")):
        s = pack.__self__
        assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([iIfPq])", s.format)) == fields(name), name


def rotary(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(B=1, L=4, H=2, Hk=2, D=64, R=64, layout=0, axes=1, s1=32, s2=32, gain=1.0, norm=0, eps=1e-6, turns=P,
             positions=P, wq=0, wk=0)
    d.update(kw)
    return _lib.PACK_ROTARY(*d.values())


def heads(data=P, b=512, t=128, h=64):
    return struct.pack("@Pqqq", data, b, t, h)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(H=0), INVALID), (dict(Hk=-1), INVALID), (dict(D=0), INVALID),
    (dict(layout=2), INVALID), (dict(norm=1), INVALID), (dict(norm=2), INVALID), (dict(axes=0), INVALID),
    (dict(axes=4), INVALID), (dict(D=65), UNSUPPORTED), (dict(D=258), UNSUPPORTED), (dict(R=63), UNSUPPORTED),
    (dict(R=66, s1=33, s2=33), INVALID), (dict(s1=31), INVALID), (dict(axes=2, s1=40, s2=32), INVALID),
    (dict(axes=3, s1=10, s2=9), INVALID), (dict(turns=0), INVALID), (dict(positions=0), INVALID),
    (dict(positions=P + 2), UNSUPPORTED), (dict(turns=P + 4), UNSUPPORTED), (dict(gain=float("nan")), INVALID),
    (dict(gain=float("inf")), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(wq=P), INVALID), (dict(norm=4, wq=P + 2), UNSUPPORTED), (dict(norm=3, Hk=0, wk=P), INVALID),
    (dict(H=5000), UNSUPPORTED), (dict(B=1 << 20, L=1 << 20), UNSUPPORTED)])
def test_rotary_refusals(lib, change, status):  # noqa: F811
    how = rotary(**change)
    assert lib.pack_rotary_fwd(how, heads(), heads(), heads(), heads(), None) == status
    assert lib.pack_rotary_bwd(how, heads(), heads(), heads(), heads(), heads(), heads(), P if change.get("wq") else None,
                               P if change.get("wk") else None, P, 1 << 30, None) == status


def test_rotary_views_and_workspace(lib):  # noqa: F811
    how = rotary()
    assert lib.pack_rotary_fwd(None, heads(), heads(), heads(), heads(), None) == INVALID
    assert lib.pack_rotary_fwd(how, None, heads(), heads(), heads(), None) == INVALID
    assert lib.pack_rotary_fwd(how, heads(), heads(0), heads(), heads(), None) == INVALID
    assert lib.pack_rotary_fwd(how, heads(P + 1), heads(), heads(), heads(), None) == UNSUPPORTED
    assert lib.pack_rotary_fwd(how, heads(h=1 << 30), heads(), heads(), heads(), None) == UNSUPPORTED
    assert lib.pack_rotary_bwd_ws_bytes(how) == 0 and lib.pack_rotary_bwd_ws_bytes(None) == 0
    normed = rotary(norm=4, wq=P, wk=P)
    need = lib.pack_rotary_bwd_ws_bytes(normed)
    assert need == 4 * 4 * 64 * 4                        # four tokens, four heads of 64
    assert lib.pack_rotary_bwd_ws_bytes(rotary(norm=3, wq=P, L=1 << 20)) == 1216 * 2 * 64 * 4
    args = [normed] + [heads()] * 6
    assert lib.pack_rotary_bwd(*args, P, P, P, need - 1, None) == INVALID
    assert lib.pack_rotary_bwd(*args, P, P, None, need, None) == INVALID
    assert lib.pack_rotary_bwd(*args, None, P, P, need, None) == INVALID          # a weight without its gradient
    assert lib.pack_rotary_bwd(*args, P, P, P + 8, need, None) == UNSUPPORTED
    assert lib.pack_rotary_bwd(normed, heads(), heads(), None, heads(), heads(), heads(), P, P, P, need, None) == INVALID
    # an output that several threads would write; an input may be broadcast (refused here for its null partner)
    for zero in ({"t": 0}, {"h": 0}):
        assert lib.pack_rotary_fwd(how, heads(), heads(), heads(**zero), heads(), None) == INVALID
        assert b"broadcast" in lib.pvl_last_error_message()
        assert lib.pack_rotary_fwd(how, heads(), heads(), heads(), heads(**zero), None) == INVALID
        assert b"broadcast" in lib.pvl_last_error_message()
        assert lib.pack_rotary_bwd(how, heads(), heads(), None, None, heads(**zero), heads(), None, None, None, 0,
                                   None) == INVALID
        assert b"broadcast" in lib.pvl_last_error_message()
        assert lib.pack_rotary_fwd(how, heads(**zero), None, heads(), heads(), None) == INVALID
        assert b"k is null" in lib.pvl_last_error_message()
    # a token that no block holds
    assert lib.pack_rotary_fwd(rotary(norm=4, H=600, Hk=0, D=66, R=66, s1=33, s2=33), heads(), None, heads(), None,
                               None) == UNSUPPORTED


def residual(**kw):
    from packed_variable_length_gb300 import _lib
    d = dict(B=2, N=4, D=64, S=2, dtype=0, norm=1, post=0, alpha=1.0, eps=1e-6, gate=P, shift=P, scale=P, w=0, b=0, w2=0,
             ids=0)
    d.update(kw)
    return _lib.PACK_RESIDUAL(*d.values())


@pytest.mark.parametrize("change,status", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(D=0), INVALID), (dict(D=60), UNSUPPORTED), (dict(D=8200), UNSUPPORTED),
    (dict(S=0, ids=P), INVALID), (dict(S=3), INVALID), (dict(S=70000, ids=P), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(norm=0), INVALID), (dict(norm=3), INVALID), (dict(post=4), INVALID), (dict(w2=P), INVALID),
    (dict(alpha=float("inf")), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(gate=P + 4), UNSUPPORTED), (dict(w=P + 8), UNSUPPORTED), (dict(ids=P + 2), UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 16), UNSUPPORTED)])
def test_residual_refusals(lib, change, status):  # noqa: F811
    how = residual(**change)
    grads = struct.pack("@PPPPPP", P, P, P, P if change.get("w") else 0, 0, P if change.get("w2") else 0)
    assert lib.adaln_residual_fwd(how, P, P, P, P, None) == status
    assert lib.adaln_residual_bwd(how, P, P, P, P, 1, P, P, grads, P, 1 << 40, None) == status


def test_residual_pointers_and_workspace(lib):  # noqa: F811
    how, none = residual(), struct.pack("@PPPPPP", 0, 0, 0, 0, 0, 0)
    grads = struct.pack("@PPPPPP", P, P, P, 0, 0, 0)
    for args in ((None, P, P, P, P), (how, None, P, P, P), (how, P, P, None, P), (how, P, P, P, None), (how, P, None, P, P),
                 (residual(gate=0, post=2), P, None, P, P), (residual(gate=0, alpha=0.5), P, None, P, P)):
        assert lib.adaln_residual_fwd(*args, None) == INVALID
    assert lib.adaln_residual_fwd(how, P + 8, P, P, P, None) == UNSUPPORTED
    need = lib.adaln_residual_bwd_ws_bytes(2, 4, 64, 2)
    assert need > 0 and lib.adaln_residual_bwd_ws_bytes(0, 4, 64, 2) == 0 == lib.adaln_residual_bwd_ws_bytes(2, 4, 64, 0)
    assert lib.adaln_residual_bwd_ws_bytes(1, 64000, 5120, 7) < 3 * (1216 + 7 + 14) * 5120 * 4 + (1 << 20)
    ok = [how, P, P, P, P, 1, P, P, grads, P, need]
    for i in (2, 3, 6, 7, 8, 9):            # dy, x_out, dx, dh, grads, ws
        assert lib.adaln_residual_bwd(*[None if j == i else a for j, a in enumerate(ok)], None) == INVALID, i
    assert lib.adaln_residual_bwd(*ok[:4], None, *ok[5:], None) == INVALID               # a gate without h
    assert lib.adaln_residual_bwd(*ok[:8], none, P, need, None) == INVALID               # tables without gradients
    assert lib.adaln_residual_bwd(*ok[:10], need - 1, None) == INVALID
    assert lib.adaln_residual_bwd(how, P, P, P, None, 0, P, None, grads, P, need, None) == INVALID   # a gate, no branch
    assert lib.adaln_residual_bwd(*ok[:6], P + 8, *ok[7:], None) == UNSUPPORTED


def test_positions_refusals(lib):  # noqa: F811
    frames = struct.pack("@2i", 3, 4)
    bad = ((None, 1, 2, 5, 1, 1, 100, P), (frames, 1, 2, 5, 1, 1, 100, None), (frames, 0, 2, 5, 1, 1, 100, P),
           (frames, 1, 2, 0, 1, 1, 100, P), (frames, 1, 2, 5, 0, 1, 100, P), (frames, 1, 2, 5, 4, 1, 100, P),
           (frames, 1, 2, 5, 3, 0, 100, P), (frames, 1, 2, 5, 1, 1, 34, P), (struct.pack("@2i", -1, 4), 1, 2, 5, 1, 1, 100, P))
    for args in bad:
        assert lib.pack_build_positions(*args, None) == INVALID, args
    assert lib.pack_build_positions(frames, 1, 3000, 5, 1, 1, 100, P, None) == UNSUPPORTED
    assert lib.pack_build_positions(frames, 1, 2, 5, 1, 1, 1 << 20, P, None) == UNSUPPORTED


def test_plan_refusals():
    import packed_variable_length_gb300 as pvl
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(layout="other"), dict(sections=(1, 2)), dict(sections=(16, 8, 4, 4)),
               dict(sections=(40, -8)), dict(scaling="dynamic"), dict(base=0.0), dict(base=float("inf")), dict(factor=0.0),
               dict(scaling="parts", factor=2.0), dict(scaling="parts", length=10, slow=3.0, fast=2.0)):
        with pytest.raises(ValueError):
            pvl.rotary_plan(**{"rotary_dim": 64, "device": "cpu", **kw})
    plan = pvl.rotary_plan(64, device="cpu", sections=(12, 10, 10))
    assert plan.turns.shape == (32,) and plan.gain == 1.0 and plan.sections == (12, 10, 10)


def test_tensors_of_the_host_are_refused():
    """Nothing of a call whose tensors are all on the host reaches the library."""
    import torch

    import packed_variable_length_gb300 as pvl
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    q, pos = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32)
    plan = pvl.rotary_plan(64, device="cpu")
    for call in (lambda: pvl.adaln_residual_fwd(x, x), lambda: pvl.adaln_residual_bwd(x, x, x, x),
                 lambda: pvl.pack_rotary_fwd(q, q, pos, plan), lambda: pvl.pack_rotary_bwd(q, q, pos, plan),
                 lambda: pvl.pack_build_positions([[1]], 4, 4, out=torch.zeros(1, 4, 1, dtype=torch.int32))):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            call()
