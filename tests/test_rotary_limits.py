"""Tokens whose heads the norm over the token cannot hold, by the widths of vectors (CPU only: every call here is to be
refused before any device work; its addresses are made up, so nothing runs where there is a device)."""

import pytest
import torch

from test_abi import lib  # noqa: F401
from test_block_abi import UNSUPPORTED, heads, rotary

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


@pytest.mark.parametrize("H,Hk,D", [(128, 8, 128), (175, 0, 96), (144, 0, 128)])
def test_a_backward_that_shared_memory_does_not_hold(lib, H, Hk, D):  # noqa: F811
    how = rotary(H=H, Hk=Hk, D=D, R=D, s1=D // 2, s2=D // 2, norm=4)
    v = heads(b=4 * H * D, t=H * D, h=D)
    w = v if Hk else None
    assert lib.pack_rotary_bwd(how, v, w, v, w, v, w, None, None, None, 0, None) == UNSUPPORTED
    assert b"does not fit" in lib.pvl_last_error_message()


def most_heads(V, D, backward):
    """The header's rule."""
    return {8: 3, 4: 4, 2: 8, 1: 16}[V] * ((352 if backward and V == 8 else 384) // (D // (2 * V)))


@pytest.mark.parametrize("V,D", [(8, 16), (8, 96), (8, 128), (8, 176), (8, 256), (4, 8), (4, 72), (4, 168), (4, 232),
                                 (2, 36), (2, 220), (2, 252), (1, 66), (1, 194), (1, 250), (1, 254)])
def test_one_head_more_than_a_block_holds(lib, V, D):  # noqa: F811
    """Both directions, one head past the limit; the largest tokens that the header says always fit are below it."""
    always = {8: 16700, 4: 11700, 2: 10700, 1: 9500}[V]
    for backward in (False, True):
        H = most_heads(V, D, backward) + 1
        assert H * D > always
        v = heads(b=2 * H * D, t=H * D, h=D)
        how = rotary(B=1, L=2, H=H, Hk=0, D=D, R=D, s1=D // 2, s2=D // 2, norm=4)
        if backward:
            st = lib.pack_rotary_bwd(how, v, None, v, None, v, None, None, None, None, 0, None)
        else:
            st = lib.pack_rotary_fwd(how, v, None, v, None, None)
        assert st == UNSUPPORTED and b"does not fit" in lib.pvl_last_error_message(), lib.pvl_last_error_message()


def test_narrow_views_have_the_narrow_limit(lib):  # noqa: F811
    """128 heads of 128 fit 8-wide, and not where a stride or an address allows 4, 2 or 1."""
    how = rotary(B=1, L=2, H=128, Hk=0, D=128, R=128, s1=64, s2=64, norm=4)
    for data, t in ((4096, 16388), (4096, 16386), (4096, 16385), (4104, 16384), (4100, 16384), (4098, 16384)):
        v = heads(data=data, b=2 * t, t=t, h=128)
        assert lib.pack_rotary_fwd(how, v, None, v, None, None) == UNSUPPORTED
        assert b"does not fit" in lib.pvl_last_error_message()
