"""Tokens that the norm over all of their heads does not fit, by the widths of vectors (CPU only: every call here is
refused before any device work)."""

import pytest

from test_abi import lib  # noqa: F401
from test_block_abi import UNSUPPORTED, heads, rotary

P = 4096


@pytest.mark.parametrize("H,Hk,D", [(128, 8, 128), (175, 0, 96), (144, 0, 128)])
def test_a_backward_that_shared_memory_does_not_hold(lib, H, Hk, D):  # noqa: F811
    how = rotary(H=H, Hk=Hk, D=D, R=D, s1=D // 2, s2=D // 2, norm=4)
    v = heads(b=4 * H * D, t=H * D, h=D)
    w = v if Hk else None
    assert lib.pack_rotary_bwd(how, v, w, v, w, v, w, None, None, None, 0, None) == UNSUPPORTED
    assert b"does not fit" in lib.pvl_last_error_message()
