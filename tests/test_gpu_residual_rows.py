"""Rows of the gated residual whose statistics are special, against the fp64 oracle (GPU)."""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_residual import check, f64, host, make, pvl  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [("layer", None), ("rms", None), ("rms", "rms"), ("layer", "layer"), ("layer", "rms")]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,post", KINDS)
@pytest.mark.parametrize("D", [64, 1536, 5120])
def test_a_value_that_is_not_finite_fills_its_row_alone(pvl, D, norm, post, stream, value):  # noqa: F811
    """One NaN or infinity in a live row: NaN where the formulas have it, forward and backward; every other row keeps
    its bits."""
    t, args, how = make(2, 60, D, "episode", norm, post, stream, D)
    ids = how["mod_id"]
    b, n = (int(i) for i in torch.nonzero(ids >= 0)[7])
    others = torch.ones_like(ids, dtype=torch.bool)
    others[b, n] = False
    which = "h" if post else "x"

    def run(t):
        x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
        return x_out, y

    a = run(t)
    g = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], a[0], t["h"], *args, **how)
    bad = {**t, which: t[which].clone()}
    bad[which][b, n, D // 3] = value
    c = run(bad)
    hh, ha = host(how, args)
    with np.errstate(invalid="ignore"):
        X, Y, _, _ = oracle.residual_fwd(bad["x"].cpu(), bad["h"].cpu(), *ha, **hh)
    assert np.isnan(Y[b, n]).any()
    for got, ref, whole in zip(c, (X, Y), a):
        assert np.array_equal(np.isnan(f64(got)), np.isnan(ref))
        assert torch.equal(got[others], whole[others])
    # backward: the value in x_out, and with a post norm also in h
    for x_out, h in ((c[0], t["h"]), (a[0], bad["h"])):
        G = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out, h, *args, **how)
        with np.errstate(invalid="ignore"):
            R = oracle.residual_bwd(t["dx_out"].cpu(), t["dy"].cpu(), x_out.cpu(), h.cpu(), *ha, **hh)
        for name in ("dx", "dh"):
            got = getattr(G, name)
            assert np.array_equal(np.isnan(f64(got)), np.isnan(R[name])), name
            assert torch.equal(got[others], getattr(g, name)[others]), name
    pvl.device_error()


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,post", [("layer", None), ("layer", "layer"), ("rms", "layer")])
@pytest.mark.parametrize("D", [1536, 5120, 8192])
@pytest.mark.parametrize("place", ["first", "third", "last"])
def test_one_outlier_channel_on_a_common_offset(pvl, D, norm, post, stream, place):  # noqa: F811
    """Rows with one large channel, as residual streams have them, and with an offset of all: the statistics are as
    near as for other rows.  The tolerances are test_gpu_residual's; they also hold for chains of 128 + 6 additions
    (the longest here, 2^-17 of the sum of magnitudes): the sums are shifted by an ordinary element of the row, so
    (mean - K)^2 is below 15 variances, the variance off by 2^-13, the root by 2^-14, xh by 2^-13 (1 + |xh|)."""
    at = {"first": 0, "third": 2, "last": D - 1}[place]
    t, args, how = make(2, 40, D, "episode", norm, post, stream, D + at)
    for name, big, offset in (("x", 1000.0, 20.0), ("h", -700.0, -9.0)):
        v = t[name].float() + offset
        v[..., at] = big
        t[name] = v.to(t[name].dtype)
    check(pvl, t, args, how)
    check(pvl, {**t, "dx_out": None}, args, how)


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_gradients_that_are_parts_of_others(pvl, stream):  # noqa: F811
    """Gradients of outputs that were joined behind one more element start off the kernels' 16-byte boundary."""
    t, args, how = make(2, 30, 256, "episode", "layer", "rms", stream, 3)
    x = t["x"].clone().requires_grad_()
    h = t["h"].clone().requires_grad_()
    x_out, y = pvl.gated_residual(x, h, *args, **how)
    ref = torch.autograd.grad([x_out, y], [x, h], [t["dx_out"], t["dy"]])
    x_out, y = pvl.gated_residual(x, h, *args, **how)
    joined, ups = [], []
    for out, up in ((x_out, t["dx_out"]), (y, t["dy"])):
        one = torch.ones(1, dtype=out.dtype, device="cuda")
        joined.append(torch.cat([one, out.flatten()]))
        ups.append(torch.cat([one, up.flatten()]))
    for a, b in zip(ref, torch.autograd.grad(joined, [x, h], ups)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,post", [("layer", None), ("rms", "layer")])
@pytest.mark.parametrize("D", [504, 512, 1280, 1328, 1528, 2304, 2344, 2560, 3584, 3800, 4096, 4608, 5616, 6912, 6920])
def test_widths(pvl, D, norm, post, stream):  # noqa: F811
    """Widths on both sides of every change of launch shape, and those between; more rows than the device has SMs."""
    check(pvl, *make(2, 90, D, "frame", norm, post, stream, seed=D))
