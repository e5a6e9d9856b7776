"""Both sides of the launch rules of the log-probabilities and of the norm's unit (GPU).

Tolerances, from the arithmetic.  Log-probabilities: a sum of V terms carries 2^-20 from exp2 and its argument and
2^-24 a term that one thread adds, V over the threads of a row, which the rule here gives; logp and lse add 2^-22 of
themselves and of the maximum, the gradient's probability 2^-22 of its exponent; it is rounded once to its type.  The
norm: a lane adds at most 32 squares in fp32, 2^-19 of their sum, and half of that of its root."""

import math

import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def threads(N, vectors):
    """Of a row, in the forward."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if vectors <= 256 and 4 * N >= sms * vectors:
        return 8
    if vectors <= 128 or (vectors <= 2048 and N >= 8 * sms):
        return 32
    return 2048 if vectors >= 4096 and 80 * N <= vectors else 256


# (rows of an SM's worth, rows beside that, vectors): both sides in vectors and in rows
RULES = [(0, 18, 128), (0, 18, 129),                                # a warp or a block, few rows
         (64, 0, 256), (64, -1, 256), (64, 0, 257), (64, 1, 257),   # 8 threads or a warp
         (32, 0, 128), (32, -1, 128), (8, 0, 32), (8, -1, 32),
         (8, 0, 2048), (8, -1, 2048), (8, 0, 2049),                 # a warp or a block, many rows
         (0, 51, 4096), (0, 52, 4096), (0, 51, 4095),               # a cluster or a block
         (16, 0, 64), (16, -1, 64), (16, 0, 65),                    # backward: 8 threads or a warp
         (8, 0, 65), (8, -1, 65), (8, 0, 1024), (8, 0, 1025), (0, 40, 64), (0, 40, 65)]     # a warp or a block


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("worth,more,vectors", RULES)
@pytest.mark.parametrize("odd", [0, 1])
def test_both_sides_of_the_rules(pvl, dtype, worth, more, vectors, odd):
    """Whole vectors, and one vector's elements more but one (odd rows lie at every alignment)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    wide = 8 if dtype == torch.bfloat16 else 4
    N, V = worth * sms + more, vectors * wide + odd * (wide - 1)
    x = (randn(1, N, V, seed=V) * 3).to(dtype)
    t = torch.randint(0, V, (1, N), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda")
    up, ue = randn(1, N, seed=1), randn(1, N, seed=2)
    logp, lse, h = pvl.pack_logprob_fwd(x, t, entropy=True)
    d = pvl.pack_logprob_bwd(up, x, t, lse, ent=h, dent=ue)
    rel = 2.0 ** -20 + V / threads(N, V // wide) * 2.0 ** -24
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    rows = range(0, N, 1000) if N > 1000 else (0,)
    for i in rows:
        at = slice(i, min(i + 1000, N))
        z = x[0, at].double()
        s = torch.logsumexp(z, 1)
        logs = z - s[:, None]
        p = logs.exp()
        pick = t[0, at, None]
        want = logs.gather(1, pick)[:, 0]
        ent = -(p * logs).sum(1)
        tol = rel + 2.0 ** -22 * (z.abs().amax(1) + s.abs())
        assert ((logp[0, at] - want).abs() <= tol + 2.0 ** -22 * want.abs()).all()
        assert ((lse[0, at] - s).abs() <= tol).all()
        assert ((h[0, at] - ent).abs() <= rel * (4 + 2 * math.log(V)) + 2.0 ** -22 * ent).all()
        g, ge = up[0, at, None].double(), ue[0, at, None].double()
        grad = -p * (g + ge * (logs + ent[:, None]))
        grad.scatter_add_(1, pick, g)
        slack = p * (tol[:, None] + 2.0 ** -22 * (2 + logs.abs())) * (g.abs() + ge.abs() * (logs.abs() + ent[:, None] + 2))
        assert ((d[0, at].double() - grad).abs() <= unit * grad.abs() + slack + 2.0 ** -120).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 511, 512, 1023, 1024, 1025, 8191, 8192, 8193])
@pytest.mark.parametrize("start", [0, 1, 4])
def test_norm_around_its_unit(pvl, dtype, n, start):
    """A warp's unit is 1024 elements, a block's turn eight of them; starts on and off a boundary; parts of zeros."""
    buf = randn(3 * n + 16, seed=n).to(dtype)
    grads = [buf[start:start + n], buf[start + n:start + 2 * n], torch.zeros(n, dtype=dtype, device="cuda")]
    grads[1][n // 2:] = 0.0
    ref = oa.grad_norm([g.double().cpu().numpy() for g in grads])
    assert abs(pvl.grad_norm(grads).item() - ref) <= 2.0 ** -19 * ref
