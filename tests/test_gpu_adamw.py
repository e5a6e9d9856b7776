"""grad_norm and adamw_step against the fp64 oracle (GPU).

Tolerances, from the arithmetic: a moment is a multiply-add of two products (three
roundings of at most |b1 m| + |c1 g|, coefficients rounded once): 2^-21 of that
sum; the update carries that over its denominator, and from exp, root, quotient
and rate 2^-19 of itself; the parameter two roundings of itself (2^-22).  bf16
parameters are rounded once (2^-8).  The norm adds fp32 squares 64 or fewer at a
time: 2^-18."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

SHAPES = [(1,), (7,), (256,), (257,), (3, 5, 11), (64, 129), (1000,), (8,), (2048,), (33, 255)]


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def to_np(t):
    return t.detach().double().cpu().numpy()


def tensors(shapes, dtype, seed, mul=1.0, flat=False):
    """Separate tensors, or neighbours in one buffer at whatever alignment they come to."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sizes = [math.prod(s) for s in shapes]
    if not flat:
        return [(torch.randn(s, generator=g, device="cuda") * mul).to(dtype) for s in shapes]
    buf = (torch.randn(sum(sizes) + 1, generator=g, device="cuda") * mul).to(dtype)
    return [part.view(s) for part, s in zip(buf[1:].split(sizes), shapes)]


def fill(state, seed, t):
    """Moments as they are in the middle of training."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i, shape in enumerate(state.shapes):
        n, at = math.prod(shape), state.blocks[i] * 256
        m = torch.randn(n, generator=g, device="cuda") * 1e-2
        v = torch.rand(n, generator=g, device="cuda") * 1e-3
        if state.bits == 8:
            whole = -(-n // 256) * 256
            um, uv = oa.chances(np.arange(state.blocks[i], state.blocks[i] + whole // 256), 0, 3)
            for key, x, u in (("m", m, um), ("v", v.sqrt(), uv)):
                rows = np.zeros(whole)
                rows[:n] = to_np(x)
                code, scale, _ = oa.encode(rows.reshape(-1, 256), u, key == "v")
                getattr(state, key)[at:at + whole] = torch.from_numpy(code.reshape(-1)).cuda().to(torch.float8_e4m3fn)
                getattr(state, key + "_scale")[state.blocks[i]:][:whole // 256] = torch.from_numpy(scale).cuda().float()
        else:
            state.m[at:at + n], state.v[at:at + n] = m, v
    state.steps.fill_(t)


def check(pvl, params, grads, state, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, decay=0.01, norm=None, max_norm=None):
    """One step, and everything it writes against the oracle."""
    decays = [decay] * len(params) if isinstance(decay, float) else decay
    p0 = [to_np(state.masters(i)) if state.master is not None else to_np(p) for i, p in enumerate(params)]
    before = [tuple(to_np(t) for t in state.moments(i)) for i in range(len(params))]
    steps = state.steps.cpu().numpy().copy()
    clip = 1.0
    if norm is not None and max_norm is not None and norm.item() > max_norm:
        clip = max_norm / norm.item()
    pvl.adamw_step(params, grads, state, lr, betas=betas, eps=eps, weight_decay=decay, grad_norm=norm, max_norm=max_norm)
    torch.cuda.synchronize()
    lr = lr.item() if isinstance(lr, torch.Tensor) else lr
    for i, (p, g) in enumerate(zip(params, grads)):
        if g is None:
            assert state.steps[i].item() == steps[i]
            continue
        t = int(steps[i]) + 1
        assert state.steps[i].item() == t
        m0, v0 = before[i]
        want, m, v, change = oa.step(p0[i], to_np(g), m0, v0, t, lr, betas, eps, decays[i], clip)
        size = np.abs(betas[0] * m0) + np.abs((1 - betas[0]) * clip * to_np(g))
        denom = np.sqrt(v / (1 - betas[1] ** t)) + eps
        tol = 2.0 ** -22 * np.abs(p0[i]) + 2.0 ** -19 * np.abs(change) + abs(lr) / (1 - betas[0] ** t) * 2.0 ** -21 * size / denom
        got = to_np(state.masters(i)) if state.master is not None else to_np(p)
        assert (np.abs(got - want) <= tol + 1e-38).all(), (i, np.abs(got - want).max())
        if state.master is not None:
            assert torch.equal(p, state.masters(i).to(torch.bfloat16))
        if state.bits == 32:
            gm, gv = state.moments(i)
            assert (np.abs(to_np(gm) - m) <= 2.0 ** -21 * size + 1e-38).all()
            assert (np.abs(to_np(gv) - v) <= 2.0 ** -21 * v + 1e-38).all()
        else:
            n = math.prod(state.shapes[i])
            whole = -(-n // 256) * 256
            b = np.arange(state.blocks[i], state.blocks[i] + whole // 256)
            um, uv = oa.chances(b, t, state.seed)
            for key, x, u, err in (("m", m, um, 2.0 ** -21 * size), ("v", np.sqrt(v), uv, 2.0 ** -20 * np.sqrt(v))):
                rows, slack = np.zeros(whole), np.zeros(whole)
                rows[:n], slack[:n] = x.reshape(-1), err.reshape(-1)
                rows, slack = rows.reshape(-1, 256), slack.reshape(-1, 256)
                code, scale, near = oa.encode(rows, u, key == "v")
                got = to_np(getattr(state, key)[b[0] * 256:][:whole]).reshape(-1, 256)
                gs = to_np(getattr(state, key + "_scale")[b[0]:][:len(b)])
                assert (np.abs(gs - scale) <= 2.0 ** -19 * scale).all()
                step = oa.e4m3_step(rows / np.where(scale > 0, scale, 1)[:, None])
                # where the value and its scale could be off far enough to round the other way, by one step
                loose = near * step * np.where(scale > 0, scale, 1)[:, None] <= slack + np.abs(rows) * 2.0 ** -18 + scale[:, None] * 2.0 ** -26
                off = np.abs(got - code)
                assert not off[~loose].any(), (i, key, off[~loose].max())
                assert (off <= 1.001 * step).all()
                assert loose.mean() < 0.05 or n < 300
    # nothing past the end of a tensor
    for i, shape in enumerate(state.shapes):
        n = math.prod(shape)
        for t in (state.m, state.v) + ((state.master,) if state.master is not None else ()):
            assert not t[state.blocks[i] * 256 + n:][:-n % 256].float().any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("flat", [False, True])
def test_step(pvl, bits, param, grad, flat):
    params = tensors(SHAPES, param, 1, flat=flat)
    grads = tensors(SHAPES, grad, 2, 1e-2, flat=flat)
    state = pvl.adamw_state(params, bits=bits, seed=11)
    for _ in range(2):          # from zero moments
        check(pvl, params, grads, state)
    fill(state, 3, 500)
    check(pvl, params, grads, state, betas=(0.8, 0.95), eps=1e-6, decay=[0.1 * (i % 3) for i in range(len(SHAPES))])
    norm = pvl.grad_norm(grads)
    check(pvl, params, grads, state, norm=norm, max_norm=0.5 * norm.item())
    check(pvl, params, grads, state, norm=norm, max_norm=2.0 * norm.item())
    check(pvl, params, grads, state, norm=norm)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(pvl, bits):
    """Both sides of what a launch takes: 32 and 512 tensors, and several launches."""
    for n in (32, 33, 512, 513, 1100):
        shapes = [SHAPES[i % len(SHAPES)] for i in range(n)]
        params, grads = tensors(shapes, torch.float32, n), tensors(shapes, torch.bfloat16, n + 1)
        state = pvl.adamw_state(params, bits=bits)
        once = [i for i in range(0, n, 97)]
        some = [None if i in once else g for i, g in enumerate(grads)]
        pvl.adamw_step(params, some, state, 1e-3)
        pvl.adamw_step(params, grads, state, 1e-3)
        torch.cuda.synchronize()
        want = [1 if i in once else 2 for i in range(n)]
        assert state.steps.tolist() == want and state.done.item() == 0
        # the same parameters one at a time
        for i in (0, 1, 31, n - 2, n - 1):
            p = tensors(shapes, torch.float32, n)[i]
            alone = pvl.adamw_state([p], bits=bits)
            for _ in range(want[i]):
                pvl.adamw_step([p], [grads[i]], alone, 1e-3)
            if bits == 32 or want[i] == 1:
                assert torch.equal(p, params[i])
        norm = pvl.grad_norm(grads)
        ref = oa.grad_norm([to_np(g) for g in grads])
        assert abs(norm.item() - ref) <= 2.0 ** -18 * ref


def test_a_gradient_that_is_not_there_and_empty_parameters(pvl):
    shapes = [(5,), (0,), (300,), (0, 4)]
    params, grads = tensors(shapes, torch.float32, 4), tensors(shapes, torch.float32, 5)
    state = pvl.adamw_state(params)
    check(pvl, params, [grads[0], None, None, None], state)
    was = [p.clone() for p in params]
    pvl.adamw_step(params, [None] * 4, state, 1e-3)
    assert all(torch.equal(a, b) for a, b in zip(was, params)) and state.steps.tolist() == [1, 0, 0, 0]
    pvl.adamw_step(params, grads, state, 1e-3)
    assert state.steps.tolist() == [2, 0, 1, 0]


def test_device_rate_and_version_counters(pvl):
    params, grads = tensors(SHAPES, torch.float32, 6), tensors(SHAPES, torch.float32, 7)
    other = [p.clone() for p in params]
    a, b = pvl.adamw_state(params), pvl.adamw_state(other)
    versions = [p._version for p in params]
    pvl.adamw_step(params, grads, a, 2.0 ** -9)
    pvl.adamw_step(other, grads, b, torch.tensor([2.0 ** -9], device="cuda"))
    assert all(torch.equal(x, y) for x, y in zip(params, other))
    pvl.adamw_step(params, grads, a, np.float32(2.0 ** -9), weight_decay=np.float32(0.5), betas=np.array([0.9, 0.999]))
    pvl.adamw_step(other, grads, b, 2.0 ** -9, weight_decay=[0.5] * len(other))
    assert all(torch.equal(x, y) for x, y in zip(params, other))
    assert all(p._version > v for p, v in zip(params, versions))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_norm_that_is_not_finite_skips_the_step(pvl, bits, bad):
    params, grads = tensors(SHAPES, torch.bfloat16, 8), tensors(SHAPES, torch.bfloat16, 9)
    state = pvl.adamw_state(params, bits=bits)
    pvl.adamw_step(params, grads, state, 1e-3)
    kept = [t.clone() for t in (*params, state.m.view(torch.uint8), state.v.view(torch.uint8), state.master, state.steps)]
    grads[3].view(-1)[77] = bad
    norm = pvl.grad_norm(grads)
    assert not math.isfinite(norm.item())
    pvl.adamw_step(params, grads, state, 1e-3, grad_norm=norm, max_norm=1.0)
    now = [*params, state.m.view(torch.uint8), state.v.view(torch.uint8), state.master, state.steps]
    assert all(torch.equal(a, b) for a, b in zip(kept, now)) and state.done.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm(pvl, dtype):
    """Sizes around a warp's unit of 2048, any alignment; values whose squares leave fp32; zeros; what is not finite."""
    for n in (1, 2, 31, 2047, 2048, 2049, 4096, 100001):
        for flat in (False, True):
            grads = tensors([(n,), (3,), (n + 1,)], dtype, n, flat=flat)
            ref = oa.grad_norm([to_np(g) for g in grads])
            assert abs(pvl.grad_norm(grads).item() - ref) <= 2.0 ** -18 * ref
    for size in (1e-30, 1e-20, 1e15, 1e30):
        for n in (100, 5000):
            grads = tensors([(n,), (n,)], dtype, n, size)
            ref = oa.grad_norm([to_np(g) for g in grads])
            assert abs(pvl.grad_norm(grads).item() - ref) <= 2.0 ** -18 * ref, size
    zero = [torch.zeros(5000, dtype=dtype, device="cuda"), torch.full((4096,), -0.0, dtype=dtype, device="cuda")]
    assert pvl.grad_norm(zero).item() == 0.0
    zero[0][4999] = 2.0 ** -130
    assert pvl.grad_norm(zero).item() == 2.0 ** -130
    zero[1][0] = math.inf
    assert pvl.grad_norm(zero).item() == math.inf
    zero[1][1] = math.nan
    assert math.isnan(pvl.grad_norm(zero).item())


def test_norm_past_32_bits(pvl):
    big = torch.ones((1 << 32) + 5, dtype=torch.bfloat16, device="cuda")
    assert pvl.grad_norm([big]).item() == pytest.approx(math.sqrt((1 << 32) + 5), rel=1e-6)


def test_step_past_32_bits(pvl):
    """One tensor of 2^32 + 300 elements in 8 bits: its end like that of a small tensor with the same place."""
    n = (1 << 32) + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-300:] = torch.linspace(-1, 1, 300, device="cuda").bfloat16()
    state = pvl.adamw_state([p], bits=8)
    pvl.adamw_step([p], [g], state, 1e-2, weight_decay=0.0)
    torch.cuda.synchronize()
    _, _, _, change = oa.step(np.zeros(300), to_np(g[-300:]), np.zeros(300), np.zeros(300), 1, 1e-2, decay=0.0)
    assert (np.abs(to_np(state.master[n - 300:n]) + change) <= 2.0 ** -19 * np.abs(change)).all()
    assert not p[:-300].any() and not state.master[n:].any()
    m = state.m[n - 300:n].float() * state.m_scale[-2:].repeat_interleave(torch.tensor([256, 44], device="cuda"))
    assert (np.abs(to_np(m) - 0.1 * to_np(g[-300:])) <= 2.0 ** -3 * 0.1 * np.abs(to_np(g[-300:])) + 0.1 * 2.0 ** -9 / 448).all()


def test_eight_bits_follow_the_averages(pvl):
    """A thousand steps with gradients of one size: rounded to nearest, a code of v would never move (a step changes the
    root by 0.05 %, half a code is 3 % and more); rounded stochastically, the mean over many elements follows.  A
    rounding adds the variance s d to a root, s <= 1/8 the distance of codes and d = 0.0005 E|g^2 / v - 1| = 0.0005 the
    change of a step, both of the root: 6e-5 of v a step, forgotten at 0.001 a step, so v's mean lies up to 6 % high.
    2 % either way for the sample (65,536 elements) and what rounding does to s."""
    p = torch.zeros(65536, device="cuda")
    state = pvl.adamw_state([p], bits=8, seed=5)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in range(1000):
        pvl.adamw_step([p], [torch.randn(65536, generator=g, device="cuda") * 1e-3], state, 0.0)
    m, v = state.moments(0)
    v_true = 1e-6 * (1 - 0.999 ** 1000)
    assert 0.98 * v_true < v.mean().item() < 1.08 * v_true
    # m of noise: deviation 1e-3 sqrt(0.1 / 1.9), and none in the mean
    assert abs(m.mean().item()) < 6 * 1e-3 / math.sqrt(65536) and 0.9 < m.std().item() / (1e-3 * math.sqrt(0.1 / 1.9)) < 1.1


def test_a_state_that_is_saved_and_copied(pvl):
    """A copy of the state goes on by itself; so does one that was written to a file."""
    import copy
    import io
    for bits in (32, 8):
        sets = [tensors(SHAPES, torch.bfloat16, 30) for _ in range(3)]
        grads = tensors(SHAPES, torch.bfloat16, 31)
        state = pvl.adamw_state(sets[0], bits=bits, seed=4)
        pvl.adamw_step(sets[0], grads, state, 1e-2)
        for p in sets[1:]:
            for a, b in zip(p, sets[0]):
                a.copy_(b)
        file = io.BytesIO()
        torch.save(state, file)
        file.seek(0)
        states = [state, copy.deepcopy(state), torch.load(file, weights_only=False)]
        del state
        for p, s in zip(sets, states):
            pvl.adamw_step(p, grads, s, 1e-2)
        torch.cuda.synchronize()
        assert all(s.steps.tolist() == [2] * len(SHAPES) for s in states)
        for p, s in zip(sets[1:], states[1:]):
            assert all(torch.equal(a, b) for a, b in zip(p, sets[0]))
            assert torch.equal(s.m.view(torch.uint8), states[0].m.view(torch.uint8)) and s.m.data_ptr() != states[0].m.data_ptr()


def test_same_bits_twice(pvl):
    for bits in (32, 8):
        out = []
        for _ in range(2):
            params, grads = tensors(SHAPES, torch.bfloat16, 20), tensors(SHAPES, torch.bfloat16, 21)
            state = pvl.adamw_state(params, bits=bits, seed=9)
            for _ in range(3):
                norm = pvl.grad_norm(grads)
                pvl.adamw_step(params, grads, state, 1e-2, grad_norm=norm, max_norm=0.1)
            out.append([*params, state.m.view(torch.uint8), state.v.view(torch.uint8), norm])
        assert all(torch.equal(a, b) for a, b in zip(*out))
