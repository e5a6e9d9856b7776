"""Parameters that a program writes between the steps, that autograd does not track, or that share memory (GPU)."""

import contextlib

import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(300,), (7, 65), (1,), (256,)]


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def tensors(seed, flat=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    sizes = [torch.Size(s).numel() for s in SHAPES]
    buf = torch.randn(sum(sizes), generator=g, device="cuda").bfloat16()
    parts = [b.view(s) for b, s in zip(buf.split(sizes), SHAPES)]
    return parts if flat else [p.clone() for p in parts]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("flat", [False, True])
def test_written_parameters_are_taken_over(pvl, bits, flat):
    """A checkpoint loaded after the state was made, and again in the middle; elements that keep their value keep the
    master's lower bits."""
    params, grads = tensors(1, flat), tensors(2)
    state = pvl.adamw_state(params, bits=bits)
    loaded = tensors(3)
    with torch.no_grad():
        for p, x in zip(params, loaded):
            p.copy_(x)
    pvl.adamw_step(params, grads, state, 0.0, weight_decay=0.0)
    assert all(torch.equal(p, x) for p, x in zip(params, loaded))
    for _ in range(3):
        pvl.adamw_step(params, grads, state, 1e-4)
    kept = [state.masters(i).clone() for i in range(len(params))]
    assert any((k != p.float()).any() for k, p in zip(kept, params))
    with torch.no_grad():
        params[0][5:9] = 2.5
    kept[0][5:9] = 2.5
    pvl.adamw_step(params, grads, state, 0.0, weight_decay=0.0)
    assert all(torch.equal(state.masters(i), k) for i, k in enumerate(kept))
    assert all(torch.equal(p, k.bfloat16()) for p, k in zip(params, kept))


def test_values_that_are_put_back_change_nothing(pvl):
    """An average swapped in and out again: bit by bit as without it."""
    runs = [tensors(1), tensors(1)]
    grads = tensors(2)
    states = [pvl.adamw_state(p) for p in runs]
    for t in range(3):
        for p, s in zip(runs, states):
            pvl.adamw_step(p, grads, s, 1e-4)
        own = [p.clone() for p in runs[0]]
        for p, x in zip(runs[0], own):
            p.zero_()
            p.copy_(x)
    for p, q in zip(*runs):
        assert torch.equal(p, q)
    assert torch.equal(states[0].master, states[1].master)


def test_a_parameter_that_does_not_step_is_taken_over_when_it_does(pvl):
    params, grads = tensors(1), tensors(2)
    state = pvl.adamw_state(params)
    params[1].fill_(3.0)
    pvl.adamw_step(params, [grads[0], None, grads[2], grads[3]], state, 1e-3)
    pvl.adamw_step(params, [None, grads[1], None, None], state, 0.0, weight_decay=0.0)
    assert (params[1] == 3.0).all() and (state.masters(1) == 3.0).all()


def test_written_on_another_stream_and_in_a_graph(pvl):
    params, grads = tensors(1), tensors(2)
    state = pvl.adamw_state(params)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        params[0].fill_(1.5)
    pvl.adamw_step(params, grads, state, 0.0, weight_decay=0.0, stream=side)
    torch.cuda.synchronize()
    assert (params[0] == 1.5).all()
    params[3].fill_(0.25)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pvl.adamw_step(params, grads, state, 0.0, weight_decay=0.0)
    graph.replay()
    torch.cuda.synchronize()
    assert (params[3] == 0.25).all() and (params[0] == 1.5).all()
    assert state.steps.tolist() == [2] * 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_inference_tensors(pvl, dtype):
    """They have no version; they step like the others beside them, in inference mode and outside it."""
    def run(make, at):
        p = [torch.ones(300, dtype=dtype, device="cuda"), make(), torch.ones(5, dtype=dtype, device="cuda")]
        g = [torch.ones_like(x, dtype=torch.float32) for x in p]
        versions = [p[0]._version, p[2]._version]
        state = pvl.adamw_state(p)
        for _ in range(3):
            with at:
                pvl.adamw_step(p, g, state, 1e-2)
        assert p[0]._version > versions[0] and p[2]._version > versions[1]
        assert state.steps.tolist() == [3] * 3
        return p

    def ordinary():
        return torch.ones(70, dtype=dtype, device="cuda")

    def free():
        with torch.inference_mode():
            return ordinary()

    want = run(ordinary, contextlib.nullcontext())
    assert free().is_inference()
    for at in (contextlib.nullcontext(), torch.inference_mode(), torch.no_grad()):
        assert all(torch.equal(a, b) for a, b in zip(run(free, at), want))


def test_parameters_that_share_memory_are_refused(pvl):
    """Two warps would write the same elements; neighbours are fine."""
    buf = torch.zeros(600, device="cuda")
    for pair in ([buf[:300], buf[299:]], [buf[100:], buf[:101]], [buf, buf[256:300]], [buf[256:300], buf]):
        with pytest.raises(ValueError, match="share memory"):
            pvl.adamw_state(pair)
    pvl.adamw_state([buf[300:], buf[:300]])
    pvl.adamw_state([buf[:0], buf[:5], buf[5:5], buf[5:]])
