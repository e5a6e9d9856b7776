"""Python binding of the parameter update: the norm of all gradients and the
AdamW step over many tensors at once.

The state of an update lives in buffers over all parameters (AdamWState); a
step passes the addresses of parameters and gradients as kernel arguments and
copies nothing to the device, so it can be captured into a CUDA graph.
"""

from __future__ import annotations

import math
from array import array
from dataclasses import dataclass, field
from numbers import Real
from operator import attrgetter

import numpy as np
import torch

from . import _lib
from .api import _addr, _check, _here, _launch, _need

BLOCK = 256     # elements that share a scale of the 8-bit moments

# pvl_adamw_tensor of include/pvl.h
_TENSOR = np.dtype([("param", np.uint64), ("grad", np.uint64), ("size", np.int64), ("block", np.int64),
                    ("slot", np.int32), ("decay", np.float32)])
_FLOATS = {torch.bfloat16: 0, torch.float32: 1}


# A model has hundreds of parameters and a step looks at each: attributes of
# whole lists are read by C loops, one list at a time.
_dtype, _shape, _version = attrgetter("dtype"), attrgetter("shape"), attrgetter("_version")
_contiguous, _index, _address, _count = (torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.data_ptr,
                                         torch.Tensor.numel)


_KINDS = {torch.Tensor, torch.nn.Parameter}


def _tensors(tensors, name: str, use=None) -> None:
    if not _KINDS.issuperset(map(type, tensors)):
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"{name}[{i if use is None else use[i]}] must be a tensor")


def _same_floats(tensors, name: str):
    """The dtype and device that all of the list share; every tensor contiguous."""
    _tensors(tensors, name)
    dtype, dev = tensors[0].dtype, tensors[0].device
    if dtype not in _FLOATS:
        raise ValueError(f"{name} must be {torch.bfloat16} or {torch.float32}, got {dtype}")
    if dev.type != "cuda":
        raise ValueError(f"{name} must be CUDA tensors, got {dev}")
    if set(map(_dtype, tensors)) != {dtype} or set(map(_index, tensors)) != {tensors[0].get_device()} or (
            not all(map(_contiguous, tensors))):
        for i, t in enumerate(tensors):
            _need(t, f"{name}[{i}]", dtype, t.shape, dev)
    return dtype, dev


def grad_norm(grads, out=None, ws=None, stream=None) -> torch.Tensor:
    """fp32 [1] device tensor: the 2-norm of all gradients together (bf16 or
    fp32 tensors of one type; None and empty ones are skipped)."""
    grads = [g for g in grads if g is not None]
    dtype, dev = _same_floats(grads, "grads") if grads else (None, None)
    counts = list(map(_count, grads))
    if 0 in counts:
        grads = [g for g, n in zip(grads, counts) if n]
        counts = [n for n in counts if n]
    if not grads:
        raise ValueError("grad_norm needs a gradient")
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_norm(grads, counts, _FLOATS[dtype], dev, out, ws, handle)
    return _run_norm(grads, counts, _FLOATS[dtype], dev, out, ws, handle)


def _run_norm(grads, counts, kind, dev, out, ws, handle):
    lib = _lib.load()
    given = out is not None
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", torch.float32, (1,), dev)
    if ws is None:
        ws = torch.empty(lib.pvl_grad_norm_ws_bytes(), dtype=torch.uint8, device=dev)
    else:
        _need(ws, "ws", torch.uint8, ws.shape, dev)
    ptrs, sizes = array("Q", map(_address, grads)), array("q", counts)
    _check(lib.pvl_grad_norm(ptrs.buffer_info()[0], sizes.buffer_info()[0], len(grads), kind, out.data_ptr(),
                             ws.data_ptr(), ws.numel(), handle))
    if given:
        torch.autograd.graph.increment_version(out)
    return out


@dataclass
class AdamWState:
    """Moments, masters and step counts of the parameters that adamw_state was
    given, in whole blocks of 256 elements a parameter.

    bits 32: m and v are fp32.  bits 8: they are torch.float8_e4m3fn, with one
    fp32 scale a block, and v holds the root: m = code m_scale, sqrt(v) = code
    v_scale, infinite where v's code is NaN and m's is not.  Rounding leaves m
    without bias and raises the mean of v by up to 6 % (betas[1] 0.999): steps are
    up to 3 % shorter than with 32 bits.  master holds bf16 parameters in fp32
    (None for fp32 ones)."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None
    v_scale: torch.Tensor | None
    master: torch.Tensor | None
    steps: torch.Tensor         # int32, one a parameter
    done: torch.Tensor          # int32 [1], the kernels' own: 0 between steps
    bits: int
    seed: int
    dtype: torch.dtype          # of the parameters
    shapes: tuple
    blocks: tuple               # first block of each parameter
    total: int                  # blocks
    empty: bool                 # whether a parameter has no elements
    table: np.ndarray = field(repr=False)
    versions: list | None = None    # of bf16 parameters, as of their masters

    def _part(self, t, i: int):
        n = math.prod(self.shapes[i])
        return t[self.blocks[i] * BLOCK:][:n]

    def moments(self, i: int):
        """(m, v) of parameter i in fp32, of its shape."""
        m, v = self._part(self.m, i).float(), self._part(self.v, i).float()
        if self.bits == 8:
            at = torch.arange(m.numel(), device=m.device) // BLOCK + self.blocks[i]
            m, v = m * self.m_scale[at], (v * self.v_scale[at]).square()
            v = torch.where(v.isnan() & m.isfinite(), math.inf, v)
        return m.view(self.shapes[i]), v.view(self.shapes[i])

    def masters(self, i: int):
        """The fp32 master of bf16 parameter i: a view of its shape."""
        return self._part(self.master, i).view(self.shapes[i])


def adamw_state(params, *, bits: int = 32, seed: int = 0) -> AdamWState:
    """State of AdamW for a list of parameters, all bf16 or all fp32: moments of
    zero in 32 or 8 bits, step counts of zero and, for bf16 parameters, fp32
    masters that start as their values.  seed chooses the random bits by which
    8-bit moments are rounded.

    Steps go from the masters and write the parameters.  A bf16 parameter that a
    program writes in between (a loaded checkpoint, say) is found by its version
    when it next steps: its master takes each value that is not the rounded
    master's already.  Writes that torch does not count, through .data or
    between replays of a captured step, are lost unless they go to masters(i)
    too."""
    params = list(params)
    if not params:
        raise ValueError("adamw_state needs a parameter")
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits!r}")
    if not 0 <= int(seed) < 1 << 32:
        raise ValueError("seed must fit in 32 bits")
    dtype, dev = _same_floats(params, "params")
    _apart([p for p in params if p.numel()])       # empty ones have no address
    table = np.zeros(len(params), dtype=_TENSOR)
    table["size"] = [p.numel() for p in params]
    table["slot"] = np.arange(len(params))
    counts = -(-table["size"] // BLOCK)
    ends = np.cumsum(counts)
    table["block"] = ends - counts
    total = int(ends[-1])
    moment = torch.float32 if bits == 32 else torch.uint8
    m, v = (torch.zeros(total * BLOCK, dtype=moment, device=dev) for _ in range(2))
    scales = (None, None)
    if bits == 8:
        m, v = m.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        scales = tuple(torch.zeros(total, dtype=torch.float32, device=dev) for _ in range(2))
    state = AdamWState(m, v, *scales, None, torch.zeros(len(params), dtype=torch.int32, device=dev),
                       torch.zeros(1, dtype=torch.int32, device=dev), bits, int(seed), dtype,
                       tuple(tuple(p.shape) for p in params), tuple(int(b) for b in table["block"]), total,
                       not table["size"].all(), table)
    if dtype is torch.bfloat16:
        state.master = torch.zeros(total * BLOCK, dtype=torch.float32, device=dev)
        for i, p in enumerate(params):
            state.masters(i).copy_(p.detach())
        state.versions = _versions(params)
    return state


def _versions(params) -> list:
    """Version of each parameter, None for what has none (tensors of inference mode)."""
    try:
        return list(map(_version, params))
    except RuntimeError:
        return [None if p.is_inference() else p._version for p in params]


def _take_written(state: AdamWState, params, use) -> None:
    """Masters of the parameters that were written since their last step, on the current stream: values that differ
    from the rounded master's are taken, the others keep the master's lower bits."""
    for i, p, version in zip(range(len(params)) if use is None else use, params, _versions(params)):
        if version != state.versions[i]:
            for master, value in zip(*(t.detach().reshape(-1).split(1 << 28) for t in (state.masters(i), p))):
                torch.where(master.to(torch.bfloat16) == value, master, value.float(), out=master)


def _keep_versions(state: AdamWState, params, use) -> None:
    if use is None:
        state.versions = _versions(params)
    else:
        for i, version in zip(use, _versions(params)):
            state.versions[i] = version


def _like(tensors, name: str, use, dtype, shapes, dev) -> None:
    """Every tensor of the list has the dtype, its shape and the device, and is contiguous; `use`: their places."""
    _tensors(tensors, name, use)
    if set(map(_dtype, tensors)) != {dtype} or set(map(_index, tensors)) != {dev.index} or (
            not all(map(_contiguous, tensors)) or list(map(_shape, tensors)) != list(shapes)):
        for i, (t, shape) in enumerate(zip(tensors, shapes)):
            _need(t, f"{name}[{i if use is None else use[i]}]", dtype, shape, dev)


def _apart(params) -> None:
    """No two of the tensors share memory, which a step would write twice, in any order."""
    _distinct(list(map(_address, params)))
    end = 0
    for start, size in sorted((p.data_ptr(), p.numel() * p.element_size()) for p in params):
        if start < end:
            raise ValueError("two parameters of the list share memory")
        end = start + size


def _distinct(ptrs):
    if len(set(ptrs)) != len(ptrs):
        raise ValueError("a parameter stands in the list twice")


def adamw_step(params, grads, state: AdamWState, lr, *, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
               grad_norm=None, max_norm: float | None = None, stream=None) -> None:
    """One AdamW step of `params` (the list that adamw_state was given) from
    `grads` (bf16 or fp32, of one type, each like its parameter; None leaves
    the parameter, its moments and its step count as they are).

    bf16 parameters step from their fp32 masters; values that were written to
    them since (see adamw_state) are taken over first.

    lr is a number or an fp32 one-element device tensor (read when the kernel
    runs); weight_decay a number or one a parameter, decoupled.  With grad_norm
    (the device tensor of grad_norm()) the gradients are scaled by min(1,
    max_norm / grad_norm), or with max_norm=None not at all, and a norm that is
    NaN or infinite leaves everything as it is."""
    params, grads = list(params), list(grads)
    n = len(state.shapes)
    if len(params) != n or len(grads) != n:
        raise ValueError(f"the state is of {n} parameters, got {len(params)} and {len(grads)} gradients")
    dev = state.m.device
    if betas is None or len(betas) != 2:
        raise ValueError("betas must be two numbers")
    blocks, elements = (state.total,), (state.total * BLOCK,)
    if state.bits == 32:
        parts = (("m", torch.float32, elements), ("v", torch.float32, elements))
    else:
        parts = (("m", torch.float8_e4m3fn, elements), ("v", torch.float8_e4m3fn, elements),
                 ("m_scale", torch.float32, blocks), ("v_scale", torch.float32, blocks))
    if state.dtype is torch.bfloat16:
        parts += (("master", torch.float32, elements),)
    for name, dtype, shape in parts + (("steps", torch.int32, (n,)), ("done", torch.int32, (1,))):
        t = getattr(state, name)
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != dev or (
                not t.is_contiguous()):
            _need(t, f"state.{name}", dtype, shape, dev)
    if grad_norm is not None:
        _need(grad_norm, "grad_norm", torch.float32, (1,), dev)
    elif max_norm is not None:
        raise ValueError("max_norm needs grad_norm")
    lr_dev = None
    if isinstance(lr, torch.Tensor):
        if lr.numel() != 1:
            raise ValueError("lr must hold one element")
        _need(lr, "lr", torch.float32, lr.shape, dev)
        lr, lr_dev = 0.0, lr
    use = None      # which parameters step: None for all
    if state.empty or type(None) in set(map(type, grads)):
        use = [i for i, g in enumerate(grads) if g is not None and state.table["size"][i]]
        if not use:
            return
    some_params = params if use is None else [params[i] for i in use]
    some_grads = grads if use is None else [grads[i] for i in use]
    some_shapes = state.shapes if use is None else [state.shapes[i] for i in use]
    _like(some_params, "params", use, state.dtype, some_shapes, dev)
    kind = some_grads[0].dtype if isinstance(some_grads[0], torch.Tensor) else None
    if kind not in _FLOATS:
        raise ValueError(f"grads must be {torch.bfloat16} or {torch.float32} tensors, got {kind}")
    _like(some_grads, "grads", use, kind, some_shapes, dev)
    table = state.table if use is None else state.table[use]
    addresses = list(map(_address, some_params))
    _distinct(addresses)
    table["param"] = addresses
    table["grad"] = list(map(_address, some_grads))
    if isinstance(weight_decay, Real):
        table["decay"] = weight_decay
    else:
        decay = [float(d) for d in weight_decay]
        if len(decay) != n:
            raise ValueError(f"weight_decay must be a number or {n} of them")
        table["decay"] = decay if use is None else [decay[i] for i in use]
    how = _lib.PACK_ADAMW(_FLOATS[state.dtype], _FLOATS[kind], state.bits, state.seed, float(betas[0]),
                          float(betas[1]), float(lr), float(eps), math.inf if max_norm is None else float(max_norm),
                          _addr(lr_dev), _addr(grad_norm), state.m.data_ptr(), state.v.data_ptr(),
                          _addr(state.m_scale), _addr(state.v_scale), _addr(state.master), state.steps.data_ptr(),
                          state.done.data_ptr())
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            _run_step(how, table, state, some_params, use, handle)
    else:
        _run_step(how, table, state, some_params, use, handle)


def _run_step(how, table, state, params, use, handle):
    tracked = state.versions is not None
    if tracked and (use is not None or _versions(params) != state.versions):
        _take_written(state, params, use)
    _check(_lib.load().pvl_adamw_step(how, table.ctypes.data, len(table), handle))
    torch.autograd.graph.increment_version(params)
    if tracked:
        _keep_versions(state, params, use)
