"""Python binding of libpvl: argument marshalling only.

Every function checks shapes/dtypes, allocates outputs with torch on the
tensors' CUDA device when the caller passes none, and calls the C entry point
of the same name on the current torch stream.  All arithmetic runs in the
library's CUDA kernels; nothing here computes attention, seq_ids or tile maps.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
from dataclasses import dataclass
from decimal import Decimal, localcontext
from typing import NamedTuple

import numpy as np
import torch

from . import _lib

PVL_OK, PVL_ERR_INVALID_ARG, PVL_ERR_UNSUPPORTED, PVL_ERR_CUDA, PVL_ERR_TIMEOUT = range(5)
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}

TM_LEVELS = 2
TM_FIELDS = ["header", "q_nv", "q_lo", "q_hi", "k_nv", "k_lo", "k_hi", "cls", "row_count", "row_full",
             "row_list", "col_count", "col_full", "col_list", "q_order", "k_order"]
EMPTY, PARTIAL, FULL = 0, 1, 2


class PvlError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pvl {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(status: int) -> None:
    if status != PVL_OK:
        raise PvlError(status, _lib.load().pvl_last_error_message().decode())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need_cuda(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, name: str, dtype: torch.dtype, shape, device: torch.device) -> None:
    """_need_cuda, on a given device, at the price of a few attribute reads where all is well."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape and (
            t.is_contiguous()):
        return
    _need_cuda(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, not on {device}")


_current_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Here:
    """The current device and stream: nothing to set, nothing to restore."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


@contextlib.contextmanager
def _there(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(_stream(stream))
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _launch(device, stream):
    """Context that makes the device current and, with a stream given, that
    stream, so that what is allocated inside belongs to the stream the kernels
    run on; gives the stream's handle.  A device that is not CUDA is refused."""
    if device.type != "cuda":
        raise ValueError(f"the kernels run on CUDA devices, not on {device}")
    if stream is None:
        index = torch.cuda.current_device()
        if device.index is None or device.index == index:
            return _Here(_current_stream_handle(index))
    return _there(device, stream)


# ------------------------------------------------------------------ seq_ids
def pack_build_seq_ids(seg_frames, seg_valid, tokens_per_frame: int, L: int, out: torch.Tensor | None = None,
                       device=None, stream=None) -> torch.Tensor:
    """int32 [B, L] seq_id on the GPU from host [B, K] frame / valid-frame tables."""
    frames = np.ascontiguousarray(np.asarray(seg_frames, dtype=np.int32))
    valid = np.ascontiguousarray(np.asarray(seg_valid, dtype=np.int32))
    if frames.ndim != 2 or frames.shape != valid.shape:
        raise ValueError("seg_frames and seg_valid must both be [B, K]")
    B, K = frames.shape
    if out is None:
        out = torch.empty((B, L), dtype=torch.int32, device=device or "cuda")
    _need_cuda(out, "out", torch.int32, (B, L))
    with torch.cuda.device(out.device):
        _check(_lib.load().pack_build_seq_ids(frames.ctypes.data, valid.ctypes.data, B, K, int(tokens_per_frame),
                                              int(L), out.data_ptr(), _stream(stream)))
    return out


def pack_build_positions(seg_frames, tokens_per_frame: int, L: int, axes: int = 1, row_width: int | None = None,
                         out: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """int32 [B, L, axes] position of each token inside its packed segment,
    from the host [B, K] frame table: its offset (axes=1), its frame and its
    token of the frame (2), or its frame, row and column with row_width tokens
    a row (3).  Positions restart in every segment; the tail gets zeros."""
    frames = np.asarray(seg_frames, dtype=np.int32)
    if frames.ndim != 2:
        raise ValueError("seg_frames must be [B, K]")
    if axes == 3 and (row_width is None or int(row_width) < 1):
        raise ValueError(f"three axes need a row_width of at least 1, got {row_width}")
    B, K = frames.shape
    device = torch.device(device or "cuda") if out is None else out.device
    with _launch(device, stream) as handle:
        if out is None:
            out = torch.empty((B, int(L), int(axes)), dtype=torch.int32, device=device)
        else:
            _need_cuda(out, "out", torch.int32, (B, int(L), int(axes)))
        _check(_lib.load().pack_build_positions(frames.tobytes(), B, K, int(tokens_per_frame), int(axes),
                                                int(row_width) if axes == 3 else 1, int(L), out.data_ptr(), handle))
    return out


# ----------------------------------------------------------------- tile map
@dataclass
class TileMap:
    """Device workspace written by tile_map_build plus typed views of its arrays.

    Level 0 is the map at (block_m, block_n); level 1 the map at
    (2 * block_m, block_n) over pairs of query tiles.  L is the query length,
    Lk the key length (equal for self attention)."""
    ws: torch.Tensor
    B: int
    L: int
    block_m: int
    block_n: int
    offsets: tuple  # LEVELS * len(TM_FIELDS) byte offsets
    Lk: int = 0     # 0: same as L

    def __post_init__(self):
        if not self.Lk:
            self.Lk = self.L

    def blocks(self, level: int = 0):
        return (self.block_m * (2 if level else 1), self.block_n)

    def n_tiles(self, level: int = 0):
        bm, bn = self.blocks(level)
        return -(-self.L // bm), -(-self.Lk // bn)

    @property
    def nTq(self) -> int:
        return self.n_tiles(0)[0]

    @property
    def nTk(self) -> int:
        return self.n_tiles(0)[1]

    def field(self, name: str, level: int = 0) -> torch.Tensor:
        i = TM_FIELDS.index(name)
        B = self.B
        nq, nk = self.n_tiles(level)
        shapes = {"header": (16,), "q_nv": (B, nq), "q_lo": (B, nq), "q_hi": (B, nq), "k_nv": (B, nk),
                  "k_lo": (B, nk), "k_hi": (B, nk), "cls": (B, nq, nk), "row_count": (B, nq),
                  "row_full": (B, nq), "row_list": (B, nq, nk), "col_count": (B, nk), "col_full": (B, nk),
                  "col_list": (B, nk, nq), "q_order": (B * nq,), "k_order": (B * nk,)}
        shape = shapes[name]
        n = int(np.prod(shape))
        off = self.offsets[level * len(TM_FIELDS) + i]
        if name == "cls":
            return self.ws[off:off + n].view(shape)
        return self.ws[off:off + 4 * n].view(torch.int32).view(shape)

    def to_host(self, level: int = 0) -> dict:
        out = {name: self.field(name, level).cpu().numpy() for name in TM_FIELDS}
        bm, bn = self.blocks(level)
        nq, nk = self.n_tiles(level)
        out.update(B=self.B, L=self.L, Lk=self.Lk, block_m=bm, block_n=bn, nTq=nq, nTk=nk)
        return out


def tile_map_ws_bytes(B: int, L: int, block_m: int = 128, block_n: int = 128, Lk: int | None = None) -> int:
    if Lk is None:
        return int(_lib.load().tile_map_ws_bytes(B, L, block_m, block_n))
    return int(_lib.load().tile_map_ws_bytes_cross(B, L, Lk, block_m, block_n))


def tile_map_build(seq_id: torch.Tensor, block_m: int = 128, block_n: int = 128,
                   ws: torch.Tensor | None = None, stream=None, k_seq_id: torch.Tensor | None = None) -> TileMap:
    """Tile map of the seq_id mask; with k_seq_id (int32 [B, Lk]) the
    cross-attention map of queries with ids seq_id against keys with ids
    k_seq_id."""
    lib = _lib.load()
    if seq_id.dim() != 2:
        raise ValueError("seq_id must be [B, L]")
    _need_cuda(seq_id, "seq_id", torch.int32)
    B, L = seq_id.shape
    Lk = L
    if k_seq_id is not None:
        if k_seq_id.dim() != 2 or k_seq_id.shape[0] != B:
            raise ValueError("k_seq_id must be [B, Lk]")
        _need_cuda(k_seq_id, "k_seq_id", torch.int32)
        Lk = k_seq_id.shape[1]
    nbytes = int(lib.tile_map_ws_bytes_cross(B, L, Lk, block_m, block_n))
    if nbytes == 0:
        raise PvlError(PVL_ERR_INVALID_ARG, "bad tile map sizes")
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=seq_id.device)
    offs = (ctypes.c_size_t * (TM_LEVELS * len(TM_FIELDS)))()
    with torch.cuda.device(seq_id.device):
        if k_seq_id is None:
            _check(lib.tile_map_layout(B, L, block_m, block_n, ctypes.addressof(offs)))
            _check(lib.tile_map_build(seq_id.data_ptr(), B, L, block_m, block_n, ws.data_ptr(), ws.numel(),
                                      _stream(stream)))
        else:
            _check(lib.tile_map_layout_cross(B, L, Lk, block_m, block_n, ctypes.addressof(offs)))
            _check(lib.tile_map_build_cross(seq_id.data_ptr(), k_seq_id.data_ptr(), B, L, Lk, block_m, block_n,
                                            ws.data_ptr(), ws.numel(), _stream(stream)))
    return TileMap(ws, B, L, block_m, block_n, tuple(offs), Lk)


# ---------------------------------------------------------------- attention
def _qkv_shape(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("q must be [B, L, H, D]")
    return tuple(q.shape)


def _key_side(q, k, seq_id, k_seq_id, tile_map):
    """Checks the key-side shapes; returns (Lk, key ids)."""
    B, L, H, D = _qkv_shape(q)
    Lk = L if k_seq_id is None else int(k.shape[1]) if k.dim() == 4 else -1
    _need_cuda(seq_id, "seq_id", torch.int32, (B, L))
    if k_seq_id is not None:
        _need_cuda(k_seq_id, "k_seq_id", torch.int32, (B, Lk))
    if (tile_map.B, tile_map.L, tile_map.Lk) != (B, L, Lk):
        raise ValueError("tile map was built for another [B, Lq, Lk]")
    return Lk, (seq_id if k_seq_id is None else k_seq_id)


def masked_attn_fwd(q, k, v, seq_id, tile_map: TileMap, scale: float | None = None, o=None, lse=None,
                    stream=None, k_seq_id=None):
    """(O bf16 [B, L, H, D], LSE fp32 [B, H, L]) of seq_id-masked softmax attention.

    With k_seq_id (int32 [B, Lk]) it is cross attention: k and v are
    [B, Lk, H, D] and query i attends key j iff seq_id[i] == k_seq_id[j] >= 0."""
    B, L, H, D = _qkv_shape(q)
    Lk, kid = _key_side(q, k, seq_id, k_seq_id, tile_map)
    _need_cuda(q, "q", torch.bfloat16, (B, L, H, D))
    for name, t in (("k", k), ("v", v)):
        _need_cuda(t, name, torch.bfloat16, (B, Lk, H, D))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _need_cuda(o, "o", torch.bfloat16, (B, L, H, D))
    _need_cuda(lse, "lse", torch.float32, (B, H, L))
    lib = _lib.load()
    with torch.cuda.device(q.device):
        if k_seq_id is None:
            _check(lib.masked_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), seq_id.data_ptr(),
                                       tile_map.ws.data_ptr(), B, L, H, D, scale, o.data_ptr(), lse.data_ptr(),
                                       _stream(stream)))
        else:
            _check(lib.masked_attn_fwd_cross(q.data_ptr(), k.data_ptr(), v.data_ptr(), seq_id.data_ptr(),
                                             kid.data_ptr(), tile_map.ws.data_ptr(), B, L, Lk, H, D, scale,
                                             o.data_ptr(), lse.data_ptr(), _stream(stream)))
    return o, lse


def masked_attn_bwd_ws_bytes(B: int, L: int, H: int, D: int, Lk: int | None = None) -> int:
    if Lk is None:
        return int(_lib.load().masked_attn_bwd_ws_bytes(B, L, H, D))
    return int(_lib.load().masked_attn_bwd_ws_bytes_cross(B, L, Lk, H, D))


def masked_attn_bwd(q, k, v, o, do, lse, seq_id, tile_map: TileMap, scale: float | None = None, dq=None,
                    dk=None, dv=None, ws=None, stream=None, k_seq_id=None):
    """(dQ, dK, dV) of the masked attention, from the saved LSE: dQ like q,
    dK and dV like k (cross attention with k_seq_id, as masked_attn_fwd)."""
    B, L, H, D = _qkv_shape(q)
    Lk, kid = _key_side(q, k, seq_id, k_seq_id, tile_map)
    for name, t in (("q", q), ("o", o), ("do", do)):
        _need_cuda(t, name, torch.bfloat16, (B, L, H, D))
    for name, t in (("k", k), ("v", v)):
        _need_cuda(t, name, torch.bfloat16, (B, Lk, H, D))
    _need_cuda(lse, "lse", torch.float32, (B, H, L))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    _need_cuda(dq, "dq", torch.bfloat16, (B, L, H, D))
    for name, t in (("dk", dk), ("dv", dv)):
        _need_cuda(t, name, torch.bfloat16, (B, Lk, H, D))
    lib = _lib.load()
    nbytes = int(lib.masked_attn_bwd_ws_bytes_cross(B, L, Lk, H, D))
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        if k_seq_id is None:
            _check(lib.masked_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                       lse.data_ptr(), seq_id.data_ptr(), tile_map.ws.data_ptr(), B, L, H, D,
                                       scale, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(),
                                       ws.numel(), _stream(stream)))
        else:
            _check(lib.masked_attn_bwd_cross(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                             lse.data_ptr(), seq_id.data_ptr(), kid.data_ptr(),
                                             tile_map.ws.data_ptr(), B, L, Lk, H, D, scale, dq.data_ptr(),
                                             dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), ws.numel(),
                                             _stream(stream)))
    return dq, dk, dv


def masked_attn_bwd_no_alloc(q, k, v, o, do, lse, seq_id, tile_map: TileMap, scale: float | None = None,
                             dq=None, dk=None, dv=None, stream=None):
    """masked_attn_bwd without a workspace argument, for callers that must not
    allocate device memory: the scratch is the library's own static device
    array (limit PVL_NO_ALLOC_SCRATCH_BYTES).  Pass dq/dk/dv to avoid the
    output allocations too.  Calls that overlap on the GPU share that scratch
    and must be serialised."""
    B, L, H, D = _qkv_shape(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _need_cuda(t, name, torch.bfloat16, (B, L, H, D))
    _need_cuda(lse, "lse", torch.float32, (B, H, L))
    _need_cuda(seq_id, "seq_id", torch.int32, (B, L))
    if (tile_map.B, tile_map.L) != (B, L):
        raise ValueError("tile map was built for another [B, L]")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need_cuda(t, name, torch.bfloat16, (B, L, H, D))
    with torch.cuda.device(q.device):
        _check(_lib.load().masked_attn_bwd_no_alloc(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
            seq_id.data_ptr(), tile_map.ws.data_ptr(), B, L, H, D, scale, dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), _stream(stream)))
    return dq, dk, dv


# -------------------------------------------------------------------- AdaLN
def adaln_fwd(x, shift, scale, eps: float = 1e-6, y=None, stats: bool = False, stream=None):
    """y = layer_norm(x) * (1 + scale) + shift ("AdaptiveLoad" §2.B): x bf16
    [B, N, D], shift / scale fp32 [B, D].  Returns y, or (y, mean, rstd) with
    stats=True."""
    if x.dim() != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = x.shape
    _need_cuda(x, "x", torch.bfloat16, (B, N, D))
    _need_cuda(shift, "shift", torch.float32, (B, D))
    _need_cuda(scale, "scale", torch.float32, (B, D))
    y = torch.empty_like(x) if y is None else y
    _need_cuda(y, "y", torch.bfloat16, (B, N, D))
    mean = rstd = None
    if stats:
        mean = torch.empty((B, N), dtype=torch.float32, device=x.device)
        rstd = torch.empty((B, N), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        _check(_lib.load().adaln_fwd(x.data_ptr(), shift.data_ptr(), scale.data_ptr(), B, N, D, float(eps),
                                     y.data_ptr(), _ptr(mean), _ptr(rstd), _stream(stream)))
    return (y, mean, rstd) if stats else y


def adaln_bwd_ws_bytes(B: int, N: int, D: int) -> int:
    return int(_lib.load().adaln_bwd_ws_bytes(B, N, D))


def adaln_bwd(x, scale, dy, eps: float = 1e-6, dx=None, dshift=None, dscale=None, ws=None, stream=None):
    """(dx bf16 [B, N, D], dshift fp32 [B, D], dscale fp32 [B, D]) of adaln_fwd."""
    if x.dim() != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = x.shape
    _need_cuda(x, "x", torch.bfloat16, (B, N, D))
    _need_cuda(dy, "dy", torch.bfloat16, (B, N, D))
    _need_cuda(scale, "scale", torch.float32, (B, D))
    dx = torch.empty_like(x) if dx is None else dx
    dshift = torch.empty((B, D), dtype=torch.float32, device=x.device) if dshift is None else dshift
    dscale = torch.empty((B, D), dtype=torch.float32, device=x.device) if dscale is None else dscale
    _need_cuda(dx, "dx", torch.bfloat16, (B, N, D))
    _need_cuda(dshift, "dshift", torch.float32, (B, D))
    _need_cuda(dscale, "dscale", torch.float32, (B, D))
    lib = _lib.load()
    nbytes = int(lib.adaln_bwd_ws_bytes(B, N, D))
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    with torch.cuda.device(x.device):
        _check(lib.adaln_bwd(x.data_ptr(), scale.data_ptr(), dy.data_ptr(), B, N, D, float(eps), dx.data_ptr(),
                             dshift.data_ptr(), dscale.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return dx, dshift, dscale


# ------------------------------------------------------- rotary positions
_NORMS = {None: 0, "layer": 1, "rms": 2, "head": 3, "token": 4}
_TWO_PI = Decimal("6.283185307179586476925286766559005768394338798750211641949889")


@dataclass
class RotaryPlan:
    """Frequencies of rotary positions, made once by rotary_plan and shared by
    all calls: turns is an int64 [rotary_dim / 2] device tensor, each pair's
    frequency in turns per position as a fraction of 2^64; sections counts the
    pairs of each position axis."""
    turns: torch.Tensor
    rotary_dim: int
    layout: str
    sections: tuple
    gain: float


def rotary_plan(rotary_dim: int, base: float = 10000.0, layout: str = "half", sections=None,
                scaling: str | None = None, factor: float = 1.0, length: int | None = None, slow: float = 1.0,
                fast: float = 32.0, gain: float | None = None, device=None) -> RotaryPlan:
    """Plan of rotary positions over the first rotary_dim features of a head.

    layout: "half" pairs feature i with i + rotary_dim / 2, "interleaved" 2 i
    with 2 i + 1.  sections: pairs of each position axis (1 to 3 of them,
    summing to rotary_dim / 2; one axis by default); pair j of an axis of n
    pairs has frequency base^(-j / n) in radians per position.

    scaling, for contexts factor times longer than trained: "linear" divides
    every frequency by factor; "ntk" raises base to base factor^(n / (n - 1)),
    which leaves the fastest pair and divides the slowest by factor; "parts"
    keeps the pairs that turn at least `fast` times within the trained
    `length`, divides by factor those that turn at most `slow` times, blends
    between, and multiplies the rotated features by 0.1 ln(factor) + 1.  gain
    overrides that multiplier (1 otherwise)."""
    R = int(rotary_dim)
    if R < 2 or R % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    sections = (R // 2,) if sections is None else tuple(int(n) for n in sections)
    if not 1 <= len(sections) <= 3 or min(sections) < 0 or sum(sections) != R // 2:
        raise ValueError(f"sections must be 1 to 3 counts that sum to {R // 2}, got {sections}")
    if scaling not in (None, "none", "linear", "ntk", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    base, factor, slow, fast = (float(v) for v in (base, factor, slow, fast))
    if not (math.isfinite(base) and base > 0.0) or not (math.isfinite(factor) and factor > 0.0):
        raise ValueError("base and factor must be positive and finite")
    if scaling == "parts" and (length is None or not 1 <= length < math.inf or not math.inf > fast > slow >= 0.0):
        raise ValueError("scaling 'parts' needs the trained length and fast > slow >= 0, all finite")
    turns = []
    with localcontext() as ctx:
        ctx.prec = 50
        s = Decimal(factor)
        for n in sections:
            b = Decimal(base)
            if scaling == "ntk" and n > 1:
                b *= (s.ln() * n / (n - 1)).exp()
            ratio, power = (-b.ln() / n).exp() if n else Decimal(1), Decimal(1)
            for j in range(n):
                t = power / _TWO_PI
                power *= ratio
                if scaling == "linear":
                    t /= s
                elif scaling == "parts":
                    keep = (Decimal(float(length)) * t - Decimal(slow)) / (Decimal(fast) - Decimal(slow))
                    keep = min(max(keep, Decimal(0)), Decimal(1))
                    t = t * keep + t / s * (1 - keep)
                whole = int((t * (1 << 64)).to_integral_value()) % (1 << 64)
                turns.append(whole - (1 << 64) if whole >> 63 else whole)
    if gain is None:
        gain = 0.1 * math.log(factor) + 1.0 if scaling == "parts" and factor > 1.0 else 1.0
    table = torch.tensor(turns, dtype=torch.int64).to(device or "cuda")
    return RotaryPlan(table, R, layout, sections, float(gain))


def _heads_view(t, name: str, shape, device) -> bytes | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    sb, sl, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    B, L, H, _ = shape  # the stride of a single entry means nothing
    return _lib.PACK_HEADS(t.data_ptr(), sb if B > 1 else 0, sl if L > 1 else 0, sh if H > 1 else 0)


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _rotary(like_q, like_k, positions, plan: RotaryPlan, norm, q_weight, k_weight, eps):
    """Checked description of a rotary call."""
    if like_q.dim() != 4 or (like_k is not None and like_k.dim() != 4):
        raise ValueError("q and k must be [B, L, heads, D]")
    B, L, H, D = like_q.shape
    device = like_q.device
    Hk = 0 if like_k is None else int(like_k.shape[2])
    if like_k is not None and (like_k.shape != (B, L, Hk, D) or Hk < 1):
        raise ValueError(f"k must be [{B}, {L}, Hk, {D}], got {tuple(like_k.shape)}")
    if norm not in (None, "head", "token"):
        raise ValueError(f"norm must be None, 'head' or 'token', got {norm!r}")
    axes = len(plan.sections)
    if axes == 1 and positions.dim() == 2:
        positions = positions.unsqueeze(2)
    _need(positions, "positions", torch.int32, (B, L, axes), device)
    for name, w, n in (("q_weight", q_weight, H), ("k_weight", k_weight, Hk)):
        if w is None:
            continue
        if norm is None or (n == 0):
            raise ValueError(f"{name} needs a norm and its heads")
        _need(w, name, torch.float32, w.shape, device)
        if w.numel() != (n * D if norm == "token" else D):
            raise ValueError(f"{name} must hold {n * D if norm == 'token' else D} values, got {w.numel()}")
    _need(plan.turns, "plan.turns", torch.int64, (plan.rotary_dim // 2,), device)
    if plan.layout not in ("half", "interleaved"):
        raise ValueError(f"the plan's layout must be 'half' or 'interleaved', got {plan.layout!r}")
    s = plan.sections
    s1 = s[0]
    s2 = s1 + (s[1] if axes > 1 else 0)
    how = _lib.PACK_ROTARY(B, L, H, Hk, D, plan.rotary_dim, 0 if plan.layout == "half" else 1, axes, s1, s2, plan.gain,
                           _NORMS[norm], float(eps), plan.turns.data_ptr(), positions.data_ptr(), _addr(q_weight),
                           _addr(k_weight))
    return how, (B, L, H, D), (B, L, Hk, D)


def pack_rotary_fwd(q, k, positions, plan: RotaryPlan, norm: str | None = None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): the rotary positions of bf16 q [B, L, H, D] and k
    [B, L, Hk, D] (or None) at int32 positions [B, L, axes] ([B, L] for one
    axis), after the RMS norm of each head (norm="head", weights fp32 [D]) or
    of all heads of the token (norm="token", weights fp32 [H * D], [Hk * D]);
    a weight of None is 1.  q and k may be slices with any strides but that of
    D; the outputs are contiguous unless given, and may be q and k."""
    how, qs, ks = _rotary(q, k, positions, plan, norm, q_weight, k_weight, eps)
    dev = q.device
    with _launch(dev, stream) as handle:
        if q_out is None:
            q_out = torch.empty(qs, dtype=torch.bfloat16, device=dev)
        if k is not None and k_out is None:
            k_out = torch.empty(ks, dtype=torch.bfloat16, device=dev)
        _check(_lib.load().pack_rotary_fwd(how, _heads_view(q, "q", qs, dev), _heads_view(k, "k", ks, dev),
                                           _heads_view(q_out, "q_out", qs, dev),
                                           None if k is None else _heads_view(k_out, "k_out", ks, dev), handle))
    return q_out, (None if k is None else k_out)


def pack_rotary_bwd(dq_out, dk_out, positions, plan: RotaryPlan, norm: str | None = None, q=None, k=None,
                    q_weight=None, k_weight=None, eps: float = 1e-6, dq=None, dk=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of pack_rotary_fwd from the gradients of
    its outputs; q, k (its inputs) are needed with a norm.  dk is None without
    keys, a weight's gradient (fp32) is None without that weight."""
    how, qs, ks = _rotary(dq_out, dk_out, positions, plan, norm, q_weight, k_weight, eps)
    keys = dk_out is not None
    if norm is not None and (q is None or (keys and k is None)):
        raise ValueError("the backward of a norm needs q and k")
    if norm is None:
        q = k = None
    lib, dev = _lib.load(), dq_out.device
    with _launch(dev, stream) as handle:
        if dq is None:
            dq = torch.empty(qs, dtype=torch.bfloat16, device=dev)
        if keys and dk is None:
            dk = torch.empty(ks, dtype=torch.bfloat16, device=dev)
        dq_weight = None if q_weight is None else torch.empty_like(q_weight)
        dk_weight = None if k_weight is None else torch.empty_like(k_weight)
        nbytes = int(lib.pack_rotary_bwd_ws_bytes(how))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        _check(lib.pack_rotary_bwd(how, _heads_view(dq_out, "dq_out", qs, dev), _heads_view(dk_out, "dk_out", ks, dev),
                                   _heads_view(q, "q", qs, dev), _heads_view(k, "k", ks, dev) if keys else None,
                                   _heads_view(dq, "dq", qs, dev), _heads_view(dk, "dk", ks, dev) if keys else None,
                                   _ptr(dq_weight), _ptr(dk_weight), _ptr(ws), nbytes, handle))
    return dq, (dk if keys else None), dq_weight, dk_weight


# ------------------------------------------------- gated residual and norms
class AdalnResidualGrads(NamedTuple):
    """Gradients of adaln_residual_fwd; None for what the call did not have."""
    dx: torch.Tensor
    dh: torch.Tensor | None
    dgate: torch.Tensor | None
    dshift: torch.Tensor | None
    dscale: torch.Tensor | None
    dweight: torch.Tensor | None
    dbias: torch.Tensor | None
    dpost_weight: torch.Tensor | None


def _residual(x, gate, shift, scale, mod_id, weight, bias, post_weight, norm, post_norm, alpha, eps):
    """Checked description of a gated residual call; returns (description, modulation rows)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = x.shape
    device = x.device
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x must be {torch.bfloat16} or {torch.float32}, got {x.dtype}")
    _need_cuda(x, "x", x.dtype)
    if norm not in ("layer", "rms"):
        raise ValueError(f"norm must be 'layer' or 'rms', got {norm!r}")
    if post_norm not in (None, "layer", "rms"):
        raise ValueError(f"post_norm must be None, 'layer' or 'rms', got {post_norm!r}")
    S = None
    for name, t in (("gate", gate), ("shift", shift), ("scale", scale)):
        if t is None:
            continue
        if t.dim() != 2:
            raise ValueError(f"{name} must be [S, D]")
        S = int(t.shape[0]) if S is None else S
        _need(t, name, torch.float32, (S, D), device)
    if mod_id is not None:
        _need(mod_id, "mod_id", torch.int32, (B, N), device)
    elif S is not None and S != B:
        raise ValueError(f"without mod_id the modulation tables must have B = {B} rows, got {S}")
    for name, t in (("weight", weight), ("bias", bias), ("post_weight", post_weight)):
        if t is not None:
            _need(t, name, torch.float32, (D,), device)
    return _lib.PACK_RESIDUAL(B, N, D, S or 1, 1 if x.dtype == torch.float32 else 0, _NORMS[norm], _NORMS[post_norm],
                         float(alpha), float(eps), _addr(gate), _addr(shift), _addr(scale), _addr(weight), _addr(bias),
                         _addr(post_weight), _addr(mod_id)), S or 1


def adaln_residual_fwd(x, h=None, gate=None, shift=None, scale=None, *, mod_id=None, weight=None, bias=None,
                       post_weight=None, norm: str = "layer", post_norm: str | None = None, alpha: float = 1.0,
                       eps: float = 1e-6, x_out=None, y=None, stream=None):
    """(x_out, y): x_out = alpha x + gate_s u with u = h, or post_norm(h)
    post_weight, and y = (norm(x_out) weight + bias)(1 + scale_s) + shift_s, the
    gated residual after a block and the modulated norm before the next.

    x [B, N, D] bf16 or fp32 (x_out alike), h and y bf16, gate / shift / scale
    fp32 [S, D], weight / bias / post_weight fp32 [D]; what is None drops out.
    mod_id int32 [B, N] is each token's row s (the seq_ids of
    pack_build_seq_ids: one modulation per packed episode), negative for
    padding: x_out = x, y = 0.  Without it row b serves batch row b (S = B).
    Without h, x_out is x itself and y its modulated norm."""
    how, _ = _residual(x, gate, shift, scale, mod_id, weight, bias, post_weight, norm, post_norm, alpha, eps)
    if h is not None:
        _need(h, "h", torch.bfloat16, x.shape, x.device)
    with _launch(x.device, stream) as handle:
        if h is None:
            x_out = x
        elif x_out is None:
            x_out = torch.empty_like(x)
        else:
            _need(x_out, "x_out", x.dtype, x.shape, x.device)
        if y is None:
            y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
        else:
            _need(y, "y", torch.bfloat16, x.shape, x.device)
        _check(_lib.load().adaln_residual_fwd(how, x.data_ptr(), _ptr(h), x_out.data_ptr(), y.data_ptr(),
                                              handle))
    return x_out, y


def adaln_residual_bwd_ws_bytes(B: int, N: int, D: int, S: int) -> int:
    return int(_lib.load().adaln_residual_bwd_ws_bytes(B, N, D, S))


def adaln_residual_bwd(dx_out, dy, x_out, h=None, gate=None, shift=None, scale=None, *, mod_id=None, weight=None,
                       bias=None, post_weight=None, norm: str = "layer", post_norm: str | None = None,
                       alpha: float = 1.0, eps: float = 1e-6, branch: bool | None = None, dx=None, dh=None, ws=None,
                       stream=None) -> AdalnResidualGrads:
    """Gradients of adaln_residual_fwd from dx_out (like x_out, or None for
    zero), dy (bf16) and the forward's x_out, h, tables and vectors (shift's
    and bias's values are not used, only whether they are there).  h is needed
    with a gate or a post norm; branch=True asks for dh without it.  The ids of
    mod_id must not decrease along the rows, padding aside; device_error
    reports a call that broke this, whose table gradients are NaN."""
    how, S = _residual(x_out, gate, shift, scale, mod_id, weight, bias, post_weight, norm, post_norm, alpha, eps)
    B, N, D = x_out.shape
    branch = h is not None if branch is None else bool(branch)
    if h is not None:
        _need(h, "h", torch.bfloat16, x_out.shape, x_out.device)
    _need(dy, "dy", torch.bfloat16, x_out.shape, x_out.device)
    if dx_out is not None:
        _need(dx_out, "dx_out", x_out.dtype, x_out.shape, x_out.device)
    lib = _lib.load()
    with _launch(x_out.device, stream) as handle:
        if dx is None:
            dx = torch.empty_like(x_out)
        else:
            _need(dx, "dx", x_out.dtype, x_out.shape, x_out.device)
        if branch and dh is None:
            dh = torch.empty(x_out.shape, dtype=torch.bfloat16, device=x_out.device)
        elif branch:
            _need(dh, "dh", torch.bfloat16, x_out.shape, x_out.device)
        params = (gate, shift, scale, weight, bias, post_weight)
        grads = [None if t is None else torch.empty_like(t) for t in params]
        if ws is not None:
            _need(ws, "ws", torch.uint8, ws.shape, x_out.device)
        else:
            ws = torch.empty(adaln_residual_bwd_ws_bytes(B, N, D, S), dtype=torch.uint8, device=x_out.device)
        out = _lib.PACK_RESIDUAL_GRADS(*(_addr(t) for t in grads))
        _check(lib.adaln_residual_bwd(how, _ptr(dx_out), dy.data_ptr(), x_out.data_ptr(), _ptr(h),
                                      int(branch), dx.data_ptr(), _ptr(dh) if branch else None, out,
                                      ws.data_ptr(), ws.numel(), handle))
    return AdalnResidualGrads(dx, dh if branch else None, *grads)


# ------------------------------------------------------------ masked loss
def masked_mse_ws_bytes(B: int, L: int, C: int) -> int:
    return int(_lib.load().masked_mse_ws_bytes(B, L, C))


def _loss_args(pred, target, seq_id):
    if pred.dim() != 3:
        raise ValueError("pred must be [B, L, C]")
    B, L, C = pred.shape
    _need_cuda(pred, "pred", torch.bfloat16, (B, L, C))
    _need_cuda(target, "target", torch.bfloat16, (B, L, C))
    _need_cuda(seq_id, "seq_id", torch.int32, (B, L))
    return B, L, C


def masked_mse_loss(pred, target, seq_id, grad: bool | torch.Tensor = False, grad_scale: float = 1.0,
                    loss=None, ws=None, stream=None):
    """Squared-error loss averaged over the valid tokens (seq_id >= 0), i.e.
    over the valid frames ("lingbot_va_packing" §2.1, compute_loss).  pred,
    target bf16 [B, L, C]; seq_id int32 [B, L].  Returns the fp32 loss as a
    one-element device tensor, or (loss, grad) when grad is True or a bf16
    [B, L, C] tensor to fill: grad = grad_scale * d loss / d pred, computed
    in the same pass."""
    B, L, C = _loss_args(pred, target, seq_id)
    want_grad = grad is not False and grad is not None
    g = None
    if want_grad:
        g = torch.empty_like(pred) if grad is True else grad
        _need_cuda(g, "grad", torch.bfloat16, (B, L, C))
    loss = torch.empty(1, dtype=torch.float32, device=pred.device) if loss is None else loss
    _need_cuda(loss, "loss", torch.float32, (1,))
    lib = _lib.load()
    nbytes = int(lib.masked_mse_ws_bytes(B, L, C))
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=pred.device)
    with torch.cuda.device(pred.device):
        _check(lib.masked_mse_loss(pred.data_ptr(), target.data_ptr(), seq_id.data_ptr(), B, L, C, loss.data_ptr(),
                                   _ptr(g), float(grad_scale), ws.data_ptr(), ws.numel(), _stream(stream)))
    return (loss, g) if want_grad else loss


def masked_mse_loss_bwd(pred, target, seq_id, dloss, grad=None, ws=None, stream=None):
    """d loss / d pred of masked_mse_loss times the device scalar dloss (fp32, one element)."""
    B, L, C = _loss_args(pred, target, seq_id)
    _need_cuda(dloss, "dloss", torch.float32)
    if dloss.numel() != 1:
        raise ValueError("dloss must hold one element")
    grad = torch.empty_like(pred) if grad is None else grad
    _need_cuda(grad, "grad", torch.bfloat16, (B, L, C))
    lib = _lib.load()
    nbytes = int(lib.masked_mse_ws_bytes(B, L, C))
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=pred.device)
    with torch.cuda.device(pred.device):
        _check(lib.masked_mse_loss_bwd(pred.data_ptr(), target.data_ptr(), seq_id.data_ptr(), B, L, C,
                                       dloss.data_ptr(), grad.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return grad


# ------------------------------------------------------------------- errors
def device_error(stream=None, raise_on_error: bool = True):
    """Synchronises the stream and returns (status, [code, where, block, thread])."""
    info = (ctypes.c_int32 * 4)()
    st = _lib.load().pvl_device_error_detail(_stream(stream), ctypes.addressof(info))
    msg = _lib.load().pvl_last_error_message().decode()
    if raise_on_error and st != PVL_OK:
        raise PvlError(st, msg)
    return st, list(info)


def set_attn_wait_timeout_ns(ns: int) -> None:
    """Bound on any single device-side wait of the attention kernels launched
    from now on, process-wide; 0 restores the default (2 s)."""
    _check(_lib.load().pvl_set_attn_wait_timeout_ns(int(ns)))


def _event_handle(ev) -> int | None:
    if ev is None:
        return None
    handle = int(ev.cuda_event)
    if handle == 0:
        raise ValueError("the event has no CUDA event yet: record it once before passing it")
    return handle


def mark_next_bwd_main(before, after) -> None:
    """Records the torch.cuda.Event objects ``before`` / ``after`` around the
    main backward kernel of this thread's next masked_attn_bwd call (one-shot;
    see pvl_mark_next_bwd_main).  Each event must have been recorded once
    already, so that its CUDA event exists."""
    _check(_lib.load().pvl_mark_next_bwd_main(_event_handle(before), _event_handle(after)))


def version() -> int:
    return int(_lib.load().pvl_version())
