"""Operators of self-attention among voxels in grid order: attention in a sliding window, the norm of queries and keys with
the rotation by their positions, and dropout that stores no mask."""
from __future__ import annotations

import ctypes
import functools
import math
import struct

import torch

from . import _lib
from ._args import _dtype_code
from ._block import _ATTENTION, _call, _heads, _ptr, _same
from ._block import _problem as _attention_problem

LAYOUTS = {"half": 0, "interleaved": 1}
_QK = struct.Struct("@iiiiiiiiffqqqqqPP")  # igc_qk_t


def _dense_like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and type (half the time of torch.empty with both given)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _window(left, right, sinks) -> tuple[int, int, int]:
    """The window's sides (None: no limit) and sinks as the library takes them."""
    for value, name in ((left, "left"), (right, "right"), (sinks, "sinks")):
        if value is not None and not 0 <= value < 1 << 31:
            raise ValueError(f"{name} must be 0 to 2^31 - 1{'' if name == 'sinks' else ', or None'}")
    return -1 if left is None else left, -1 if right is None else right, sinks


@functools.lru_cache(maxsize=256)
def _window_workspace(backward: int, window: tuple, code: int, batch: int, heads: int, kv_heads: int, dim: int, nq: int,
                      nk: int) -> int:
    # The offsets' addresses only have to be there: the size depends on the counts alone.
    p = _ATTENTION.pack(code, batch, heads, kv_heads, dim, 1.0, nq, nk, 0, 0, 0, 0, 0, 0, 16, 16, 0)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().igc_window_attention_workspace(p, *window, backward, ctypes.byref(n)))
    return n.value


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, left: int | None = None, right: int | None = None,
                     sinks: int = 0, q_offsets: torch.Tensor | None = None, kv_offsets: torch.Tensor | None = None,
                     key_mask: torch.Tensor | None = None, scale: float | None = None, kv_lengths: torch.Tensor | None = None):
    """cross_attention among rows in order, where a query sees a window of keys and a few first ones: query i of a
    sequence of lq queries and lk keys stands at p = i + lk - lq and sees key j if j <= p + right and (j >= p - left or j < sinks) and
    key_mask keeps it. None: no limit to that side; right 0 is causal. With as many queries as keys this is attention within
    a sequence, with fewer that of its last rows to a cache (single tokens); kv_lengths (int32 [batch] on the device) says how many
    of a sequence's key rows are in use where a cache has room for more (its lk then; without gradients). k and v in use must be finite where
    key_mask keeps them, and for gradients q and dout of rows that see a key; masked keys and rows without keys may hold anything.
    Returns (out, lse) as cross_attention (igc_window_attention)."""
    window = _window(left, right, sinks)
    p, sizes = _attention_problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dev = q.device
    if kv_lengths is not None:
        _same(kv_lengths, "kv_lengths", torch.int32, (sizes[1],), dev.index)
        if window[0] < 0 and window[1] < 0:  # lengths need a limit: one that leaves nothing out
            window = (2 ** 31 - 1, -1, 0)
    out = _dense_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    n = _window_workspace(0, window, *sizes)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _call("igc_window_attention", dev.index, p, *window, _ptr(kv_lengths), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
          _ptr(ws), n)
    return out, lse


def window_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                              lse: torch.Tensor, left: int | None = None, right: int | None = None, sinks: int = 0,
                              q_offsets: torch.Tensor | None = None, kv_offsets: torch.Tensor | None = None,
                              key_mask: torch.Tensor | None = None, scale: float | None = None, need_dq: bool = True,
                              need_dkv: bool = True):
    """Gradients (dq, dk, dv) of window_attention for the output gradient dout, from its inputs and results; None for those
    not needed (igc_window_attention_backward)."""
    window = _window(left, right, sinks)
    p, sizes = _attention_problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dt, dev = q.dtype, q.device
    _same(dout, "dout", dt, q.shape, dev.index), _same(out, "out", dt, q.shape, dev.index)
    _same(lse, "lse", torch.float32, q.shape[:2], dev.index)
    dq = _dense_like(q) if need_dq else None
    dk = _dense_like(k) if need_dkv else None
    dv = _dense_like(k) if need_dkv else None
    n = _window_workspace(1, window, *sizes)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _call("igc_window_attention_backward", dev.index, p, *window, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), dout.data_ptr(), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), n)
    return dq, dk, dv


def rotary_frequencies(dim: int, base: float = 10000.0, axes: int = 1, scaling: str | None = None, factor: float = 1.0,
                       original: int | None = None, low: float = 1.0, high: float = 32.0) -> torch.Tensor:
    """Frequencies float32 [axes, pairs] (on the host) for rotating `dim` channels of a head, pairs = dim // 2 // axes
    on each of 1 to 3 position axes: base ** (-i / pairs). For positions up to `factor` times those trained on:
    scaling="linear" divides all by factor; "base" raises the base so that the slowest frequency is divided by factor and the
    fastest stays (at least two pairs); "parts" divides those that make fewer than `low` turns over the `original` length, keeps
    those that make more than `high`, and blends in between."""
    if not 1 <= axes <= 3 or dim < 2 * axes:
        raise ValueError("axes must be 1 to 3, and dim at least 2 a axis")
    if not base > 0 or not factor > 0 or not math.isfinite(base) or not math.isfinite(factor):
        raise ValueError("base and factor must be positive and finite")
    pairs = dim // 2 // axes
    i = torch.arange(pairs, dtype=torch.float64)
    if scaling == "base" and factor != 1:
        if pairs < 2:
            raise ValueError("scaling by the base needs at least two pairs: one is the fastest and the slowest")
        base = base * factor ** (pairs / (pairs - 1))
    f = base ** (-i / pairs)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original is None or original < 1 or not 0 <= low < high:
            raise ValueError("scaling in parts needs the original length and 0 <= low < high")
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    return f.float().expand(axes, -1).contiguous()


def _turn(positions, frequencies, n: int, layout: str, index: int) -> tuple[int, int, int]:
    """Checks positions and frequencies and returns (axes, pairs, layout code)."""
    if layout not in LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if (positions is None) != (frequencies is None):
        raise ValueError("positions and frequencies come together")
    if positions is None:
        return 0, 0, LAYOUTS[layout]
    if not isinstance(frequencies, torch.Tensor) or frequencies.dim() not in (1, 2):
        raise ValueError("frequencies must have shape [pairs] or [axes, pairs]")
    axes, pairs = (1, frequencies.shape[0]) if frequencies.dim() == 1 else frequencies.shape
    if axes < 1:
        raise ValueError("frequencies must have at least one axis")
    _same(frequencies, "frequencies", torch.float32, frequencies.shape, index)
    flat = axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1
    _same(positions, "positions", torch.int32, (n,) if flat else (n, axes), index)
    return axes, pairs, LAYOUTS[layout]


def _weights(q_weight, k_weight, dim: int, dtype: torch.dtype, index: int) -> int:
    """Checks the weights and returns the type code they share."""
    first = q_weight if q_weight is not None else k_weight
    if first is None:
        return _dtype_code(dtype)
    dt = first.dtype if isinstance(first, torch.Tensor) else None
    if dt != torch.float32 and dt != dtype:
        raise TypeError(f"weights must be float32 or {dtype}, got {dt}")
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _same(t, name, dt, (dim,), index)
    return _dtype_code(dt)


def _problem(q, k, positions, frequencies, eps, layout, amplitude, norm, name="q") -> tuple[bytes, tuple]:
    """The problem as an igc_qk_t, and the sizes its workspace depends on."""
    dt = q.dtype
    code, index = _dtype_code(dt), q.get_device()
    _heads(q, name, dt, index)
    n, heads, dim = q.shape
    kv_heads, ks = 0, (0, 0, 0)
    if k is not None:
        _heads(k, "k", dt, index)
        if k.shape[0] != n or k.shape[2] != dim or k.shape[1] < 1:
            raise ValueError(f"k must have shape [{n}, kv_heads, {dim}], got {tuple(k.shape)}")
        kv_heads, ks = k.shape[1], k.stride()
    axes, pairs, how = _turn(positions, frequencies, n, layout, index)
    sizes = (code, heads, kv_heads, dim, axes, pairs, how, int(norm))
    qs = q.stride()
    p = _QK.pack(*sizes, eps, amplitude, n, qs[0], qs[1], ks[0], ks[1], _ptr(positions) or 0, _ptr(frequencies) or 0)
    return p, sizes + (n,)


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                   frequencies: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                   k_weight: torch.Tensor | None = None, eps: float = 1e-6, layout: str = "half", amplitude: float = 1.0):
    """Root-mean-square norm of each head of q [n, heads, dim] and k [n, kv_heads, dim] (None: queries alone) with weights [dim]
    (float32 or q's type; None: ones), and the rotation of its channel pairs by positions (int32 [n] or [n, axes], up to three
    axes: voxel coordinates) times frequencies (float32 [pairs] or [axes, pairs], see rotary_frequencies; both None: the norm
    alone). layout "half": pair t is channels t and axes * pairs + t; "interleaved": 2 t and 2 t + 1; channels behind the pairs do not
    turn. amplitude scales the pairs. dim is up to 128, row and head strides are free. Returns new (q, k), rounded once
    (igc_qk_norm_rotary)."""
    p, sizes = _problem(q, k, positions, frequencies, eps, layout, amplitude, True)
    dt, dev = q.dtype, q.device
    wd = _weights(q_weight, k_weight, q.shape[2], dt, dev.index)
    yq = _dense_like(q)
    yk = _dense_like(k) if k is not None else None
    _call("igc_qk_norm_rotary", dev.index, p, q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), wd, yq.data_ptr(), _ptr(yk))
    return yq, yk


@functools.lru_cache(maxsize=256)
def _qk_workspace(*sizes: int) -> int:
    n = ctypes.c_size_t(0)
    # eps and the addresses do not matter to the size.
    _lib.check(_lib.load().igc_qk_norm_rotary_workspace(_QK.pack(*sizes[:-1], 0.0, 1.0, sizes[-1], 0, 0, 0, 0, 0, 0), ctypes.byref(n)))
    return n.value


def qk_norm_rotary_backward(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                            positions: torch.Tensor | None = None, frequencies: torch.Tensor | None = None,
                            q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                            layout: str = "half", amplitude: float = 1.0, need_dweight: bool = True):
    """Gradients of qk_norm_rotary for its outputs' gradients dq and dk (contiguous), from its inputs: (dq, dk of q's
    type, dq_weight, dk_weight [dim] float32; the last two None without need_dweight, those of keys None without keys)
    (igc_qk_norm_rotary_backward)."""
    p, sizes = _problem(q, k, positions, frequencies, eps, layout, amplitude, True)
    dt, dev = q.dtype, q.device
    wd = _weights(q_weight, k_weight, q.shape[2], dt, dev.index)
    _same(dq, "dq", dt, q.shape, dev.index)
    if k is not None:
        _same(dk, "dk", dt, k.shape, dev.index)
    gq = _dense_like(q)
    gk = _dense_like(k) if k is not None else None
    dqw = dkw = ws = None
    nbytes = 0
    if need_dweight:
        nbytes = _qk_workspace(*sizes)
        dqw = torch.empty(q.shape[2], dtype=torch.float32, device=dev)
        dkw = torch.empty(q.shape[2], dtype=torch.float32, device=dev) if k is not None else None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call("igc_qk_norm_rotary_backward", dev.index, p, dq.data_ptr(), _ptr(dk) if k is not None else None, q.data_ptr(), _ptr(k),
          _ptr(q_weight), _ptr(k_weight), wd, gq.data_ptr(), _ptr(gk), _ptr(dqw), _ptr(dkw), _ptr(ws), nbytes)
    return gq, gk, dqw, dkw


def rotary(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, layout: str = "half", amplitude: float = 1.0):
    """The rotation of qk_norm_rotary alone: x [n, heads, dim] turned by its positions (igc_qk_norm_rotary without the norm)."""
    if positions is None or frequencies is None:
        raise ValueError("the rotation needs positions and frequencies")
    p, _ = _problem(x, None, positions, frequencies, 0.0, layout, amplitude, False, "x")
    y = _dense_like(x)
    _call("igc_qk_norm_rotary", x.get_device(), p, x.data_ptr(), None, None, None, _dtype_code(x.dtype), y.data_ptr(), None)
    return y


def rotary_backward(dy: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, layout: str = "half",
                    amplitude: float = 1.0):
    """Gradient of rotary for the output gradient dy (contiguous): the rotation back, times amplitude."""
    if positions is None or frequencies is None:
        raise ValueError("the rotation needs positions and frequencies")
    p, _ = _problem(dy, None, positions, frequencies, 0.0, layout, amplitude, False, "dy")
    _same(dy, "dy", dy.dtype, dy.shape, dy.get_device())
    dx = _dense_like(dy)
    _call("igc_qk_norm_rotary_backward", dy.get_device(), p, dy.data_ptr(), None, None, None, None, None, _dtype_code(dy.dtype),
          dx.data_ptr(), None, None, None, None, 0)
    return dx


def _dropout(x, p: float, seed: int, offset, residual, counter):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    code, index = _dtype_code(x.dtype), x.get_device()
    _same(x, "x", x.dtype, x.shape, index)
    if residual is not None:
        _same(residual, "residual", x.dtype, x.shape, index)
    if isinstance(offset, torch.Tensor):
        if counter is not None:
            raise ValueError("with a counter the offset is a number")
        _same(offset, "offset", torch.int64, (1,), index)
        counter, offset = offset, 0
    elif counter is not None:
        _same(counter, "counter", torch.int64, (1,), index)
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset must be 0 to 2^64 - 1")
    y = torch.empty_like(x)
    _call("igc_dropout", index, x.data_ptr(), _ptr(residual), x.numel(), code, p, seed, offset, _ptr(counter), y.data_ptr())
    return y


def dropout(x: torch.Tensor, p: float, seed: int, offset: int | torch.Tensor = 0, residual: torch.Tensor | None = None,
            counter: torch.Tensor | None = None):
    """x (any shape, contiguous) with each element dropped with probability p (a multiple of 2^-16 is taken) and the others scaled so that
    the expected value stays, plus residual. What is dropped depends on (p, seed, offset) and the element's index alone: no
    mask is kept, and dropout_backward computes it again. Give every call of a step an offset of its own. counter, an int64
    tensor of one element on the device, is added to the offset (modulo 2^64), so that a captured graph can count its steps; calls that
    share a counter take offsets further apart than it counts, for example layer << 32. An offset that is such a tensor itself is a
    counter on the offset 0 (igc_dropout)."""
    return _dropout(x, p, seed, offset, residual, counter)


def dropout_backward(dy: torch.Tensor, p: float, seed: int, offset: int | torch.Tensor = 0, counter: torch.Tensor | None = None):
    """Gradient of dropout with the same p, seed, offset and counter for the output gradient dy; residual's is dy itself."""
    return _dropout(dy, p, seed, offset, None, counter)
