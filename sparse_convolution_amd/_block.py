"""Operators between convolutions: layer norm and 8-bit activation checkpoints over voxel
features [n, channels], and cross attention of voxel or object queries to another set of rows."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._args import _device_tensor, _dtype_code

Q8_GROUP = 64  # channels of a row that share a checkpoint scale (IGC_Q8_GROUP)


class Checkpoint8:
    """Features held in 8 bits (igc_checkpoint_pack): codes int8 [n, c], scales float32
    [n, ceil(c / 64)] and the type the values are restored in; value = code * scale of its group
    of 64 channels."""

    __slots__ = ("codes", "scales", "dtype")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32):
        _dtype_code(dtype)
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError("codes must have shape [n, c]")
        _device_tensor(codes, "codes", torch.int8)
        _device_tensor(scales, "scales", torch.float32, -(-codes.shape[1] // Q8_GROUP))
        if scales.shape[0] != codes.shape[0] or scales.device != codes.device:
            raise ValueError("codes and scales must have the same rows and device")
        self.codes, self.scales, self.dtype = codes, scales, dtype

    @property
    def shape(self) -> torch.Size:
        return self.codes.shape

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


# The current stream's handle without building a Stream object (3 us of a 13 us call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _call(name: str, device: torch.device, *args) -> None:
    """lib.name(*args, stream) on the current stream of `device`, with that device current."""
    index = device.index
    fn = getattr(_lib.load(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(status)


def _rows(x: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must have shape [n, channels]")
    _dtype_code(x.dtype)
    return _device_tensor(x, name, x.dtype)


def _same(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: torch.device) -> torch.Tensor:
    _device_tensor(t, name, dtype)
    if tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    return t


def _params(weight, bias, c: int, x_dtype: torch.dtype, device: torch.device) -> int:
    """Checks weight and bias and returns the type code they share."""
    dt = x_dtype
    for p in (weight, bias):
        if p is not None:
            dt = p.dtype
            break
    if dt not in (torch.float32, x_dtype):
        raise TypeError(f"weight and bias must be float32 or {x_dtype}, got {dt}")
    for p, name in ((weight, "weight"), (bias, "bias")):
        if p is not None:
            _same(p, name, dt, (c,), device)
    return _dtype_code(dt)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5):
    """Layer norm of each row of x [n, c] (c up to 4096): (y of x's type, mean [n] float32,
    rstd [n] float32). weight and bias [c] are float32 or of x's type (igc_layer_norm)."""
    x = _rows(x, "x")
    n, c = x.shape
    wd = _params(weight, bias, c, x.dtype, x.device)
    y = torch.empty_like(x)
    stats = torch.empty((2, n), dtype=torch.float32, device=x.device)
    mean, rstd = stats.unbind(0)
    _call("igc_layer_norm", x.device, _ptr(x), n, c, _dtype_code(x.dtype), _ptr(weight), _ptr(bias), wd, eps, _ptr(y),
          _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def _backward(name, dy, source, rstd, weight, need_dweight, c):
    n = dy.shape[0]
    dev = dy.device
    wd = _params(weight, None, c, dy.dtype, dev)
    _same(rstd, "rstd", torch.float32, (n,), dev)
    dx = torch.empty_like(dy)
    dw = db = ws = None
    nbytes = ctypes.c_size_t(0)
    if need_dweight:
        dw, db = torch.empty((2, c), dtype=torch.float32, device=dev).unbind(0)
        _lib.check(_lib.load().igc_layer_norm_workspace(n, c, ctypes.byref(nbytes)))
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
    _call(name, dev, _ptr(dy), *source, _ptr(rstd), n, c, _dtype_code(dy.dtype), _ptr(weight), wd, _ptr(dx), _ptr(dw),
          _ptr(db), _ptr(ws), nbytes)
    return dx, dw, db


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, need_dweight: bool = True):
    """Gradients of layer_norm for the output gradient dy: (dx of x's type, dweight [c] float32,
    dbias [c] float32; the last two None without need_dweight) (igc_layer_norm_backward)."""
    x = _rows(x, "x")
    dy = _same(dy, "dy", x.dtype, x.shape, x.device)
    mean = _same(mean, "mean", torch.float32, (x.shape[0],), x.device)
    return _backward("igc_layer_norm_backward", dy, (_ptr(x), _ptr(mean)), rstd, weight, need_dweight, x.shape[1])


def layer_norm_checkpoint(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                          eps: float = 1e-5):
    """layer_norm that keeps what its backward pass needs in 8 bits: (y, Checkpoint8 of the normalised
    rows before weight and bias, rstd [n] float32) (igc_layer_norm_q8)."""
    x = _rows(x, "x")
    n, c = x.shape
    wd = _params(weight, bias, c, x.dtype, x.device)
    y = torch.empty_like(x)
    codes = torch.empty((n, c), dtype=torch.int8, device=x.device)
    scales = torch.empty((n, -(-c // Q8_GROUP)), dtype=torch.float32, device=x.device)
    rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("igc_layer_norm_q8", x.device, _ptr(x), n, c, _dtype_code(x.dtype), _ptr(weight), _ptr(bias), wd, eps, _ptr(y),
          _ptr(codes), _ptr(scales), _ptr(rstd))
    return y, Checkpoint8(codes, scales, x.dtype), rstd


def layer_norm_checkpoint_backward(dy: torch.Tensor, ckpt: Checkpoint8, rstd: torch.Tensor,
                                   weight: torch.Tensor | None = None, need_dweight: bool = True):
    """layer_norm_backward from the checkpoint of layer_norm_checkpoint (igc_layer_norm_q8_backward)."""
    dy = _same(_rows(dy, "dy"), "dy", dy.dtype, ckpt.shape, ckpt.device)
    return _backward("igc_layer_norm_q8_backward", dy, (_ptr(ckpt.codes), _ptr(ckpt.scales)), rstd, weight, need_dweight,
                     dy.shape[1])


def checkpoint_pack(x: torch.Tensor) -> Checkpoint8:
    """x [n, c] in 8 bits, one scale per row and 64 channels (igc_checkpoint_pack)."""
    x = _rows(x, "x")
    n, c = x.shape
    codes = torch.empty((n, c), dtype=torch.int8, device=x.device)
    scales = torch.empty((n, -(-c // Q8_GROUP)), dtype=torch.float32, device=x.device)
    _call("igc_checkpoint_pack", x.device, _ptr(x), n, c, _dtype_code(x.dtype), _ptr(codes), _ptr(scales))
    return Checkpoint8(codes, scales, x.dtype)


def checkpoint_unpack(ckpt: Checkpoint8, dtype: torch.dtype | None = None) -> torch.Tensor:
    """The values a checkpoint stands for, in its own type or `dtype` (igc_checkpoint_unpack)."""
    dt = ckpt.dtype if dtype is None else dtype
    n, c = ckpt.shape
    x = torch.empty((n, c), dtype=dt, device=ckpt.device)
    _call("igc_checkpoint_unpack", ckpt.device, _ptr(ckpt.codes), _ptr(ckpt.scales), n, c, _dtype_code(dt), _ptr(x))
    return x


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype) -> torch.Tensor:
    """Checks a [rows, heads, dim] operand; row and head strides are free."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [rows, heads, dim], got {tuple(t.shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return t


def _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale) -> _lib.Attention:
    dt, dev = q.dtype, q.device
    _dtype_code(dt)
    _heads(q, "q", dt), _heads(k, "k", dt), _heads(v, "v", dt)
    (nq, heads, dim), (nk, kv_heads, _) = q.shape, k.shape
    if k.shape != v.shape or k.shape[2] != dim:
        raise ValueError(f"k and v must have shape [n, kv_heads, {dim}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"heads ({heads}) must be a multiple of kv_heads ({kv_heads})")
    if (q_offsets is None) != (kv_offsets is None):
        raise ValueError("q_offsets and kv_offsets come together")
    batch = 1
    if q_offsets is not None:
        batch = q_offsets.shape[0] - 1 if q_offsets.dim() == 1 else -1
        for t, name in ((q_offsets, "q_offsets"), (kv_offsets, "kv_offsets")):
            _device_tensor(t, name, torch.int32)
            if batch < 1 or tuple(t.shape) != (batch + 1,):
                raise ValueError("q_offsets and kv_offsets must have shape [batch + 1]")
    if key_mask is not None:
        if isinstance(key_mask, torch.Tensor) and key_mask.dtype == torch.bool:
            key_mask = key_mask.view(torch.uint8)
        _same(key_mask, "key_mask", torch.uint8, (nk,), dev)
    for t in (k, v, q_offsets, kv_offsets):
        if t is not None and t.device != dev:
            raise ValueError("all operands must be on one device")
    pair = ctypes.c_int64 * 2
    return _lib.Attention(_dtype_code(dt), batch, heads, kv_heads, dim, dim ** -0.5 if scale is None else scale, nq, nk,
                          pair(*q.stride()[:2]), pair(*k.stride()[:2]), pair(*v.stride()[:2]), _ptr(q_offsets),
                          _ptr(kv_offsets), _ptr(key_mask))


def _workspace(p: _lib.Attention, backward: int, device: torch.device):
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().igc_cross_attention_workspace(ctypes.byref(p), backward, ctypes.byref(n)))
    return (torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None), n


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor | None = None,
                    kv_offsets: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                    scale: float | None = None):
    """Attention of q [nq, heads, dim] to k and v [nk, kv_heads, dim] (kv_heads divides heads, dim up to 128,
    any row and head strides), sequence by sequence: rows q_offsets[b] .. q_offsets[b+1] of q attend to rows
    kv_offsets[b] .. kv_offsets[b+1] of k and v (int32 [batch + 1] on the device; None: one sequence).
    key_mask (bool or uint8 [nk]): false rows are left out. scale defaults to dim ** -0.5. Returns (out
    [nq, heads, dim], lse [nq, heads] float32); a row without keys gets zeros and -inf (igc_cross_attention)."""
    p = _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dev = q.device
    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    ws, n = _workspace(p, 0, dev)
    _call("igc_cross_attention", dev, ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(ws), n)
    return out, lse


def cross_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                             lse: torch.Tensor, q_offsets: torch.Tensor | None = None,
                             kv_offsets: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                             scale: float | None = None, need_dq: bool = True, need_dkv: bool = True):
    """Gradients (dq, dk, dv) of cross_attention for the output gradient dout, from its inputs and results;
    None for those not needed (igc_cross_attention_backward)."""
    p = _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dev = q.device
    _same(dout, "dout", q.dtype, q.shape, dev), _same(out, "out", q.dtype, q.shape, dev)
    _same(lse, "lse", torch.float32, q.shape[:2], dev)
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev) if need_dq else None
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev) if need_dkv else None
    dv = torch.empty(k.shape, dtype=q.dtype, device=dev) if need_dkv else None
    ws, n = _workspace(p, 1, dev)
    _call("igc_cross_attention_backward", dev, ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
          _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), n)
    return dq, dk, dv
