"""Operators between convolutions: layer norm and 8-bit activation checkpoints over voxel
features [n, channels], and cross attention of voxel or object queries to another set of rows."""
from __future__ import annotations

import ctypes
import functools
import struct

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


# The current stream's handle without building a Stream object, where torch has it. The calls below take 6 to 20 us of
# host time, as much as their kernels on small grids, so the checks read each attribute once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _call(name: str, index: int, *args) -> None:
    """lib.name(*args, stream) on the current stream of device `index`, with that device current."""
    fn = getattr(_lib.load(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(status)


def _rows(x: torch.Tensor, name: str) -> int:
    """Checks features [n, channels] and returns their type code."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must have shape [n, channels]")
    code = _dtype_code(x.dtype)
    if not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def _same(t: torch.Tensor, name: str, dtype: torch.dtype, shape, index: int) -> None:
    """Checks type, shape, device and contiguity of an operand."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must have shape {tuple(shape)} on device {index}, got {tuple(t.shape)} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _params(weight, bias, c: int, x_dtype: torch.dtype, index: int) -> int:
    """Checks weight and bias and returns the type code they share."""
    first = weight if weight is not None else bias
    if first is None:
        return _dtype_code(x_dtype)
    dt = first.dtype if isinstance(first, torch.Tensor) else None
    if dt != torch.float32 and dt != x_dtype:
        raise TypeError(f"weight and bias must be float32 or {x_dtype}, got {dt}")
    if weight is not None:
        _same(weight, "weight", dt, (c,), index)
    if bias is not None:
        _same(bias, "bias", dt, (c,), index)
    return _dtype_code(dt)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5):
    """Layer norm of each row of x [n, c] (c up to 4096): (y of x's type, mean [n] float32,
    rstd [n] float32). weight and bias [c] are float32 or of x's type (igc_layer_norm)."""
    code = _rows(x, "x")
    (n, c), dev = x.shape, x.device
    wd = _params(weight, bias, c, x.dtype, dev.index)
    y = torch.empty_like(x)
    mean = torch.empty(n, dtype=torch.float32, device=dev)
    rstd = torch.empty(n, dtype=torch.float32, device=dev)
    _call("igc_layer_norm", dev.index, x.data_ptr(), n, c, code, _ptr(weight), _ptr(bias), wd, eps, y.data_ptr(),
          mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def _norm_workspace(n: int, c: int) -> int:
    size = ctypes.c_size_t(0)
    _lib.check(_lib.load().igc_layer_norm_workspace(n, c, ctypes.byref(size)))
    return size.value


def _backward(name, dy, code, source, rstd, weight, need_dweight):
    (n, c), dev = dy.shape, dy.device
    wd = _params(weight, None, c, dy.dtype, dev.index)
    _same(rstd, "rstd", torch.float32, (n,), dev.index)
    dx = torch.empty_like(dy)
    dw = db = ws = None
    nbytes = 0
    if need_dweight:
        nbytes = _norm_workspace(n, c)
        dw = torch.empty(c, dtype=torch.float32, device=dev)
        db = torch.empty(c, dtype=torch.float32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call(name, dev.index, dy.data_ptr(), *source, rstd.data_ptr(), n, c, code, _ptr(weight), wd, dx.data_ptr(), _ptr(dw),
          _ptr(db), _ptr(ws), nbytes)
    return dx, dw, db


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, need_dweight: bool = True):
    """Gradients of layer_norm for the output gradient dy: (dx of x's type, dweight [c] float32,
    dbias [c] float32; the last two None without need_dweight) (igc_layer_norm_backward)."""
    code, index = _rows(x, "x"), x.get_device()
    _same(dy, "dy", x.dtype, x.shape, index)
    _same(mean, "mean", torch.float32, (x.shape[0],), index)
    return _backward("igc_layer_norm_backward", dy, code, (x.data_ptr(), mean.data_ptr()), rstd, weight, need_dweight)


def _new_checkpoint(n: int, c: int, dtype: torch.dtype, dev: torch.device) -> Checkpoint8:
    ckpt = Checkpoint8.__new__(Checkpoint8)  # its parts need no checks
    ckpt.codes = torch.empty((n, c), dtype=torch.int8, device=dev)
    ckpt.scales = torch.empty((n, -(-c // Q8_GROUP)), dtype=torch.float32, device=dev)
    ckpt.dtype = dtype
    return ckpt


def layer_norm_checkpoint(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                          eps: float = 1e-5):
    """layer_norm that keeps what its backward pass needs in 8 bits: (y, Checkpoint8 of the normalised
    rows before weight and bias, rstd [n] float32) (igc_layer_norm_q8)."""
    code = _rows(x, "x")
    (n, c), dev = x.shape, x.device
    wd = _params(weight, bias, c, x.dtype, dev.index)
    y = torch.empty_like(x)
    ckpt = _new_checkpoint(n, c, x.dtype, dev)
    rstd = torch.empty(n, dtype=torch.float32, device=dev)
    _call("igc_layer_norm_q8", dev.index, x.data_ptr(), n, c, code, _ptr(weight), _ptr(bias), wd, eps, y.data_ptr(),
          ckpt.codes.data_ptr(), ckpt.scales.data_ptr(), rstd.data_ptr())
    return y, ckpt, rstd


def layer_norm_checkpoint_backward(dy: torch.Tensor, ckpt: Checkpoint8, rstd: torch.Tensor,
                                   weight: torch.Tensor | None = None, need_dweight: bool = True):
    """layer_norm_backward from the checkpoint of layer_norm_checkpoint (igc_layer_norm_q8_backward)."""
    code = _rows(dy, "dy")
    _same(dy, "dy", dy.dtype, ckpt.shape, ckpt.codes.get_device())
    return _backward("igc_layer_norm_q8_backward", dy, code, (ckpt.codes.data_ptr(), ckpt.scales.data_ptr()), rstd, weight,
                     need_dweight)


def checkpoint_pack(x: torch.Tensor) -> Checkpoint8:
    """x [n, c] in 8 bits, one scale per row and 64 channels (igc_checkpoint_pack)."""
    code = _rows(x, "x")
    (n, c), dev = x.shape, x.device
    ckpt = _new_checkpoint(n, c, x.dtype, dev)
    _call("igc_checkpoint_pack", dev.index, x.data_ptr(), n, c, code, ckpt.codes.data_ptr(), ckpt.scales.data_ptr())
    return ckpt


def checkpoint_unpack(ckpt: Checkpoint8, dtype: torch.dtype | None = None) -> torch.Tensor:
    """The values a checkpoint stands for, in its own type or `dtype` (igc_checkpoint_unpack)."""
    dt = ckpt.dtype if dtype is None else dtype
    code = _dtype_code(dt)
    (n, c), dev = ckpt.codes.shape, ckpt.codes.device
    x = torch.empty((n, c), dtype=dt, device=dev)
    _call("igc_checkpoint_unpack", dev.index, ckpt.codes.data_ptr(), ckpt.scales.data_ptr(), n, c, code, x.data_ptr())
    return x


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype, index: int) -> None:
    """Checks a [rows, heads, dim] operand; row and head strides are free."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [rows, heads, dim], got {tuple(t.shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    if t.get_device() != index:
        raise ValueError("all operands must be on one device")


_ATTENTION = struct.Struct("@iiiiifqqqqqqqqPPP")  # igc_attention_t


def _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale) -> tuple[bytes, tuple]:
    """The problem as an igc_attention_t, and the sizes its workspace depends on."""
    dt = q.dtype
    code = _dtype_code(dt)
    index = q.get_device()
    _heads(q, "q", dt, index), _heads(k, "k", dt, index), _heads(v, "v", dt, index)
    (nq, heads, dim), (nk, kv_heads, kdim) = q.shape, k.shape
    if k.shape != v.shape or kdim != dim:
        raise ValueError(f"k and v must have shape [n, kv_heads, {dim}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"heads ({heads}) must be a multiple of kv_heads ({kv_heads})")
    if (q_offsets is None) != (kv_offsets is None):
        raise ValueError("q_offsets and kv_offsets come together")
    batch = 1
    if q_offsets is not None:
        batch = q_offsets.shape[0] - 1 if q_offsets.dim() == 1 else 0
        if batch < 1 or q_offsets.shape != kv_offsets.shape:
            raise ValueError("q_offsets and kv_offsets must have shape [batch + 1]")
        _same(q_offsets, "q_offsets", torch.int32, (batch + 1,), index)
        _same(kv_offsets, "kv_offsets", torch.int32, (batch + 1,), index)
    if key_mask is not None:
        mask_type = torch.bool if getattr(key_mask, "dtype", None) == torch.bool else torch.uint8
        _same(key_mask, "key_mask", mask_type, (nk,), index)
    (q0, q1, _), (k0, k1, _), (v0, v1, _) = q.stride(), k.stride(), v.stride()
    sizes = (code, batch, heads, kv_heads, dim)
    p = _ATTENTION.pack(*sizes, dim ** -0.5 if scale is None else scale, nq, nk, q0, q1, k0, k1, v0, v1,
                        _ptr(q_offsets) or 0, _ptr(kv_offsets) or 0, _ptr(key_mask) or 0)
    return p, sizes + (nq, nk)


@functools.lru_cache(maxsize=256)
def _attention_workspace(backward: int, code: int, batch: int, heads: int, kv_heads: int, dim: int, nq: int,
                         nk: int) -> int:
    # The offsets' addresses only have to be there: the size depends on the counts alone.
    p = _ATTENTION.pack(code, batch, heads, kv_heads, dim, 1.0, nq, nk, 0, 0, 0, 0, 0, 0, 16, 16, 0)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().igc_cross_attention_workspace(p, backward, ctypes.byref(n)))
    return n.value


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor | None = None,
                    kv_offsets: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                    scale: float | None = None):
    """Attention of q [nq, heads, dim] to k and v [nk, kv_heads, dim] (kv_heads divides heads, dim up to 128,
    any row and head strides), sequence by sequence: rows q_offsets[b] .. q_offsets[b+1] of q attend to rows
    kv_offsets[b] .. kv_offsets[b+1] of k and v (int32 [batch + 1] on the device; None: one sequence).
    key_mask (bool or uint8 [nk]): false rows are left out. scale defaults to dim ** -0.5. Returns (out
    [nq, heads, dim], lse [nq, heads] float32); a row without keys gets zeros and -inf, a row of no sequence is left
    unwritten, in the gradients too (igc_cross_attention)."""
    p, sizes = _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dev = q.device
    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    n = _attention_workspace(0, *sizes)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _call("igc_cross_attention", dev.index, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
          _ptr(ws), n)
    return out, lse


def cross_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                             lse: torch.Tensor, q_offsets: torch.Tensor | None = None,
                             kv_offsets: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                             scale: float | None = None, need_dq: bool = True, need_dkv: bool = True):
    """Gradients (dq, dk, dv) of cross_attention for the output gradient dout, from its inputs and results;
    None for those not needed (igc_cross_attention_backward)."""
    p, sizes = _problem(q, k, v, q_offsets, kv_offsets, key_mask, scale)
    dt, dev = q.dtype, q.device
    _same(dout, "dout", dt, q.shape, dev.index), _same(out, "out", dt, q.shape, dev.index)
    _same(lse, "lse", torch.float32, q.shape[:2], dev.index)
    dq = torch.empty(q.shape, dtype=dt, device=dev) if need_dq else None
    dk = torch.empty(k.shape, dtype=dt, device=dev) if need_dkv else None
    dv = torch.empty(k.shape, dtype=dt, device=dev) if need_dkv else None
    n = _attention_workspace(1, *sizes)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _call("igc_cross_attention_backward", dev.index, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), dout.data_ptr(), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), n)
    return dq, dk, dv
