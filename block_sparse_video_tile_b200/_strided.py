"""Checks that the strided-tensor calls (norm_rope.py, window.py) share.

These calls take tensors by strides, so views of a fused projection and caches
with room to grow are passed as they are; the C ABI checks alignment and
strides, and what is only known here (types, devices, shapes) is checked here.
"""
from __future__ import annotations

import contextlib

import torch

from ._native import DTYPE_BF16, DTYPE_F16

DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
# axes of b, n, h in each layout
AXES = {"bhnd": (0, 2, 1), "bnhd": (0, 1, 2)}


def dims(name: str, x: torch.Tensor, layout: str):
    """(B, N, H, d) of a head tensor."""
    if layout not in AXES:
        raise ValueError(f"layout must be 'bhnd' or 'bnhd', got {layout!r}")
    if x.dim() != 4:
        raise ValueError(f"{name}: expected a 4-D tensor, got shape {tuple(x.shape)}")
    b, n, h = AXES[layout]
    s = x.shape
    return s[b], s[n], s[h], s[3]


def head_tensor(name: str, x: torch.Tensor, want, layout: str, dtype, device) -> None:
    """x has (B, N, H, d) = want (None: any), the type and the device, and contiguous channels."""
    if not x.is_cuda or x.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {x.device}")
    if x.dtype is not dtype:
        raise ValueError(f"{name} is {x.dtype}, expected {dtype}")
    if x.dim() != 4 or x.stride(3) != 1:
        raise ValueError(f"{name} must be 4-D with contiguous channels")
    if want is not None and dims(name, x, layout) != want:
        raise ValueError(f"{name} has (B, N, H, d) = {dims(name, x, layout)} in layout {layout}, expected {want}")


def strides(x: torch.Tensor, layout: str):
    b, n, h = AXES[layout]
    s = x.stride()
    return s[b], s[n], s[h]


def _span(x: torch.Tensor):
    """First and last-plus-one byte of a tensor."""
    n = sum((e - 1) * s for e, s in zip(x.shape, x.stride()))
    p = x.data_ptr()
    return p, p + (n + 1) * x.element_size()


def apart(outs, ins) -> None:
    """No output given by the caller shares memory with an input or another output."""
    for i, (name, o) in enumerate(outs):
        a, b = _span(o)
        for other, x in list(ins) + list(outs[:i]):
            c, e = _span(x)
            if a < e and c < b:
                raise ValueError(f"{name} overlaps {other}")


@contextlib.contextmanager
def _other(device, stream, tensors):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
            return
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):            # what the call allocates belongs to its stream
            yield stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)            # not reused before the stream is done with it


# The handle of a device's current stream, without an object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def on(device, stream, tensors, run):
    """run(stream handle) on the tensors' device and the given stream (None: that device's current one).  Inputs and
    outputs of a given stream are kept until it is done with them."""
    if stream is None and device.index == torch.cuda.current_device():
        return run(_raw_stream(device.index))
    with _other(device, stream, tensors) as st:
        return run(st)


def spread(x, stream):
    """A gradient as it is, or copied out (on the call's stream) where it was broadcast: o.sum().backward() gives one
    value with strides of 0, which the kernels do not take."""
    if x is None or 0 not in x.stride() or not x.is_cuda or all(s or n == 1 for s, n in zip(x.stride(), x.shape)):
        return x
    return on(x.device, stream, (x,), lambda st: x.contiguous())


_F32 = {}


def empty_f32(device, *shape):
    """A new float32 tensor (new_empty of a tensor at hand takes half of torch.empty's host time)."""
    e = _F32.get(device.index)
    if e is None:
        e = _F32[device.index] = torch.empty(0, dtype=torch.float32, device=device)
    return e.new_empty(*shape)


def sig(x):
    """What the checks of a call look at in a tensor: shape, strides, type and device (never its address)."""
    return None if x is None else (x.shape, x.stride(), x.dtype, x.get_device())


class Plans(dict):
    """Checked argument structures by the signatures of a call's tensors and its other arguments; a call copies its
    structure and fills in the addresses.  Emptied when it has grown large."""

    def keep(self, key, plan):
        if len(self) >= 512:
            self.clear()
        self[key] = plan
        return plan
