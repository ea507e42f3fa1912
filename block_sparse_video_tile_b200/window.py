"""Attention over a sliding window of units (latent frames, or single tokens) with the first units kept, its form for
a few query tokens against a long cache, and its gradient (vsa_window_attn of include/vsa.h)."""
from __future__ import annotations

import math

import torch

from ._native import VsaWindow, check, lib
from ._strided import DTYPES, apart, dims, head_tensor, new_heads, on, strides

__all__ = ["window_attn", "window_attn_bwd"]

_NO = (0, 0, 0)
_MAX_POS = 1 << 30


def _positions(name, x, lo, hi, B, device):
    """A device int32 [B] tensor as it is, an int as such a tensor, None as None."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if not (x.device == device and x.dtype is torch.int32 and x.is_contiguous() and x.shape == (B,)):
            raise ValueError(f"{name} must be a contiguous int32 [{B}] tensor on {device}, or an int")
        return x
    if not lo <= x <= hi:
        raise ValueError(f"{name} must lie in [{lo}, {hi}], got {x}")
    return torch.full((B,), int(x), dtype=torch.int32, device=device)


def _common(q, k, v, window, sink, unit, layout, scale):
    B, Nq, Hq, d = dims("q", q, layout)
    Bk, Nk, Hkv, _ = dims("k", k, layout)
    if q.dtype not in DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    device, dtype = q.device, q.dtype
    head_tensor("q", q, None, layout, dtype, device)
    head_tensor("k", k, (B, Nk, Hkv, d), layout, dtype, device)
    head_tensor("v", v, (B, Nk, Hkv, d), layout, dtype, device)
    for name, x, lo in (("window", window, 1), ("sink", sink, 0), ("unit", unit, 1)):
        if not lo <= x < 1 << 31:
            raise ValueError(f"{name} must be at least {lo} (and fit 32 bits), got {x}")
    return B, Nq, Hq, d, Nk, Hkv, 1.0 / math.sqrt(d) if scale is None else scale


def window_attn(q, k, v, window: int, *, sink: int = 0, unit: int = 1, kv_len=None, q_start=None,
                layout: str = "bhnd", scale=None, out=None, lse=None, stream=None):
    """(O, LSE) of attention over a sliding window: position p sees key j if j < kv_len, j // unit <= p // unit, and
    p // unit - j // unit < window or j // unit < sink.  unit: tokens of a unit (Hh * W for latent frames: a frame's
    tokens see each other); 1 is token-causal attention over the last `window` tokens and the first `sink`.

    q: [B, Hq, Nq, d], k and v: [B, Hkv, Nk, d] (or the "bnhd" order), views with contiguous channels; Hq a multiple
    of Hkv.  kv_len: keys held of each sequence (device int32 [B], or an int; default Nk); rows behind it may hold
    anything.  q_start: position of the first query (default kv_len - Nq: the queries are the last tokens).  A query
    that sees nothing gets O = 0 and LSE = -inf.  O is like q, LSE float32 [B, Hq, Nq]; both can be given, apart from
    the inputs."""
    B, Nq, Hq, d, Nk, Hkv, scale = _common(q, k, v, window, sink, unit, layout, scale)
    device = q.device
    with on(device, stream, (q, k, v, kv_len if isinstance(kv_len, torch.Tensor) else None,
                             q_start if isinstance(q_start, torch.Tensor) else None, out, lse)) as st:
        n = _positions("kv_len", kv_len, 0, Nk, B, device)
        p0 = _positions("q_start", q_start, -_MAX_POS, _MAX_POS, B, device)
        given = [(name, x) for name, x in (("out", out), ("lse", lse)) if x is not None]
        if out is None:
            out = new_heads(B, Nq, Hq, d, layout, q.dtype, device)
        else:
            head_tensor("out", out, (B, Nq, Hq, d), layout, q.dtype, device)
        if lse is None:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device)
        elif not (lse.device == device and lse.dtype is torch.float32 and lse.is_contiguous()
                  and tuple(lse.shape) == (B, Hq, Nq)):
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(B, Hq, Nq)} on {device}")
        if given:
            apart(given, [("q", q), ("k", k), ("v", v)])
        if not (B and Nq and Hq):
            return out, lse
        if not (Nk and Hkv):
            return out.zero_(), lse.fill_(-math.inf)
        w = VsaWindow(B, Hq, Hkv, Nq, Nk, d, DTYPES[q.dtype], window, sink, unit, 0 if n is None else n.data_ptr(),
                      0 if p0 is None else p0.data_ptr(), strides(q, layout), strides(k, layout), strides(v, layout),
                      strides(out, layout), _NO, _NO, _NO, _NO)
        size = lib().vsa_window_attn_workspace_bytes(w)
        ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        check("vsa_window_attn", lib().vsa_window_attn(
            w, q.data_ptr(), k.data_ptr(), v.data_ptr(), scale, out.data_ptr(), lse.data_ptr(),
            ws.data_ptr() if size else None, size, st))
    return out, lse


def window_attn_bwd(do, q, k, v, out, lse, window: int, *, sink: int = 0, unit: int = 1, kv_len=None, q_start=None,
                    layout: str = "bhnd", scale=None, stream=None):
    """Gradient of window_attn: (dq, dk, dv) from the gradient of O, the inputs and the (O, LSE) that it gave, with
    the same window.  A key/value head's gradient is the sum over its query heads; keys that no query sees get
    zeros.  Every sum has a fixed order (the same bits each time)."""
    B, Nq, Hq, d, Nk, Hkv, scale = _common(q, k, v, window, sink, unit, layout, scale)
    device, dtype = q.device, q.dtype
    head_tensor("do", do, (B, Nq, Hq, d), layout, dtype, device)
    head_tensor("out", out, (B, Nq, Hq, d), layout, dtype, device)
    if not (lse.device == device and lse.dtype is torch.float32 and lse.is_contiguous()
            and tuple(lse.shape) == (B, Hq, Nq)):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {(B, Hq, Nq)} on {device}")
    with on(device, stream, (do, q, k, v, out, lse, kv_len if isinstance(kv_len, torch.Tensor) else None,
                             q_start if isinstance(q_start, torch.Tensor) else None)) as st:
        n = _positions("kv_len", kv_len, 0, Nk, B, device)
        p0 = _positions("q_start", q_start, -_MAX_POS, _MAX_POS, B, device)
        dq = new_heads(B, Nq, Hq, d, layout, dtype, device)
        dk, dv = (new_heads(B, Nk, Hkv, d, layout, dtype, device) for _ in range(2))
        if not (B and Nq and Hq and Nk and Hkv):
            return dq.zero_(), dk.zero_(), dv.zero_()
        w = VsaWindow(B, Hq, Hkv, Nq, Nk, d, DTYPES[dtype], window, sink, unit, 0 if n is None else n.data_ptr(),
                      0 if p0 is None else p0.data_ptr(), strides(q, layout), strides(k, layout), strides(v, layout),
                      strides(out, layout), strides(do, layout), strides(dq, layout), strides(dk, layout),
                      strides(dv, layout))
        size = lib().vsa_window_attn_bwd_workspace_bytes(w)
        ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        check("vsa_window_attn_bwd", lib().vsa_window_attn_bwd(
            w, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), scale,
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr() if size else None, size, st))
    return dq, dk, dv
