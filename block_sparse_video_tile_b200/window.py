"""Attention over a sliding window of units (latent frames, or single tokens) with the first units kept, its form for
a few query tokens against a long cache, and its gradient (vsa_window_attn of include/vsa.h)."""
from __future__ import annotations

import math

import torch

from ._native import VsaWindow, check, lib
from ._strided import AXES, DTYPES, Plans, apart, dims, empty_f32, head_tensor, on, sig, spread, strides

__all__ = ["window_attn", "window_attn_bwd"]

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


_PLANS = Plans()


def _plan(q, k, v, window, sink, unit, layout, scale, do=None, out=None, lse=None):
    """(vsa_window without addresses, shape of O, shape of dK and dV, scale, workspace bytes) of checked arguments;
    the backward call gives do, out and lse."""
    key = (sig(q), sig(k), sig(v), window, sink, unit, layout, scale, sig(do), sig(out), sig(lse))
    plan = _PLANS.get(key)
    if plan is not None:
        return plan
    B, Nq, Hq, d = dims("q", q, layout)
    _, Nk, Hkv, _ = dims("k", k, layout)
    if q.dtype not in DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    device, dtype = q.device, q.dtype
    head_tensor("q", q, None, layout, dtype, device)
    head_tensor("k", k, (B, Nk, Hkv, d), layout, dtype, device)
    head_tensor("v", v, (B, Nk, Hkv, d), layout, dtype, device)
    for name, x, lo in (("window", window, 1), ("sink", sink, 0), ("unit", unit, 1)):
        if not lo <= x < 1 << 31:
            raise ValueError(f"{name} must be at least {lo} (and fit 32 bits), got {x}")
    oshape = (B, Hq, Nq, d) if layout == "bhnd" else (B, Nq, Hq, d)
    kshape = (B, Hkv, Nk, d) if layout == "bhnd" else (B, Nk, Hkv, d)
    no, nk = (strides(torch.empty(x, device="meta"), layout) for x in (oshape, kshape))
    if do is not None:
        head_tensor("do", do, (B, Nq, Hq, d), layout, dtype, device)
        head_tensor("out", out, (B, Nq, Hq, d), layout, dtype, device)
        _check_lse(lse, (B, Hq, Nq), device)
    w = VsaWindow(B, Hq, Hkv, Nq, Nk, d, DTYPES[dtype], window, sink, unit, 0, 0, strides(q, layout), strides(k, layout),
                  strides(v, layout), no if do is None else strides(out, layout), no if do is None else strides(do, layout),
                  no, nk, nk)
    size = 0
    if B and Nq and Hq and Nk and Hkv:
        size = (lib().vsa_window_attn_workspace_bytes if do is None else lib().vsa_window_attn_bwd_workspace_bytes)(w)
    return _PLANS.keep(key, (w, oshape, kshape, 1.0 / math.sqrt(d) if scale is None else scale, size))


def _check_lse(lse, shape, device):
    if not (lse.device == device and lse.dtype is torch.float32 and lse.is_contiguous() and tuple(lse.shape) == shape):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {shape} on {device}")


def _tensor(x):
    return x if isinstance(x, torch.Tensor) else None


def window_attn(q, k, v, window: int, *, sink: int = 0, unit: int = 1, kv_len=None, q_start=None,
                layout: str = "bhnd", scale=None, out=None, lse=None, stream=None):
    """(O, LSE) of attention over a sliding window: position p sees key j if j < kv_len, j // unit <= p // unit, and
    p // unit - j // unit < window or j // unit < sink.  unit: tokens of a unit (Hh * W for latent frames: a frame's
    tokens see each other); 1 is token-causal attention over the last `window` tokens and the first `sink`.

    q: [B, Hq, Nq, d], k and v: [B, Hkv, Nk, d] (or the "bnhd" order), views with contiguous channels; Hq a multiple
    of Hkv.  kv_len: keys held of each sequence (device int32 [B], or an int; default Nk); rows behind it may hold
    anything.  q_start: position of the first query (default kv_len - Nq: the queries are the last tokens).  A query
    that sees nothing gets O = 0 and LSE = -inf.  What some query sees must be finite (a NaN there makes the rows that
    see it NaN, and may make others NaN too).  O is like q, LSE float32 [B, Hq, Nq]; both can be given, apart from the
    inputs and each other (from first to last byte)."""
    t, oshape, _, scale, size = _plan(q, k, v, window, sink, unit, layout, scale)
    device, B, Nk = q.device, t.B, t.Nk
    if out is not None or lse is not None:
        if out is not None:
            b, n, h = AXES[layout]
            head_tensor("out", out, (oshape[b], oshape[n], oshape[h], oshape[3]), layout, q.dtype, device)
        if lse is not None:
            _check_lse(lse, (B, t.Hq, t.Nq), device)
        apart([(name, x) for name, x in (("out", out), ("lse", lse)) if x is not None],
              [("q", q), ("k", k), ("v", v)] + [(name, x) for name, x in (("kv_len", kv_len), ("q_start", q_start))
                                                if isinstance(x, torch.Tensor)])
    def run(st):
        n = _positions("kv_len", kv_len, 0, Nk, B, device)
        p0 = _positions("q_start", q_start, -_MAX_POS, _MAX_POS, B, device)
        w = VsaWindow.from_buffer_copy(t)
        if out is None:
            o = q.new_empty(*oshape)
        else:
            o = out
            w.o_s = strides(o, layout)
        ls = empty_f32(device, B, t.Hq, t.Nq) if lse is None else lse
        if not (B and t.Nq and t.Hq):
            return o, ls
        if not (Nk and t.Hkv):
            return o.zero_(), ls.fill_(-math.inf)
        if n is not None:
            w.kv_len = n.data_ptr()
        if p0 is not None:
            w.q_start = p0.data_ptr()
        ws = empty_f32(device, (size + 3) // 4) if size else None
        check("vsa_window_attn", lib().vsa_window_attn(
            w, q.data_ptr(), k.data_ptr(), v.data_ptr(), scale, o.data_ptr(), ls.data_ptr(),
            ws.data_ptr() if size else None, size, st))
        return o, ls

    return on(device, stream, (q, k, v, _tensor(kv_len), _tensor(q_start), out, lse), run)


def window_attn_bwd(do, q, k, v, out, lse, window: int, *, sink: int = 0, unit: int = 1, kv_len=None, q_start=None,
                    layout: str = "bhnd", scale=None, stream=None):
    """Gradient of window_attn: (dq, dk, dv) from the gradient of O, the inputs and the (O, LSE) that it gave, with
    the same window.  A key/value head's gradient is the sum over its query heads; keys that no query sees get
    zeros.  Every sum has a fixed order (the same bits each time).  A broadcast gradient (strides of 0) is copied
    first."""
    do = spread(do, stream)
    t, oshape, kshape, scale, size = _plan(q, k, v, window, sink, unit, layout, scale, do, out, lse)
    device, B = q.device, t.B
    def run(st):
        n = _positions("kv_len", kv_len, 0, t.Nk, B, device)
        p0 = _positions("q_start", q_start, -_MAX_POS, _MAX_POS, B, device)
        dq, dk, dv = q.new_empty(*oshape), k.new_empty(*kshape), k.new_empty(*kshape)
        if not (B and t.Nq and t.Hq and t.Nk and t.Hkv):
            return dq.zero_(), dk.zero_(), dv.zero_()
        w = VsaWindow.from_buffer_copy(t)
        if n is not None:
            w.kv_len = n.data_ptr()
        if p0 is not None:
            w.q_start = p0.data_ptr()
        ws = empty_f32(device, (size + 3) // 4)
        check("vsa_window_attn_bwd", lib().vsa_window_attn_bwd(
            w, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), scale,
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), size, st))
        return dq, dk, dv

    return on(device, stream, (do, q, k, v, out, lse, _tensor(kv_len), _tensor(q_start)), run)
