"""RMS norm of query and key heads with the 3-D position rotation in the same pass, and its gradient
(vsa_qk_norm_rope of include/vsa.h): what a video transformer's layer does to q and k before its attention."""
from __future__ import annotations

import ctypes

import torch

from ._native import VsaNormRope, VsaQkSide, check, lib
from ._strided import DTYPES, apart, dims, head_tensor, new_heads, on, strides

__all__ = ["rope_split", "rope_table", "qk_norm_rope", "qk_norm_rope_bwd"]


def rope_split(d: int):
    """Channels rotated by (t, y, x): y and x get the even third 2 * (d // 6), t the rest ((44, 42, 42) of 128)."""
    s = 2 * (d // 6)
    return d - 2 * s, s, s


def rope_table(grid, d: int, *, split=None, theta: float = 10000.0, first=(0, 0, 0), device="cuda") -> torch.Tensor:
    """cos and sin of every axis position and channel pair, float32 [rows, 2]: T rows of the t pairs, then Hh rows
    of the y pairs, then W rows of the x pairs; pair i of an axis with s channels turns by (position + first) *
    theta^(-2i/s), in 64 bits.  first: where the grid begins (latent frames generated before this chunk)."""
    parts = []
    for n, s, off in zip(grid, rope_split(d) if split is None else split, first):
        pos = torch.arange(off, off + n, dtype=torch.float64, device=device)
        freq = theta ** (-torch.arange(0, s, 2, dtype=torch.float64, device=device) / max(s, 1))
        ang = pos[:, None] * freq
        parts.append(torch.stack((ang.cos(), ang.sin()), -1).reshape(-1, 2))
    return torch.cat(parts).float()


def _table(name, table, grid, split, device):
    if table is None:
        return 0
    rows = sum(n * (s // 2) for n, s in zip(grid, split))
    if not (table.device == device and table.dtype is torch.float32 and table.is_contiguous()
            and tuple(table.shape) == (rows, 2)):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(rows, 2)} on {device}")
    return table.data_ptr()


def _weight(name, w, d, dtype, device):
    if w is None:
        return 0, 0
    if not (w.device == device and w.dtype in (dtype, torch.float32) and w.shape == (d,) and w.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous [{d}] tensor of type {dtype} or float32 on {device}")
    return w.data_ptr(), int(w.dtype is torch.float32)


def _common(q, k, grid, grid_k, split, eps, interleaved, layout):
    B, N, H, d = dims("q", q, layout)
    if q.dtype not in DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    grid_k = grid if grid_k is None else grid_k
    split = rope_split(d) if split is None else split
    for name, x, g in (("q", q, grid), ("k", k, grid_k)):
        if x is None:
            continue
        if len(g) != 3:
            raise ValueError("a grid is (T, Hh, W)")
        head_tensor(name, x, None, layout, q.dtype, q.device)
        b, n, _, dd = dims(name, x, layout)
        if (n, dd) != (g[0] * g[1] * g[2], d):
            raise ValueError(f"{name} has {n} tokens of {dd} channels, the grid {tuple(g)} and q ask for "
                             f"{g[0] * g[1] * g[2]} of {d}")
    p = VsaNormRope(d, DTYPES[q.dtype], int(bool(interleaved)), tuple(split), eps)
    return p, grid_k, split


def qk_norm_rope(q, k, grid, *, table=None, table_k=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 split=None, grid_k=None, interleaved: bool = True, layout: str = "bhnd", out=None, stream=None):
    """(q', k') = rotation of the RMS-normed rows of q and k, for each token and head:
    R(position) (weight * x / sqrt(mean(x^2) + eps)), rounded once to the type of q.

    q, k: [B, H, N, d] or [B, N, H, d] views with contiguous channels (k may be None, and have its own batch, heads
    and grid).  table: rope_table(grid, d, ...), None for no rotation; table_k: the keys' (default: table, when the
    keys have the queries' grid).  q_weight, k_weight: [d], the type of q or float32; None for ones.  interleaved: a
    pair is channels (2p, 2p + 1), else (p, p + d/2).  out: (q', k') to write to, apart from the inputs."""
    p, grid_k, split = _common(q, k, grid, grid_k, split, eps, interleaved, layout)
    device, dtype, d = q.device, q.dtype, p.d
    if table_k is None and table is not None and k is not None:
        if tuple(grid_k) != tuple(grid):
            raise ValueError("keys on their own grid need table_k")
        table_k = table
    with on(device, stream, (q, k, table, table_k, q_weight, k_weight) + tuple(out or ())) as st:
        sides, outs = [], []
        for i, (name, x, g, t, w) in enumerate((("q", q, grid, table, q_weight), ("k", k, grid_k, table_k, k_weight))):
            if x is None:
                outs.append(None)
                continue
            B, N, H, _ = dims(name, x, layout)
            if out is None:
                y = new_heads(B, N, H, d, layout, dtype, device)
            else:
                y = out[i]
                head_tensor("out", y, (B, N, H, d), layout, dtype, device)
            wp, wf = _weight(name + "_weight", w, d, dtype, device)
            outs.append(y)
            if B and N and H:
                sides.append(VsaQkSide(B, H, *g, wf, x.data_ptr(), strides(x, layout), y.data_ptr(), strides(y, layout),
                                       0, (0, 0, 0), wp, _table("table", t, g, split, device), 0))
        if out is not None:
            apart([("out", o) for o in outs if o is not None],
                  [(n, x) for n, x in (("q", q), ("k", k), ("table", table), ("q_weight", q_weight),
                                       ("k_weight", k_weight)) if x is not None])
        if sides:
            check("vsa_qk_norm_rope", lib().vsa_qk_norm_rope(p, sides[0], sides[1] if len(sides) > 1 else None, st))
    return outs[0], outs[1]


def qk_norm_rope_bwd(dq_out, dk_out, q, k, grid, *, table=None, table_k=None, q_weight=None, k_weight=None,
                     eps: float = 1e-6, split=None, grid_k=None, interleaved: bool = True, layout: str = "bhnd",
                     stream=None):
    """Gradient of qk_norm_rope: (dq, dk, dq_weight, dk_weight) from the gradients of its results and its inputs.
    The weights' gradients are float32 [d], None where the weight is None, summed in a fixed order."""
    p, grid_k, split = _common(q, k, grid, grid_k, split, eps, interleaved, layout)
    device, dtype, d = q.device, q.dtype, p.d
    if (k is None) != (dk_out is None):
        raise ValueError("give k and dk_out, or neither")
    if table_k is None and table is not None and k is not None:
        if tuple(grid_k) != tuple(grid):
            raise ValueError("keys on their own grid need table_k")
        table_k = table
    with on(device, stream, (q, k, dq_out, dk_out, table, table_k, q_weight, k_weight)) as st:
        sides, dx, dw = [], [], []
        for name, x, dy, g, t, w in (("q", q, dq_out, grid, table, q_weight), ("k", k, dk_out, grid_k, table_k, k_weight)):
            if x is None:
                dx.append(None)
                dw.append(None)
                continue
            B, N, H, _ = dims(name, x, layout)
            head_tensor(f"d{name}_out", dy, (B, N, H, d), layout, dtype, device)
            wp, wf = _weight(name + "_weight", w, d, dtype, device)
            gx = new_heads(B, N, H, d, layout, dtype, device)
            some = B and N and H
            gw = None if w is None else (torch.empty if some else torch.zeros)(d, dtype=torch.float32, device=device)
            dx.append(gx)
            dw.append(gw)
            if some:
                sides.append(VsaQkSide(B, H, *g, wf, x.data_ptr(), strides(x, layout), dy.data_ptr(),
                                       strides(dy, layout), gx.data_ptr(), strides(gx, layout), wp,
                                       _table("table", t, g, split, device), 0 if gw is None else gw.data_ptr()))
        if sides:
            sk = sides[1] if len(sides) > 1 else None
            n = lib().vsa_qk_norm_rope_bwd_workspace_bytes(p, sides[0], sk)
            ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
            check("vsa_qk_norm_rope_bwd", lib().vsa_qk_norm_rope_bwd(p, sides[0], sk, ws.data_ptr() if n else None, n, st))
    return dx[0], dx[1], dw[0], dw[1]
