"""RMS norm of query and key heads with the 3-D position rotation in the same pass, and its gradient
(vsa_qk_norm_rope of include/vsa.h): what a video transformer's layer does to q and k before its attention."""
from __future__ import annotations

import torch

from ._native import VsaNormRope, VsaQkSide, check, lib
from ._strided import AXES, DTYPES, Plans, apart, dims, empty_f32, head_tensor, on, sig, spread, strides

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


def _check_table(name, table, grid, split, device):
    if table is None:
        return
    rows = sum(n * (s // 2) for n, s in zip(grid, split))
    if not (table.device == device and table.dtype is torch.float32 and table.is_contiguous()
            and tuple(table.shape) == (rows, 2)):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(rows, 2)} on {device}")


def _check_weight(name, w, d, dtype, device):
    if w is None:
        return
    if not (w.device == device and w.dtype in (dtype, torch.float32) and w.shape == (d,) and w.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous [{d}] tensor of type {dtype} or float32 on {device}")


_PLANS = Plans()


def _plan(key, q, k, grid, grid_k, split, eps, interleaved, layout, table, table_k, q_weight, k_weight, dy):
    """(vsa_norm_rope, [for q and for k: (vsa_qk_side without addresses, shape of a result)]) of checked arguments.
    dy: gradients of the results for the backward call, else None."""
    plan = _PLANS.get(key)
    if plan is not None:
        return plan
    _, _, _, d = dims("q", q, layout)
    if q.dtype not in DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    device, dtype = q.device, q.dtype
    split = rope_split(d) if split is None else tuple(split)
    if k is not None and table is not None and table_k is None and grid_k != grid:
        raise ValueError("keys on their own grid need table_k")
    p = VsaNormRope(d, DTYPES[dtype], int(bool(interleaved)), split, eps)
    sides = []
    for name, x, g, t, w, gy in (("q", q, grid, table, q_weight, dy and dy[0]),
                                 ("k", k, grid_k, table if table_k is None else table_k, k_weight, dy and dy[1])):
        if x is None:
            sides.append(None)
            continue
        if len(g) != 3:
            raise ValueError("a grid is (T, Hh, W)")
        head_tensor(name, x, None, layout, dtype, device)
        B, N, H, dd = dims(name, x, layout)
        if (N, dd) != (g[0] * g[1] * g[2], d):
            raise ValueError(f"{name} has {N} tokens of {dd} channels, the grid {g} and q ask for "
                             f"{g[0] * g[1] * g[2]} of {d}")
        if dy is not None:
            head_tensor(f"d{name}_out", gy, (B, N, H, d), layout, dtype, device)
        _check_table("table", t, g, split, device)
        _check_weight(name + "_weight", w, d, dtype, device)
        shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
        new = strides(torch.empty(shape, device="meta"), layout)
        side = VsaQkSide(B, H, *g, int(w is not None and w.dtype is torch.float32), 0, strides(x, layout), 0,
                         new if dy is None else strides(gy, layout), 0, new, 0, 0, 0)
        sides.append((side, shape) if B and N and H else (None, shape))
    return _PLANS.keep(key, (p, sides))


def _key(q, k, grid, grid_k, split, eps, interleaved, layout, table, table_k, q_weight, k_weight, dy):
    return (sig(q), sig(k), grid, grid_k, None if split is None else tuple(split), eps, interleaved, layout, sig(table),
            sig(table_k), sig(q_weight), sig(k_weight), None if dy is None else (sig(dy[0]), sig(dy[1])))


def _side(side, x, y, t, w):
    """A side's argument structure with its addresses (None where it has no rows)."""
    if side is None or side[0] is None:
        return None
    c = VsaQkSide.from_buffer_copy(side[0])
    c.x = x.data_ptr()
    c.y = y.data_ptr()
    if w is not None:
        c.weight = w.data_ptr()
    if t is not None:
        c.table = t.data_ptr()
    return c


def qk_norm_rope(q, k, grid, *, table=None, table_k=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 split=None, grid_k=None, interleaved: bool = True, layout: str = "bhnd", out=None, stream=None):
    """(q', k') = rotation of the RMS-normed rows of q and k, for each token and head:
    R(position) (weight * x / sqrt(mean(x^2) + eps)), rounded once to the type of q.

    q, k: [B, H, N, d] or [B, N, H, d] views with contiguous channels (k may be None, and have its own batch, heads
    and grid).  table: rope_table(grid, d, ...), None for no rotation; table_k: the keys' (default: table, when the
    keys have the queries' grid).  q_weight, k_weight: [d], the type of q or float32; None for ones.  interleaved: a
    pair is channels (2p, 2p + 1), else (p, p + d/2).  out: (q', k') to write to, apart from the inputs and each other
    (from first to last byte: interleaved views of one buffer are refused).  The norm is over the d channels of each
    head; a norm over all heads' channels together is not this call."""
    grid = tuple(grid)
    args = (q, k, grid, grid if grid_k is None else tuple(grid_k), split, eps, interleaved, layout, table, table_k,
            q_weight, k_weight, None)
    p, sides = _plan(_key(*args), *args)
    device = q.device
    if out is not None:
        for y, side in zip(out, sides):
            if side is not None:
                b, n, h = AXES[layout]
                s = side[1]
                head_tensor("out", y, (s[b], s[n], s[h], s[3]), layout, q.dtype, device)
        apart([("out", y) for y in out if y is not None],
              [(n, x) for n, x in (("q", q), ("k", k), ("table", table), ("table_k", table_k), ("q_weight", q_weight),
                                  ("k_weight", k_weight))
               if x is not None])
    def run(st):
        sq, sk = sides
        yq, yk = out if out is not None else (q.new_empty(*sq[1]), None if sk is None else k.new_empty(*sk[1]))
        cq = _side(sq, q, yq, table, q_weight)
        ck = _side(sk, k, yk, table if table_k is None else table_k, k_weight)
        if out is not None:
            for c, y in ((cq, yq), (ck, yk)):
                if c is not None:
                    c.y_s = strides(y, layout)
        if cq is None:
            cq, ck = ck, None
        if cq is not None:
            check("vsa_qk_norm_rope", lib().vsa_qk_norm_rope(p, cq, ck, st))
        return yq, yk

    return on(device, stream, (q, k, table, table_k, q_weight, k_weight, *(out or ())), run)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, grid, *, table=None, table_k=None, q_weight=None, k_weight=None,
                     eps: float = 1e-6, split=None, grid_k=None, interleaved: bool = True, layout: str = "bhnd",
                     stream=None):
    """Gradient of qk_norm_rope: (dq, dk, dq_weight, dk_weight) from the gradients of its results and its inputs.
    The weights' gradients are float32 [d], None where the weight is None, summed in a fixed order.  Broadcast gradients
    (strides of 0) are copied first."""
    grid = tuple(grid)
    if (k is None) != (dk_out is None):
        raise ValueError("give k and dk_out, or neither")
    dq_out, dk_out = spread(dq_out, stream), spread(dk_out, stream)
    args = (q, k, grid, grid if grid_k is None else tuple(grid_k), split, eps, interleaved, layout, table, table_k,
            q_weight, k_weight, (dq_out, dk_out))
    p, sides = _plan(_key(*args), *args)
    device = q.device
    def grad(side, x, dy, t, w):
        """(argument structure, dx, dweight) of a side."""
        if side is None:
            return None, None, None
        gx = x.new_empty(*side[1])
        gw = None if w is None else empty_f32(device, p.d)
        c = _side(side, x, dy, t, w)
        if c is not None:
            c.dx = gx.data_ptr()
            if w is not None:
                c.dweight = gw.data_ptr()
        elif gw is not None:
            gw.zero_()
        return c, gx, gw

    def run(st):
        cq, gq, gwq = grad(sides[0], q, dq_out, table, q_weight)
        ck, gk, gwk = grad(sides[1], k, dk_out, table if table_k is None else table_k, k_weight)
        if cq is None:
            cq, ck = ck, None
        if cq is not None:
            n = lib().vsa_qk_norm_rope_bwd_workspace_bytes(p, cq, ck)
            ws = empty_f32(device, (n + 3) // 4) if n else None
            check("vsa_qk_norm_rope_bwd", lib().vsa_qk_norm_rope_bwd(p, cq, ck, ws.data_ptr() if n else None, n, st))
        return gq, gk, gwq, gwk

    return on(device, stream, (q, k, dq_out, dk_out, table, table_k, q_weight, k_weight), run)
