"""float64 restatements of qk_norm_rope and window_attn with their gradients, and bounds on what 16-bit tensors and
float32 arithmetic may differ from them.  Head tensors are [B, H, N, d] float64 arrays here."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
# Scores come from fp32 accumulators whose additions may truncate: an error of at most d * 2^-23 of sum |q k|
# (d <= 128), doubled for the subtraction of the maximum; ex2 adds 2^-22 relative.
SCORE = 2.0 ** -15


# ------------------------------------------------------------------ norm and rotation
def angles(grid, d, split=None, theta=10000.0, first=(0, 0, 0)):
    """[N, d / 2] rotation angles of the raster-ordered tokens."""
    if split is None:
        s = 2 * (d // 6)
        split = (d - 2 * s, s, s)
    T, Hh, W = grid
    out = np.zeros((T * Hh * W, d // 2))
    for n in range(T * Hh * W):
        pos = (n // (Hh * W), n // W % Hh, n % W)
        row = []
        for a in range(3):
            row += [(pos[a] + first[a]) * theta ** (-2.0 * i / split[a]) for i in range(split[a] // 2)]
        out[n] = row
    return out


def _split(x, interleaved):
    h = x.shape[-1] // 2
    return (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])


def _join(a, b, interleaved):
    if not interleaved:
        return np.concatenate((a, b), -1)
    out = np.empty(a.shape[:-1] + (2 * a.shape[-1],))
    out[..., 0::2], out[..., 1::2] = a, b
    return out


def rotate(x, ang, interleaved, sign=1.0):
    a, b = _split(x, interleaved)
    c, s = np.cos(ang), sign * np.sin(ang)
    return _join(a * c - b * s, a * s + b * c, interleaved)


def norm_rope(x, w, eps, ang, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r * w
    return y if ang is None else rotate(y, ang, interleaved)


def norm_rope_bwd(dy, x, w, eps, ang, interleaved):
    """(dx, dw, scale of dx's terms, sum of |dw terms|)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    g = dy if ang is None else rotate(dy, ang, interleaved, -1.0)
    h = g * w
    m = (h * u).mean(-1, keepdims=True)
    terms = r * (np.abs(h) + np.abs(u) * np.abs(h * u).mean(-1, keepdims=True))
    return r * (h - u * m), (g * u).sum((0, 1, 2)), terms, np.abs(g * u).sum((0, 1, 2))


# ------------------------------------------------------------------ window attention
def visible(Nq, Nk, length, start, window, sink, unit):
    """bool [Nq, Nk]: the definition, pair by pair."""
    see = np.zeros((Nq, Nk), bool)
    for i in range(Nq):
        p = start + i
        if p < 0:
            continue
        for j in range(min(length, Nk)):
            u, w = p // unit, j // unit
            see[i, j] = w <= u and (u - w < window or w < sink)
    return see


def window_head(q, k, v, see, scale):
    """O, LSE, P and sum of P |v| of one head."""
    z = np.where(see, scale * (q @ np.where(see.any(0)[:, None], k, 0.0).T), -np.inf)
    m = z.max(-1, keepdims=True)
    m[~np.isfinite(m)] = 0.0
    e = np.exp(z - m)
    l = e.sum(-1, keepdims=True)
    P = e / np.where(l == 0, 1.0, l)
    v = np.where(see.any(0)[:, None], v, 0.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return P @ v, lse, P, P @ np.abs(v)


def window_fwd(q, k, v, sees, scale, u):
    """(O, LSE, bound on |O - o|, bound on |LSE - lse|) over [B, Hq, N, d]; u: half a step of the 16-bit type.  P is
    rounded once to that type before it meets V, O once at the end."""
    B, Hq, Nq, d = q.shape
    g = Hq // k.shape[1]
    O, L = np.zeros(q.shape), np.zeros(q.shape[:3])
    bo, bl = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        rows = sees[b].any(1)
        for h in range(Hq):
            Q = np.where(rows[:, None], q[b, h], 0.0)
            O[b, h], L[b, h], P, pv = window_head(Q, k[b, h // g], v[b, h // g], sees[b], scale)
            K = np.where(sees[b].any(0)[:, None], k[b, h // g], 0.0)
            s = SCORE * np.where(sees[b], scale * (np.abs(Q) @ np.abs(K).T), 0.0).max(-1, initial=0.0)
            bl[b, h] = s + 2.0 ** -20 * np.maximum(1.0, np.abs(np.where(rows, L[b, h], 0.0)))
            bo[b, h] = u * np.abs(O[b, h]) * 1.01 + (u + 2 * s + 2.0 ** -18)[:, None] * pv + 2.0 ** -24
    return O, L, bo, bl


def window_bwd(do, q, k, v, sees, scale, u):
    """(dq, dk, dv) and bounds on what they may differ by: P and dS are rounded once to the 16-bit type (fp16, half a
    step u = 2^-11, has no steps finer than 2^-24, so values below its normal range are off by up to 2^-25), O (inside
    delta) is the forward's."""
    low = 2.0 ** -25 if u == 2.0 ** -11 else 0.0
    B, Hq, Nq, d = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    _, _, bo, bl = window_fwd(q, k, v, sees, scale, u)
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    tol = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    for b in range(B):
        see, rows, cols = sees[b], sees[b].any(1)[:, None], sees[b].any(0)[:, None]
        for h in range(Hq):
            Q, G = np.where(rows, q[b, h], 0.0), np.where(rows, do[b, h], 0.0)
            K, V = np.where(cols, k[b, h // g], 0.0), np.where(cols, v[b, h // g], 0.0)
            O, _, P, _ = window_head(Q, K, V, see, scale)
            dP = G @ V.T
            delta = (G * O).sum(-1, keepdims=True)
            dS = P * (dP - delta) * scale
            rel = (2 * bl[b, h])[:, None]                          # of P, from its score and its LSE
            E = scale * P * ((u + rel) * np.abs(dP - delta) + SCORE * (np.abs(G) @ np.abs(V).T)
                             + (np.abs(G) * bo[b, h]).sum(-1, keepdims=True)) + scale * low * see
            out[0][b, h] = dS @ K
            out[1][b, h // g] += dS.T @ Q
            out[2][b, h // g] += P.T @ G
            tol[0][b, h] = E @ np.abs(K)
            tol[1][b, h // g] += E.T @ np.abs(Q)
            tol[2][b, h // g] += (P * (u + rel) + low * see).T @ np.abs(G)
    return out, [t + u * 1.01 * np.abs(o) + 2.0 ** -23 for t, o in zip(tol, out)]
