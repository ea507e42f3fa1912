"""The measured calls of two operators: qk_norm_rope (RMS norm of query and key heads with the 3-D position
rotation in the same pass, and its gradient) and window_attn (attention over a sliding window of units with a few
first units that stay visible, its form for a few query tokens against a long cache, and its gradient)."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 10000.0


def _norm_case(name, op, grid, H, d, dtype, layout, *, B=1, fused=False, interleaved=True, first=0):
    """grid: latent frames, rows, columns as "TxHxW"; fused: q and k are views of one [B, N, 3, H, d] projection;
    first: latent frames generated before this chunk (the rotation goes on from there)."""
    return {"name": name, "op": op, "grid": grid, "B": B, "H": H, "d": d, "dtype": dtype, "layout": layout,
            "fused": fused, "interleaved": interleaved, "first": first}


def _win_case(name, op, B, Hq, Hkv, Nq, Nk, d, window, sink, unit, dtype, layout, *, ragged=False):
    """Nq query tokens are the last ones of each sequence; ragged: sequences of the batch end at different places of
    the cache."""
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d, "window": window,
            "sink": sink, "unit": unit, "dtype": dtype, "layout": layout, "ragged": ragged}


def listed():
    return [
        # every query and key of one layer of the Wan-5B grid (31, 22, 40), straight from the fused projection
        _norm_case("norm_rope_wan5b", "norm", "31x22x40", 24, 128, "bf16", "bnhd", fused=True),
        # one new latent frame of a video that is generated frame by frame: the smallest call, latency counts
        _norm_case("norm_rope_frame", "norm", "1x22x40", 24, 128, "bf16", "bnhd", fused=True, first=30),
        # the same layer in training: gradients of q, k and both weights
        _norm_case("norm_rope_bwd_wan5b", "norm_bwd", "31x22x40", 24, 128, "bf16", "bhnd"),
        # a small odd grid, two videos, heads of 64 rotated as halves
        _norm_case("norm_rope_bwd_odd", "norm_bwd", "9x13x21", 8, 64, "f16", "bnhd", B=2, interleaved=False),
        # training forward of a frame-causal video model: 6 of 24 heads (one of four sequence-parallel ranks), 8
        # latent frames of 880 tokens in sight and the first frame
        _win_case("window_wan5b", "win", 1, 6, 6, 27280, 27280, 128, 8, 1, 880, "bf16", "bhnd"),
        # streaming: three new latent frames against a cache of 31, all heads
        _win_case("window_chunk", "win", 1, 24, 24, 2640, 27280, 128, 12, 3, 880, "bf16", "bnhd"),
        # token-causal, shared key heads, an odd length, sequences that end at different places
        _win_case("window_tokens", "win", 2, 16, 4, 8191, 8191, 64, 1024, 4, 1, "f16", "bhnd", ragged=True),
        # one new token for each of 8 long sequences
        _win_case("window_step", "win", 8, 32, 8, 1, 32768, 128, 16384, 16, 1, "bf16", "bnhd", ragged=True),
        # one new token of one short sequence: latency counts
        _win_case("window_step_small", "win", 1, 24, 24, 1, 1000, 128, 512, 4, 1, "bf16", "bhnd"),
        # training backward of window_wan5b
        _win_case("window_bwd_wan5b", "win_bwd", 1, 6, 6, 27280, 27280, 128, 8, 1, 880, "bf16", "bhnd"),
        # token-causal backward, gradients of shared key heads summed over their query heads
        _win_case("window_bwd_tokens", "win_bwd", 2, 8, 2, 4095, 4095, 64, 1024, 4, 1, "f16", "bnhd", ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "win", "win", "step", "win_bwd"))
    dtype, layout, d = rng.choice(("bf16", "f16")), rng.choice(("bhnd", "bnhd")), rng.choice((64, 128))
    if op in ("norm", "norm_bwd"):
        B, H = rng.randint(1, 3), rng.randint(1, 24)
        T, Hh, W = _log(rng, 1, 31), rng.randint(3, 40), rng.randint(3, 48)
        T = max(1, min(T, 27280 * 24 // (B * H * Hh * W)))
        fused = layout == "bnhd" and rng.random() < 0.5
        c = _norm_case("", op, "%dx%dx%d" % (T, Hh, W), H, d, dtype, layout, B=B, fused=fused,
                       interleaved=rng.random() < 0.5, first=rng.randint(0, 200))
    else:
        Hkv, g = rng.randint(1, 8), rng.choice((1, 1, 2, 4, 7))
        unit = 1 if rng.random() < 0.5 else rng.randint(30, 1000)
        if op == "step":
            B, Nq, Nk = rng.randint(1, 8), rng.choice((1, 1, 1, 2, 5, 16)), _log(rng, 64, 32768)
        else:
            B = rng.randint(1, 2)
            Nk = _log(rng, 200, 12000)
            Nq = Nk if op == "win_bwd" or rng.random() < 0.5 else rng.randint(17, Nk)
            Hkv = max(1, min(Hkv, int(1.2e9) // (B * g * Nq * Nk)))
            g = max(1, min(g, int(1.2e9) // (B * Hkv * Nq * Nk)))
        Nq = min(Nq, Nk)
        window = max(1, _log(rng, 64, 16384) // unit)
        sink = rng.choice((0, 1, 4)) if unit > 1 else rng.choice((0, 4, 16, 130))
        c = _win_case("", "win_bwd" if op == "win_bwd" else "win", B, Hkv * g, Hkv, Nq, Nk, d, window, sink, unit,
                      dtype, layout, ragged=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ shared facts of a case
def _grid(case):
    return tuple(int(x) for x in case["grid"].split("x"))


def _splits(d):
    """Channels rotated by frame, row and column: what is left of two equal even thirds goes to the frame."""
    s = 2 * (d // 6)
    return d - 2 * s, s, s


def _table(case, device):
    """cos and sin of every axis position and channel pair, float32 [rows, 2]: T rows of the frame's pairs, then Hh
    of the row's, then W of the column's, from angles in 64 bits."""
    parts = []
    for n, s, off in zip(_grid(case), _splits(case["d"]), (case["first"], 0, 0)):
        pos = torch.arange(off, off + n, dtype=torch.float64, device=device)
        freq = THETA ** (-torch.arange(0, s, 2, dtype=torch.float64, device=device) / s)
        ang = pos[:, None] * freq
        parts.append(torch.stack((ang.cos(), ang.sin()), -1).reshape(-1, 2))
    return torch.cat(parts).float()


def _lengths(case):
    """Tokens of each sequence in the cache."""
    step = case["Nk"] // (3 * case["B"]) if case["ragged"] else 0
    return [case["Nk"] - b * step for b in range(case["B"])]


def _rows(case, b_len):
    """First and last-plus-one key of the window, and the end of the first units, for each query of a sequence."""
    pos = torch.arange(b_len - case["Nq"], b_len)
    u = torch.div(pos, case["unit"], rounding_mode="floor")
    hi = ((u + 1) * case["unit"]).clamp(0, b_len)
    lo = torch.minimum(((u - case["window"] + 1) * case["unit"]).clamp(min=0), hi)
    first = torch.minimum(torch.full_like(lo, case["sink"] * case["unit"]), hi)
    return lo, hi, first


def work(case):
    d = case["d"]
    if case["op"] in ("norm", "norm_bwd"):
        T, Hh, W = _grid(case)
        n = 2 * case["B"] * T * Hh * W * case["H"]              # rows of q and k
        if case["op"] == "norm":
            return {"bytes": n * d * 4, "flops": n * d * 8}
        return {"bytes": n * d * 6, "flops": n * d * 16}
    pairs = keys = 0
    for n in _lengths(case):
        lo, hi, first = _rows(case, n)
        pairs += int((hi - lo + torch.minimum(first, lo)).sum())
        a, f = int(lo.min()), int(first.max())
        keys += int(hi.max()) - a + min(a, f)
    q_rows, kv_rows = case["B"] * case["Hq"] * case["Nq"], case["Hkv"] * keys
    if case["op"] == "win":
        return {"bytes": (q_rows * 2 + kv_rows * 2) * d * 2 + q_rows * 4, "flops": 4 * d * pairs * case["Hq"]}
    all_kv = case["B"] * case["Hkv"] * case["Nk"]                # gradients of keys that nobody sees are written too
    return {"bytes": (q_rows * 4 + kv_rows * 2 + all_kv * 2) * d * 2 + q_rows * 4,
            "flops": 10 * d * pairs * case["Hq"]}


# ------------------------------------------------------------------ inputs
def _heads(g, case, H, N, scale=1.0):
    """Normal values in the case's layout and type."""
    shape = (case["B"], H, N, case["d"]) if case["layout"] == "bhnd" else (case["B"], N, H, case["d"])
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("norm", "norm_bwd"):
        T, Hh, W = _grid(case)
        N, H, d, dt = T * Hh * W, case["H"], case["d"], DT[case["dtype"]]
        s = {"case": case, "table": _table(case, "cuda")}
        if case["fused"]:
            qkv = torch.randn((case["B"], N, 3, H, d), generator=g, device="cuda").to(dt)
            s["q"], s["k"] = qkv[:, :, 0], qkv[:, :, 1]
        else:
            s["q"], s["k"] = _heads(g, case, H, N, 1.5), _heads(g, case, H, N, 0.7)
        s["wq"], s["wk"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        if case["op"] == "norm_bwd":
            s["dq"], s["dk"] = _heads(g, case, H, N), _heads(g, case, H, N)
        return s
    s = {"case": case, "q": _heads(g, case, case["Hq"], case["Nq"]), "k": _heads(g, case, case["Hkv"], case["Nk"]),
         "v": _heads(g, case, case["Hkv"], case["Nk"]), "kv_len": None}
    if case["ragged"]:
        s["kv_len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["op"] == "win_bwd":
        s["o"], s["lse"] = _window(s)
        s["do"] = _heads(g, case, case["Hq"], case["Nq"])
    return s


# ------------------------------------------------------------------ plain forms
def _angles(s):
    """cos and sin [N, d / 2] of every token of the grid, from the axis table."""
    case, table = s["case"], s["table"]
    T, Hh, W = _grid(case)
    ct, cy, cx = (x // 2 for x in _splits(case["d"]))
    n = torch.arange(T * Hh * W, device=table.device)
    t = table[:T * ct].view(T, ct, 2)[n // (Hh * W)]
    y = table[T * ct:T * ct + Hh * cy].view(Hh, cy, 2)[n // W % Hh]
    x = table[T * ct + Hh * cy:].view(W, cx, 2)[n % W]
    return torch.cat((t, y, x), 1).unbind(-1)


def _pairs(x, case):
    return (x[..., 0::2], x[..., 1::2]) if case["interleaved"] else x.chunk(2, -1)


def _joined(a, b, case):
    return torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)


def _by_token(c, case):
    """[N, d / 2] against [B, H, N, d / 2] or [B, N, H, d / 2]."""
    return c if case["layout"] == "bhnd" else c[:, None]


def _norm_rope(x, w, cos, sin, case):
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w
    a, b = _pairs(y, case)
    return _joined(a * cos - b * sin, a * sin + b * cos, case).to(x.dtype)


def _norm_rope_bwd(dy, x, w, cos, sin, case):
    f, d = x.float(), dy.float()
    a, b = _pairs(d, case)
    gy = _joined(a * cos + b * sin, b * cos - a * sin, case)
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    u = f * r
    dw = (gy * u).double().sum((0, 1, 2)).float()
    h = gy * w
    return (r * (h - u * (h * u).mean(-1, keepdim=True))).to(x.dtype), dw


def _by_head(x, case):
    return x if case["layout"] == "bhnd" else x.transpose(1, 2)


def _visible(case, kv_len, device):
    """[B, Nq, Nk]: which keys a query sees."""
    B, Nq, Nk, unit = case["B"], case["Nq"], case["Nk"], case["unit"]
    n = torch.full((B,), Nk, device=device) if kv_len is None else kv_len.long()
    j = torch.arange(Nk, device=device)
    u = torch.div(n[:, None] - Nq + torch.arange(Nq, device=device), unit, rounding_mode="floor")[:, :, None]
    uj = torch.div(j, unit, rounding_mode="floor")
    return (uj <= u) & ((uj > u - case["window"]) | (uj < case["sink"])) & (j < n[:, None, None])


def _scores(s):
    """Scaled scores [B, Hkv, g, Nq, Nk] with -inf where nothing is seen."""
    case = s["case"]
    q, k = _by_head(s["q"], case).float(), _by_head(s["k"], case).float()
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    z = torch.matmul(q.reshape(B, Hkv, -1, d) * d ** -0.5, k.transpose(2, 3)).view(B, Hkv, -1, Nq, Nk)
    return z.masked_fill_(~_visible(case, s["kv_len"], q.device)[:, None, None], -math.inf)


def _window(s):
    case = s["case"]
    z = _scores(s)
    B, Hkv, g, Nq, Nk = z.shape
    m = z.amax(-1, keepdim=True)
    m.masked_fill_(m == -math.inf, 0.0)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, g * Nq, Nk), _by_head(s["v"], case).float()).view(B, Hkv, g, Nq, -1)
    o = (o / l.masked_fill(l == 0, 1.0)).view(B, Hkv * g, Nq, -1)
    lse = (m + l.log()).view(B, Hkv * g, Nq)
    return _by_head(o, case).to(s["q"].dtype).contiguous(), lse


def _window_bwd(s):
    case = s["case"]
    z = _scores(s)
    B, Hkv, g, Nq, Nk = z.shape
    q, k, v, o, do = (_by_head(s[n], case).float() for n in ("q", "k", "v", "o", "do"))
    d = q.shape[-1]
    lse = s["lse"].view(B, Hkv, g, Nq, 1)
    p = z.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_().view(B, Hkv, g * Nq, Nk)
    rows = do.reshape(B, Hkv, g * Nq, d)
    dv = torch.matmul(p.transpose(2, 3), rows)
    delta = (do * o).sum(-1).view(B, Hkv, g * Nq, 1)
    ds = torch.matmul(rows, v.transpose(2, 3)).sub_(delta).mul_(p).mul_(d ** -0.5)
    dk = torch.matmul(ds.transpose(2, 3), q.reshape(B, Hkv, g * Nq, d))
    dq = torch.matmul(ds, k).view(B, Hkv * g, Nq, d)
    return tuple(_by_head(x, case).to(s["q"].dtype).contiguous() for x in (dq, dk, dv))


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from block_sparse_video_tile_b200 import api
        if op in ("norm", "norm_bwd"):
            how = dict(table=s["table"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, layout=case["layout"],
                       interleaved=case["interleaved"])
            if op == "norm":
                return api.qk_norm_rope(s["q"], s["k"], _grid(case), **how)
            return api.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], _grid(case), **how)
        how = dict(sink=case["sink"], unit=case["unit"], kv_len=s["kv_len"], layout=case["layout"])
        if op == "win":
            return api.window_attn(s["q"], s["k"], s["v"], case["window"], **how)
        return api.window_attn_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], case["window"], **how)
    if op in ("norm", "norm_bwd"):
        cos, sin = (_by_token(c, case) for c in _angles(s))
        if op == "norm":
            return _norm_rope(s["q"], s["wq"], cos, sin, case), _norm_rope(s["k"], s["wk"], cos, sin, case)
        dq, dwq = _norm_rope_bwd(s["dq"], s["q"], s["wq"], cos, sin, case)
        dk, dwk = _norm_rope_bwd(s["dk"], s["k"], s["wk"], cos, sin, case)
        return dq, dk, dwq, dwk
    return _window(s) if op == "win" else _window_bwd(s)


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_norm(case, s):
    """y = R (w x / rms(x)), the rotation as a product with e^{i angle}; gradients by the chain rule on complex
    pairs."""
    T, Hh, W = _grid(case)
    d = case["d"]
    place = torch.stack(torch.meshgrid(*(torch.arange(n, dtype=torch.float64, device="cuda") for n in (T, Hh, W)),
                                       indexing="ij"), -1).reshape(-1, 3)
    place[:, 0] += case["first"]
    axis = torch.cat([torch.full((s // 2,), a, device="cuda") for a, s in enumerate(_splits(d))])
    freq = torch.cat([torch.exp(-math.log(THETA) * 2 * torch.arange(s // 2, dtype=torch.float64, device="cuda") / s)
                      for s in _splits(d)])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), place[:, axis] * freq)
    turn = turn if case["layout"] == "bhnd" else turn[:, None]

    def to_c(x):
        x = x.unflatten(-1, (-1, 2)) if case["interleaved"] else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        return torch.view_as_complex(x.contiguous())

    def from_c(z):
        x = torch.view_as_real(z)
        return (x if case["interleaved"] else x.transpose(-1, -2)).flatten(-2)

    outs, dws = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        rms = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        if dy is None:
            outs.append(from_c(to_c(w * x / rms) * turn))
            continue
        back = from_c(to_c(dy.double()) * turn.conj())
        dws.append((back * x / rms).sum((0, 1, 2)))
        inner = (back * w * x).sum(-1, keepdim=True) / (d * rms ** 3)
        outs.append(back * w / rms - x * inner)
    return tuple(outs + dws)


def _exact_window(case, s):
    """Softmax attention head by head; its gradient from the Jacobian of the softmax."""
    hd = (lambda x: x) if case["layout"] == "bhnd" else (lambda x: x.transpose(1, 2))
    q, k, v = hd(s["q"]), hd(s["k"]), hd(s["v"])
    do = hd(s["do"]) if "do" in s else None
    B, Hq, Nq, d = q.shape
    g = Hq // case["Hkv"]
    o, lse = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v))
    for b, n in enumerate(_lengths(case)):
        lo, hi, first = (x.cuda()[:, None] for x in _rows(case, n))
        j = torch.arange(n, device="cuda")
        seen = (j < hi) & ((j >= lo) | (j < first))
        for h in range(Hq):
            Q, K, V = q[b, h].double(), k[b, h // g, :n].double(), v[b, h // g, :n].double()
            z = (Q @ K.T) / math.sqrt(d)
            z = torch.where(seen, z, -math.inf)
            L = torch.logsumexp(z, -1, keepdim=True)
            P = torch.where(seen, torch.exp(z - L), 0.0)
            del z
            lse[b, h] = L[:, 0]
            o[b, h] = P @ V
            if do is not None:
                G = do[b, h].double()
                dv[b, h // g, :n] += P.T @ G
                dP = G @ V.T
                dZ = P * (dP - (P * dP).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[b, h] = dZ @ K
                dk[b, h // g, :n] += dZ.T @ Q
    return (hd(o), lse) if do is None else (hd(dq), hd(dk), hd(dv))


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] in ("norm", "norm_bwd") else _exact_window(case, s)
