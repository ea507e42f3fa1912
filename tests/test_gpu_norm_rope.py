"""qk_norm_rope and its gradient on the GPU against float64 (oracle/layer_ops.py).

Bounds: a result is rounded once (half a step, u = eps / 2 of the type, relative) from float32 arithmetic whose own
error is a few 2^-24 of its terms: 32 of them for the rotated row (one sum of squares in a tree, rsqrt, the products),
64 for dx (two such sums).  fp16 results below its normal range are off by up to 2^-25 more.  A weight's gradient is a
float32 sum; a lane adds at most 200 terms here before the tree, so it is off by at most 256 * 2^-24 of sum |terms|."""
import numpy as np
import pytest
import torch

from block_sparse_video_tile_b200 import api
from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def f64(x):
    return x.double().cpu().numpy()


def bhnd(x, layout):
    x = f64(x)
    return x if layout == "bhnd" else x.transpose(0, 2, 1, 3)


def rand(g, B, H, N, d, dtype, layout, scale=1.0):
    shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def check(got, ref, terms, dtype, n, layout):
    u = torch.finfo(DT[dtype]).eps / 2
    tol = 1.01 * u * np.abs(ref) + n * 2.0 ** -24 * terms + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = np.abs(bhnd(got, layout) - ref)
    assert (err <= tol).all(), f"off by {err.max()}, {(err / tol).max()} of the bound"


def row_terms(x, w, eps):
    """Largest magnitude that enters a rotated pair, for every channel."""
    y = np.abs(lo.norm_rope(x, w, eps, None, True))
    return np.broadcast_to(y.max(-1, keepdims=True), y.shape)


CASES = [
    # grid, B, Hq, Hk, d, dtype, layout, interleaved, weight, first, split
    ((1, 1, 1), 1, 1, 1, 128, "bf16", "bhnd", True, "f32", (0, 0, 0), None),
    ((1, 1, 1), 1, 1, 1, 64, "f16", "bnhd", False, "same", (5, 0, 0), None),
    ((3, 5, 7), 2, 3, 3, 128, "bf16", "bnhd", True, "same", (100, 0, 0), None),
    ((3, 5, 7), 2, 5, 2, 128, "f16", "bhnd", False, "f32", (0, 0, 0), None),
    ((2, 9, 11), 1, 24, 24, 64, "bf16", "bhnd", False, None, (0, 3, 4), None),
    ((2, 9, 11), 3, 7, 1, 64, "f16", "bnhd", True, "f32", (0, 0, 0), (32, 16, 16)),
    ((2, 5, 9), 2, 17, 19, 64, "f16", "bnhd", True, "f32", (0, 0, 0), None),      # several heads of a token side by side
    ((3, 4, 3), 1, 9, 13, 128, "bf16", "bnhd", False, "same", (0, 0, 0), None),
    ((257, 1, 1), 1, 4, 4, 128, "bf16", "bnhd", False, "same", (100000, 0, 0), (128, 0, 0)),
    ((4, 13, 21), 1, 13, 13, 128, "bf16", "bhnd", True, "f32", (0, 0, 0), (0, 64, 64)),
]


def inputs(case, seed=0):
    grid, B, Hq, Hk, d, dtype, layout, il, weight, first, split = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = grid[0] * grid[1] * grid[2]
    q, k = rand(g, B, Hq, N, d, dtype, layout, 1.5), rand(g, B, Hk, N, d, dtype, layout, 0.5)
    wt = {"f32": torch.float32, "same": DT[dtype], None: None}[weight]
    wq, wk = (None if wt is None else (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(wt) for _ in range(2))
    how = dict(table=api.rope_table(grid, d, split=split, first=first), split=split, q_weight=wq, k_weight=wk, eps=1e-5,
               interleaved=il, layout=layout)
    return q, k, wq, wk, how, lo.angles(grid, d, split, first=first), g


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    grid, dtype, layout, il = case[0], case[5], case[6], case[7]
    q, k, wq, wk, how, ang, _ = inputs(case)
    for got, x, w in zip(api.qk_norm_rope(q, k, grid, **how), (q, k), (wq, wk)):
        w = 1.0 if w is None else f64(w)
        X = bhnd(x, layout)
        check(got, lo.norm_rope(X, w, 1e-5, ang, il), row_terms(X, w, 1e-5), dtype, 32, layout)


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    grid, B, Hq, Hk, d, dtype, layout, il = case[:8]
    q, k, wq, wk, how, ang, g = inputs(case)
    N = grid[0] * grid[1] * grid[2]
    dq, dk = rand(g, B, Hq, N, d, dtype, layout), rand(g, B, Hk, N, d, dtype, layout)
    got = api.qk_norm_rope_bwd(dq, dk, q, k, grid, **how)
    for dx, dw, x, w, dy in ((got[0], got[2], q, wq, dq), (got[1], got[3], k, wk, dk)):
        W = 1.0 if w is None else f64(w)
        rx, rw, terms, sums = lo.norm_rope_bwd(bhnd(dy, layout), bhnd(x, layout), W, 1e-5, ang, il)
        terms = np.broadcast_to(terms.max(-1, keepdims=True), terms.shape)
        check(dx, rx, terms, dtype, 64, layout)
        assert (dw is None) == (w is None)
        if w is not None:
            assert dw.dtype == torch.float32 and (np.abs(f64(dw) - rw) <= 256 * 2.0 ** -24 * sums).all()
    again = api.qk_norm_rope_bwd(dq, dk, q, k, grid, **how)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, again))


def test_views_of_a_fused_projection_and_strided_outputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    grid, H, d = (2, 5, 6), 3, 128
    qkv = torch.randn(2, 60, 3, H, d, generator=g, device="cuda").bfloat16()
    table = api.rope_table(grid, d)
    w = torch.rand(d, generator=g, device="cuda")
    kw = dict(table=table, q_weight=w, k_weight=w, layout="bnhd")
    want = api.qk_norm_rope(qkv[:, :, 0].contiguous(), qkv[:, :, 1].contiguous(), grid, **kw)
    got = api.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], grid, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    room = torch.full((2, 70, 2, H + 1, d), 7.0, device="cuda", dtype=torch.bfloat16)      # rows behind stay as they were
    out = (room[:, :60, 0, :H], room[:, 10:, 1, 1:])
    with pytest.raises(ValueError, match="overlaps"):
        api.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], grid, out=out, **kw)                   # interleaved spans: refused
    room2 = room.clone()
    out = (room[:, :60, 0, :H], room2[:, 10:, 1, 1:])
    api.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], grid, out=out, **kw)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert (room[:, 60:] == 7).all() and (room[:, :, 1] == 7).all() and (room[:, :, :, H] == 7).all()
    assert (room2[:, :10] == 7).all() and (room2[:, :, 0] == 7).all() and (room2[:, :, :, 0] == 7).all()
    dy = (room[:, :60, 0, :H], room2[:, 10:, 1, 1:])
    got = api.qk_norm_rope_bwd(*dy, qkv[:, :, 0], qkv[:, :, 1], grid, **kw)
    ref = api.qk_norm_rope_bwd(*(x.contiguous() for x in dy), *(qkv[:, :, i].contiguous() for i in (0, 1)), grid, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_one_side_own_key_grid_and_no_rotation():
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k = rand(g, 2, 3, 24, 64, "bf16", "bhnd"), rand(g, 1, 2, 30, 64, "bf16", "bhnd")
    tq, tk = api.rope_table((2, 3, 4), 64), api.rope_table((5, 2, 3), 64, first=(2, 0, 0))
    a, b = api.qk_norm_rope(q, k, (2, 3, 4), grid_k=(5, 2, 3), table=tq, table_k=tk)
    only, none = api.qk_norm_rope(q, None, (2, 3, 4), table=tq)
    assert none is None and torch.equal(a, only)
    assert torch.equal(b, api.qk_norm_rope(k, None, (5, 2, 3), table=tk)[0])
    with pytest.raises(ValueError, match="table_k"):
        api.qk_norm_rope(q, k, (2, 3, 4), grid_k=(5, 2, 3), table=tq)
    plain, _ = api.qk_norm_rope(q, None, (2, 3, 4))
    X = f64(q)
    check(plain, lo.norm_rope(X, 1.0, 1e-6, None, True), row_terms(X, 1.0, 1e-6), "bf16", 32, "bhnd")
    dx = api.qk_norm_rope_bwd(plain, None, q, None, (2, 3, 4), q_weight=torch.ones(64, device="cuda"))
    assert dx[1] is None and dx[3] is None and dx[2].shape == (64,)


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(5)
    q = rand(g, 1, 2, 24, 64, "bf16", "bhnd")
    t = api.rope_table((2, 3, 4), 64)
    for bad in (dict(table=t[:-1]), dict(table=t.double()), dict(q_weight=torch.ones(63, device="cuda")),
                dict(q_weight=torch.ones(64)), dict(q_weight=torch.ones(64, device="cuda").half())):
        with pytest.raises(ValueError):
            api.qk_norm_rope(q, None, (2, 3, 4), **bad)
    with pytest.raises(ValueError, match="tokens"):
        api.qk_norm_rope(q, None, (2, 3, 5))
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, rand(g, 1, 2, 24, 64, "f16", "bhnd"), (2, 3, 4))
    with pytest.raises(ValueError, match="channels"):
        api.qk_norm_rope(q.transpose(2, 3), None, (2, 4, 8))
    with pytest.raises(ValueError, match="overlaps"):
        api.qk_norm_rope(q, None, (2, 3, 4), out=(q, None))
    with pytest.raises(RuntimeError):
        api.qk_norm_rope(q.expand(3, 2, 24, 64), None, (2, 3, 4))      # a batch stride of 0


def test_empty_batch():
    q = torch.empty(0, 2, 24, 64, dtype=torch.bfloat16, device="cuda")
    assert api.qk_norm_rope(q, q, (2, 3, 4))[0].shape == q.shape
    w = torch.ones(64, device="cuda")
    got = api.qk_norm_rope_bwd(q, q, q, q, (2, 3, 4), q_weight=w, k_weight=w)
    assert got[0].shape == q.shape and (got[2] == 0).all()


def test_other_stream_and_graph():
    g = torch.Generator(device="cuda").manual_seed(6)
    grid = (2, 9, 8)
    q, k = rand(g, 1, 4, 144, 128, "bf16", "bnhd"), rand(g, 1, 4, 144, 128, "bf16", "bnhd")
    w = torch.rand(128, device="cuda", generator=g)
    kw = dict(table=api.rope_table(grid, 128), q_weight=w, k_weight=w, layout="bnhd")
    want, bwant = api.qk_norm_rope(q, k, grid, **kw), api.qk_norm_rope_bwd(q, k, q, k, grid, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.qk_norm_rope(q, k, grid, stream=s, **kw)
    bgot = api.qk_norm_rope_bwd(q, k, q, k, grid, stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + bgot, want + bwant))
    graphs = []
    for _ in range(2):                                    # two captured graphs, replayed in turn
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = api.qk_norm_rope(q, k, grid, **kw) + api.qk_norm_rope_bwd(q, k, q, k, grid, **kw)
        graphs.append((gr, r))
    q.copy_(rand(g, 1, 4, 144, 128, "bf16", "bnhd"))
    for gr, _ in graphs + graphs:
        gr.replay()
    want = api.qk_norm_rope(q, k, grid, **kw) + api.qk_norm_rope_bwd(q, k, q, k, grid, **kw)
    for _, r in graphs:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_large_call_against_torch():
    """Many tokens and heads (the whole-head loop), against the same formula in float64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(7)
    grid, H, d = (9, 22, 40), 24, 128
    N = 9 * 22 * 40
    q = rand(g, 1, H, N, d, "bf16", "bnhd")
    dy = rand(g, 1, H, N, d, "bf16", "bnhd")
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    kw = dict(table=api.rope_table(grid, d), q_weight=w, layout="bnhd")
    y, _ = api.qk_norm_rope(q, None, grid, **kw)
    dx, _, dw, _ = api.qk_norm_rope_bwd(dy, None, q, None, grid, **kw)
    ang = torch.from_numpy(lo.angles(grid, d)).cuda()[:, None]
    x, G, W = q.double(), dy.double(), w.double()
    turn = torch.polar(torch.ones_like(ang), ang)
    r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    ref = torch.view_as_real(torch.view_as_complex((x * r * W).unflatten(-1, (-1, 2))) * turn).flatten(-2)
    u = 2.0 ** -8
    big = ref.abs().amax(-1, keepdim=True) * 1.5
    assert ((y.double() - ref).abs() <= 1.01 * u * ref.abs() + 32 * 2.0 ** -24 * big).all()
    back = torch.view_as_real(torch.view_as_complex(G.unflatten(-1, (-1, 2))) * turn.conj()).flatten(-2)
    un = x * r
    h = back * W
    refdx = r * (h - un * (h * un).mean(-1, keepdim=True))
    big = refdx.abs().amax(-1, keepdim=True) * 4
    assert ((dx.double() - refdx).abs() <= 1.01 * u * refdx.abs() + 64 * 2.0 ** -24 * big).all()
    terms = back * un
    # a lane adds at most ceil(495 groups / 592 CTAs) * 24 rows, then 16 + 8 + 592 / 8 + 8 partial sums
    assert ((dw.double() - terms.sum((0, 1, 2))).abs() <= 256 * 2.0 ** -24 * terms.abs().sum((0, 1, 2))).all()


def test_offsets_beyond_32_bits():
    """Two videos further apart than 2^31 elements."""
    g = torch.Generator(device="cuda").manual_seed(8)
    N, H, d, grid = 24, 3, 128, (2, 3, 4)
    far = (1 << 31) + 64
    room = torch.zeros(far + N * H * d, dtype=torch.bfloat16, device="cuda")
    q = room.as_strided((2, N, H, d), (far, H * d, d, 1))
    q.copy_(rand(g, 2, H, N, d, "bf16", "bnhd"))
    kw = dict(table=api.rope_table(grid, d), q_weight=torch.rand(d, device="cuda", generator=g), layout="bnhd")
    near = q.contiguous()
    assert torch.equal(api.qk_norm_rope(q, None, grid, **kw)[0], api.qk_norm_rope(near, None, grid, **kw)[0])
    a, b = (api.qk_norm_rope_bwd(x, None, x, None, grid, **kw) for x in (q, near))
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("interleaved", [True, False])
def test_gradient_against_differences(interleaved):
    """dx and dw against central differences of the call's own result along the gradient (fp16; the rounding of y, 2^-11
    of a value, is a random 1e-4 of the rise that it hides; the curvature of a step of 0.1 about 1 %)."""
    g = torch.Generator(device="cuda").manual_seed(9)
    grid, d = (2, 3, 5), 64
    x, dy = rand(g, 1, 4, 30, d, "f16", "bhnd", 1.5), rand(g, 1, 4, 30, d, "f16", "bhnd")
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    kw = dict(table=api.rope_table(grid, d), interleaved=interleaved)
    dx, _, dw, _ = api.qk_norm_rope_bwd(dy, None, x, None, grid, q_weight=w, **kw)
    for gr, at, f in ((dx, x, lambda t: api.qk_norm_rope(t, None, grid, q_weight=w, **kw)[0]),
                      (dw, w, lambda t: api.qk_norm_rope(x, None, grid, q_weight=t, **kw)[0])):
        step = gr.double() / gr.double().abs().max()
        a, b = ((at.double() + sign * 0.1 * step).to(at.dtype) for sign in (1, -1))
        rise = ((f(a).double() - f(b).double()) * dy.double()).sum()
        slope = ((a.double() - b.double()) * gr.double()).sum()
        assert abs(rise - slope) <= 0.03 * abs(slope)
