"""window_attn and its gradient on the GPU against float64 (oracle/layer_ops.py, which also derives the bounds: P, dS
and the results are rounded once to the 16-bit type, scores and sums are float32)."""
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


def rand(g, B, H, N, d, dtype, layout):
    shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


def c(B, Hq, Hkv, Nq, Nk, d, window, sink=0, unit=1, dtype="bf16", layout="bhnd", kv_len=None, q_start=None, scale=None):
    return dict(B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, window=window, sink=sink, unit=unit, dtype=dtype, layout=layout,
                kv_len=kv_len, q_start=q_start, scale=scale)


CASES = {
    "one_key": c(1, 1, 1, 1, 1, 128, 1),
    "one_query": c(2, 4, 4, 1, 300, 128, 100, 4, layout="bnhd"),
    "one_query_group": c(3, 8, 2, 1, 700, 64, 256, 16, dtype="f16", kv_len=[700, 3, 401]),
    "one_query_long": c(1, 6, 2, 1, 9000, 128, 8000, 130, layout="bnhd"),
    "one_query_frames": c(1, 3, 3, 1, 1000, 128, 2, 1, 88),
    "few_queries": c(2, 6, 2, 5, 513, 128, 64, 4, layout="bnhd", kv_len=[513, 130]),
    "sixteen_queries": c(1, 7, 1, 16, 385, 64, 100, 0, dtype="f16"),
    "seventeen_queries": c(1, 2, 2, 17, 260, 128, 50, 3),
    "square": c(1, 2, 2, 128, 128, 128, 1 << 20),
    "square_64": c(1, 2, 1, 256, 256, 64, 1 << 20, dtype="f16", layout="bnhd"),
    "odd": c(1, 3, 1, 257, 259, 128, 100, 7),
    "token_window": c(2, 4, 2, 511, 511, 128, 37, 0, dtype="f16", layout="bnhd"),
    "window_of_one": c(1, 2, 2, 200, 200, 64, 1),
    "window_and_far_sinks": c(1, 2, 2, 700, 700, 128, 64, 4),
    "many_sinks": c(1, 2, 2, 600, 600, 64, 30, 300, dtype="f16"),
    "frames": c(1, 2, 2, 352, 352, 128, 2, 1, 88),
    "frames_no_sink": c(1, 2, 1, 700, 700, 64, 1, 0, 100, layout="bnhd"),
    "frames_chunk": c(1, 3, 3, 176, 880, 128, 3, 2, 88, layout="bnhd"),
    "frame_over_everything": c(1, 2, 2, 300, 300, 128, 1, 0, 4096),
    "long_frames": c(1, 2, 1, 1500, 1500, 64, 1, 0, 500),
    "long_frames_sink": c(1, 1, 1, 1300, 1300, 128, 2, 1, 350, layout="bnhd", kv_len=[1290]),
    "few_ctas": c(1, 1, 1, 100, 3000, 128, 2900, 5),
    "few_ctas_64": c(1, 2, 1, 130, 2500, 64, 3000, 0, dtype="f16", layout="bnhd"),
    "sinks_seen_by_all": c(1, 4, 1, 1100, 1100, 64, 40, 3, layout="bnhd"),
    "partial_frames": c(2, 2, 2, 130, 530, 128, 2, 1, 130, kv_len=[530, 399]),
    "ragged": c(3, 2, 2, 300, 400, 128, 90, 5, kv_len=[400, 0, 131]),
    "fewer_keys_than_queries": c(2, 2, 2, 300, 300, 64, 60, 2, kv_len=[40, 300], dtype="f16"),
    "starts": c(3, 2, 1, 150, 400, 128, 50, 3, kv_len=[400, 400, 200], q_start=[0, 300, -70]),
    "past_the_end": c(2, 2, 2, 140, 200, 128, 20, 0, kv_len=[200, 90], q_start=[100, 150]),
    "future_keys": c(1, 2, 2, 100, 900, 128, 30, 1, q_start=[200]),
    "scale": c(1, 2, 2, 140, 140, 64, 1000, scale=0.9),
    "small_scale": c(1, 1, 1, 140, 140, 64, 1000, scale=1e-3),
    "group_of_seven": c(1, 14, 2, 190, 190, 64, 77, 3, layout="bnhd"),
}


def make(case, seed=0, poison=True):
    """Tensors and the call's arguments; rows behind kv_len hold NaN and infinities, and so do queries that see
    nothing."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Nq, Nk, d, layout = case["B"], case["Nq"], case["Nk"], case["d"], case["layout"]
    q = rand(g, B, case["Hq"], Nq, d, case["dtype"], layout)
    k, v = (rand(g, B, case["Hkv"], Nk, d, case["dtype"], layout) for _ in range(2))
    lens = case["kv_len"] or [Nk] * B
    starts = case["q_start"] or [n - Nq for n in lens]
    sees = [lo.visible(Nq, Nk, lens[b], starts[b], case["window"], case["sink"], case["unit"]) for b in range(B)]
    do = rand(g, B, case["Hq"], Nq, d, case["dtype"], layout)
    if poison:
        for b in range(B):
            for x, bad in ((k, float("nan")), (v, float("inf"))):
                (x[b].transpose(0, 1) if layout == "bhnd" else x[b])[lens[b]:] = bad
            gone = torch.from_numpy(~sees[b].any(0)).cuda()          # between first units and window, too
            (k[b].transpose(0, 1) if layout == "bhnd" else k[b])[gone] = float("inf")
            (v[b].transpose(0, 1) if layout == "bhnd" else v[b])[gone] = float("nan")
            dead = torch.from_numpy(~sees[b].any(1)).cuda()
            for x in (q, do):
                (x[b].transpose(0, 1) if layout == "bhnd" else x[b])[dead] = float("nan")
    how = dict(window=case["window"], sink=case["sink"], unit=case["unit"], layout=layout, scale=case["scale"],
               kv_len=torch.tensor(case["kv_len"], dtype=torch.int32, device="cuda") if case["kv_len"] else None,
               q_start=torch.tensor(case["q_start"], dtype=torch.int32, device="cuda") if case["q_start"] else None)
    return q, k, v, do, sees, how, case["scale"] or d ** -0.5, torch.finfo(DT[case["dtype"]]).eps / 2


def within(got, ref, tol, what):
    assert np.isfinite(got[np.isfinite(ref)]).all(), f"{what}: not finite"
    inf = ~np.isfinite(ref)
    assert (got[inf] == ref[inf]).all(), f"{what}: -inf expected"
    err = np.abs(np.where(inf, 0, got) - np.where(inf, 0, ref))
    assert (err <= tol).all(), f"{what}: off by {err.max()}, {(err / tol).max()} of the bound"


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    case = CASES[name]
    q, k, v, _, sees, how, scale, u = make(case)
    o, lse = api.window_attn(q, k, v, **how)
    assert o.shape == q.shape and o.dtype == q.dtype and lse.shape == (case["B"], case["Hq"], case["Nq"])
    O, Lse, bo, bl = lo.window_fwd(*(bhnd(x, case["layout"]) for x in (q, k, v)), sees, scale, u)
    within(bhnd(o, case["layout"]), O, bo, "O")
    within(f64(lse), Lse, bl, "LSE")
    again = api.window_attn(q, k, v, **how)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert api.device_error() == 0


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    case = CASES[name]
    q, k, v, do, sees, how, scale, u = make(case, seed=1)
    o, lse = api.window_attn(q, k, v, **how)
    got = api.window_attn_bwd(do, q, k, v, o, lse, **how)
    ref, tol = lo.window_bwd(*(bhnd(x, case["layout"]) for x in (do, q, k, v)), sees, scale, u)
    for what, x, r, t in zip(("dq", "dk", "dv"), got, ref, tol):
        within(bhnd(x, case["layout"]), r, t, what)
    again = api.window_attn_bwd(do, q, k, v, o, lse, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert api.device_error() == 0


def test_views_and_given_outputs():
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn(2, 300, 3, 4, 128, generator=g, device="cuda").bfloat16()
    cache = torch.full((2, 2, 900, 4, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    cache[:, :, :300] = qkv[:, :, 1:].transpose(1, 2)
    q, k, v = qkv[:, :, 0], cache[:, 0], cache[:, 1]
    kw = dict(sink=3, layout="bnhd")
    want = api.window_attn(q.contiguous(), qkv[:, :, 1].contiguous(), qkv[:, :, 2].contiguous(), 70, **kw)
    got = api.window_attn(q, k, v, 70, kv_len=300, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    room = torch.full((2, 310, 5, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(2, 4, 300, device="cuda")
    out, l2 = api.window_attn(q, k, v, 70, kv_len=300, out=room[:, :300, :4], lse=lse, **kw)
    assert out.data_ptr() == room.data_ptr() and l2 is lse
    assert torch.equal(room[:, :300, :4], want[0]) and (room[:, 300:] == 7).all() and (room[:, :, 4] == 7).all()
    do = torch.randn(2, 300, 6, 128, generator=g, device="cuda").bfloat16()[:, :, :4]
    a = api.window_attn_bwd(do, q, k, v, out, lse, 70, kv_len=300, **kw)
    b = api.window_attn_bwd(do.contiguous(), q.contiguous(), qkv[:, :, 1].contiguous(), qkv[:, :, 2].contiguous(),
                            *want, 70, **kw)
    assert torch.equal(a[0], b[0])
    assert all(torch.equal(x[:, :300], y) and (x[:, 300:] == 0).all() for x, y in zip(a[1:], b[1:]))


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = rand(g, 2, 4, 8, 64, "bf16", "bhnd"), rand(g, 2, 2, 16, 64, "bf16", "bhnd")
    o, lse = api.window_attn(q, k, k, 4)
    for bad in (dict(window=0), dict(window=1 << 31), dict(sink=-1), dict(unit=0), dict(kv_len=17), dict(kv_len=-1),
                dict(q_start=1 << 31), dict(kv_len=torch.tensor([1, 2])), dict(out=q), dict(lse=lse[:1]),
                dict(kv_len=torch.tensor([1, 2], device="cuda")), dict(out=o[:1])):
        with pytest.raises(ValueError):
            api.window_attn(q, k, k, **{"window": 4, **bad})
    with pytest.raises(ValueError):
        api.window_attn(q, k, k[:, :, :8], 4)
    with pytest.raises(ValueError):
        api.window_attn(q, k, k.half(), 4)
    with pytest.raises(RuntimeError):
        api.window_attn(q, rand(g, 2, 3, 16, 64, "bf16", "bhnd"), rand(g, 2, 3, 16, 64, "bf16", "bhnd"), 4)
    with pytest.raises(RuntimeError):
        api.window_attn(q, k[:1].expand(2, 2, 16, 64), k, 4)
    with pytest.raises(RuntimeError):
        api.window_attn(q, k, k, 4, layout="bnhd")         # 8 query heads of 16 key heads
    with pytest.raises(RuntimeError):
        api.window_attn(q, k, k, 4, scale=-1.0)
    with pytest.raises(ValueError):
        api.window_attn_bwd(q[:1], q, k, k, o, lse, 4)
    with pytest.raises(ValueError):
        api.window_attn_bwd(o, q, k, k, o, lse.double(), 4)


def test_lengths_of_zero():
    q = torch.randn(2, 4, 8, 64, device="cuda").bfloat16()
    none = torch.empty(2, 2, 0, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = api.window_attn(q, none, none, 4)
    assert (o == 0).all() and (lse == -float("inf")).all()
    dq, dk, dv = api.window_attn_bwd(q, q, none, none, o, lse, 4)
    assert (dq == 0).all() and dk.shape == none.shape == dv.shape
    k = torch.randn(2, 2, 16, 64, device="cuda").bfloat16()
    o, lse = api.window_attn(q[:, :, :0], k, k, 4)
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    dq, dk, dv = api.window_attn_bwd(o, q[:, :, :0], k, k, o, lse, 4)
    assert (dk == 0).all() and (dv == 0).all()
    assert api.window_attn(q[:0], k[:0], k[:0], 4)[0].shape == (0, 4, 8, 64)


@pytest.mark.parametrize("Nq", [1, 200])
def test_other_stream_and_graphs(Nq):
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = rand(g, 2, 4, Nq, 128, "bf16", "bnhd"), *(rand(g, 2, 2, 900, 128, "bf16", "bnhd") for _ in range(2))
    n = torch.tensor([900, 500], dtype=torch.int32, device="cuda")
    kw = dict(sink=4, layout="bnhd", kv_len=n)

    def both(**more):
        o, lse = api.window_attn(q, k, v, 300, **kw, **more)
        return (o, lse) + api.window_attn_bwd(q, q, k, v, o, lse, 300, **kw, **more)

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = both()
        graphs.append((gr, r))
    q.copy_(rand(g, 2, 4, Nq, 128, "bf16", "bnhd"))
    n.copy_(torch.tensor([630, 899], dtype=torch.int32))          # lengths are read when the graph runs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0][0].replay()
    with torch.cuda.stream(side):
        graphs[1][0].replay()                                     # two graphs at once
    torch.cuda.synchronize()
    want = both()
    for _, r in graphs:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_streaming_equals_one_call():
    """Chunks of frames, each against the cache that grew so far, give what one call over the video gives (each within
    its bound of the other)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    unit, frames = 60, 7
    N = unit * frames
    q, k, v = (rand(g, 1, 3, N, 128, "bf16", "bnhd") for _ in range(3))
    kw = dict(window=3, sink=1, unit=unit, layout="bnhd")
    whole, lse = api.window_attn(q, k, v, **kw)
    cache = [torch.full_like(x, float("nan")) for x in (k, v)]
    sees = [lo.visible(N, N, N, 0, 3, 1, unit)]
    _, _, bo, bl = lo.window_fwd(*(bhnd(x, "bnhd") for x in (q, k, v)), sees, 128 ** -0.5, 2.0 ** -8)
    at = 0
    for n in (2, 1, 3, 1):
        a, b = at * unit, (at + n) * unit
        cache[0][:, a:b], cache[1][:, a:b] = k[:, a:b], v[:, a:b]
        o, l = api.window_attn(q[:, a:b], *cache, kv_len=b, **kw)
        assert (np.abs(bhnd(o, "bnhd") - bhnd(whole[:, a:b], "bnhd")) <= 2 * bo[:, :, a:b]).all()
        assert (np.abs(f64(l) - f64(lse[:, :, a:b])) <= 2 * bl[:, :, a:b]).all()
        at += n


def test_layer_forward_and_gradients():
    """Projection rows -> qk_norm_rope -> window_attn and back, as a training step of a layer runs them, against
    float64 autograd of the formulas.  The bf16 tensors between the calls are rounded once each (2^-9 of a value on
    average, 2^-8 at most); errors of single values add up at random, so the gradients' 2-norms are compared: q', k', P,
    dS, o, dq' and the results each add at most 2^-8 of the norm, 7 * 2^-8 in all."""
    g = torch.Generator(device="cuda").manual_seed(6)
    grid, H, d, unit = (6, 5, 8), 2, 128, 40
    N = 240
    qkv = torch.randn(1, N, 3, H, d, generator=g, device="cuda").bfloat16()
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    do = torch.randn(1, N, H, d, generator=g, device="cuda").bfloat16()
    how = dict(table=api.rope_table(grid, d), q_weight=wq, k_weight=wk, layout="bnhd")
    win = dict(window=2, sink=1, unit=unit, layout="bnhd")
    q, k = api.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], grid, **how)
    o, lse = api.window_attn(q, k, qkv[:, :, 2], **win)
    dq, dk, dv = api.window_attn_bwd(do, q, k, qkv[:, :, 2], o, lse, **win)
    dxq, dxk, dwq, dwk = api.qk_norm_rope_bwd(dq, dk, qkv[:, :, 0], qkv[:, :, 1], grid, **how)

    x = qkv.double().requires_grad_()
    w = [t.double().requires_grad_() for t in (wq, wk)]
    ang = torch.from_numpy(lo.angles(grid, d)).cuda()[:, None]
    turn = torch.polar(torch.ones_like(ang), ang)

    def prep(t, wt):
        y = t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wt
        return torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (-1, 2))) * turn).flatten(-2)

    see = torch.from_numpy(lo.visible(N, N, N, 0, 2, 1, unit)).cuda()
    Q, K = prep(x[:, :, 0], w[0]), prep(x[:, :, 1], w[1])
    z = torch.einsum("bnhd,bmhd->bhnm", Q, K) * d ** -0.5
    O = torch.einsum("bhnm,bmhd->bnhd", z.masked_fill(~see, -float("inf")).softmax(-1), x[:, :, 2])
    O.backward(do.double())
    for got, ref in ((o, O), (dxq, x.grad[:, :, 0]), (dxk, x.grad[:, :, 1]), (dv, x.grad[:, :, 2]), (dwq, w[0].grad),
                     (dwk, w[1].grad)):
        assert (got.double() - ref).norm() <= 7 * 2.0 ** -8 * ref.norm()


def test_block_sparse_forward_with_norm_rope():
    """api.forward(norm_rope=...) is qk_norm_rope followed by the forward."""
    g = torch.Generator(device="cuda").manual_seed(7)
    grid, tile, d = (8, 8, 8), (4, 4, 4), 64
    q, k, v = (torch.randn(1, 512, 2, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    how = dict(table=api.rope_table(grid, d), q_weight=torch.rand(d, device="cuda", generator=g))
    got = api.forward(q, k, v, grid, tile, 3, layout="bnhd", norm_rope=how)
    q2, k2 = api.qk_norm_rope(q, k, grid, layout="bnhd", **how)
    assert all(torch.equal(a, b) for a, b in zip(got, api.forward(q2, k2, v, grid, tile, 3, layout="bnhd")))


@pytest.mark.parametrize("Nq", [1, 5, 200])
def test_cache_beyond_32_bit_offsets(Nq):
    """The window lies behind 2^31 elements of the cache; the answer is that of a short copy (whose keys may be split
    and blocked differently: each within its bound)."""
    H, d, Nk, tail = 8, 128, (1 << 21) + 4096, 1024
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.empty(1, Nk, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (k, v):
        x[:, -tail:] = torch.randn(1, tail, H, d, generator=g, device="cuda").bfloat16()
    q = rand(g, 1, H, Nq, d, "bf16", "bnhd")
    o, lse = api.window_attn(q, k, v, 300, layout="bnhd")
    ks, vs = k[:, -tail:].contiguous(), v[:, -tail:].contiguous()
    ref = api.window_attn(q, ks, vs, 300, layout="bnhd")
    sees = [lo.visible(Nq, tail, tail, tail - Nq, 300, 0, 1)]
    _, _, bo, bl = lo.window_fwd(*(bhnd(x, "bnhd") for x in (q, ks, vs)), sees, d ** -0.5, 2.0 ** -8)
    within(bhnd(o, "bnhd"), bhnd(ref[0], "bnhd"), 2 * bo, "O")
    within(f64(lse), f64(ref[1]), 2 * bl, "LSE")
    if Nq == 200:
        do = rand(g, 1, H, Nq, d, "bf16", "bnhd")
        got = api.window_attn_bwd(do, q, k, v, o, lse, 300, layout="bnhd")
        want = api.window_attn_bwd(do, q, ks, vs, *ref, 300, layout="bnhd")
        _, tol = lo.window_bwd(*(bhnd(x, "bnhd") for x in (do, q, ks, vs)), sees, d ** -0.5, 2.0 ** -8)
        for what, a, b, t in zip(("dq", "dk", "dv"), (got[0], got[1][:, -tail:], got[2][:, -tail:]), want, tol):
            within(bhnd(a, "bnhd"), bhnd(b, "bnhd"), 2 * t, what)
        assert not got[1][:, :-tail].any() and not got[2][:, :-tail].any()


def test_two_streams_at_once():
    g = torch.Generator(device="cuda").manual_seed(9)
    calls = []
    for Nq in (1, 333):
        q, k, v = rand(g, 2, 4, Nq, 128, "bf16", "bhnd"), *(rand(g, 2, 2, 5000, 128, "bf16", "bhnd") for _ in range(2))
        calls.append((q, k, v))
    want = [api.window_attn(*c, 4000, sink=3) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [api.window_attn(*calls[i % 2], 4000, sink=3, stream=streams[i % 4]) for i in range(24)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert torch.equal(r[0], want[i % 2][0]) and torch.equal(r[1], want[i % 2][1])


def test_gradient_against_differences():
    """dq, dk and dv against central differences of the call's own O (fp16 inputs moved by a step h that fp16 holds
    exactly).  O is rounded to fp16 (2^-11 of a value, and P's rounding the same), so a difference of sums over n values
    is off by at most (2 * 2^-11 * sum |o do|) / (2 h) -- far too much for one entry; averaged over a random direction
    of all entries it is that divided by about sqrt(n) while the derivative along it grows with the norm, so whole
    directions are compared, to 3 %."""
    g = torch.Generator(device="cuda").manual_seed(10)
    q, k, v = rand(g, 1, 4, 200, 64, "f16", "bhnd"), *(rand(g, 1, 2, 200, 64, "f16", "bhnd") for _ in range(2))
    do = rand(g, 1, 4, 200, 64, "f16", "bhnd")
    kw = dict(window=2, sink=1, unit=40)
    o, lse = api.window_attn(q, k, v, **kw)
    grads = api.window_attn_bwd(do, q, k, v, o, lse, **kw)
    for i, gr in enumerate(grads):
        step = gr.double() / gr.double().abs().max()                # along the gradient: the largest derivative
        args = [q, k, v]
        ends = []
        for sign in (1, -1):
            moved = (args[i].double() + sign * 0.25 * step).half()
            ends.append((moved.double(), api.window_attn(*(moved if j == i else x for j, x in enumerate(args)), **kw)[0]))
        rise = ((ends[0][1].double() - ends[1][1].double()) * do.double()).sum()
        slope = ((ends[0][0] - ends[1][0]) * gr.double()).sum()      # the steps as fp16 took them
        assert abs(rise - slope) <= 0.03 * abs(slope), (i, float(rise), float(slope))
