"""Range of the fp16 window_attn_bwd (GPU, against float64): gradients far below and far above 1, and probabilities below
fp16's normal numbers (2^-14), lose nothing but roundings of half a step, u = 2^-11, of the value at hand.

A result is a sum of products with one factor rounded to fp16 (dS for dq and dk, P for dv), rounded once: errors of
single values add up at random, so 2-norms are compared, at most u of the norm for each of the two roundings.  Scores,
LSE, delta and sums are float32, and the forward's O, whose rounding enters delta, is an average over all the keys:
together below half of u here.  Where a result of size r is near the end of fp16's normal range, its own rounding may
be off by 2^-25: inputs are chosen so that r is above 2^-14 (then 2^-25 / r is at most u again, and is counted once
more).  In all 4 u."""
import math

import pytest
import torch

from block_sparse_video_tile_b200 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


def reference(do, q, k, v, see=None):
    """dq, dk, dv in float64, head by head; see: [Nq, Nk] or None for everything."""
    out = [torch.zeros_like(x, dtype=torch.float64) for x in (q, k, v)]
    group = q.shape[1] // k.shape[1]
    s = 1 / math.sqrt(q.shape[-1])
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            Q, K, V, G = (x.double() for x in (q[b, h], k[b, h // group], v[b, h // group], do[b, h]))
            z = (Q @ K.T) * s
            P = (z if see is None else z.masked_fill(~see, -math.inf)).softmax(-1)
            dP = G @ V.T
            dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * s
            out[0][b, h] = dS @ K
            out[1][b, h // group] += dS.T @ Q
            out[2][b, h // group] += P.T @ G
    return out


def norm_error(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def make(B, Hq, Hkv, Nq, Nk, d, size, qs=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda H, N, s: (s * torch.randn(B, H, N, d, generator=g, device="cuda")).half()  # noqa: E731
    return rand(Hq, Nq, size), rand(Hq, Nq, qs), rand(Hkv, Nk, 1 / qs), rand(Hkv, Nk, 1.0)


# Hq, Hkv: a key block's queries walked by several CTAs, and by one
@pytest.mark.parametrize("heads", [(1, 1), (6, 6), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
def test_small_gradients_of_long_rows(size, d, heads):
    """4480 keys for every query: P is about 2e-4, dS that times dO.  dq is held by large keys (and small queries, so
    that the scores stay), dk the other way round."""
    for which, qs in ((0, 2.0 ** -8), (1, 2.0 ** 8)):
        do, q, k, v = make(1, *heads, 4480, 4480, d, size, qs)
        o, lse = api.window_attn(q, k, v, 1, unit=4480)
        got = api.window_attn_bwd(do, q, k, v, o, lse, 1, unit=4480)
        ref = reference(do, q, k, v)
        assert float(ref[which].square().mean().sqrt()) > 2.0 ** -14
        assert norm_error(got[which], ref[which]) <= 4 * U


def test_probabilities_below_normal_numbers():
    """400000 keys: P is about 2.5e-6.  dv of 128 queries."""
    do, q, k, v = make(1, 1, 1, 128, 400000, 64, 64.0)
    o, lse = api.window_attn(q, k, v, 1, unit=400000)
    got = api.window_attn_bwd(do, q, k, v, o, lse, 1, unit=400000)
    ref = reference(do, q, k, v)
    assert float(ref[2].square().mean().sqrt()) > 2.0 ** -14
    assert norm_error(got[2], ref[2]) <= 4 * U


@pytest.mark.parametrize("heads", [(1, 1), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_large_gradients(d, heads):
    """dO of 1e4 against two visible keys: dP and dS pass 65504, the results (of small queries and keys) do not."""
    do, q, k, v = make(2, *heads, 300, 300, d, 1e4)
    do.clamp_(-6e4, 6e4)
    q, k = (q * 0.05).half(), (k * 0.05).half()
    o, lse = api.window_attn(q, k, v, 2)
    got = api.window_attn_bwd(do, q, k, v, o, lse, 2)
    i = torch.arange(300, device="cuda")
    see = (i <= i[:, None]) & (i > i[:, None] - 2)
    ref = reference(do, q, k, v, see)
    assert all(float(r.abs().max()) < 6e4 for r in ref)
    G, V = do.double(), v.repeat_interleave(heads[0] // heads[1], 1).double()
    assert float((G @ V.transpose(2, 3)).masked_fill(~see, 0).abs().max()) > 65504
    # here O is not an average: its rounding, u of it, is of delta's own size and enters dS once more; P is about 1/2,
    # so that dS = P (dP - delta) is a difference of values of dP's size
    for x, r in zip(got, ref):
        assert x.isfinite().all() and norm_error(x, r) <= 8 * U


def test_one_large_query_leaves_the_others_alone():
    """One query's gradient is 1000 times the others': keys that it does not see keep their gradients' precision."""
    do, q, k, v = make(1, 2, 1, 2048, 2048, 64, 1e-2, 16.0)
    do[0, 1, 2047] *= 1000
    o, lse = api.window_attn(q, k, v, 1, unit=1024)
    got = api.window_attn_bwd(do, q, k, v, o, lse, 1, unit=1024)
    i = torch.arange(2048, device="cuda") // 1024
    ref = reference(do, q, k, v, i == i[:, None])
    for part in (slice(0, 1024), slice(1024, 2048)):
        for n in (0, 1, 2):
            if float(ref[n][:, :, part].square().mean().sqrt()) > 2.0 ** -14:
                assert norm_error(got[n][:, :, part], ref[n][:, :, part]) <= 4 * U
        assert float(ref[1][:, :, part].square().mean().sqrt()) > 2.0 ** -14


def test_gradients_of_zero_and_of_unseen_rows():
    """A gradient of zeros gives zeros; rows that nothing sees may hold NaN and do not touch the factors."""
    do, q, k, v = make(2, 2, 1, 200, 300, 128, 1e-3)
    n = torch.tensor([300, 150], dtype=torch.int32, device="cuda")
    kw = dict(sink=3, kv_len=n)
    o, lse = api.window_attn(q, k, v, 40, **kw)
    for x in api.window_attn_bwd(torch.zeros_like(do), q, k, v, o, lse, 40, **kw):
        assert (x == 0).all()
    want = api.window_attn_bwd(do, q, k, v, o, lse, 40, **kw)
    for x in (k, v):
        x[1, :, 150:] = float("nan")
    do[1, :, :50] = q[1, :, :50] = float("nan")                     # positions -50 .. -1
    o, lse = api.window_attn(q, k, v, 40, **kw)
    got = api.window_attn_bwd(do, q, k, v, o, lse, 40, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed_and_on_several_streams():
    """The three or four launches of the fp16 gradient in two graphs that run at once, with inputs changed after the
    capture, and eagerly on four streams."""
    do, q, k, v = make(2, 4, 2, 700, 900, 64, 1e-2)
    n = torch.tensor([900, 500], dtype=torch.int32, device="cuda")
    kw = dict(sink=4, kv_len=n)

    def both(**more):
        o, lse = api.window_attn(q, k, v, 300, **kw, **more)
        return (o, lse) + api.window_attn_bwd(do, q, k, v, o, lse, 300, **kw, **more)

    want = both()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = both()
        graphs.append((gr, r))
    do.mul_(64.0)
    v.mul_(0.25)
    n.copy_(torch.tensor([630, 899], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    now = both()
    assert not torch.equal(now[3], want[3])
    for _, r in graphs:
        assert all(torch.equal(a, b) for a, b in zip(r, now))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [both(stream=streams[i % 4]) for i in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, now))
