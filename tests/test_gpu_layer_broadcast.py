"""Gradients that were broadcast (what o.sum().backward() gives) are taken like any others (GPU)."""
import pytest
import torch

from block_sparse_video_tile_b200 import api

pytestmark = pytest.mark.gpu


def kinds(B, H, N, d):
    """Broadcast bf16 tensors of shape [B, H, N, d]: one value, one row, one head, one sequence."""
    g = torch.Generator(device="cuda").manual_seed(0)
    for shape in ((1, 1, 1, 1), (1, 1, 1, d), (B, 1, N, d), (1, H, N, d)):
        yield torch.randn(shape, generator=g, device="cuda").bfloat16().expand(B, H, N, d)


@pytest.mark.parametrize("other", [False, True])
def test_broadcast_gradients(other):
    q, k, v = (torch.randn(2, 3, 24, 64, device="cuda").bfloat16() for _ in range(3))
    w = torch.rand(64, device="cuda")
    o, lse = api.window_attn(q, k, v, 5)
    s = torch.cuda.Stream() if other else None
    if other:
        s.wait_stream(torch.cuda.current_stream())
    for do in kinds(2, 3, 24, 64):
        got = api.window_attn_bwd(do, q, k, v, o, lse, 5, stream=s)
        got += api.qk_norm_rope_bwd(do, do, q, k, (2, 3, 4), q_weight=w, k_weight=w, stream=s)
        if other:
            s.synchronize()
        do = do.contiguous()
        want = api.window_attn_bwd(do, q, k, v, o, lse, 5)
        want += api.qk_norm_rope_bwd(do, do, q, k, (2, 3, 4), q_weight=w, k_weight=w)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_lengths_of_one_are_not_copied():
    """A stride of 0 beside an extent of 1 is no broadcast."""
    q = torch.randn(24, 64, device="cuda").bfloat16().as_strided((1, 1, 24, 64), (0, 0, 64, 1))
    o, lse = api.window_attn(q, q, q, 5)
    dq, dk, dv = api.window_attn_bwd(q, q, q, q, o, lse, 5)
    c = q.contiguous()
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), api.window_attn_bwd(c, c, c, c, o, lse, 5)))


def test_other_broadcast_tensors_are_still_refused():
    q = torch.randn(2, 3, 24, 64, device="cuda").bfloat16()
    o, lse = api.window_attn(q, q, q, 5)
    with pytest.raises(RuntimeError):
        api.window_attn_bwd(o, q[:1].expand(2, 3, 24, 64), q, q, o, lse, 5)
    with pytest.raises(ValueError):
        api.window_attn_bwd(torch.zeros(2, 3, 24, 64, device="cuda").half()[:1, :1, :1, :1].expand(2, 3, 24, 64), q, q, q,
                            o, lse, 5)
