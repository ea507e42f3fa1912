"""Given outputs that share memory with anything a call reads are refused before it starts (GPU tensors, host checks)."""
import pytest
import torch

from block_sparse_video_tile_b200 import api

pytestmark = pytest.mark.gpu


def test_norm_rope_out_over_a_table():
    q, k = torch.randn(1, 2, 24, 64, device="cuda").bfloat16(), torch.randn(1, 2, 30, 64, device="cuda").bfloat16()
    tq, tk = api.rope_table((2, 3, 4), 64), api.rope_table((5, 2, 3), 64)
    kw = dict(grid_k=(5, 2, 3), table=tq)
    yq = torch.empty_like(q)
    room = torch.empty(k.numel() + 2 * tk.numel(), dtype=torch.bfloat16, device="cuda")
    yk = room[:k.numel()].view(k.shape)
    inside = room[:2 * tk.numel()].view(torch.float32).view(tk.shape)
    behind = room[k.numel():].view(torch.float32).view(tk.shape)
    for t in (inside, behind):
        t.copy_(tk)
    with pytest.raises(ValueError, match="overlaps table_k"):
        api.qk_norm_rope(q, k, (2, 3, 4), table_k=inside, out=(yq, yk), **kw)
    behind.copy_(tk)
    got = api.qk_norm_rope(q, k, (2, 3, 4), table_k=behind, out=(yq, yk), **kw)
    want = api.qk_norm_rope(q, k, (2, 3, 4), table_k=tk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(behind, tk)


@pytest.mark.parametrize("name", ["kv_len", "q_start"])
def test_window_outputs_over_lengths(name):
    q, k = torch.randn(2, 2, 24, 64, device="cuda").bfloat16(), torch.randn(2, 2, 30, 64, device="cuda").bfloat16()
    lse = torch.zeros(2, 2, 24, device="cuda")
    n = lse.view(torch.int32).flatten()[5:7]
    n.copy_(torch.tensor([30, 7], dtype=torch.int32))
    with pytest.raises(ValueError, match="lse overlaps " + name):
        api.window_attn(q, k, k, 4, lse=lse, **{name: n})
    out = torch.zeros_like(q)
    n = out.view(torch.int32).flatten()[-2:]
    with pytest.raises(ValueError, match="out overlaps " + name):
        api.window_attn(q, k, k, 4, out=out, **{name: n})
