"""qk_norm_rope_bwd for rows of unusual size (GPU, against float64): whatever the size of a row, as long as its sum of
squares fits float32, dx is as exact as for rows of size 1.

Bounds as in test_gpu_norm_rope.py: dx is rounded once (half a step, 2^-8 of it) from float32 arithmetic that is off by
at most 64 * 2^-24 of its terms r |h| and r |u| mean |h u|; bf16 holds every dx here as a normal number."""
import numpy as np
import pytest
import torch

from block_sparse_video_tile_b200 import api
from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,interleaved", [(128, True), (64, False)])
@pytest.mark.parametrize("size", [1e-17, 1e-14, 1e-13, 1e13, 1e14, 1e15, 1e17])
def test_backward_of_rows_of_any_size(size, d, interleaved):
    g = torch.Generator(device="cuda").manual_seed(0)
    grid, B, H = (2, 3, 4), 1, 3
    x = (size * torch.randn(B, H, 24, d, generator=g, device="cuda")).bfloat16()
    dy = torch.randn(B, H, 24, d, generator=g, device="cuda").bfloat16()
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    table = api.rope_table(grid, d)
    y, _ = api.qk_norm_rope(x, None, grid, table=table, q_weight=w, eps=0.0, interleaved=interleaved)
    dy[:, 1] = y[:, 1]                           # a gradient along the row: the two terms of dx nearly cancel
    dx, _, dw, _ = api.qk_norm_rope_bwd(dy, None, x, None, grid, table=table, q_weight=w, eps=0.0,
                                        interleaved=interleaved)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref, rw, terms, sums = lo.norm_rope_bwd(f64(dy), f64(x), f64(w), 0.0, lo.angles(grid, d), interleaved)
    tol = 1.01 * 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * terms.max(-1, keepdims=True)
    err = np.abs(f64(dx) - ref)
    assert (err <= tol).all(), f"off by {(err / tol).max()} of the bound"
    assert (np.abs(f64(dw) - rw) <= 256 * 2.0 ** -24 * sums).all()
