"""Every way window_attn and its gradient are launched, against float64 (oracle/layer_ops.py): clusters of 2 to 8 splits,
split keys with the combine kernel, several row tiles, key blocks shared among CTAs, each with sequences of the batch
that leave splits and CTAs without work.  test_launches checks that the cases are launched as their names say."""
import json

import pytest
import torch
from torch.profiler import ProfilerActivity, profile

from block_sparse_video_tile_b200 import api
from oracle import layer_ops as lo
from tests.test_gpu_window import bhnd, c, f64, make, within

pytestmark = pytest.mark.gpu

# name: (case, kernel, grid)
FORWARD = {
    "cluster_2": (c(2, 4, 2, 1, 300, 128, 290, 4, kv_len=[300, 17]), "window_step_kernel<128, false, true>", (2, 2, 2)),
    "cluster_3": (c(2, 4, 2, 3, 400, 64, 500, 0, dtype="f16", kv_len=[0, 400]), "window_step_kernel<64, true, true>", (3, 2, 2)),
    "cluster_4_tiles": (c(1, 8, 2, 9, 600, 128, 520, 20, layout="bnhd"), "window_step_kernel<128, false, true>", (4, 6, 1)),
    "cluster_5": (c(2, 3, 3, 5, 700, 128, 640, 3, dtype="f16", kv_len=[700, 90]), "window_step_kernel<128, true, true>", (5, 3, 2)),
    "cluster_6_tiles": (c(2, 7, 1, 7, 800, 64, 790, 0, kv_len=[33, 800], layout="bnhd"), "window_step_kernel<64, false, true>",
                        (6, 4, 2)),
    "cluster_7": (c(1, 2, 1, 16, 1000, 128, 900, 9, dtype="f16"), "window_step_kernel<128, true, true>", (7, 2, 1)),
    "cluster_8_frames": (c(1, 4, 4, 3, 1100, 64, 12, 1, 88, layout="bnhd"), "window_step_kernel<64, false, true>", (8, 4, 1)),
    # 80 row tiles: 6 splits asked for, 7 leave less of the last round of CTAs empty
    "cluster_one_more": (c(5, 32, 8, 5, 1100, 64, 1000, 4, dtype="f16", kv_len=[1100, 1099, 700, 5, 1]),
                         "window_step_kernel<64, true, true>", (7, 16, 5)),
    "combine_tiles": (c(2, 8, 2, 10, 2600, 64, 2500, 3, dtype="f16", kv_len=[2600, 0]), "window_step_kernel<64, true, false>",
                      (19, 6, 2)),
    "combine_dead_rows": (c(2, 4, 1, 16, 3000, 128, 2800, 0, kv_len=[3000, 50], q_start=[2990, -8], layout="bnhd"),
                          "window_step_kernel<128, false, false>", (22, 4, 2)),
    "split_forward": (c(2, 2, 2, 100, 3000, 128, 2900, 5, kv_len=[3000, 40]), "window_fwd_kernel<128, false>", (1, 2, 12)),
    "split_forward_dead_rows": (c(2, 4, 2, 130, 3000, 64, 2900, 0, dtype="f16", kv_len=[3000, 40], q_start=[2870, -60],
                                  layout="bnhd"), "window_fwd_kernel<64, true>", (1, 4, 12)),
    "split_forward_f16": (c(3, 1, 1, 70, 2000, 128, 3000, 0, dtype="f16", kv_len=[2000, 0, 1300]),
                          "window_fwd_kernel<128, true>", (1, 1, 12)),
}

SHARED = {
    "all_blocks_128": (c(2, 14, 2, 400, 400, 128, 77, 3, kv_len=[400, 131]), "window_dkv_kernel<128, false, true>", (9, 2, 2)),
    "all_blocks_128_f16": (c(2, 14, 2, 400, 400, 128, 77, 3, dtype="f16", kv_len=[131, 400], layout="bnhd"),
                           "window_dkv_kernel<128, true, true>", (9, 2, 2)),
    "all_blocks_64_f16": (c(2, 14, 2, 400, 400, 64, 77, 3, dtype="f16", kv_len=[400, 0]), "window_dkv_kernel<64, true, true>",
                          (9, 2, 2)),
    "no_first_units": (c(2, 16, 2, 390, 390, 128, 500, 0, dtype="f16", q_start=[-20, 60]), "window_dkv_kernel<128, true, true>",
                       (12, 2, 2)),
    "first_blocks_only": (c(2, 4, 1, 1100, 1100, 128, 40, 3, kv_len=[1100, 1000]), "window_dkv_kernel<128, false, true>",
                          (11, 1, 2)),
    "first_blocks_only_f16": (c(2, 4, 1, 1100, 1100, 128, 40, 3, dtype="f16", kv_len=[1000, 1100], layout="bnhd"),
                              "window_dkv_kernel<128, true, true>", (11, 1, 2)),
    "first_blocks_only_64_f16": (c(1, 4, 1, 1100, 1100, 64, 40, 140, dtype="f16"), "window_dkv_kernel<64, true, true>",
                                 (13, 1, 1)),
}


@pytest.mark.parametrize("name", FORWARD)
def test_forward(name):
    case = FORWARD[name][0]
    q, k, v, _, sees, how, scale, u = make(case, seed=2)
    o, lse = api.window_attn(q, k, v, **how)
    O, Lse, bo, bl = lo.window_fwd(*(bhnd(x, case["layout"]) for x in (q, k, v)), sees, scale, u)
    within(bhnd(o, case["layout"]), O, bo, "O")
    within(f64(lse), Lse, bl, "LSE")
    again = api.window_attn(q, k, v, **how)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert api.device_error() == 0


@pytest.mark.parametrize("name", SHARED)
def test_shared_key_blocks(name):
    case = SHARED[name][0]
    q, k, v, do, sees, how, scale, u = make(case, seed=3)
    o, lse = api.window_attn(q, k, v, **how)
    got = api.window_attn_bwd(do, q, k, v, o, lse, **how)
    ref, tol = lo.window_bwd(*(bhnd(x, case["layout"]) for x in (do, q, k, v)), sees, scale, u)
    for what, x, r, t in zip(("dq", "dk", "dv"), got, ref, tol):
        within(bhnd(x, case["layout"]), r, t, what)
    again = api.window_attn_bwd(do, q, k, v, o, lse, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert api.device_error() == 0


def launches(run, path):
    run()
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        run()
        torch.cuda.synchronize()
    p.export_chrome_trace(str(path))
    with open(path) as f:
        return [(e["name"], tuple(e["args"]["grid"])) for e in json.load(f)["traceEvents"] if e.get("cat") == "kernel"]


@pytest.mark.parametrize("name", list(FORWARD) + list(SHARED))
def test_launches(name, tmp_path):
    case, kernel, grid = {**FORWARD, **SHARED}[name]
    q, k, v, do, _, how, _, _ = make(case)
    o, lse = api.window_attn(q, k, v, **how)
    run = (lambda: api.window_attn_bwd(do, q, k, v, o, lse, **how)) if name in SHARED else (
        lambda: api.window_attn(q, k, v, **how))
    seen = launches(run, tmp_path / "trace.json")
    if not seen:
        pytest.skip("the profiler sees no kernels here")
    assert any(kernel in n and g == grid for n, g in seen), seen
    combine = any("window_combine_kernel" in n for n, _ in seen)
    assert combine == (name.startswith("combine") or name.startswith("split"))
    assert any("window_dkv_sum_kernel" in n for n, _ in seen) == (name in SHARED)
