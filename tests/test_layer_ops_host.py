"""qk_norm_rope and window_attn without a GPU: their float64 restatements against differences and independent forms,
and every refusal of the C ABI and of the Python calls that comes before a device is touched."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_video_tile_b200 import _native, api
from block_sparse_video_tile_b200._native import VsaNormRope, VsaQkSide, VsaWindow
from oracle import layer_ops as lo

L = _native.lib()


# ------------------------------------------------------------------ the restatements
def _diff(f, x, dy, eps=1e-5):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = ((f(a) - f(b)) * dy).sum() / (2 * eps)
    return g


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_gradient_against_differences(interleaved):
    r = np.random.default_rng(0)
    x, dy, w = r.normal(size=(1, 2, 4, 12)), r.normal(size=(1, 2, 4, 12)), r.normal(size=12)
    ang = lo.angles((1, 2, 2), 12, first=(3, 0, 0))
    dx, dw, _, _ = lo.norm_rope_bwd(dy, x, w, 1e-3, ang, interleaved)
    assert np.abs(dx - _diff(lambda t: lo.norm_rope(t, w, 1e-3, ang, interleaved), x, dy)).max() < 1e-8
    assert np.abs(dw - _diff(lambda t: lo.norm_rope(x, t, 1e-3, ang, interleaved), w, dy)).max() < 1e-8


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    r = np.random.default_rng(1)
    ang = lo.angles((9, 1, 1), 16, split=(16, 0, 0))
    a, b = r.normal(size=16), r.normal(size=16)
    q, k = (lo.rotate(np.tile(x, (9, 1)), ang, interleaved) for x in (a, b))
    assert np.abs((q * q).sum(-1) - (a * a).sum()).max() < 1e-12
    s = q @ k.T
    for i in range(8):
        assert abs(s[i, i + 1] - s[0, 1]) < 1e-12


def test_rope_table_holds_the_angles():
    grid, d, first = (3, 4, 5), 64, (7, 0, 1)
    t = api.rope_table(grid, d, first=first, device="cpu").double().numpy()
    ct, cy, cx = (s // 2 for s in api.rope_split(d))
    assert api.rope_split(d) == (24, 20, 20) and api.rope_split(128) == (44, 42, 42)
    ang = lo.angles(grid, d, first=first)
    for n in range(60):
        rows = np.concatenate((t[n // 20 * ct:][:ct], t[3 * ct + n // 5 % 4 * cy:][:cy],
                               t[3 * ct + 4 * cy + n % 5 * cx:][:cx]))
        assert np.abs(rows - np.stack((np.cos(ang[n]), np.sin(ang[n])), -1)).max() <= 2.0 ** -24


@pytest.mark.parametrize("window,sink,unit", [(2, 0, 1), (1, 1, 3), (3, 2, 2), (99, 0, 4)])
def test_window_gradient_against_differences(window, sink, unit):
    r = np.random.default_rng(2)
    q, k, v, do = (r.normal(size=(1, h, n, 4)) for h, n in ((2, 5), (1, 8), (1, 8), (2, 5)))
    sees = [lo.visible(5, 8, 7, 2, window, sink, unit)]
    (dq, dk, dv), _ = lo.window_bwd(do, q, k, v, sees, 0.5, 0.0)
    for x, g, f in ((q, dq, lambda t: lo.window_fwd(t, k, v, sees, 0.5, 0.0)[0]),
                    (k, dk, lambda t: lo.window_fwd(q, t, v, sees, 0.5, 0.0)[0]),
                    (v, dv, lambda t: lo.window_fwd(q, k, t, sees, 0.5, 0.0)[0])):
        assert np.abs(g - _diff(f, x, do)).max() < 1e-8


def test_window_covering_everything_is_causal_attention():
    r = np.random.default_rng(3)
    q, k, v = (torch.from_numpy(r.normal(size=(1, 2, 9, 8))) for _ in range(3))
    sees = [lo.visible(9, 9, 9, 0, 1 << 20, 0, 1)]
    ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True).numpy()
    assert np.abs(lo.window_fwd(q.numpy(), k.numpy(), v.numpy(), sees, 8 ** -0.5, 0.0)[0] - ref).max() < 1e-12


def test_visible_ranges_by_hand():
    see = lo.visible(6, 12, 11, 5, 2, 1, 3)          # positions 5 .. 10, units of 3
    want = {5: range(0, 6), 6: range(0, 9), 8: range(0, 9), 9: [0, 1, 2] + list(range(6, 11)),
            10: [0, 1, 2] + list(range(6, 11))}
    for p, js in want.items():
        assert sorted(np.flatnonzero(see[p - 5])) == list(js)


# ------------------------------------------------------------------ refusals of the C ABI
def _side(**kw):
    a = dict(B=1, H=2, T=2, Hh=3, W=4, weight_f32=1, x=256, x_s=(24 * 256, 256, 128), y=1 << 20, y_s=(24 * 256, 256, 128),
             dx=0, dx_s=(24 * 256, 256, 128), weight=4096, table=8192, dweight=0)
    a.update(kw)
    return VsaQkSide(*a.values())


def _nr(d=128, dtype=0, interleaved=1, split=(44, 42, 42), eps=1e-6):
    return VsaNormRope(d, dtype, interleaved, split, eps)


@pytest.mark.parametrize("nr,side,status", [
    (dict(d=96), {}, 3), (dict(dtype=2), {}, 3), (dict(eps=-1.0), {}, 1), (dict(eps=float("nan")), {}, 1),
    (dict(eps=float("inf")), {}, 1), (dict(split=(44, 42, 44)), {}, 1), (dict(split=(45, 41, 42)), {}, 1),
    (dict(split=(170, -84, 42)), {}, 1), ({}, dict(B=0), 1), ({}, dict(W=-1), 1), ({}, dict(x=0), 1), ({}, dict(y=0), 1),
    ({}, dict(x=264), 4), ({}, dict(y=(1 << 20) + 8), 4), ({}, dict(weight=4100), 4), ({}, dict(table=8196), 4),
    ({}, dict(x_s=(0, 0, 128)), 1), ({}, dict(x_s=(0, -256, 128)), 1), ({}, dict(x_s=(0, 256, 132)), 4),
    ({}, dict(T=1 << 16, Hh=1 << 16), 8), ({}, dict(x_s=(0, 1 << 39, 128)), 8),
])
def test_norm_rope_refusals(nr, side, status):
    p, s = _nr(**nr), _side(**side)
    assert L.vsa_qk_norm_rope(p, s, None, None) == status
    assert L.vsa_qk_norm_rope(p, s, s, None) == status
    if not nr:
        assert L.vsa_qk_norm_rope(p, _side(), s, None) == status
    b = _side(**{**dict(dx=1 << 21, dweight=1 << 22), **side})
    assert L.vsa_qk_norm_rope_bwd(p, b, None, 1 << 23, 1 << 30, None) == status
    assert L.vsa_qk_norm_rope_bwd_workspace_bytes(p, b, None) == 0


def test_norm_rope_bwd_refusals():
    p, s = _nr(), _side(dx=1 << 21, dweight=1 << 22)
    need = L.vsa_qk_norm_rope_bwd_workspace_bytes(p, s, s)
    assert need > 0 and need == 2 * L.vsa_qk_norm_rope_bwd_workspace_bytes(p, s, None)
    call = L.vsa_qk_norm_rope_bwd
    assert call(p, s, s, 1 << 23, need - 1, None) == 5
    assert call(p, s, s, None, need, None) == 5
    assert call(p, s, s, (1 << 23) + 4, need, None) == 4
    assert call(p, _side(dx=0, dweight=1 << 22), None, 1 << 23, need, None) == 1
    assert call(p, _side(dx=1 << 21, dweight=0), None, 1 << 23, need, None) == 1       # a weight asks for its gradient
    assert call(p, _side(dx=1 << 21, dweight=1 << 22, weight=0), None, 1 << 23, need, None) == 1
    assert call(p, _side(dx=(1 << 21) + 2, dweight=1 << 22), None, 1 << 23, need, None) == 4
    assert L.vsa_qk_norm_rope_bwd_workspace_bytes(p, _side(dx=1 << 21, weight=0), None) == 0
    assert call(None, s, s, 1 << 23, need, None) == 1 and call(p, None, s, 1 << 23, need, None) == 1


def _win(**kw):
    s = (1 << 20, 256, 128)
    a = dict(B=2, Hq=4, Hkv=2, Nq=10, Nk=20, d=128, dtype=0, window=4, sink=1, unit=2, kv_len=0, q_start=0, q_s=s, k_s=s,
             v_s=s, o_s=s, do_s=s, dq_s=s, dk_s=s, dv_s=s)
    a.update(kw)
    return VsaWindow(*a.values())


def _fwd(w, q=256, k=512, v=768, scale=0.1, o=1024, lse=2048, ws=4096, n=1 << 30):
    return L.vsa_window_attn(w, q, k, v, scale, o, lse, ws, n, None)


def _bwd(w, do=256, q=512, k=768, v=1024, o=1280, lse=2048, scale=0.1, dq=4096, dk=8192, dv=12288, ws=1 << 20, n=1 << 30):
    return L.vsa_window_attn_bwd(w, do, q, k, v, o, lse, scale, dq, dk, dv, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(Nq=0), 1), (dict(Nk=-1), 1), (dict(Hq=3), 1), (dict(window=0), 1), (dict(sink=-1), 1),
    (dict(unit=0), 1), (dict(d=80), 3), (dict(dtype=5), 3), (dict(kv_len=6), 4), (dict(q_start=6), 4),
    (dict(Nq=(1 << 30) + 1), 8), (dict(B=65536), 8), (dict(Hq=65536), 8), (dict(k_s=(1 << 20, 0, 128)), 1),
    (dict(v_s=(1 << 20, -256, 128)), 1), (dict(q_s=(1 << 20, 250, 128)), 4), (dict(o_s=(1 << 40, 256, 128)), 8),
])
def test_window_refusals(kw, status):
    w = _win(**kw)
    assert _fwd(w) == status and _bwd(w) == status
    assert L.vsa_window_attn_workspace_bytes(w) == 0 and L.vsa_window_attn_bwd_workspace_bytes(w) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(q=264), 4), (dict(o=1032), 4),
    (dict(lse=2050), 4), (dict(ws=4100), 4),
])
def test_window_argument_refusals(kw, status):
    assert _fwd(_win(), **kw) == status
    assert _bwd(_win(), **kw) == status


def test_window_bwd_refusals():
    w = _win()
    need = L.vsa_window_attn_bwd_workspace_bytes(w)
    assert need >= 2 * 4 * 10 * 4
    assert _bwd(w, n=need - 1) == 5 and _bwd(w, ws=None) == 5
    for name in ("do", "dq", "dk", "dv"):
        assert _bwd(w, **{name: 0}) == 1
        assert _bwd(w, **{name: 4104}) == 4
    assert _bwd(_win(dk_s=(1 << 20, 0, 128))) == 1
    assert L.vsa_window_attn(None, 256, 512, 768, 0.1, 1024, 2048, None, 0, None) == 1


# ------------------------------------------------------------------ refusals of the Python calls
def test_python_calls_refuse_cpu_tensors_and_bad_arguments():
    q = torch.zeros(1, 2, 24, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.qk_norm_rope(q, q, (2, 3, 4))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        api.qk_norm_rope(q.float(), None, (2, 3, 4))
    with pytest.raises(ValueError, match="layout"):
        api.window_attn(q, q, q, 4, layout="nbhd")
    with pytest.raises(ValueError, match="CUDA"):
        api.window_attn(q, q, q, 4)
    with pytest.raises(ValueError, match="4-D"):
        api.window_attn(q[0], q, q, 4)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        api.window_attn(q.double(), q, q, 4)


def test_only_broadcast_gradients_are_copied():
    from block_sparse_video_tile_b200._strided import spread
    x = torch.zeros(1, 1, 4, 8)
    for same in (None, x, x.as_strided((1, 1, 4, 8), (0, 0, 8, 1)), x.expand(2, 3, 4, 8)):      # (a CPU tensor is refused later)
        assert spread(same, None) is same
