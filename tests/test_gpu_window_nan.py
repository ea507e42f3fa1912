"""window_attn never turns a NaN among the keys and values that a query sees into a plausible answer (GPU)."""
import pytest
import torch

from block_sparse_video_tile_b200 import api

pytestmark = pytest.mark.gpu

# Nq, Nk, heads: the step kernel with one split, as a cluster, and with the combine kernel; the tcgen05 kernel whole and
# with its keys split
FORMS = {"step": (1, 100, 2), "cluster": (1, 1000, 2), "combine": (1, 40000, 2), "whole": (300, 300, 2),
         "split": (100, 3000, 1)}


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("form", FORMS)
def test_nan_in_a_visible_key(form, what):
    Nq, Nk, H = FORMS[form]
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(1, H, Nq, 128, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(1, H, Nk, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    (k if what == "k" else v)[0, 0, 3, 5] = float("nan")        # every query sees the first 8 keys, and those of its window
    o, lse = api.window_attn(q, k, v, Nk, sink=8)
    rows = slice(3, None) if Nq == Nk else slice(None)          # (of a square call, those from key 3 on)
    if what == "k":
        assert o[0, 0, rows].isnan().all() and lse[0, 0, rows].isnan().all()
    else:
        assert o[0, 0, rows, 5].isnan().all() and lse.isfinite().all()
    if H > 1:
        assert o[0, 1].isfinite().all() and lse[0, 1].isfinite().all()


@pytest.mark.parametrize("form", FORMS)
def test_only_nan_is_not_nothing(form):
    """A query whose visible keys all hold NaN gets NaN, not the O = 0 and LSE = -inf of one that sees nothing."""
    Nq, Nk, H = FORMS[form]
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(1, H, Nq, 128, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, H, Nk, 128, generator=g, device="cuda").bfloat16()
    o, lse = api.window_attn(q, torch.full_like(v, float("nan")), v, Nk)
    assert o.isnan().all() and lse.isnan().all()
