"""fp16 window_attn where a first key draws nearly all of the weight and the answer comes from the others (GPU, against
float64).

One key stands e^14 above the others and its V is 0, as models use first tokens: the others' P is then about 2^-20 of
the largest.  O is a sum of products with P rounded once to fp16 and is rounded once, half a step u = 2^-11 each; scores,
sums and LSE are float32.  Errors of single values add up at random, so 2-norms are compared: two roundings of at most
u of the norm, and half of u for the rest.  V is 64 times a normal value, so that O (about 2^-7) is a normal number of
fp16.  LSE is the dominating key's: off by float32 errors of the score, 2^-15 of sum |q k| (oracle/layer_ops.py)."""
import math

import pytest
import torch

from block_sparse_video_tile_b200 import api

pytestmark = pytest.mark.gpu


# queries, keys, heads: the step kernel with one split, as a cluster and with the combine kernel; the tcgen05 kernel whole
# and with its keys split
@pytest.mark.parametrize("Nq,Nk,H", [(1, 250, 4), (4, 1000, 2), (1, 8000, 2), (1100, 8000, 40), (100, 8000, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_answer_beside_a_dominating_key(Nq, Nk, H, d):
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(1, H, n, d, generator=g, device="cuda") for n in (Nq, Nk, Nk))
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, :, 0] = 0.0
    k[:, :, 0, 0] = 14 / 4 * math.sqrt(d)
    v *= 64
    v[:, :, 0] = 0.0
    q, k, v = q.half(), k.half(), v.half()
    o, lse = api.window_attn(q, k, v, 1, unit=Nk)
    z = (q.double() @ k.double().transpose(2, 3)) / math.sqrt(d)
    ref = z.softmax(-1) @ v.double()
    assert float(ref.square().mean().sqrt()) > 2.0 ** -12
    assert float((o.double() - ref).norm() / ref.norm()) <= 2.5 * 2.0 ** -11
    assert float((lse.double() - z.logsumexp(-1)).abs().max()) <= 2.0 ** -15 * 24 + 2.0 ** -20 * 15
