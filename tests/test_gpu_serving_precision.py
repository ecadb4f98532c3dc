"""The precision that the operators of a server's batch promise, at inputs where the outputs show it."""
import math

import pytest
import torch

import int8_weight_quantized_amd as ck
from tests import serving_ref as ref
from tests.gpu_util import cuda_device

pytestmark = pytest.mark.gpu
DT = ref.TYPES


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=cuda_device())


# ---------------------------------------------------- shared_prefix_attention

@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("members,hq,d", [(2, 8, 64), (8, 8, 64), (16, 8, 128), (8, 4, 192), (16, 16, 256)])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16")])
def test_prefix_weights_to_32_bits(cache, dtype, members, hq, d, own):
    """Values that almost cancel, so that the output shows the weights' own precision: groups of few and of many
    rows, and the same tokens as the sequences' own.

    Tokens 0 and 2 have score 0 and, in column r, the values -hi and -lo; token 1 has the value 1 and for row r of the
    queries the weight e = exp(score), hi + lo = e to 14 bits or more: out = (e - hi - lo) / (2 + e), almost nothing
    in column r.  Allowed, in units of 2^-24 of (e + hi + |lo|) / (2 + e): 12 for the weight (three roundings of the
    score's change to base 2, at most 1 in magnitude, one of its offset from M, at most 8 in magnitude, the
    exponential's 2, a value scale's 3, its own to 32 bits), 8 for the products and sums, 4 for the division."""
    dev = cuda_device()
    rows, t = members * hq, DT[dtype]
    score = -torch.linspace(0.02, 0.69, rows).to(t)
    e = torch.exp(score.double())
    k, v = torch.zeros((1, 1, 4, d)), torch.zeros((1, 1, 4, d))
    k[0, 0, 1, 0] = 1
    ks = vs = None
    if cache == "int8":
        v[0, 0, 1], v[0, 0, 0, :rows] = 64, -torch.round(e * 128).float()
        v[0, 0, 2, :rows] = -torch.round((e + v[0, 0, 0, :rows].double() / 128) * 2 ** 14).float()
        vs = torch.tensor([2.0 ** -7, 2.0 ** -6, 2.0 ** -14, 0.0]).view(1, 1, 4)
        ks = torch.ones((1, 1, 4))
        values = v[0, 0, :3].double() * vs[0, 0, :3, None].double()
        k, v = k.to(torch.int8), v.to(torch.int8)
    else:
        v[0, 0, 1], v[0, 0, 0, :rows] = 1, -e.to(t).float()
        v[0, 0, 2, :rows] = -(e - e.to(t).double()).to(t).float()
        values = v[0, 0, :3].to(t).double()
        k, v = k.to(t), v.to(t)
    c = ck.KVCache(*(None if x is None else x.to(dev) for x in (k, v, ks, vs)))
    q = torch.zeros((members, hq, d), dtype=t)
    q[:, :, 0] = score.view(members, hq)
    table = torch.zeros((members, 1), dtype=torch.int32, device=dev)
    lens = torch.full((members,), 3 if own else 0, dtype=torch.int32, device=dev)
    out = ck.shared_prefix_attention(q.to(dev), c, i32([0]), i32(3), i32(0, 0 if own else members), table, lens, 1.0)
    weight = torch.stack([torch.ones_like(e), e, torch.ones_like(e)], -1)
    want = weight @ values / (2 + e[:, None])
    slack = 24 * ref.U32 * (weight @ values.abs()) / (2 + e[:, None])
    ref.assert_within(out.view(rows, d), want, slack, "almost nothing")
