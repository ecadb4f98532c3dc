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


@pytest.mark.parametrize("members", [2, 20])
@pytest.mark.parametrize("up", [27.3, 33.3, 37.3, 39.3, 40.3])
def test_prefix_lightest_fp16_weights(members, up):
    """What is held of weights far below the largest in an fp16 cache: 2^-23 of a weight or 2^-42 of the largest.

    One token of value 0 has weight 1, 4095 others the weight 2^-up and the value 2^15, whose sum is the output (at
    least 2^-13 here).  Beside the weights' parts the score's offset, of at most 48, is rounded (2^-24 of it, twice with its
    scale), the exponential is off by 2 units and the sums by 4096 + 8."""
    dev = cuda_device()
    n, page, d = 4096, 64, 64
    k, v = torch.zeros((n // page, 1, page, d)), torch.full((n // page, 1, page, d), 2.0 ** 15)
    k[0, 0, 5, 0], v[0, 0, 5] = 1, 0
    c = ck.KVCache(k.half().to(dev), v.half().to(dev))
    q = torch.zeros((members, 4, d), dtype=torch.float16)
    q[:, :, 0] = up
    x = q[0, 0, 0].double().item()
    table = torch.zeros((members, 1), dtype=torch.int32, device=dev)
    pages = torch.arange(n // page, dtype=torch.int32, device=dev)[None]
    out = ck.shared_prefix_attention(q.to(dev), c, pages, i32(n), i32(0, members), table, torch.zeros_like(table[:, 0]), math.log(2.0))
    light = 2.0 ** -x
    want = torch.full(out.shape, (n - 1) * light * 2.0 ** 15 / (1 + (n - 1) * light), dtype=torch.float64)
    held = (n - 1) * 2.0 ** 15 * max(2.0 ** -23 * light, 2.0 ** -42)
    ref.assert_within(out, want, held + (2 * 48 + 2 + 4096 + 8) * ref.U32 * want, f"2^-{x}")


# -------------------------------------------------------------------- lora_add

@pytest.mark.parametrize("m", [1, 3, 17, 70, 600])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128, 256])
def test_lora_bf16_holds_24_bits_of_v(m, rank):
    """Ranks that cancel: what is left are the last 8 of 22 to 23 bits of v, exactly.

    Rank 2 i has v = p + c 2^-8, p of 14 or 15 bits (a product of a 7- and an 8-bit number) and c an odd number of 8, rank
    2 i + 1 v = p and b the opposite: the output is c 2^-8.  Three parts of bf16 hold these bits, two hold 17 of them and
    never c's last one.  Each column of b has one such pair, so all sums are whole multiples of 2^-8 below 2^24 of them,
    which fp32 holds in any order."""
    dev = cuda_device()
    pairs, adapters, g = rank // 2, 3, torch.Generator().manual_seed(rank)
    odd = lambda lo, hi, *s: torch.randint(lo // 2, hi // 2, s, generator=g) * 2.0 + 1  # noqa: E731
    x, a = torch.zeros((m, 16)), torch.zeros((adapters, rank, 16))
    x[:, 0], x[:, 9] = odd(64, 128, m), 2.0 ** -8
    a[:, ::2, 0] = odd(128, 256, adapters, pairs)
    a[:, 1::2, 0] = a[:, ::2, 0]
    a[:, ::2, 9] = odd(128, 256, adapters, pairs)
    b = torch.zeros((adapters, pairs, rank))
    for i in range(pairs):
        b[:, i, 2 * i], b[:, i, 2 * i + 1] = 1, -1
    ids = torch.arange(m) % (adapters + 1) - 1
    want = torch.zeros((m, pairs))
    for i, t in enumerate(ids.tolist()):
        if t >= 0:
            want[i] = a[t, ::2, 9] * 2.0 ** -8
    w = ck.LoraWeight(a.bfloat16().to(dev), b.bfloat16().to(dev))
    got = ck.lora_add(torch.zeros((m, pairs), device=dev), x.bfloat16().to(dev), w, ids.int().to(dev))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("m", [1, 3, 17, 70, 600])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128, 256])
def test_lora_fp16_holds_22_bits_of_v(m, rank):
    """As above with v = p, a product of two 11-bit numbers with 21 or 22 bits, and v = h, p's leading bits: p - h is exact.
    (One part of fp16 holds 11 bits.)"""
    dev = cuda_device()
    pairs, adapters, g = rank // 2, 3, torch.Generator().manual_seed(rank)
    odd = lambda *s: torch.randint(512, 1024, s, generator=g) * 2.0 + 1  # noqa: E731
    x, a = torch.zeros((m, 16)), torch.zeros((adapters, rank, 16))
    x[:, 0] = odd(1)                     # (of all rows: h goes by the product)
    a[:, ::2, 0] = odd(adapters, pairs)
    p = x[0, 0] * a[:, ::2, 0]
    h = torch.floor(p / 2048)            # below 2^11, to be multiplied by 2048
    x[:, 9], a[:, 1::2, 9] = 2048.0, h
    b = torch.zeros((adapters, pairs, rank))
    for i in range(pairs):
        b[:, i, 2 * i], b[:, i, 2 * i + 1] = 1, -1
    ids = torch.arange(m) % (adapters + 1) - 1
    want = torch.zeros((m, pairs))
    for i, t in enumerate(ids.tolist()):
        if t >= 0:
            want[i] = p[t] - h[t] * 2048
    w = ck.LoraWeight(a.half().to(dev), b.half().to(dev))
    got = ck.lora_add(torch.zeros((m, pairs), device=dev), x.half().to(dev), w, ids.int().to(dev))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("m", [1, 17, 70, 600])
@pytest.mark.parametrize("rank", [8, 32, 64, 256])
def test_lora_fp16_small_ranks_beside_a_large_one(m, rank):
    """v of a rank far below the row's largest is held to 2^-38 of that: rank 0 has v = 1 (2^13 after the power of two
    that the row is multiplied by, its lowest place), the others 2^-20 to 2^-36, each with a column of b of its own.
    v itself is exact, and so are the product with b = 1 and the sum."""
    dev = cuda_device()
    g = torch.Generator().manual_seed(rank)
    x, a = torch.zeros((m, 16)), torch.zeros((1, rank, 16))
    x[:, 0], x[:, 9] = 1.0, 2.0 ** -13
    a[0, 0, 0] = 1
    a[0, 1:, 9] = (1 + torch.rand(rank - 1, generator=g)) * 2.0 ** (-7 - torch.arange(rank - 1) % 17).float()
    a = a.half()
    b = torch.eye(rank).view(1, rank, rank).half()
    w = ck.LoraWeight(a.to(dev), b.to(dev))
    got = ck.lora_add(torch.zeros((m, rank), device=dev), x.half().to(dev), w, torch.zeros(m, dtype=torch.int32, device=dev)).cpu().double()
    want = a[0, :, 9].double() * 2.0 ** -13
    want[0] = 1
    assert ((got - want).abs() <= torch.maximum(torch.tensor(2.0 ** -38, dtype=torch.float64), 2.0 ** -22 * want)).all()
    assert (got[:, 0] == 1).all()


# -------------------------------------------------------------- token_logprobs

@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("vocab", [3001, 20000, 60000])
def test_logprobs_are_not_off_to_one_side(vocab, top):
    """The mean error of 256 rows: what all terms share does not average out.

    One logit is 0, the others about -log(vocab) - 1.6: the sum is about 1.2.  A change to base 2 by a factor that is r
    too small makes every e^d too large by r |d| of it: a log probability by r sum p |d|, the entropy by about r sum p d^2.
    With one fp32 constant for log2(e), r is 1.3e-8.  Allowed is a third of that, and what the rows' own errors leave in
    the mean: the lane that has the largest logit adds its other terms to 1, up to 16 times, each sum off by 2^-24 at
    most and evenly, so by 4 2^-24 / sqrt(3) as a standard deviation, a 16th of that in the mean of 256, three of those.
    That is as much as r does to a log probability.  The entropy log S - W / S, W = sum e^d d, shows r alone: of a relative
    error of S it takes 1 - |W| / S, here from -0.7 to -1.3 times, and r makes 2e-7 of it or more."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn((256, vocab), generator=g) * 0.5 - (math.log(vocab) + 1.6)
    x[:, 7] = 0
    tokens = torch.full((256,), 7, dtype=torch.int64, device=cuda_device())
    r = ck.token_logprobs(x.to(cuda_device()), tokens, top)
    d = x.double()
    p = torch.softmax(d, -1)
    want, entropy = torch.log(p[:, 7]), -(p * torch.log(p)).sum(-1)
    third, noise = 1.3e-8 / 3, 3 * 4 * ref.U32 / math.sqrt(3) / 16
    assert abs((r.logprob.cpu().double() - want).mean()) <= third * (p * d.abs()).sum(-1).mean() + noise
    assert abs((r.entropy.cpu().double() - entropy).mean()) <= third * (p * d * d).sum(-1).mean() + 1.3 * noise
