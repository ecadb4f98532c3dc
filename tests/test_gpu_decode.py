"""The decode-step operators on the GPU against plain references in 64 bits:
qk_norm_rope, paged_attention, int4_pack and int4_linear."""
import pytest
import torch

import int8_weight_quantized_amd as ck
from tests import decode_ref as ref
from tests.gpu_util import cuda_device

pytestmark = pytest.mark.gpu
DT = ref.TYPES


def rand(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 7919 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g) * scale).to(dtype)


# ------------------------------------------------------------- qk_norm_rope

def rope_inputs(tokens, hq, hk, d, rot, dtype, far, seed=1):
    dev = cuda_device()
    qkv = rand(tokens, (hq + 2 * hk) * d, dtype=DT[dtype], seed=seed).to(dev)
    q = qkv[:, :hq * d].view(tokens, hq, d)
    k = qkv[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
    v = qkv[:, (hq + hk) * d:].view(tokens, hk, d)
    qw, kw = (1 + 0.3 * rand(d, seed=seed + 8)).to(dev), (1 + 0.3 * rand(d, seed=seed + 9)).to(dev)
    pos = torch.randint(0, far, (tokens,), generator=torch.Generator().manual_seed(seed)).to(dev)
    return q, k, v, qw, kw, pos, ck.rope_table(far, rot, device=dev) if rot else None


@pytest.mark.parametrize("tokens,hq,hk,d,rot,interleaved,dtype,cache,page,norm", [
    (1, 32, 8, 128, 128, False, "bf16", "bf16", 16, True),
    (3, 4, 4, 64, 64, False, "fp16", "int8", 1, True),
    (65, 7, 1, 96, 48, False, "bf16", "int8", 8, True),
    (33, 16, 2, 256, 128, True, "fp16", "fp16", 32, True),
    (17, 2, 1, 512, 512, True, "bf16", "bf16", 64, False),
    (9, 5, 5, 80, 32, False, "fp16", "fp16", 16, True),
    (31, 3, 1, 8, 0, False, "bf16", "int8", 16, True),
    (20, 6, 2, 192, 192, True, "bf16", "int8", 128, False),
    (700, 24, 8, 128, 64, False, "bf16", "bf16", 16, True),
])
def test_rope(tokens, hq, hk, d, rot, interleaved, dtype, cache, page, norm):
    dev = cuda_device()
    q, k, v, qw, kw, pos, table = rope_inputs(tokens, hq, hk, d, rot, dtype, 5000)
    qw, kw = (qw, kw) if norm else (None, None)
    pages = -(-tokens // page) + 2
    c = ck.KVCache.empty(pages, hk, page, d, cache, dev)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(7)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:tokens]
    if tokens > 2:
        slots[1] = -1
        slots[2] = pages * page          # outside: not written
    qo, ko = ck.qk_norm_rope(q, k, v, pos if rot else None, table, qw, kw, eps=1e-5, interleaved=interleaved,
                             cache=c, slots=slots.to(dev), k_out=torch.empty_like(k))
    want_q, slack_q = ref.rope(q, qw, table, pos, rot, interleaved, 1e-5)
    want_k, slack_k = ref.rope(k, kw, table, pos, rot, interleaved, 1e-5)
    ref.assert_within(qo, want_q, slack_q, "q")
    ref.assert_within(ko, want_k, slack_k, "k_out")
    used = (slots >= 0) & (slots < pages * page)
    for name, t, sc, want, slack in (("k", c.k, c.k_scale, want_k, slack_k),
                                     ("v", c.v, c.v_scale, v.cpu().double(), torch.zeros(()))):
        flat = t.cpu().transpose(1, 2).reshape(pages * page, hk, d)
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[slots[used]] = False
        assert (flat[rest] == 7).all(), f"{name}: a row of the cache that no token has was written"
        got, w = flat[slots[used]], want[used]
        if cache != "int8":
            ref.assert_within(got, w, slack[used] if slack.dim() else torch.zeros_like(w), f"cache {name}")
            continue
        scale = sc.cpu().transpose(1, 2).reshape(pages * page, hk)[slots[used]].double()
        if name == "v":                  # given values: the row quantisation's codes and scales, bit for bit
            x = v.cpu()[used].float()
            scales = x.abs().amax(-1) * (torch.ones(()) / 127)
            assert torch.equal(scale, scales.double())
            assert torch.equal(got, torch.round(x / scales[..., None]).clamp(-127, 127).to(torch.int8))
            continue
        amax = w.abs().amax(-1)
        e = slack[used].amax(-1)
        assert ((scale - amax / 127).abs() <= (e + amax * 2 * ref.U32) / 127 + 2.0 ** -149).all(), f"scale of {name}"
        # a code is the nearest: half a scale off, and what the value and the scale are off themselves
        off = (got.double() * scale[..., None] - w).abs()
        assert (off <= 0.5 * scale[..., None] * (1 + 2.0 ** -20) + 2 * e[..., None]).all(), f"codes of {name}"
        assert got.abs().max() <= 127


@pytest.mark.parametrize("hk,d,rot,interleaved", [(8, 96, 96, False), (4, 128, 64, True), (2, 64, 64, False),
                                                  (8, 192, 192, False), (8, 256, 128, True)])
def test_rope_int8_codes_are_the_formulas(hk, d, rot, interleaved):
    """An int8 cache's codes and scales, keys' and values', are bit for bit
    those of the same formula in fp32 torch operations on this device; a row
    of zeros has scale 0 and codes 0."""
    dev = cuda_device()
    q, k, v, qw, kw, pos, table = rope_inputs(40, 4, hk, d, rot, "bf16", 100)
    v[5, 1] = 0
    k[6, 0] = 0
    c = ck.KVCache.empty(5, hk, 8, d, "int8", dev)
    ck.qk_norm_rope(q, k, v, pos, table, qw, kw, interleaved=interleaved, cache=c, slots=torch.arange(40, device=dev))
    y = k.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * kw
    cos, sin = table[pos][:, None].split(rot // 2, -1)
    x, z = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    turned = x * cos - z * sin, z * cos + x * sin
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    for got, scale, y in ((c.k, c.k_scale, torch.cat([turned, y[..., rot:]], -1)), (c.v, c.v_scale, v.float())):
        s = y.abs().amax(-1) * (torch.ones((), device=dev) / 127)
        codes = torch.where(s[..., None] > 0, torch.round(y / s[..., None]), torch.zeros_like(y))
        assert torch.equal(scale.transpose(1, 2).reshape(40, hk), s)
        assert torch.equal(got.transpose(1, 2).reshape(40, hk, d), codes.clamp(-127, 127).to(torch.int8))


def test_rope_in_place_and_queries_alone():
    q, k, v, qw, kw, pos, table = rope_inputs(50, 6, 2, 128, 128, "bf16", 300)
    want_q, want_k = ck.qk_norm_rope(q, k, None, pos, table, qw, kw)
    alone, none = ck.qk_norm_rope(q, None, None, pos, table, qw)
    assert none is None and torch.equal(alone, want_q)
    qq, kk = ck.qk_norm_rope(q, k, None, pos, table, qw, kw, q_out=q, k_out=k)
    assert qq is q and kk is k and torch.equal(q, want_q) and torch.equal(k, want_k)


def test_rope_positions_outside_the_table():
    """Such a token's rows are NaN and the cache keeps its rows; the others are not touched."""
    dev = cuda_device()
    q, k, v, qw, kw, pos, table = rope_inputs(6, 3, 1, 96, 48, "bf16", 64)
    good, good_k = ck.qk_norm_rope(q, k, None, pos, table, qw, kw)
    pos[1], pos[4] = -1, 64
    c = ck.KVCache.empty(1, 1, 8, 96, "bf16", dev)
    c.k.fill_(7)
    c.v.fill_(7)
    qo, ko = ck.qk_norm_rope(q, k, v, pos, table, qw, kw, cache=c, slots=torch.arange(6, device=dev), k_out=torch.empty_like(k))
    for t in range(6):
        if t in (1, 4):
            assert qo[t].isnan().all() and ko[t].isnan().all()
            assert (c.k[0, 0, t] == 7).all() and (c.v[0, 0, t] == 7).all()
        else:
            assert torch.equal(qo[t], good[t]) and torch.equal(ko[t], good_k[t])
            assert torch.equal(c.k[0, 0, t], good_k[t, 0]) and torch.equal(c.v[0, 0, t], v[t, 0])


def test_rope_zero_tokens_and_zero_rows():
    q, k, v, qw, kw, pos, table = rope_inputs(4, 2, 2, 64, 64, "fp16", 64)
    qo, ko = ck.qk_norm_rope(q[:0], k[:0], None, pos[:0], table, qw, kw)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 2, 64)
    q.zero_()
    qo, _ = ck.qk_norm_rope(q, k, None, pos, table, qw, kw)
    assert (qo == 0).all()


def test_rope_far_cache_rows():
    """A row past 2^31 elements of the cache."""
    dev = cuda_device()
    pages = (1 << 31) // (16 * 128) + 3
    c = ck.KVCache(*(torch.zeros((pages, 1, 16, 128), dtype=torch.int8, device=dev) for _ in range(2)),
                   *(torch.zeros((pages, 1, 16), device=dev) for _ in range(2)))
    q, k, v, qw, kw, pos, table = rope_inputs(2, 1, 1, 128, 128, "bf16", 64)
    slots = torch.tensor([pages * 16 - 1, 0], device=dev)
    ck.qk_norm_rope(q, k, v, pos, table, qw, kw, cache=c, slots=slots)
    near = ck.KVCache.empty(1, 1, 2, 128, "int8", dev)
    ck.qk_norm_rope(q, k, v, pos, table, qw, kw, cache=near, slots=torch.arange(2, device=dev))
    for far, t in ((c.k, near.k), (c.v, near.v), (c.k_scale, near.k_scale), (c.v_scale, near.v_scale)):
        assert torch.equal(far[-1, 0, 15], t[0, 0, 0]) and torch.equal(far[0, 0, 0], t[0, 0, 1])
    assert int((c.v_scale != 0).sum()) == 2


# ---------------------------------------------------------- paged_attention

def make_cache(pages, hk, page, d, cache, dtype, layout="hnd", seed=5):
    dev = cuda_device()
    shape = (pages, hk, page, d) if layout == "hnd" else (pages, page, hk, d)
    k, v = rand(*shape, seed=seed).to(dev), rand(*shape, seed=seed + 1).to(dev)
    if cache == "int8":
        ks, vs = (t.abs().amax(-1) / 127 for t in (k, v))
        k, v = (torch.round(t / s[..., None]).to(torch.int8) for t, s in ((k, ks), (v, vs)))
    else:
        k, v, ks, vs = k.to(DT[dtype]), v.to(DT[dtype]), None, None
    if layout != "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
        ks, vs = (None if t is None else t.transpose(1, 2) for t in (ks, vs))
    return ck.KVCache(k, v, ks, vs)


def tables(lens, page, pages, seed=11):
    """Every sequence's pages, all different, the table's unused entries far outside the cache."""
    width = max(1, max(-(-n // page) for n in lens))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lens):
        c = -(-n // page)
        t[i, :c] = order[at:at + c]
        at += c
    return t.to(cuda_device()), torch.tensor(lens, dtype=torch.int32, device=cuda_device())


def poison(cache, table, lens, window=0, sinks=0):
    """Rows that no sequence sees become NaN (codes 127 with a NaN scale)."""
    page = cache.page_size
    seen = torch.zeros((cache.pages, page), dtype=torch.bool)
    for i, n in enumerate(lens.tolist()):
        at = ref.visible_tokens(n, window, sinks)
        seen[table[i].cpu().long()[at // page], at % page] = True
    hide = ~seen.to(cache.device)[:, None, :].expand(-1, cache.heads, -1)
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        t[hide] = 127 if s is not None else float("nan")
        if s is not None:
            s[hide] = float("nan")


def check_attention(q, cache, table, lens, scale=None, window=0, sinks=0, **kw):
    out = ck.paged_attention(q, cache, table, lens, scale, window=window, sinks=sinks, **kw)
    want, slack = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lens,
                                q.shape[2] ** -0.5 if scale is None else scale, window, sinks)
    ref.assert_within(out, want, slack, "attention")
    return out


@pytest.mark.parametrize("hq,hk,d,dtype,cache,page", [
    (8, 8, 128, "bf16", "bf16", 16),
    (32, 8, 128, "bf16", "int8", 16),
    (6, 2, 64, "fp16", "fp16", 8),
    (7, 1, 96, "fp16", "int8", 1),
    (16, 1, 192, "bf16", "bf16", 32),
    (16, 2, 256, "fp16", "int8", 64),
    (20, 1, 128, "bf16", "bf16", 128),
    (33, 1, 64, "bf16", "int8", 2),
    (40, 2, 256, "bf16", "bf16", 4),
])
def test_attention_lengths(hq, hk, d, dtype, cache, page):
    """Lengths about the borders of pages, tiles and splits, 0 and 1 among them; unseen rows are NaN."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1500]
    pages = sum(-(-n // page) for n in lens) + 1
    c = make_cache(pages, hk, page, d, cache, dtype)
    table, n = tables(lens, page, pages)
    poison(c, table, n)
    q = rand(len(lens), hq, d, dtype=DT[dtype], scale=2.0).to(cuda_device())
    out = check_attention(q, c, table, n)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 16), (100, 4), (333, 37), (1000, 2000), (4096, 4)])
@pytest.mark.parametrize("cache,d", [("bf16", 128), ("int8", 64)])
def test_attention_window_and_sinks(window, sinks, cache, d):
    lens = [0, 1, 4, 5, 6, 50, 104, 105, 333, 370, 371, 1001, 2500]
    pages = sum(-(-n // 16) for n in lens) + 1
    c = make_cache(pages, 2, 16, d, cache, "bf16")
    table, n = tables(lens, 16, pages)
    poison(c, table, n, window, sinks)
    check_attention(rand(len(lens), 8, d, dtype=torch.bfloat16, scale=2.0).to(cuda_device()), c, table, n,
                    window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_long(dtype):
    """One long sequence among short ones: many splits, most of them empty for the short ones."""
    lens = [40000, 3, 9000, 0]
    pages = sum(-(-n // 16) for n in lens)
    c = make_cache(pages, 2, 16, 128, dtype, dtype)
    table, n = tables(lens, 16, pages)
    check_attention(rand(4, 8, 128, dtype=DT[dtype], scale=2.0).to(cuda_device()), c, table, n)


def test_attention_peaked_and_growing_scores():
    """Scores that rise along the sequence by hundreds, and one token that outweighs all others."""
    c = make_cache(40, 1, 16, 128, "bf16", "bf16")
    table, n = tables([640], 16, 40)
    order = table[0].long()
    ramp = torch.linspace(-6, 6, 640, device=cuda_device()).to(torch.bfloat16)
    c.k[order, 0] = ramp.view(40, 16, 1).expand(40, 16, 128)
    q = torch.ones((1, 4, 128), dtype=torch.bfloat16, device=cuda_device())
    q[0, 1] = -1
    q[0, 2] = 0.01
    q[0, 3] = 0
    check_attention(q, c, table, n, scale=0.5)
    check_attention(q, c, table, n, scale=-0.5)
    check_attention(q, c, table, n, scale=0.0)


def test_attention_lowest_finite_scores():
    """Scores near the lowest that fp32 holds, all alike: the mean of the values."""
    c = make_cache(10, 1, 16, 64, "bf16", "bf16")
    table, n = tables([100], 16, 10)
    c.k.fill_(-1.0)
    q = torch.full((1, 2, 64), 2.0 ** 60, dtype=torch.bfloat16, device=cuda_device())
    out = ck.paged_attention(q, c, table, n, 2.0 ** 60)
    want, slack = ref.attention(q * 0, c.k, c.v, None, None, table, n, 1.0, 0, 0)
    ref.assert_within(out, want, slack, "mean")


@pytest.mark.parametrize("hidden", [16, 32, 304])
def test_attention_scores_of_minus_infinity(hidden):
    """Leading tokens whose score is -inf have no weight, be they a tile, a wave's share or whole
    chunks; a sequence of nothing else is 0 / 0."""
    c = make_cache(80, 1, 16, 128, "bf16", "bf16")
    table, n = tables([700, 500], 16, 80)
    c.k[table[0, :hidden // 16].long(), :, :, 0] = -float("inf")
    c.k[table[1, :32].long(), :, :, 0] = -float("inf")      # 500 tokens: the row's other entries are no pages
    q = rand(2, 4, 128, dtype=torch.bfloat16).to(cuda_device())
    q[:, :, 0] = 1
    out = ck.paged_attention(q, c, table, n)
    want, slack = ref.attention(q[:1], c.k, c.v, None, None, table[:1, hidden // 16:], n[:1] - hidden, 128 ** -0.5, 0, 0)
    ref.assert_within(out[:1], want, slack, "visible scores")
    assert out[1].isnan().all()


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16")])
def test_attention_weights_to_32_bits(cache, dtype):
    """Values that almost cancel, so that the output shows the weights' own precision.

    Tokens 0 and 2 have score 0 and the values -hi and -lo, token 1 the value 1 and the weight
    e = exp(score) with hi + lo = e to 14 bits or more: out = (e - hi - lo) / (2 + e).
    Allowed, in units of 2^-24 of (e + hi + |lo|) / (2 + e): 12 for the weight (three roundings of the
    score's change to base 2, at most 1 in magnitude, one of its offset from M, at most 8 in
    magnitude, the exponential's 2, a value scale's 3, its own to 32 bits), 8 for the products and
    sums, 4 for the division."""
    dev = cuda_device()
    hq, d, n = 16, 64, 8
    t = DT[dtype]
    score = -torch.linspace(0.02, 0.69, n * hq).to(t).view(n, hq)
    e = torch.exp(score.double())
    k, v = torch.zeros((n, 1, 4, d)), torch.zeros((n, 1, 4, d))
    k[:, 0, 1, 0] = 1
    ks = vs = None
    if cache == "int8":
        v[:, 0, 1], v[:, 0, 0, :hq] = 64, -torch.round(e * 128)
        v[:, 0, 2, :hq] = -torch.round((e + v[:, 0, 0, :hq].double() / 128) * 2 ** 14).float()
        vs = torch.tensor([2.0 ** -7, 2.0 ** -6, 2.0 ** -14, 0.0]).expand(n, 1, 4).contiguous()
        ks = torch.ones((n, 1, 4))
        parts = v[:, 0, :3].double() * vs[:, 0, :3, None].double()
        k, v = k.to(torch.int8), v.to(torch.int8)
    else:
        v[:, 0, 1], v[:, 0, 0, :hq] = 1, -e.to(t).float()
        v[:, 0, 2, :hq] = -(e - e.to(t).double()).to(t).float()
        parts = v[:, 0, :3].to(t).double()
        k, v = k.to(t), v.to(t)
    c = ck.KVCache(*(None if x is None else x.to(dev) for x in (k, v, ks, vs)))
    q = torch.zeros((n, hq, d), dtype=t)
    q[:, :, 0] = score
    table = torch.arange(n, dtype=torch.int32, device=dev)[:, None]
    lens = torch.full((n,), 3, dtype=torch.int32, device=dev)
    out = ck.paged_attention(q.to(dev), c, table, lens, 1.0)
    weight = torch.stack([torch.ones_like(e), e, torch.ones_like(e)], -1)
    want = weight @ parts / (2 + e[..., None])
    ref.assert_within(out, want, 24 * ref.U32 * (weight @ parts.abs()) / (2 + e[..., None]), "almost nothing")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("exponent", [-149, -140, -130, -127, -100, 0, 90])
def test_attention_value_scales_of_any_size(exponent, dtype):
    """An int8 cache whose value scales are subnormal, small or large, all of them finite."""
    c = make_cache(40, 2, 16, 128, "int8", dtype)
    c.v_scale.fill_(2.0 ** exponent)
    c.v.abs_()
    table, n = tables([500, 20], 16, 40)
    q = rand(2, 8, 128, dtype=DT[dtype]).to(cuda_device())
    if dtype == "fp16" and exponent > 9:
        assert ck.paged_attention(q, c, table, n).isinf().any()
    else:
        check_attention(q, c, table, n)


def check_light_tokens(cache, dtype):
    """600 tokens in several chunks.  Head h gives the first one a score `nats[h]` above all others',
    and its values are zero.  The others' values are large enough for what is left to be normal
    numbers of the output's type."""
    nats = torch.tensor([4.0, 8.0, 11.0, 14.0, 16.0, 16.75, 18.0, 18.5, 20.0, 22.0, 23.5, 24.0, 26.0, 28.0, 31.0, 35.0])
    dev = cuda_device()
    c = make_cache(40, 1, 16, 64, cache, dtype)
    table, n = tables([600, 30], 16, 40)
    for i in range(2):
        at = table[i, :-(-int(n[i]) // 16)].long()
        c.k[at, 0], c.k[at[0], 0, 0, 0] = 0, 1
        if cache == "int8":
            c.k_scale[at, 0] = 1.0
            c.v_scale[at, 0] *= 2.0 ** 12
        else:
            c.v[at, 0] *= 2.0 ** 12
        c.v[at, 0] = c.v[at, 0].abs()
        c.v[at[0], 0, 0] = 0
    q = torch.zeros((2, 16, 64), dtype=DT[dtype], device=dev)
    q[:, :, 0] = nats.to(dev)
    check_attention(q, c, table, n, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_int8_light_tokens_beside_a_heavy_one_without_value(dtype):
    """The first token outweighs all others and its values are zero: the output is the others', of
    weights down to 2^-51."""
    check_light_tokens("int8", dtype)


@pytest.mark.parametrize("spread", [16, 22, 26, 30, 40])
def test_attention_int8_value_scales_far_apart(spread):
    """One row's value scale is 2^spread (in the second sequence 2^(2 spread)) times the others' and
    its weight e^-40 or less: the others' mean is as exact as without it."""
    c = make_cache(40, 2, 16, 128, "int8", "fp16")
    table, n = tables([500, 100], 16, 40)
    heads = torch.arange(2, device=cuda_device())
    for i in range(2):
        page = table[i, 0].long()
        c.k[page, heads, 3], c.v[page, heads, 3] = 127, 127
        c.k_scale[page, heads, 3], c.v_scale[page, heads, 3] = 0.05, 2.0 ** spread * float(c.v_scale.max())
    q = rand(2, 8, 128, dtype=torch.float16).abs().to(cuda_device())
    check_attention(-q, c, table, n)


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16")])
def test_attention_light_tokens_beside_a_heavy_one_without_value(cache, dtype):
    """As for the int8 cache above."""
    check_light_tokens(cache, dtype)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_attention_bad_pages_of_a_split_sequence(cache):
    """A bad page in the first, a middle or the last chunk of a sequence in several chunks makes that
    sequence NaN whatever the workspace held, and no other."""
    lens = [3000, 3000, 3000, 3000, 40]
    pages = sum(-(-n // 16) for n in lens)
    c = make_cache(pages, 2, 16, 128, cache, "bf16")
    table, n = tables(lens, 16, pages)
    q = rand(5, 8, 128, dtype=torch.bfloat16).to(cuda_device())
    good = check_attention(q, c, table, n)
    bad = table.clone()
    bad[0, 0], bad[1, 90], bad[2, 187] = -1, pages, 1 << 30
    ws = ck.paged_attention_workspace(q, c, table)
    assert ws is not None
    for byte in (0, 127, 255):
        ws.fill_(byte)
        out = ck.paged_attention(q, c, bad, n, workspace=ws)
        assert out[:3].isnan().all()
        assert torch.equal(out[3:], good[3:])


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("width", [1, 300])
def test_attention_cache_without_pages(cache, width):
    """No page is inside a cache of none: NaN where a token is visible, zeros where none is."""
    dev = cuda_device()
    c = ck.KVCache.empty(0, 2, 16, 128, cache, dev)
    table = torch.zeros((3, width), dtype=torch.int32, device=dev)
    n = torch.tensor([5, 0, 16 * width], dtype=torch.int32, device=dev)
    out = ck.paged_attention(rand(3, 4, 128, dtype=torch.bfloat16).to(dev), c, table, n)
    assert out[0].isnan().all() and out[2].isnan().all() and (out[1] == 0).all()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16")])
def test_attention_every_head_dim(d, cache, dtype):
    """Each head_dim with each type of cache: a sequence of several chunks, one of a few tiles, one token."""
    lens = [3000, 70, 1]
    pages = sum(-(-n // 16) for n in lens)
    c = make_cache(pages, 2, 16, d, cache, dtype)
    table, n = tables(lens, 16, pages)
    poison(c, table, n)
    check_attention(rand(3, 10, d, dtype=DT[dtype], scale=2.0).to(cuda_device()), c, table, n)


def test_attention_bad_pages():
    """A visible page outside the cache makes that sequence NaN, and no other."""
    lens = [100, 100, 100, 100]
    c = make_cache(28, 2, 16, 128, "bf16", "bf16")
    table, n = tables(lens, 16, 28)
    q = rand(4, 4, 128, dtype=torch.bfloat16).to(cuda_device())
    good = check_attention(q, c, table, n)
    bad = table.clone()
    bad[1, 3] = -1
    bad[2, 6] = 28                       # tokens 96 .. 99
    out = ck.paged_attention(q, c, bad, n)
    assert out[1].isnan().all() and out[2].isnan().all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    out = ck.paged_attention(q, c, bad, n, window=4)         # tokens 96 .. 99 only
    assert out[2].isnan().all() and not out[1].isnan().any()
    c8 = make_cache(28, 2, 16, 128, "int8", "bf16")
    out = ck.paged_attention(q, c8, bad, n)
    assert out[1].isnan().all() and out[2].isnan().all() and not out[0].isnan().any()


def test_attention_lens_outside_the_table():
    c = make_cache(8, 1, 16, 128, "bf16", "bf16")
    table, _ = tables([32, 32, 32], 16, 8)
    q = rand(3, 2, 128, dtype=torch.bfloat16).to(cuda_device())
    n = torch.tensor([1000, -5, 32], dtype=torch.int32, device=cuda_device())
    out = check_attention(q, c, table, n)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_attention_strides(cache):
    """[page, head] inner layouts, strided q, out and table: the same bits as contiguous ones."""
    lens = [70, 9, 300]
    c = make_cache(40, 4, 16, 128, cache, "bf16", layout="nhd")
    flat = ck.KVCache(c.k.contiguous(), c.v.contiguous(), *(None if t is None else t.contiguous() for t in (c.k_scale, c.v_scale)))
    table, n = tables(lens, 16, 40)
    q = rand(3, 12, 128, dtype=torch.bfloat16).to(cuda_device())
    want = check_attention(q, flat, table, n)
    wide = torch.zeros((3, 20, 136), dtype=torch.bfloat16, device=q.device)[:, 3:15, :128]
    wide.copy_(q)
    t2 = torch.zeros((3, table.shape[1] + 5), dtype=torch.int32, device=q.device)[:, :table.shape[1]]
    t2.copy_(table)
    out = torch.zeros((3, 24, 128), dtype=torch.bfloat16, device=q.device)[:, ::2]
    got = ck.paged_attention(wide, c, t2, n, out=out)
    assert got is out and torch.equal(out, want)


def test_attention_far_pages():
    """Rows past 2^31 elements of the cache."""
    dev = cuda_device()
    pages = (1 << 31) // (64 * 128) + 4
    k, v = (torch.zeros((pages, 1, 64, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    k[-2:], v[-2:] = rand(2, 1, 64, 128, dtype=torch.bfloat16).to(dev), rand(2, 1, 64, 128, dtype=torch.bfloat16, seed=4).to(dev)
    c = ck.KVCache(k, v)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=dev)
    n = torch.tensor([100], dtype=torch.int32, device=dev)
    q = rand(1, 4, 128, dtype=torch.bfloat16).to(dev)
    out = ck.paged_attention(q, c, table, n)
    small = ck.KVCache(k[-2:].contiguous(), v[-2:].contiguous())
    want, slack = ref.attention(q, small.k, small.v, None, None, table - (pages - 2), n, 128 ** -0.5, 0, 0)
    ref.assert_within(out, want, slack, "far pages")


def test_attention_same_bits_each_call_and_dirty_workspace():
    lens = [3000, 100, 0]
    c = make_cache(220, 2, 16, 128, "int8", "bf16")
    table, n = tables(lens, 16, 220)
    q = rand(3, 16, 128, dtype=torch.bfloat16).to(cuda_device())
    ws = ck.paged_attention_workspace(q, c, table)
    want = check_attention(q, c, table, n)
    for byte in (0, 255):
        if ws is not None:
            ws.fill_(byte)
        for _ in range(3):
            assert torch.equal(ck.paged_attention(q, c, table, n, workspace=ws), want)


def test_decode_on_a_side_stream_and_in_a_graph():
    """All three operators captured into one graph, replayed over changed
    inputs with eager calls between, each replay against the eager result."""
    dev = cuda_device()
    q, k, v, qw, kw, pos, table = rope_inputs(4, 8, 2, 128, 128, "bf16", 500)
    lens = [90, 33, 1, 700]
    c = make_cache(60, 2, 16, 128, "bf16", "bf16")
    pt, n = tables(lens, 16, 60)
    slots = torch.stack([pt[i, (x - 1) // 16].long() * 16 + (x - 1) % 16 for i, x in enumerate(lens)])
    codes = torch.randint(0, 256, (200, 512), dtype=torch.uint8, device=dev)
    w = ck.int4_pack(codes, (rand(200, 8).abs() * 0.01).to(torch.bfloat16).to(dev), group=128)
    ws = ck.paged_attention_workspace(q, c, pt)

    def step():
        qo, _ = ck.qk_norm_rope(q, k, v, pos, table, qw, kw, cache=c, slots=slots)
        o = ck.paged_attention(qo, c, pt, n, workspace=ws)
        return ck.int4_linear(o.view(4, 1024), w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(first, step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        q.copy_(rand(4, 8, 128, dtype=torch.bfloat16, seed=50 + i))
        v.copy_(rand(4, 2, 128, dtype=torch.bfloat16, seed=60 + i))
        want = step().clone()
        torch.cuda.synchronize()
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i


# -------------------------------------------------------------- int4_linear

def int4_inputs(m, n, k, group, zeros, bias, dtype, out_dtype=None, seed=2):
    dev = cuda_device()
    g = torch.Generator().manual_seed(seed + m + n + k)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).to(dev)
    groups = -(-k // group)
    scales = (0.02 * (0.5 + torch.rand((n, groups), generator=g))).to(DT[dtype]).to(dev)
    z = torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8).to(dev) if zeros else None
    b = rand(n, dtype=DT[out_dtype or dtype], seed=seed).to(dev) if bias else None
    return rand(m, k, dtype=DT[dtype], seed=seed).to(dev), codes, scales, z, b


@pytest.mark.parametrize("m,n,k,group,zeros,bias,dtype,out", [
    (1, 64, 128, 128, False, False, "bf16", None),
    (1, 4096, 4096, 128, False, False, "bf16", None),
    (1, 1000, 2048, 32, True, True, "fp16", None),
    (2, 17, 136, 32, True, False, "bf16", "fp32"),
    (3, 1, 8, 64, True, True, "bf16", None),
    (5, 33, 1000, 128, True, True, "fp16", "fp32"),
    (8, 300, 5376, 64, False, True, "bf16", "fp16"),
    (15, 257, 4104, 128, True, False, "bf16", None),
    (16, 512, 2048, 32, False, False, "fp16", "bf16"),
    (17, 272, 2056, 64, True, True, "bf16", None),
    (33, 1040, 1024, 128, False, True, "fp16", None),
    (64, 160, 5376, 32, True, True, "bf16", None),
    (65, 100, 640, 64, True, False, "bf16", "fp32"),
    (128, 528, 1928, 128, True, True, "bf16", None),
    (200, 48, 384, 32, False, False, "fp16", None),
    (513, 80, 256, 128, True, True, "bf16", None),
])
def test_int4(m, n, k, group, zeros, bias, dtype, out):
    x, codes, scales, z, b = int4_inputs(m, n, k, group, zeros, bias, dtype, out)
    w = ck.int4_pack(codes, scales, z, group=group)
    got = ck.int4_linear(x, w, b, out_dtype=out)
    assert got.dtype == DT[out or dtype]
    want, slack = ref.int4(x, codes, scales, z, b, group)
    ref.assert_within(got, want, slack, "int4_linear")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 16, 40, 130])
def test_int4_exact_on_whole_numbers(m, group):
    """Small whole x and scales of powers of two: every sum is exact in fp32, and so is the output."""
    dev = cuda_device()
    n, k = 70, 1000
    _, codes, scales, z, _ = int4_inputs(m, n, k, group, True, False, "bf16")
    g = torch.Generator().manual_seed(m)
    x = torch.randint(-3, 4, (m, k), generator=g).to(torch.bfloat16).to(dev)
    scales = (2.0 ** torch.randint(-2, 2, scales.shape, generator=g)).to(torch.bfloat16).to(dev)
    got = ck.int4_linear(x, ck.int4_pack(codes, scales, z, group=group), out_dtype="fp32")
    want, _ = ref.int4(x, codes, scales, z, None, group)
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [
    (1, 20501, 392), (7, 20501, 392), (16, 24001, 264), (3, 9007, 520), (6, 9007, 520), (16, 9007, 520),
    (21, 8230, 392), (21, 17003, 264), (37, 9007, 136), (37, 8230, 392), (70, 9007, 136), (70, 8230, 648),
    (70, 20501, 264), (130, 17003, 264),
])
def test_int4_exact_for_every_block_shape(m, n, k, group, zeros):
    """Wide outputs, where blocks of each shape are chosen: whole numbers, as above."""
    dev = cuda_device()
    _, codes, scales, z, _ = int4_inputs(m, n, k, group, zeros, False, "fp16")
    g = torch.Generator().manual_seed(m + n)
    x = torch.randint(-3, 4, (m, k), generator=g).to(torch.float16).to(dev)
    scales = (2.0 ** torch.randint(-2, 2, scales.shape, generator=g)).to(torch.float16).to(dev)
    got = ck.int4_linear(x, ck.int4_pack(codes, scales, z, group=group), out_dtype="fp32")
    want, _ = ref.int4(x, codes, scales, z, None, group)
    assert torch.equal(got.cpu().double(), want)


def test_int4_pack_layout():
    """The layout that include/ck_int8.h gives, word by word."""
    n, k, group = 37, 200, 64
    _, codes, scales, z, _ = int4_inputs(1, n, k, group, True, False, "fp16")
    w = ck.int4_pack(codes, scales, z, group=group)
    full = torch.zeros((48, 256), dtype=torch.int64)
    full[:n, :k] = ref.unpack_codes(codes).long()
    got = w.w.cpu().view(torch.int32).long().view(3, 2, 64, 4) & 0xffffffff
    lane = torch.arange(64)
    for e, at in enumerate((0, 4, 1, 5, 2, 6, 3, 7)):        # column e of a word is nibble `at`
        nib = (got >> (4 * at)) & 15
        for i in range(4):
            cols = 32 * i + 8 * (lane // 16) + e
            for t in range(3):
                for c in range(2):
                    assert torch.equal(nib[t, c, :, i], full[16 * t + lane % 16, 128 * c + cols])
    groups = -(-k // group)
    ws, wz = torch.zeros((48, groups)), torch.zeros((48, groups), dtype=torch.uint8)
    ws[:n], wz[:n] = scales.cpu().float(), z.cpu()
    assert torch.equal(w.scales.cpu().float(), ws.view(3, 16, groups).transpose(1, 2))
    assert torch.equal(w.zeros.cpu(), wz.view(3, 16, groups).transpose(1, 2))


def test_int4_strides_and_empty():
    """Rows of x and out further apart, strided codes and scales; no rows; no columns of K."""
    dev = cuda_device()
    x, codes, scales, z, b = int4_inputs(9, 50, 264, 32, True, True, "bf16")
    want = ck.int4_linear(x, ck.int4_pack(codes, scales, z, group=32), b)
    wx = torch.full((9, 320), float("nan"), dtype=torch.bfloat16, device=dev)[:, 16:280]
    wx.copy_(x)
    out = torch.full((9, 61), 7.0, dtype=torch.bfloat16, device=dev)
    wide = [torch.zeros((t.shape[0], t.shape[1] + 5), dtype=t.dtype, device=dev)[:, :t.shape[1]] for t in (codes, scales, z)]
    for a, t in zip(wide, (codes, scales, z)):
        a.copy_(t)
    ck.int4_linear(wx, ck.int4_pack(*wide, group=32), b, out=out[:, 3:53])
    assert torch.equal(out[:, 3:53], want)
    assert (out[:, :3] == 7).all() and (out[:, 53:] == 7).all()
    w = ck.int4_pack(codes, scales, z, group=32)
    assert ck.int4_linear(x[:0], w).shape == (0, 50)
    empty = ck.int4_pack(codes[:, :0], scales[:, :0], group=32)
    got = ck.int4_linear(x[:, :0], empty, b)
    assert torch.equal(got, b.expand(9, 50))


def test_int4_same_bits_each_call():
    x, codes, scales, z, b = int4_inputs(24, 2000, 4096, 64, True, True, "bf16")
    w = ck.int4_pack(codes, scales, z, group=64)
    want = ck.int4_linear(x, w, b)
    for _ in range(3):
        assert torch.equal(ck.int4_linear(x, w, b), want)


def test_int4_row_results_do_not_depend_on_the_batch_tile():
    """The rows of a batch within one row tile give the bits that they give on the same kernel in another order."""
    x, codes, scales, z, b = int4_inputs(16, 300, 1024, 128, True, True, "bf16")
    w = ck.int4_pack(codes, scales, z, group=128)
    order = torch.randperm(16, generator=torch.Generator().manual_seed(1)).to(x.device)
    assert torch.equal(ck.int4_linear(x[order].contiguous(), w, b), ck.int4_linear(x, w, b)[order])


# -------------------------------------------------------------- all together

@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_example_block_against_its_parts(cache):
    """examples/decode_attention.py's block, prompt and two decode steps:
    its output is that of plain 64-bit forms on the operators' own inputs."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from decode_attention import AttentionBlock
    dev = cuda_device()
    hidden, page, prompt = 512, 8, 43
    block = AttentionBlock(hidden, 8, 2, 64, 20, page, cache, rows=256, device=dev)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(2)).int().view(2, 10).to(dev)
    at = torch.arange(prompt, device=dev)
    for b in range(2):
        x = rand(prompt, hidden, dtype=torch.bfloat16, seed=b).to(dev)
        assert block(x, at, table[b].long()[at // page] * page + at % page) is None
    pos = torch.full((2,), prompt, device=dev)
    for step in range(2):
        x = rand(2, hidden, dtype=torch.bfloat16, seed=10 + step).to(dev)
        slots = table.long().gather(1, (pos // page)[:, None])[:, 0] * page + pos % page
        lens = (pos + 1).int()
        y = block(x, pos, slots, table, lens)
        qkv = ck.int8_linear(x, block.w_qkv, block.s_qkv)
        q = ck.qk_norm_rope(qkv[:, :512].view(2, 8, 64), None, None, pos, block.table, block.q_norm)[0]
        want_q, slack_q = ref.rope(qkv[:, :512].view(2, 8, 64), block.q_norm, block.table, pos, 64, False, 1e-6)
        ref.assert_within(q, want_q, slack_q, "q")
        c = block.cache
        o = check_attention(q, c, table, lens)
        w = block.w_out
        got = ck.int4_linear(o.view(2, 512), w)
        assert torch.equal(got, y)
        # the newest row of the cache is this step's value
        v = qkv[:, 640:].view(2, 2, 64).float()
        row = c.v[slots // page, :, slots % page].float()
        if cache == "int8":
            row = row * c.v_scale[slots // page, :, slots % page][..., None]
            assert ((row - v).abs() <= v.abs().amax(-1, keepdim=True) / 127).all()
        else:
            assert torch.equal(row, v)
        pos += 1
