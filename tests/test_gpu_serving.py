"""The operators of a server's batch on the GPU against plain references in 64
bits: shared_prefix_attention, lora_add and token_logprobs."""
import math

import pytest
import torch

import int8_weight_quantized_amd as ck
from tests import serving_ref as ref
from tests.gpu_util import cuda_device
from tests.test_gpu_decode import make_cache, rand

pytestmark = pytest.mark.gpu
DT = ref.TYPES


# ---------------------------------------------------- shared_prefix_attention

def prefix_inputs(prefix, starts, lens, hq, hk, d, dtype, cache, page, layout="hnd", seed=3):
    """A cache, tables whose unused entries are far outside of it, and queries; rows that nobody sees are NaN."""
    dev = cuda_device()
    every = list(prefix) + list(lens)
    pages = sum(-(-n // page) for n in every) + 1
    c = make_cache(pages, hk, page, d, cache, dtype, layout)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    seen = torch.zeros((pages, page), dtype=torch.bool)
    at, tables = 0, []
    for group in (prefix, lens):
        t = torch.full((len(group), max([1] + [-(-n // page) for n in group])), 1 << 30, dtype=torch.int32)
        for i, n in enumerate(group):
            k = -(-n // page)
            t[i, :k] = order[at:at + k]
            tok = torch.arange(n)
            seen[t[i].long()[tok // page], tok % page] = True
            at += k
        tables.append(t.to(dev))
    hide = ~seen.to(dev)[:, None, :].expand(-1, hk, -1)
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        t[hide] = 127 if s is not None else float("nan")
        if s is not None:
            s[hide] = float("nan")
    q = rand(len(lens), hq, d, dtype=DT[dtype], scale=2.0).to(dev)
    i32 = [torch.tensor(v, dtype=torch.int32, device=dev) for v in (prefix, starts, lens)]
    return q, c, tables[0], i32[0], i32[1], tables[1], i32[2]


def check_prefix(q, c, pt, pl, starts, table, lens, scale=None, **kw):
    out = ck.shared_prefix_attention(q, c, pt, pl, starts, table, lens, scale, **kw)
    want, slack = ref.shared_prefix(q, c, pt, pl, starts, table, lens, q.shape[2] ** -0.5 if scale is None else scale)
    ref.assert_within(out, want, slack, "shared_prefix_attention")
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
    (20, 2, 256, "bf16", "bf16", 4),
])
def test_prefix_lengths(hq, hk, d, dtype, cache, page):
    """Prefixes and sequences of lengths about the borders of pages and tiles, 0 and 1 among them; groups of
    no, one and several sequences, and sequences without a prefix at both ends."""
    prefix = [0, 1, 31, 33, 64, 129, 300, 700]
    lens = [5, 0, 1, 31, 32, 33, 0, 1, 63, 64, 65, 17, 16, 15, 127, 129, 300, 2, 0, 40]
    starts = [1, 3, 4, 6, 6, 9, 10, 16, 18]
    check_prefix(*prefix_inputs(prefix, starts, lens, hq, hk, d, dtype, cache, page))


@pytest.mark.parametrize("members", [1, 2, 4, 5, 8, 15, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "int8")])
def test_prefix_group_sizes(members, dtype, cache):
    """Groups of one to many sequences: rows of queries about the borders of the row tiles."""
    lens = [1 + i % 7 for i in range(members)]
    check_prefix(*prefix_inputs([517], [0, members], lens, 8, 2, 128, dtype, cache, 16))


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16")])
def test_prefix_every_head_dim(d, cache, dtype):
    """Each head_dim with each type of cache: a long prefix of several chunks, a large and a small group."""
    lens = [300, 1, 40] + [9] * 22
    check_prefix(*prefix_inputs([2900, 1100], [0, 2, 25], lens, 10, 2, d, dtype, cache, 16))


def test_prefix_long():
    """A long prefix, many splits; and a table far wider than any length."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([20000, 37], [0, 6, 8], [10, 700, 1, 3, 50, 9, 1, 2000], 8, 2, 128,
                                                      "bf16", "bf16", 64)
    want = check_prefix(q, c, pt, pl, starts, table, lens)
    wide = torch.full((2, 4000), -7, dtype=torch.int32, device=q.device)
    wide[:, :pt.shape[1]] = pt
    got = check_prefix(q, c, wide, pl, starts, table, lens)
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -6, atol=2.0 ** -10)


def test_prefix_is_paged_attention_over_the_whole():
    """The same tokens in a page table of each sequence's own give the same values (a bf16 step apart)."""
    page, dev = 16, cuda_device()
    q, c, pt, pl, starts, table, lens = prefix_inputs([320], [0, 9], [3 + 20 * i for i in range(9)], 8, 2, 128, "bf16",
                                                      "bf16", page)
    whole = torch.cat([pt.expand(9, -1), table], 1).contiguous()
    a = ck.shared_prefix_attention(q, c, pt, pl, starts, table, lens).float()
    b = ck.paged_attention(q, c, whole, lens + 320).float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-5).all()
    # and without any prefix
    none = torch.zeros((0, 0), dtype=torch.int32, device=dev)
    got = check_prefix(q, c, none, pl[:0], starts[:1], table, lens)
    b = ck.paged_attention(q, c, table, lens).float()
    assert ((got.float() - b).abs() <= 2.0 ** -7 * b.abs() + 1e-5).all()


def test_prefix_starts_that_are_wrong():
    """Entries that decrease, are negative or past the batch: every output is NaN, and nothing outside is read."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([50, 60], [0, 3, 5], [4] * 6, 4, 2, 64, "bf16", "bf16", 16)
    for bad in ([-1, 3, 5], [3, 2, 5], [0, 3, 7], [0, 1 << 30, 5], [5, 3, 0], [-(1 << 31), 0, (1 << 31) - 1]):
        out = ck.shared_prefix_attention(q, c, pt, pl, torch.tensor(bad, dtype=torch.int32, device=q.device), table, lens)
        assert out.isnan().all(), bad
    for fine in ([0, 0, 0], [6, 6, 6], [2, 2, 4]):
        check_prefix(q, c, pt, pl, torch.tensor(fine, dtype=torch.int32, device=q.device), table, lens)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("members", [2, 20])
def test_prefix_bad_pages(cache, members):
    """A bad page of a prefix makes its group NaN, one of a sequence that sequence, whatever the workspace held."""
    n = 2 * members
    q, c, pt, pl, starts, table, lens = prefix_inputs([2100, 2100], [0, members, n], [40] * n, 8, 2, 128, "bf16", cache, 16)
    good = check_prefix(q, c, pt, pl, starts, table, lens)
    ws = ck.shared_prefix_attention_workspace(q, c, pt, table)
    for where in (0, 70, 131):
        for byte in (0, 127, 255):
            if ws is not None:
                ws.fill_(byte)
            bad = pt.clone()
            bad[0, where] = (-1, c.pages, 1 << 30)[where % 3]
            out = ck.shared_prefix_attention(q, c, bad, pl, starts, table, lens, workspace=ws)
            assert out[:members].isnan().all()
            assert torch.equal(out[members:], good[members:])
    bad = table.clone()
    bad[1, 2] = c.pages
    out = ck.shared_prefix_attention(q, c, pt, pl, starts, bad, lens, workspace=ws)
    keep = [i for i in range(n) if i != 1]
    assert out[1].isnan().all() and torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_prefix_cache_without_pages_and_lens_outside(cache):
    dev = cuda_device()
    c = ck.KVCache.empty(0, 2, 16, 128, cache, dev)
    q = rand(3, 4, 128, dtype=torch.bfloat16).to(dev)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    t = torch.zeros((3, 2), dtype=torch.int32, device=dev)
    out = ck.shared_prefix_attention(q, c, t[:1], i32(5), i32(0, 1), t, i32(0, 0, 3))
    assert out[0].isnan().all() and (out[1] == 0).all() and out[2].isnan().all()
    q, c, pt, pl, starts, table, lens = prefix_inputs([32, 32], [0, 2, 3], [32, 32, 32], 4, 2, 64, "bf16", cache, 16)
    check_prefix(q, c, pt, i32(1000, -5), starts, table, i32(-3, 1 << 30, 7))


def test_prefix_lowest_lengths():
    """The lowest int32 as a length is 0 for every chunk, of a prefix and of a sequence."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([3000, 3000], [0, 20, 22], [2000] * 24, 8, 2, 128, "bf16", "bf16", 16)
    low = -(1 << 31)
    for i in (0, 20, 23):
        few = lens.clone()
        few[i] = low
        check_prefix(q[[i]], c, pt, pl, starts.clamp(0, 0), table[[i]], few[[i]])
    check_prefix(q, c, pt, torch.tensor([low, 3000], dtype=torch.int32, device=q.device), starts, table, lens)
    few = torch.full_like(lens, low)
    none = ck.shared_prefix_attention(q, c, pt, torch.full_like(pl, low), starts, table, few)
    assert (none == 0).all()


@pytest.mark.parametrize("prefixes,sequences", [(70, 200), (300, 90), (65, 64)])
def test_prefix_many(prefixes, sequences):
    """More prefixes than a wave has lanes, groups of none to many sequences."""
    g = torch.Generator().manual_seed(prefixes)
    starts = torch.sort(torch.randint(0, sequences + 1, (prefixes + 1,), generator=g)).values.tolist()
    prefix = torch.randint(0, 150, (prefixes,), generator=g).tolist()
    lens = torch.randint(0, 40, (sequences,), generator=g).tolist()
    check_prefix(*prefix_inputs(prefix, starts, lens, 12, 2, 64, "bf16", "bf16", 16))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16")])
def test_prefix_blocks_with_several_chunks(d, cache, dtype):
    """So many sequences and prefixes that a block goes through several chunks of a long one, of both kinds; a bad
    page in one of them makes what sees it NaN and nothing else."""
    prefix = [2500 if i in (3, 40) else 1025 if i == 63 else i % 70 for i in range(64)]
    lens = [1700 if i in (5, 66) else 513 if i == 6 else 1 + i % 40 for i in range(70)]
    starts = [2 + i for i in range(65)]
    q, c, pt, pl, starts, table, lens = prefix_inputs(prefix, starts, lens, 16, 8, d, dtype, cache, 16)
    good = check_prefix(q, c, pt, pl, starts, table, lens)
    for where, who in ((10, 5), (75, 5), (100, 42)):         # of table, table and pt
        bad, one = table.clone(), pt.clone()
        (one if where == 100 else bad)[40 if where == 100 else who, where] = c.pages
        out = ck.shared_prefix_attention(q, c, one, pl, starts, bad, lens)
        keep = [i for i in range(70) if i != who]
        assert out[who].isnan().all() and torch.equal(out[keep], good[keep])


def test_prefix_wide_tables_give_the_same_bits():
    """Tables far wider than any length, in which as many blocks share a list: the same bits."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([1000, 300], [0, 20, 30], [700 - 20 * i for i in range(33)], 8, 8, 64,
                                                      "bf16", "bf16", 16)
    got = []
    for more in (2000, 3000):
        wide = [torch.full((len(t), more), -7, dtype=torch.int32, device=q.device) for t in (pt, table)]
        for w, t in zip(wide, (pt, table)):
            w[:, :t.shape[1]] = t
        got.append(check_prefix(q, c, wide[0], pl, starts, wide[1], lens))
    assert torch.equal(*got)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("members", [17, 66])
def test_prefix_long_chunks(cache, members):
    """So many heads that a block goes through well over 1024 tokens; of an int8 cache scales that rise and fall by
    powers of two along the way; a bad page late in such a chunk."""
    hk, n = 256, 3000
    q, c, pt, pl, starts, table, lens = prefix_inputs([n], [0, members], [3] * members, hk, hk, 64, "bf16", cache, 8)
    pick = [0, 100, 255]
    steps = [[0] * 6] if cache == "bf16" else [[0, 12, -12, 5, 20, 3], [20, 3, -20, -40, 8, 0], [-40, -41, -30, -30, -28, -10]]
    for ups in steps:
        if cache == "int8":
            vs = c.v_scale.clone()
            for i, up in enumerate(ups):
                at = pt[0, i * 64:(i + 1) * 64].long()
                vs[at] *= 2.0 ** up
            now = ck.KVCache(c.k, c.v, c.k_scale, vs)
            some = ck.KVCache(*(t[:, pick].contiguous() for t in (c.k, c.v, c.k_scale, vs)))
        else:
            now, some = c, ck.KVCache(c.k[:, pick].contiguous(), c.v[:, pick].contiguous())
        out = ck.shared_prefix_attention(q, now, pt, pl, starts, table, lens)
        want, slack = ref.shared_prefix(q[:, pick], some, pt, pl, starts, table, lens, 64 ** -0.5)
        ref.assert_within(out[:, pick], want, slack, str(ups))
    for where in (150, 190, 374):
        bad = pt.clone()
        bad[0, where] = -1
        assert ck.shared_prefix_attention(q, c, bad, pl, starts, table, lens).isnan().all()


def test_prefix_scores_of_minus_infinity_and_large_ones():
    """Tokens of the prefix whose score is -inf have no weight; scores that differ by hundreds; one token that
    outweighs all others, in the prefix or in the sequence."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([1500], [0, 20], [33] * 20, 8, 1, 128, "bf16", "bf16", 16)
    q[:, :, 0] = 1
    hidden = c.k.clone()
    hidden[pt[0, :40].long(), :, :, 0] = -float("inf")
    check_prefix(q, ck.KVCache(hidden, c.v), pt, pl, starts, table, lens)
    for where in (pt[0, 50], table[3, 1]):
        heavy = c.k.clone()
        heavy[where.long(), 0, 0] = 40 * q[3, 2]
        check_prefix(q, ck.KVCache(heavy, c.v), pt, pl, starts, table, lens, scale=0.5)
    check_prefix(q, c, pt, pl, starts, table, lens, scale=0.0)
    check_prefix(q, c, pt, pl, starts, table, lens, scale=-1.0)


@pytest.mark.parametrize("members", [2, 20])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16")])
def test_prefix_light_tokens_beside_a_heavy_one_without_value(members, cache, dtype):
    """A heavy token whose value is zero leaves the light ones' mean, however light they are."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([600], [0, members], [20] * members, 4, 1, 128, dtype, cache, 16)
    heavy = pt[0, 7].long()
    for up in (8.0, 16.0, 22.0, 30.0):
        if cache == "int8":
            c.k.fill_(0)
            c.k[heavy, 0, 5, 0] = 127
            c.k_scale.fill_(1.0 / 127)
            c.v[heavy, 0, 5] = 0
        else:
            c.k.fill_(0)
            c.k[heavy, 0, 5, 0] = 1
            c.v[heavy, 0, 5] = 0
        q.fill_(0)
        q[:, :, 0] = up
        out = ck.shared_prefix_attention(q, c, pt, pl, starts, table, lens, math.log(2.0))
        want, _ = ref.shared_prefix(q, c, pt, pl, starts, table, lens, math.log(2.0))
        # relative to the light tokens' own values: the bound of the weights' parts, not of the largest weight; and
        # half a step of the output's type where it is subnormal (fp16 at 2^-30)
        got = out.double().cpu()
        big = want.abs().amax()
        tol = (ref.HALF[DT[dtype]] * 2 + 2.0 ** -9) * want.abs() + 2.0 ** -9 * big + ref.TINY[DT[dtype]]
        assert ((got - want).abs() <= tol).all(), up


def test_prefix_strides():
    """[page, head] inner layouts, strided q, out and tables: the same bits as contiguous ones."""
    q, c, pt, pl, starts, table, lens = prefix_inputs([300, 70], [1, 4, 9], [20] * 9, 12, 4, 128, "bf16", "int8", 16, "nhd")
    flat = ck.KVCache(*(t.contiguous() for t in (c.k, c.v, c.k_scale, c.v_scale)))
    want = check_prefix(q, flat, pt, pl, starts, table, lens)
    wide = torch.zeros((9, 20, 136), dtype=torch.bfloat16, device=q.device)[:, 3:15, :128]
    wide.copy_(q)
    t2, pt2 = (torch.zeros((t.shape[0], t.shape[1] + 5), dtype=torch.int32, device=q.device)[:, :t.shape[1]] for t in (table, pt))
    t2.copy_(table)
    pt2.copy_(pt)
    out = torch.zeros((9, 24, 128), dtype=torch.bfloat16, device=q.device)
    got = ck.shared_prefix_attention(wide, c, pt2, pl, starts, t2, lens, out=out[:, ::2])
    assert torch.equal(got, want) and (out[:, 1::2] == 0).all()


def test_prefix_far_pages():
    """Rows past 2^31 elements of the cache."""
    dev = cuda_device()
    pages = (1 << 31) // (64 * 128) + 4
    k, v = (torch.zeros((pages, 1, 64, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    k[-3:], v[-3:] = rand(3, 1, 64, 128, dtype=torch.bfloat16).to(dev), rand(3, 1, 64, 128, dtype=torch.bfloat16, seed=4).to(dev)
    c, small = ck.KVCache(k, v), ck.KVCache(k[-3:].contiguous(), v[-3:].contiguous())
    i32 = lambda *s: torch.tensor(s, dtype=torch.int32, device=dev)  # noqa: E731
    q = rand(30, 4, 128, dtype=torch.bfloat16).to(dev)
    pt, table = i32([2, 0]), i32([1]).expand(30, 1).contiguous()
    lens = i32(*[1 + i for i in range(30)])
    out = ck.shared_prefix_attention(q, c, pt + (pages - 3), i32(100), i32(0, 30), table + (pages - 3), lens)
    want, slack = ref.shared_prefix(q, small, pt, i32(100), i32(0, 30), table, lens, 128 ** -0.5)
    ref.assert_within(out, want, slack, "far pages")


def test_prefix_same_bits_each_call_and_dirty_workspace():
    a = prefix_inputs([3000, 90], [0, 20, 23], [400] + [60] * 23, 16, 2, 128, "bf16", "int8", 16)
    ws = ck.shared_prefix_attention_workspace(a[0], a[1], a[2], a[5])
    want = check_prefix(*a)
    for byte in (0, 255):
        if ws is not None:
            ws.fill_(byte)
        for _ in range(3):
            assert torch.equal(ck.shared_prefix_attention(*a, workspace=ws), want)


# -------------------------------------------------------------------- lora_add

def lora_inputs(m, n, k, rank, adapters, dtype, out, ids=None, scale=True, seed=5):
    dev = cuda_device()
    y = rand(m, n, dtype=DT[out], seed=seed).to(dev)
    x = rand(m, k, dtype=DT[dtype], seed=seed + 1).to(dev)
    a = (rand(adapters, rank, k, seed=seed + 2) * max(k, 1) ** -0.5).to(DT[dtype]).to(dev)
    b = (rand(adapters, n, rank, seed=seed + 3) * rank ** -0.5).to(DT[dtype]).to(dev)
    s = (0.5 + rand(adapters, seed=seed + 4).abs()).to(dev) if scale else None
    if ids is None:
        ids = torch.randint(-1, adapters, (m,), generator=torch.Generator().manual_seed(seed))
    return y, x, ck.LoraWeight(a, b, s), torch.as_tensor(ids, dtype=torch.int32).to(dev)


def check_lora(y, x, w, ids, **kw):
    had = y.clone()
    got = ck.lora_add(y, x, w, ids, **kw)
    want, slack = ref.lora(had, x, w.a, w.b, w.scale, ids)
    ref.assert_within(got, want, slack, "lora_add")
    off = (ids < 0) | (ids >= w.adapters)
    assert torch.equal(got[off], had[off])
    if kw.get("out") is not y:
        assert torch.equal(y, had)
    return got


@pytest.mark.parametrize("m,n,k,rank,adapters,dtype,out", [
    (1, 64, 64, 8, 1, "bf16", "bf16"),
    (1, 4096, 4096, 16, 8, "bf16", "bf16"),
    (1, 1, 8, 8, 1, "fp16", "fp16"),
    (2, 129, 520, 24, 3, "fp16", "fp32"),
    (15, 1000, 1032, 16, 40, "bf16", "fp32"),
    (16, 333, 264, 32, 2, "fp16", "fp16"),
    (17, 2050, 4096, 64, 5, "bf16", "bf16"),
    (33, 511, 128, 40, 7, "fp16", "bf16"),
    (61, 1024, 2056, 16, 48, "fp16", "fp16"),
    (64, 77, 96, 256, 3, "bf16", "bf16"),
    (65, 640, 1000, 128, 4, "bf16", "fp32"),
    (130, 300, 776, 8, 3, "fp16", "fp16"),
    (300, 700, 512, 16, 6, "bf16", "bf16"),
    (1030, 257, 136, 72, 9, "fp16", "fp32"),
    (600, 200, 264, 256, 5, "bf16", "bf16"),
    (513, 130, 136, 136, 70, "fp16", "fp16"),
    (512, 64, 72, 104, 100, "bf16", "fp32"),
])
def test_lora(m, n, k, rank, adapters, dtype, out):
    check_lora(*lora_inputs(m, n, k, rank, adapters, dtype, out))


@pytest.mark.parametrize("rank", range(8, 257, 8))
def test_lora_every_rank(rank):
    check_lora(*lora_inputs(19, 100, 200, rank, 3, "bf16", "fp32"))
    check_lora(*lora_inputs(150, 100, 200, rank, 3, "fp16", "fp16"))


@pytest.mark.parametrize("m", [1, 16, 40, 64, 65, 200, 515])
@pytest.mark.parametrize("kind", ["one", "runs", "none", "alternating", "outside"])
def test_lora_orders_of_ids(m, kind):
    """One adapter for all, prompts behind each other, no adapter at all, every second row, numbers outside."""
    at = torch.arange(m)
    ids = {"one": torch.full((m,), 2), "runs": at * 4 // m, "none": torch.full((m,), -1), "alternating": at % 2 * 3 - at % 3 // 2,
           "outside": torch.tensor([0, 4, -1, 1, 1 << 30, -(1 << 31), 3])[at % 7]}[kind]
    y, x, w, ids = lora_inputs(m, 330, 264, 16, 4, "bf16", "bf16", ids)
    got = check_lora(y, x, w, ids)
    assert check_lora(y, x, w, ids, out=y) is y and torch.equal(got, y)


@pytest.mark.parametrize("m", [1, 7, 100])
def test_lora_exact_on_whole_numbers(m):
    """Small whole numbers: every product and sum is exact, so is the result."""
    dev = cuda_device()
    g = torch.Generator().manual_seed(m)
    pick = lambda *s: torch.randint(-2, 3, s, generator=g).float()  # noqa: E731
    x, a, b, y = pick(m, 136), pick(3, 24, 136), pick(3, 90, 24), pick(m, 90)
    ids = torch.randint(-1, 3, (m,), generator=g)
    scale = torch.tensor([1.0, 2.0, 0.5])
    want = y.clone()
    for i, t in enumerate(ids.tolist()):
        if t >= 0:
            want[i] += scale[t] * (x[i] @ a[t].t() @ b[t].t())
    for dt in (torch.bfloat16, torch.float16):
        w = ck.LoraWeight(a.to(dt).to(dev), b.to(dt).to(dev), scale.to(dev))
        got = ck.lora_add(y.to(dev), x.to(dt).to(dev), w, ids.int().to(dev))
        assert torch.equal(got.cpu(), want)


def test_lora_small_and_large_values():
    """v far from one: the parts that it enters the second product in keep its precision and range."""
    for dtype, sizes in (("bf16", (2.0 ** -60, 2.0 ** -20, 2.0 ** 40)), ("fp16", (2.0 ** -14, 2.0 ** -8, 2.0 ** 8))):
        for m in (3, 90):
            for size in sizes:
                y, x, w, ids = lora_inputs(m, 200, 256, 16, 3, dtype, "fp32")
                check_lora(y * 0, (x.float() * size).to(x.dtype), w, ids)
    # rows of one tile, and ranks of one row, that lie far apart
    y, x, w, ids = lora_inputs(32, 64, 128, 16, 2, "fp16", "fp32", scale=False)
    x[::2] *= 2.0 ** -10
    w.a[:, ::2] *= 2.0 ** -10
    w.b[:, :, 1::2] = 0
    check_lora(y * 0, x, w, ids)


def test_lora_rows_with_infinities_and_nan_keep_to_themselves():
    """What a row without an adapter or of another adapter holds does not reach the others."""
    for m in (12, 100):
        y, x, w, ids = lora_inputs(m, 100, 128, 16, 3, "bf16", "bf16", torch.arange(m) % 3)
        want = ck.lora_add(y, x, w, ids)
        ids2 = ids.clone()
        ids2[5] = -1
        x[5], y[7, 3] = float("nan"), float("inf")
        x[6, 2] = float("nan")
        got = ck.lora_add(y, x, w, ids2)
        assert torch.equal(got[5], y[5]) and got[6].isnan().all()
        keep = [i for i in range(m) if i not in (5, 6, 7)]
        assert torch.equal(got[keep], want[keep])
        keep = [j for j in range(100) if j != 3]
        assert torch.equal(got[7, keep], want[7, keep]) and got[7, 3].isinf()
    # an adapter of NaN that no row asks for
    y, x, w, ids = lora_inputs(20, 100, 128, 16, 3, "bf16", "bf16", torch.arange(20) % 2 * 2)
    want = ck.lora_add(y, x, w, ids)
    w.a[1], w.b[1] = float("nan"), float("nan")
    assert torch.equal(ck.lora_add(y, x, w, ids), want)


def test_lora_strides_empty_and_places():
    dev = cuda_device()
    for m in (9, 90):
        y, x, w, ids = lora_inputs(m, 50, 128, 16, 4, "bf16", "bf16")
        want = check_lora(y, x, w, ids)
        wide = torch.zeros((m, 200), dtype=torch.bfloat16, device=dev)
        wide[:, 3:53] = y
        xw = torch.zeros((m, 160), dtype=torch.bfloat16, device=dev)
        xw[:, 8:136] = x
        assert torch.equal(ck.lora_add(wide[:, 3:53], xw[:, 8:136], w, ids), want)
        out = torch.zeros((m, 77), dtype=torch.bfloat16, device=dev)
        ck.lora_add(y, x, w, ids, out=out[:, 1:51])
        assert torch.equal(out[:, 1:51], want) and (out[:, 0] == 0).all() and (out[:, 51:] == 0).all()
        view = wide[:, 3:53]
        assert ck.lora_add(view, x, w, ids, out=view) is view
        assert torch.equal(view, want) and (wide[:, :3] == 0).all() and (wide[:, 53:] == 0).all()
        # adapters at a stride, and another one written into a place
        pool_a, pool_b = (torch.zeros((4,) + s, dtype=torch.bfloat16, device=dev) for s in ((20, 128), (60, 16)))
        pool_a[:, :16], pool_b[:, :50] = w.a, w.b
        w2 = ck.LoraWeight(pool_a[:, :16], pool_b[:, :50], w.scale)
        assert torch.equal(ck.lora_add(y, x, w2, ids), want)
        pool_a[1, :16], pool_b[1, :50] = w.a[0], w.b[0]
        w2.scale[1] = w2.scale[0]
        assert torch.equal(ck.lora_add(y, x, w2, ids), ck.lora_add(y, x, w, torch.where(ids == 1, 0, ids).int()))
    y, x, w, ids = lora_inputs(0, 50, 128, 16, 4, "bf16", "bf16", [])
    assert ck.lora_add(y, x, w, ids).shape == (0, 50)
    y, x, w, ids = lora_inputs(5, 50, 0, 16, 4, "bf16", "bf16")
    assert torch.equal(ck.lora_add(y, x, w, ids), y)
    y, x, w, ids = lora_inputs(5, 50, 64, 16, 0, "bf16", "bf16", [0, 0, -1, 2, 0])
    assert torch.equal(ck.lora_add(y, x, w, ids), y)


def test_lora_same_bits_each_call_and_dirty_workspace():
    for m in (24, 400):
        y, x, w, ids = lora_inputs(m, 2000, 1024, 32, 5, "bf16", "fp32")
        want = check_lora(y, x, w, ids)
        ws = ck.lora_add_workspace(x, w)
        for byte in (0, 255):
            if ws is not None:
                ws.fill_(byte)
            assert torch.equal(ck.lora_add(y, x, w, ids, workspace=ws), want)


# -------------------------------------------------------------- token_logprobs

def check_logprobs(x, tokens, top, **kw):
    r = ck.token_logprobs(x, tokens, top, **kw)
    want, ids = ref.logprobs(x, tokens, top)
    assert r.top_ids.dtype == torch.int64 and torch.equal(r.top_ids.cpu(), ids)
    for name, got in (("logprob", r.logprob), ("entropy", r.entropy), ("top", r.top_logprobs)):
        if got is None:
            assert name == "logprob" and tokens is None
            continue
        assert got.dtype == torch.float32
        value, slack = want[name]
        g = got.double().cpu()
        assert torch.equal(g.isnan(), value.isnan()) and torch.equal(g[~value.isfinite() & ~value.isnan()], value[~value.isfinite() & ~value.isnan()]), name
        off = torch.where(value.isfinite(), (g - value).abs() - slack - 2.0 ** -24 * value.abs(), 0.0)
        assert not (off > 0).any(), (name, off.max().item(), (g - value).abs().nan_to_num().max().item())
    return r


def logits(rows, vocab, dtype, seed=1, spread=4.0):
    x = rand(rows, vocab, seed=seed) * (1 + spread * torch.rand((rows, 1), generator=torch.Generator().manual_seed(seed)))
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(seed + 1))
    return x.to(DT[dtype]).to(cuda_device()), tokens.to(cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (3, 2, 2), (2, 7, 5), (1, 63, 63), (5, 64, 64), (2, 65, 64), (4, 255, 1), (3, 1000, 20), (1, 4096, 5), (9, 5003, 8),
    (1, 32000, 5), (2, 32001, 20), (7, 65537, 0), (1, 131072, 64), (40, 20001, 12), (300, 3001, 5), (600, 1023, 64), (1, 200000, 1),
    (2, 4096, 64), (2, 4097, 64), (3, 32767, 64), (1, 32768, 3), (1, 32769, 3), (256, 5000, 9), (257, 5000, 9),
])
def test_logprobs(rows, vocab, top, dtype):
    x, tokens = logits(rows, vocab, dtype)
    tokens[::2] = x.float().argmax(1)[::2]
    check_logprobs(x, tokens, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(2, 50), (3, 5000), (1, 70001), (200, 9000)])
def test_logprobs_ties(rows, vocab, dtype):
    """Equal logits, a few values or one: the lowest indices, in their order; +0 and -0 are equal."""
    dev = cuda_device()
    top = min(64, vocab)
    tokens = torch.zeros(rows, dtype=torch.int64, device=dev)
    x = torch.randint(0, 3, (rows, vocab), generator=torch.Generator().manual_seed(vocab)).to(DT[dtype]).to(dev)
    check_logprobs(x, tokens, top)
    check_logprobs(torch.full_like(x, 2.5), tokens, top)
    x = torch.where(torch.arange(vocab, device=dev) % 2 == 0, 0.0, -0.0).to(DT[dtype]).expand(rows, -1).contiguous()
    r = check_logprobs(x, tokens, top)
    assert torch.equal(r.top_ids[0].cpu(), torch.arange(top))
    x = torch.arange(vocab, device=dev).to(DT[dtype]).expand(rows, -1).contiguous()     # rising: each beats all before
    check_logprobs(x, tokens, top)
    check_logprobs(x.flip(1).contiguous(), tokens, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 5000, 90001])
def test_logprobs_masks(dtype, vocab):
    """Masks of -inf and of the type's lowest value: most of a row, all but one, all."""
    x, tokens = logits(12, vocab, dtype, spread=1.0)
    low = torch.finfo(DT[dtype]).min
    keep = torch.rand((12, vocab), generator=torch.Generator().manual_seed(3)).to(x.device) < 0.1
    top = min(20, vocab)
    for fill in (-math.inf, low):
        y = torch.where(keep, x, fill)
        y[3] = fill
        y[3, vocab // 2] = 1.0
        y[4] = fill
        y[5, :] = fill
        y[5, 0] = low
        y[6, 1:] = fill
        y[7, :-1] = fill
        check_logprobs(y, tokens, top)
    y = torch.full_like(x, -math.inf)
    r = ck.token_logprobs(y, tokens, top)
    assert r.logprob.isnan().all() and r.entropy.isnan().all() and r.top_logprobs.isnan().all()
    assert torch.equal(r.top_ids.cpu(), torch.arange(top).expand(12, -1))


@pytest.mark.parametrize("vocab", [40, 5000, 90001])
def test_logprobs_nan_infinity_and_tokens_outside(vocab):
    """A row with NaN or +inf is NaN and no other is; NaN comes first; a token outside the vocabulary gives NaN."""
    x, tokens = logits(6, vocab, "bf16")
    want = check_logprobs(x, tokens, 5)
    y = x.clone()
    y[1, 30], y[2, 17] = math.nan, math.inf
    y[4, 33], y[4, 3] = -math.nan, math.inf
    r = ck.token_logprobs(y, tokens, 5)
    for i in (1, 2, 4):
        assert r.logprob[i].isnan() and r.entropy[i].isnan() and r.top_logprobs[i].isnan().all()
    assert r.top_ids[1, 0] == 30 and r.top_ids[2, 0] == 17 and r.top_ids[4, :2].tolist() == [33, 3]
    for i in (0, 3, 5):
        assert all(torch.equal(a[i], b[i]) for a, b in zip(r, want))
    bad = tokens.clone()
    bad[0], bad[2], bad[5] = -1, vocab, 1 << 40
    r = ck.token_logprobs(x, bad, 5)
    assert r.logprob[[0, 2, 5]].isnan().all()
    assert torch.equal(r.logprob[[1, 3, 4]], want.logprob[[1, 3, 4]]) and torch.equal(r.top_logprobs, want.top_logprobs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_logprobs_sharp_even_and_far_rows(dtype):
    """One token that has nearly all of the probability, rows of equal logits, and logits far from zero."""
    x, tokens = logits(8, 30000, dtype)
    x[0, 700] = 60.0
    x[1] *= 0
    x[2] += 1000.0
    x[3] -= 1000.0
    x[4] *= 100.0
    x[5] *= 0.001
    tokens[0] = 700
    r = check_logprobs(x, tokens, 10)
    assert abs(r.entropy[1].item() - math.log(30000)) < 1e-5 and r.logprob[0] <= 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_strides_and_alignment(dtype):
    """Rows that start anywhere, at any stride, and what lies between them."""
    for rows, vocab in ((5, 3001), (2, 40009), (300, 2049)):
        x, tokens = logits(rows, vocab, dtype)
        want = check_logprobs(x, tokens, 7)
        for lead, gap in ((1, 0), (3, 5), (8, 8), (2, 1)):
            wide = torch.full((rows, lead + vocab + gap), math.nan, dtype=x.dtype, device=x.device)
            wide[:, lead:lead + vocab] = x
            r = check_logprobs(wide[:, lead:lead + vocab], tokens, 7)
            assert torch.equal(r.top_ids, want.top_ids)


def test_logprobs_without_tokens_empty_and_same_bits():
    x, tokens = logits(3, 50000, "fp16")
    want = check_logprobs(x, tokens, 9)
    r = check_logprobs(x, None, 9)
    assert r.logprob is None and torch.equal(r.entropy, want.entropy)
    ws = ck.token_logprobs_workspace(x, 9)
    for byte in (0, 255):
        if ws is not None:
            ws.fill_(byte)
        r = ck.token_logprobs(x, tokens, 9, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    r = ck.token_logprobs(x[:0], tokens[:0], 4)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 4)


def test_logprobs_far_rows():
    """Rows past 2^31 elements."""
    dev = cuda_device()
    vocab = 1 << 17
    rows = (1 << 31) // vocab + 3
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device=dev)
    tail, tokens = logits(3, vocab, "bf16")
    x[-3:] = tail
    r = ck.token_logprobs(x, torch.cat([torch.zeros(rows - 3, dtype=torch.int64, device=dev), tokens]), 3)
    want = check_logprobs(tail, tokens, 3)
    assert torch.equal(r.top_ids[-3:], want.top_ids) and (r.top_ids[:-3] == torch.arange(3, device=dev)).all()
    assert (r.logprob[-3:] - want.logprob).abs().max() < 1e-4
    assert (r.entropy[:-3] - 17 * math.log(2)).abs().max() < 1e-4


# -------------------------------------------------------------- all together

def calls_of_three():
    """Calls of the three operators, some of them with chunks and a second launch: (call with a workspace, its workspace)."""
    a = prefix_inputs([1500, 90], [0, 20, 23], [400] + [60] * 23, 16, 2, 128, "bf16", "int8", 16)
    few, many = lora_inputs(24, 2000, 1024, 64, 5, "bf16", "fp32"), lora_inputs(600, 300, 264, 16, 5, "fp16", "fp16")
    (x, tokens), (z, told) = logits(3, 50000, "fp16"), logits(40, 5000, "bf16")
    return [
        (lambda ws: [ck.shared_prefix_attention(*a, workspace=ws)], ck.shared_prefix_attention_workspace(a[0], a[1], a[2], a[5])),
        (lambda ws: [ck.lora_add(*few, workspace=ws)], ck.lora_add_workspace(few[1], few[2])),
        (lambda ws: [ck.lora_add(*many, workspace=ws)], ck.lora_add_workspace(many[1], many[2])),
        (lambda ws: list(ck.token_logprobs(x, tokens, 9, workspace=ws)), ck.token_logprobs_workspace(x, 9)),
        (lambda ws: list(ck.token_logprobs(z, told, 9, workspace=ws)), ck.token_logprobs_workspace(z, 9)),
    ]


def test_two_streams_at_once():
    """Calls on two streams, each with workspaces of its own or of the call's, interleaved without waiting."""
    calls = calls_of_three()
    want = [[t.clone() for t in call(None)] for call, _ in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    own = [[None if ws is None else torch.empty_like(ws) for _, ws in calls] for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got += [(j, call(own[s][j] if i % 2 else None)) for j, (call, _) in enumerate(calls)]
    torch.cuda.synchronize()
    for j, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[j])), j


def test_two_graphs_with_one_workspace():
    """Two captured graphs that use the same workspaces, replayed in turn with eager calls between."""
    calls = calls_of_three()
    want = [[t.clone() for t in call(ws)] for call, ws in calls]
    graphs, got = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append([call(ws) for call, ws in calls])
    for i in range(6):
        for r in got[i % 2]:
            for t in r:
                t.zero_()
        for _, ws in calls:
            if ws is not None:
                ws.fill_(255 * (i % 3 == 0))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for r, w in zip(got[i % 2], want):
            assert all(torch.equal(a, b) for a, b in zip(r, w)), i
        for (call, ws), w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(call(ws), w)), i

def server_step(x, qkv_w, lora_qkv, ids, pos, rope, cache, slots, pt, pl, starts, table, lens, w_out, lora_out, head, tokens):
    qkv = ck.int8_linear(x, *qkv_w)
    ck.lora_add(qkv, x, lora_qkv, ids, out=qkv)
    q, k, v = (t.view(len(x), -1, 64) for t in qkv.split([512, 128, 128], 1))
    q, _ = ck.qk_norm_rope(q, k, v, pos, rope, cache=cache, slots=slots)
    o = ck.shared_prefix_attention(q, cache, pt, pl, starts, table, lens).view(len(x), -1)
    y = ck.lora_add(ck.int4_linear(o, w_out), o, lora_out, ids)
    z = ck.int8_linear(y, *head, out_dtype="fp32")
    return qkv, q, o, y, z, ck.token_logprobs(z, tokens, 4)


def test_a_servers_step_eager_and_in_a_graph():
    """All of a step's operators in a row: each against its reference on its own inputs, on a side stream, and
    captured into two graphs that are replayed over changed inputs with eager calls between."""
    dev = cuda_device()
    b, hidden, page = 6, 256, 8
    g = torch.Generator().manual_seed(1)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=g).to(torch.int8).to(dev)  # noqa: E731
    qkv_w = (i8(768, hidden), torch.full((768,), 0.001, device=dev))
    head = (i8(1000, hidden), torch.full((1000,), 0.002, device=dev))
    codes = torch.randint(0, 256, (hidden, 256), generator=g).to(torch.uint8).to(dev)
    w_out = ck.int4_pack(codes, torch.full((hidden, 4), 0.01, dtype=torch.bfloat16, device=dev), group=128)
    lora_qkv = lora_inputs(1, 768, hidden, 16, 3, "bf16", "bf16")[2]
    lora_out = lora_inputs(1, hidden, 512, 8, 3, "bf16", "bf16")[2]
    ids = torch.tensor([0, 2, -1, 1, 1, 0], dtype=torch.int32, device=dev)
    q, cache, pt, pl, starts, table, lens = prefix_inputs([45, 20], [1, 4, 6], [1, 9, 30, 16, 8, 3], 8, 2, 64, "bf16", "bf16", page)
    slots = torch.stack([table[i, (n - 1) // page].long() * page + (n - 1) % page for i, n in enumerate(lens.tolist())])
    pos = lens.long() - 1 + torch.tensor([0, 45, 45, 45, 20, 20], device=dev)
    rope = ck.rope_table(200, 64, device=dev)
    x = rand(b, hidden, dtype=torch.bfloat16).to(dev)
    tokens = torch.randint(0, 1000, (b,), generator=g).to(dev)
    args = (x, qkv_w, lora_qkv, ids, pos, rope, cache, slots, pt, pl, starts, table, lens, w_out, lora_out, head, tokens)

    def flat(r):
        return list(r[:-1]) + list(r[-1])

    qkv, q, o, y, z, r = server_step(*args)
    want, slack = ref.lora(ck.int8_linear(x, *qkv_w), x, lora_qkv.a, lora_qkv.b, lora_qkv.scale, ids)
    ref.assert_within(qkv, want, slack, "qkv")
    check_prefix(q, cache, pt, pl, starts, table, lens)
    want, slack = ref.lora(ck.int4_linear(o, w_out), o, lora_out.a, lora_out.b, lora_out.scale, ids)
    ref.assert_within(y, want, slack, "y")
    check_logprobs(z, tokens, 4)
    eager = [t.clone() for t in flat((qkv, q, o, y, z, r))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = flat(server_step(*args))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))
    graphs, got = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(flat(server_step(*args)))
    for i in range(6):
        x.copy_(rand(b, hidden, dtype=torch.bfloat16, seed=70 + i))
        tokens.copy_(torch.randint(0, 1000, (b,), generator=g))
        ids.copy_(torch.randint(-1, 3, (b,), generator=g).int())
        want = [t.clone() for t in flat(server_step(*args))]
        torch.cuda.synchronize()
        for t in got[i % 2]:
            t.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i % 2], want)), i
