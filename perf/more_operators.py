"""The operators of a server's batch: what is measured.

What a step of many requests at once needs beside the int8 layers and the
decode step's operators:

  shared_prefix_attention  attention of one new token per sequence, where the
                           sequences of a group begin with the same tokens,
                           whose keys and values are read once for the group;
  lora_add                 y + s (x A^T) B^T with the low-rank adapter that
                           each row's request asks for, beside the projection
                           that all of them share;
  token_logprobs           log probabilities of the chosen tokens, with the
                           entropy and the most likely alternatives.

A case names its operator in "op".  `run` computes the plain form with
elementary torch operations in 32 bits, or, where `own` is true, makes the
calls of the framework.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # A few answers to one short prompt: the step's latency.
        dict(name="prefix 4 of 1000", op="shared_prefix_attention", batch=4, prefixes=1, prefix=1000, own=60,
             ragged=False, hq=32, hk=8, d=128, dtype="bf16", cache="bf16", page=16),
        # A server's batch: three instructions of different lengths, conversations of different lengths behind
        # them and some without any, keys and values as int8 codes.
        dict(name="prefix 48 of three int8", op="shared_prefix_attention", batch=48, prefixes=3, prefix=6001, own=1500,
             ragged=True, hq=32, hk=8, d=128, dtype="bf16", cache="int8", page=16),
        # Questions to one document, wide heads.
        dict(name="prefix 24 of 20000 d256", op="shared_prefix_attention", batch=24, prefixes=1, prefix=20000, own=700,
             ragged=True, hq=16, hk=2, d=256, dtype="fp16", cache="fp16", page=32),
        # Many samples about one very long document: the largest, bound by the products.
        dict(name="prefix 128 of 65536", op="shared_prefix_attention", batch=128, prefixes=1, prefix=65536, own=500,
             ragged=True, hq=64, hk=8, d=128, dtype="bf16", cache="bf16", page=64),
        # One request's token beside a small square projection.
        dict(name="lora 1x4096x4096 r16", op="lora_add", m=1, n=4096, k=4096, rank=16, adapters=8, runs=False,
             dtype="bf16", out="bf16"),
        # A decode batch in which nearly every request has an adapter of its own, beside a wide projection.
        dict(name="lora 61x16384x4096 r16", op="lora_add", m=61, n=16384, k=4096, rank=16, adapters=48, runs=False,
             dtype="fp16", out="fp16"),
        # A few large adapters beside the widest projection.
        dict(name="lora 17x28672x5376 r64", op="lora_add", m=17, n=28672, k=5376, rank=64, adapters=5, runs=False,
             dtype="bf16", out="bf16"),
        # The prompts of a few requests in one call, into a 32-bit sum.
        dict(name="lora 4001x5376x5376 r32", op="lora_add", m=4001, n=5376, k=5376, rank=32, adapters=6, runs=True,
             dtype="bf16", out="fp32"),
        # One token's choice, with the five best alternatives.
        dict(name="logprobs 1x32000", op="token_logprobs", rows=1, vocab=32000, top=5, masked=False, dtype="bf16"),
        # A few rows of an odd width, a grammar's mask over most of them, no alternatives wanted.
        dict(name="logprobs 7x65537 masked", op="token_logprobs", rows=7, vocab=65537, top=0, masked=True,
             dtype="fp16"),
        # A decode batch with 32-bit logits and many alternatives.
        dict(name="logprobs 48x128000 fp32", op="token_logprobs", rows=48, vocab=128000, top=20, masked=False,
             dtype="fp32"),
        # The log probabilities of a long prompt: the largest.
        dict(name="logprobs 2048x131072", op="token_logprobs", rows=2048, vocab=131072, top=8, masked=False,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared_prefix_attention", "lora_add", "token_logprobs"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "token_logprobs":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        vocab = _log(rng, 1000, 200000)
        most = 2048 * 131072 // (2 if dtype == "fp32" else 1)
        return dict(op=op, rows=_log(rng, 1, min(2048, most // vocab)), vocab=vocab, top=rng.choice([0, 1, 5, 8, 20, 64]),
                    masked=rng.random() < 0.3, dtype=dtype)
    if op == "lora_add":
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        n, k = _log(rng, 500, 21504), 8 * _log(rng, 64, 672)
        m = _log(rng, 1, max(1, min(4001, 4001 * 32 * 10752 // (rank * (n + k)), 4001 * 5376 * 5 // (4 * n + k))))
        return dict(op=op, m=m, n=n, k=k, rank=rank, adapters=_log(rng, 1, 4 * 64 // rank if rank > 32 else 64),
                    runs=rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]))
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 7, 8])
    d = rng.choice([64, 96, 128, 192, 256])
    batch = _log(rng, 1, 128)
    return dict(op=op, batch=batch, prefixes=_log(rng, 1, min(8, batch)),
                prefix=_log(rng, 16, min(65536, 128 * 64 * 65536 * 128 // (batch * hq * d * 2))),
                own=_log(rng, 1, min(4096, 65536 // batch)), ragged=rng.random() < 0.7, hq=hq, hk=hk, d=d, dtype=dtype,
                cache=rng.choice([dtype, dtype, "int8"]), page=rng.choice([8, 16, 32, 64, 128]))


# ----------------------------------------------------------------- the inputs

def _ragged(g, count, top):
    """Lengths even over the logarithm, from a tenth of the longest on; one of them the longest."""
    lens = (top * torch.exp(torch.rand(count, generator=g, dtype=torch.float64) * math.log(0.1))).long().clamp(1, top)
    lens[int(torch.randint(count, (1,), generator=g))] = top
    return lens.tolist()


def _lens(case, seed):
    """What the host's program knows: the lengths of the prefixes and of the sequences, and where each prefix's
    sequences begin."""
    b, p = case["batch"], case["prefixes"]
    if not case["ragged"]:
        return [case["prefix"]] * p, [case["own"]] * b, [b * i // p for i in range(p + 1)]
    g = torch.Generator().manual_seed(seed)
    prefix, lens = _ragged(g, p, case["prefix"]), _ragged(g, b, case["own"])
    # the first sixteenth of the batch has no prefix; the others go to the prefixes in shares of any size
    free = b // 16 if p > 1 else 0
    inner = torch.randperm(b - free - 1, generator=g)[:p - 1].add(free + 1).sort().values.tolist() if p > 1 else []
    return prefix, lens, [free] + inner + [b]


def _codes(x):
    """int8 codes and the scale of each row of the last dimension: s = amax / 127, rint(x / s)."""
    s = x.abs().amax(-1) / 127
    return torch.where(s[..., None] > 0, torch.round(x / s[..., None]), 0.0).clamp(-127, 127).to(torch.int8), s


def _pages(lens, page, order):
    """A page table [len(lens), pages of the longest] from the pages in `order`, and how many it used."""
    counts = torch.tensor([-(-n // page) for n in lens])
    start = torch.cumsum(counts, 0) - counts
    col = torch.arange(max(1, int(counts.max())))
    at = torch.where(col < counts[:, None], start[:, None] + col, 0)
    return order[at.to(DEV)].contiguous(), int(counts.sum())


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    if own:
        import int8_weight_quantized_amd as ck

    t = TYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "token_logprobs":
        rows, vocab = case["rows"], case["vocab"]
        # rows from nearly even to sharp
        x = normal(rows, vocab) * (1 + 4 * torch.rand((rows, 1), generator=g, device=DEV))
        if case["masked"]:
            x.masked_fill_(torch.rand((rows, vocab), generator=g, device=DEV) < 0.9, -math.inf)
        s["logits"] = x.to(t)
        # a likely token for every other row, any for the others
        s["tokens"] = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        s["tokens"][::2] = s["logits"][::2].float().argmax(-1)
        return s
    if case["op"] == "lora_add":
        m, n, k, r, count = (case[i] for i in ("m", "n", "k", "rank", "adapters"))
        s["x"], s["y"] = normal(m, k, dtype=t), normal(m, n, dtype=TYPES[case["out"]])
        s["a"] = normal(count, r, k).mul_(k ** -0.5).to(t)
        s["b"] = normal(count, n, r).mul_(r ** -0.5).to(t)
        s["scale"] = 0.5 + torch.rand(count, generator=g, device=DEV)
        if case["runs"]:        # prompts one behind the other, in shares of any size
            edge = torch.rand(count, generator=g, device=DEV).mul_(m).long().sort().values
            s["ids"] = ((torch.arange(m, device=DEV)[:, None] >= edge).sum(1) % count).int()
        else:                   # any request in any row, one in sixteen without an adapter
            s["ids"] = torch.randint(0, count, (m,), generator=g, device=DEV).int()
            s["ids"][5::16] = -1
        if own:
            s["lora"] = ck.LoraWeight(s["a"], s["b"], s["scale"])
        return s

    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    prefix, lens, starts = _lens(case, seed)
    pages = sum(-(-n // page) for n in prefix + lens) + 1
    order = torch.randperm(pages, generator=g, device=DEV).int()
    s["prefix_table"], used = _pages(prefix, page, order)
    s["table"], _ = _pages(lens, page, order[used:])
    s["prefix_lens"], s["lens"], s["starts"] = (torch.tensor(v, dtype=torch.int32, device=DEV)
                                                for v in (prefix, lens, starts))
    s["most"] = max(b - a for a, b in zip(starts, starts[1:]))
    s["q"] = (2 * normal(case["batch"], hq, d)).to(t)
    s["scale"] = d ** -0.5
    shape = (pages, hk, page, d)
    if case["cache"] == "int8":
        (k, ks), (v, vs) = (_codes(normal(*shape)) for _ in range(2))
    else:
        (k, ks), (v, vs) = ((normal(*shape, dtype=TYPES[case["cache"]]), None) for _ in range(2))
    s.update(kc=k, vc=v, ks=ks, vs=vs)
    if own:
        s["cache"] = ck.KVCache(k, v, ks, vs)
    return s


# ------------------------------------------------------------ the plain forms

def _plain_part(q, s, table, lens):
    """Scores' largest, sum of weights and weighted values of q [n, hk, rows, d] over the n token lists of table."""
    n, hk, d = q.shape[0], q.shape[1], q.shape[3]
    page = table.long()

    def whole(x, scale):
        x = x[page].float() if scale is None else x[page].float() * scale[page][..., None]
        return x.transpose(1, 2).reshape(n, hk, -1, d)         # [n, hk, tokens, d]

    score = torch.matmul(q, whole(s["kc"], s["ks"]).transpose(2, 3).contiguous()) * s["scale"]
    seen = torch.arange(score.shape[3], device=DEV) < lens[:, None]
    score = score.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = score.amax(3, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score.sub_(top))
    return top, p.sum(3, keepdim=True), torch.matmul(p, whole(s["vc"], s["vs"]))


def _plain_shared_prefix_attention(s):
    c = s["case"]
    b, hq, hk, d, p = (c[i] for i in ("batch", "hq", "hk", "d", "prefixes"))
    g = hq // hk
    q = s["q"].float().view(b, hk, g, d)
    # every prefix's sequences side by side, as many places as the largest group has
    starts, most = s["starts"].long(), s["most"]
    rows = (starts[:-1, None] + torch.arange(most, device=DEV)).clamp_max(b - 1)
    qp = q[rows].transpose(1, 2).reshape(p, hk, most * g, d)
    shared = [x.view(p, hk, most, g, -1).transpose(1, 2) for x in _plain_part(qp, s, s["prefix_table"], s["prefix_lens"])]
    # and back to the sequences
    seq = torch.arange(b, device=DEV)
    group = (starts <= seq[:, None]).sum(1) - 1
    has = (group >= 0) & (group < p)
    group = group.clamp(0, p - 1)
    place = (seq - starts[group]).clamp(0, most - 1)
    top, total, out = (x[group, place] for x in shared)
    top = torch.where(has[:, None, None, None], top, -1e30)
    total, out = total * has[:, None, None, None], out * has[:, None, None, None]
    top2, total2, out2 = _plain_part(q, s, s["table"], s["lens"])
    high = torch.maximum(top, top2)
    f, f2 = torch.exp(top - high), torch.exp(top2 - high)
    return ((out * f + out2 * f2) / (total * f + total2 * f2)).reshape(b, hq, d).to(s["q"].dtype)


def _plain_lora_add(s):
    x, a, b, ids = s["x"].float(), s["a"].float(), s["b"].float(), s["ids"].long()
    m, count, r, n = x.shape[0], a.shape[0], a.shape[1], b.shape[1]
    # every adapter's part of every row, all but the row's own one cleared
    v = torch.matmul(x, a.view(count * r, -1).t()).view(m, count, r)
    mine = (torch.arange(count, device=DEV) == ids[:, None]).float() * s["scale"]
    v = (v * mine[..., None]).view(m, count * r)
    return (s["y"].float() + torch.matmul(v, b.transpose(1, 2).reshape(count * r, n))).to(s["y"].dtype)


def _plain_token_logprobs(s):
    x, top = s["logits"].float(), s["case"]["top"]
    high = x.amax(1, keepdim=True)
    y = x - high
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    # a masked token's e (x - max) is 0 times infinity: it adds nothing
    entropy = torch.log(total) - torch.where(e > 0, e * y, 0.0).sum(1, keepdim=True) / total
    norm = high + torch.log(total)
    ids = s["tokens"].new_empty((x.shape[0], 0))
    if top:     # the largest values, and among equal ones the lowest index: whole numbers that order both
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32
        ids = torch.topk(order - torch.arange(x.shape[1], device=DEV), top, 1).indices
    return dict(logprob=(x.gather(1, s["tokens"][:, None]) - norm)[:, 0], entropy=entropy[:, 0], ids=ids,
                top=x.gather(1, ids) - norm)


def run(state):
    c = state["case"]
    if own:
        import int8_weight_quantized_amd as ck
        if c["op"] == "shared_prefix_attention":
            return ck.shared_prefix_attention(state["q"], state["cache"], state["prefix_table"], state["prefix_lens"],
                                              state["starts"], state["table"], state["lens"], state["scale"])
        if c["op"] == "lora_add":
            return ck.lora_add(state["y"], state["x"], state["lora"], state["ids"])
        r = ck.token_logprobs(state["logits"], state["tokens"], c["top"])
        return dict(logprob=r.logprob, entropy=r.entropy, ids=r.top_ids, top=r.top_logprobs)
    if c["op"] == "shared_prefix_attention":
        return _plain_shared_prefix_attention(state)
    if c["op"] == "lora_add":
        return _plain_lora_add(state)
    return _plain_token_logprobs(state)


# ----------------------------------------------------------------- the floors

def work(case):
    if case["op"] == "token_logprobs":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        # of each logit: the largest, the difference, its exponential, two sums and a product
        return dict(bytes=rows * (vocab * (4 if case["dtype"] == "fp32" else 2) + 16 + 12 * top), flops=6 * rows * vocab)
    if case["op"] == "lora_add":
        m, n, k, r, count = (case[i] for i in ("m", "n", "k", "rank", "adapters"))
        used = count if case["runs"] and m >= count else count * (1 - (1 - 1 / count) ** m)     # as many as are asked for
        return dict(bytes=m * (2 * k + 2 * n * (4 if case["out"] == "fp32" else 2) + 4) + 2 * used * r * (n + k),
                    flops=2 * m * r * (n + k))
    # The lengths of a ragged batch go by the seed: their mean is 0.39 of the longest, which one of them has.
    b, p, hq, hk, d = (case[i] for i in ("batch", "prefixes", "hq", "hk", "d"))
    row = (d + 4) if case["cache"] == "int8" else 2 * d        # one head's key or value in the cache
    share = 0.39 if case["ragged"] else 1.0
    shared = case["prefix"] * (1 + (p - 1) * share)
    alone = case["own"] * (1 + (b - 1) * share)
    with_prefix = b - (b // 16 if case["ragged"] and p > 1 else 0)
    return dict(bytes=2 * (shared + alone) * hk * row + 4 * b * hq * d + 4 * (shared + alone) / case["page"] + 4 * (b + 2 * p),
                flops=4 * hq * d * (with_prefix * shared / p + alone))


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "token_logprobs":
        x = s["logits"].double()
        log_p = x - torch.logsumexp(x, 1)[:, None]
        entropy = -torch.special.xlogy(log_p.exp(), log_p.exp()).sum(1)
        value, ids = torch.sort(log_p, dim=1, descending=True, stable=True)
        return dict(logprob=log_p[torch.arange(case["rows"]), s["tokens"]], entropy=entropy, ids=ids[:, :case["top"]],
                    top=value[:, :case["top"]].contiguous())
    if case["op"] == "lora_add":
        out = s["y"].double()
        for j in range(case["adapters"]):
            mine = (s["ids"] == j).nonzero()[:, 0]
            v = s["x"][mine].double() @ s["a"][j].double().t()
            out[mine] += s["scale"][j].double() * (v @ s["b"][j].double().t())
        return out
    out = torch.zeros((case["batch"], case["hq"], case["d"]), dtype=torch.float64, device=DEV)
    g, page = case["hq"] // case["hk"], case["page"]
    starts, prefix = s["starts"].tolist(), s["prefix_lens"].tolist()

    def rows(table, n, h):
        at = torch.arange(n, device=DEV)
        where = (table[at // page].long(), h, at % page)
        k, v = s["kc"][where].double(), s["vc"][where].double()
        if s["ks"] is not None:
            k, v = k * s["ks"][where].double()[:, None], v * s["vs"][where].double()[:, None]
        return k, v

    for h in range(case["hk"]):
        first = [rows(s["prefix_table"][i], n, h) for i, n in enumerate(prefix)]
        for i, n in enumerate(s["lens"].tolist()):
            parts = [first[j] for j in range(case["prefixes"]) if starts[j] <= i < starts[j + 1]]
            parts.append(rows(s["table"][i], n, h))
            q = s["q"][i, h * g:(h + 1) * g].double()
            p = torch.softmax(torch.cat([q @ k.t() for k, _ in parts], 1) * s["scale"], 1)
            at = 0
            for k, v in parts:
                out[i, h * g:(h + 1) * g] += p[:, at:at + len(k)] @ v
                at += len(k)
    return out
