"""The decode step's operators beside the int8 projections: what is measured.

Three operators that a model served with this framework's int8 layers runs
between its projections, and the 4-bit projection itself:

  qk_norm_rope     RMS norm of every query and key head, the position
                   rotation, and the write of keys and values into a paged
                   cache, in one pass;
  paged_attention  attention of one new token per sequence over that cache;
  int4_linear      x W^T with 4-bit weights and a scale (and zero point) for
                   every group of weights along K, for few rows of x.

A case names its operator in "op".  `run` computes the plain form with
elementary torch operations in 32 bits, or, where `own` is true, makes the
calls of the framework.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One new token of one sequence: the step's latency, 32 query and 8 key heads of 128.
        dict(name="rope 1 token", op="qk_norm_rope", tokens=1, hq=32, hk=8, d=128, rot=128, interleaved=False,
             dtype="bf16", cache="bf16", page=16, far=8192, norm=True),
        # A decode batch with wide heads, half of each rotated in neighbouring pairs, far positions.
        dict(name="rope 61 tokens d256", op="qk_norm_rope", tokens=61, hq=16, hk=2, d=256, rot=128, interleaved=True,
             dtype="fp16", cache="fp16", page=32, far=131072, norm=True),
        # A prompt's chunk into a cache that holds int8 codes with a scale for each token and head.
        dict(name="rope 515 tokens int8 cache", op="qk_norm_rope", tokens=515, hq=24, hk=8, d=96, rot=96,
             interleaved=False, dtype="bf16", cache="int8", page=16, far=32768, norm=True),
        # A long prompt in one call.
        dict(name="rope 8192 tokens", op="qk_norm_rope", tokens=8192, hq=32, hk=8, d=128, rot=128, interleaved=False,
             dtype="bf16", cache="bf16", page=64, far=8192, norm=True),
        # One short conversation.
        dict(name="attention 1x1000", op="paged_attention", batch=1, longest=1000, ragged=False, hq=32, hk=8, d=128,
             dtype="bf16", cache="bf16", page=16, window=0, sinks=0),
        # A server's batch: sequences of very different lengths, keys and values as int8 codes.
        dict(name="attention 48 ragged int8", op="paged_attention", batch=48, longest=9001, ragged=True, hq=32, hk=8,
             d=128, dtype="bf16", cache="int8", page=16, window=0, sinks=0),
        # A layer that sees the last 4096 tokens and the first four, wide heads.
        dict(name="attention window sinks d256", op="paged_attention", batch=16, longest=20000, ragged=True, hq=16,
             hk=2, d=256, dtype="fp16", cache="fp16", page=32, window=4096, sinks=4),
        # Few very long documents: the largest cache.
        dict(name="attention 4x131072", op="paged_attention", batch=4, longest=131072, ragged=False, hq=64, hk=8,
             d=128, dtype="bf16", cache="bf16", page=64, window=0, sinks=0),
        # One row through a small square projection.
        dict(name="int4 1x4096x4096", op="int4_linear", m=1, n=4096, k=4096, group=128, zeros=False, bias=False,
             dtype="bf16"),
        # One row through the wide projection, small groups with zero points.
        dict(name="int4 1x28672x5376 g32", op="int4_linear", m=1, n=28672, k=5376, group=32, zeros=True, bias=False,
             dtype="fp16"),
        # A decode batch of an odd number of rows.
        dict(name="int4 17x16384x4096 g64", op="int4_linear", m=17, n=16384, k=4096, group=64, zeros=True, bias=True,
             dtype="bf16"),
        # The largest decode batch.
        dict(name="int4 128x21504x5376", op="int4_linear", m=128, n=21504, k=5376, group=128, zeros=False, bias=True,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "paged_attention", "int4_linear"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "int4_linear":
        return dict(op=op, m=_log(rng, 1, 128), n=_log(rng, 1000, 28672 if rng.random() < 0.5 else 16384),
                    k=8 * _log(rng, 128, 640), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                    bias=rng.random() < 0.5, dtype=dtype)
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 7, 8])
    d = rng.choice([64, 96, 128, 192, 256])
    cache = rng.choice([dtype, dtype, "int8"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "qk_norm_rope":
        tokens = _log(rng, 1, 4096)
        return dict(op=op, tokens=tokens, hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3, dtype=dtype, cache=cache, page=page,
                    far=_log(rng, max(64, tokens), 131072), norm=rng.random() < 0.8)
    longest = _log(rng, 1, 65536)
    batch = _log(rng, 1, max(1, min(64, 131072 // longest)))
    windowed = rng.random() < 0.4
    return dict(op=op, batch=batch, longest=longest, ragged=rng.random() < 0.7, hq=hq, hk=hk, d=d, dtype=dtype,
                cache=cache, page=page, window=_log(rng, 1, 8192) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 37]) if windowed else 0)


# ----------------------------------------------------------------- the inputs

def _lens(case, seed):
    """The sequences' lengths, as the host's program knows them."""
    b, top = case["batch"], case["longest"]
    if not case["ragged"]:
        return [top] * b
    g = torch.Generator().manual_seed(seed)
    # even over the logarithm, from a hundredth of the longest on; one of them the longest
    lens = (top * torch.exp(torch.rand(b, generator=g, dtype=torch.float64) * math.log(0.01))).long().clamp(1, top)
    lens[int(torch.randint(b, (1,), generator=g))] = top
    return lens.tolist()


def _visible(case, n):
    """How many tokens of a sequence of n the new one sees."""
    if not case["window"]:
        return n
    return min(n, min(case["window"], n) + min(case["sinks"], max(0, n - case["window"])))


def _codes(x):
    """int8 codes and the scale of each row of the last dimension: s = amax / 127, rint(x / s)."""
    s = x.abs().amax(-1) / 127
    return torch.where(s[..., None] > 0, torch.round(x / s[..., None]), 0.0).clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    if own:
        import int8_weight_quantized_amd as ck

    t = TYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "int4_linear":
        n, k, group = case["n"], case["k"], case["group"]
        groups = -(-k // group)
        # two codes a byte, the lower half the even one, as checkpoints hold them
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((n, groups), generator=g, device=DEV)) * 0.01).to(t)
        s["zeros"] = (torch.randint(0, 16, (n, groups), generator=g, device=DEV, dtype=torch.uint8)
                      if case["zeros"] else None)
        s["x"] = normal(case["m"], k, dtype=t)
        s["bias"] = normal(n, dtype=t) if case["bias"] else None
        if own:
            s["weight"] = ck.int4_pack(s["codes"], s["scales"], s["zeros"], group=group)
        return s

    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    ct = torch.int8 if case["cache"] == "int8" else TYPES[case["cache"]]
    if case["op"] == "qk_norm_rope":
        tokens, rot = case["tokens"], case["rot"]
        pages = -(-tokens // page) + 3
        qkv = normal(tokens, (hq + 2 * hk) * d, dtype=t)       # what a fused projection returns
        s["q"] = qkv[:, :hq * d].view(tokens, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(tokens, hk, d)
        s["qw"] = 1 + 0.2 * normal(d) if case["norm"] else None
        s["kw"] = 1 + 0.2 * normal(d) if case["norm"] else None
        first = int(torch.randint(0, case["far"] - tokens + 1, (1,), generator=torch.Generator().manual_seed(seed)))
        s["positions"] = torch.arange(first, first + tokens, device=DEV)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        angle = torch.arange(case["far"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(tokens, device=DEV)
        s["slots"] = order[at // page] * page + at % page
    else:
        lens = _lens(case, seed)
        width = -(-max(lens) // page)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 1
        order = torch.randperm(pages, generator=g, device=DEV).int()
        used = torch.tensor(counts)
        start = torch.cumsum(used, 0) - used
        col = torch.arange(width)
        at = torch.where(col < used[:, None], start[:, None] + col, pages - 1)
        s["table"] = order[at.to(DEV)].contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = 2 * normal(case["batch"], hq, d)
        s["q"] = s["q"].to(t)
        s["scale"] = d ** -0.5

    shape = (pages, hk, page, d)
    if case["op"] == "qk_norm_rope":
        k, v = (torch.zeros(shape, dtype=ct, device=DEV) for _ in range(2))
        ks, vs = ((torch.zeros(shape[:3], device=DEV) for _ in range(2)) if ct == torch.int8 else (None, None))
    elif ct == torch.int8:
        (k, ks), (v, vs) = (_codes(normal(*shape)) for _ in range(2))
    else:
        (k, ks), (v, vs) = ((normal(*shape, dtype=ct), None) for _ in range(2))
    s.update(kc=k, vc=v, ks=ks, vs=vs)
    if own:
        s["cache"] = ck.KVCache(k, v, ks, vs)
    return s


# ------------------------------------------------------------ the plain forms

def _plain_rotated(x, w, table, positions, rot, interleaved):
    """The normed and rotated heads of x [tokens, heads, d], in 32 bits."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
    cos, sin = table[positions][:, None].split(rot // 2, -1)
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r.split(rot // 2, -1)
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_qk_norm_rope(s):
    c = s["case"]
    q = _plain_rotated(s["q"], s["qw"], s["table"], s["positions"], c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _plain_rotated(s["k"], s["kw"], s["table"], s["positions"], c["rot"], c["interleaved"])
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    if s["ks"] is None:
        s["kc"][page, :, at] = k.to(s["kc"].dtype)
        s["vc"][page, :, at] = s["v"]
    else:
        s["kc"][page, :, at], s["ks"][page, :, at] = _codes(k)
        s["vc"][page, :, at], s["vs"][page, :, at] = _codes(s["v"].float())
    return q


def _plain_paged_attention(s):
    c = s["case"]
    b, hk, d = c["batch"], c["hk"], c["d"]
    g = c["hq"] // hk
    page = s["table"].long()

    def whole(x, scale):
        x = x[page].float() if scale is None else x[page].float() * scale[page][..., None]
        return x.transpose(1, 2).reshape(b, hk, -1, d)         # [b, hk, tokens, d]

    k = whole(s["kc"], s["ks"])
    q = s["q"].float().view(b, hk, g, d).transpose(2, 3).contiguous()
    score = torch.matmul(k, q) * s["scale"]                    # [b, hk, tokens, g]
    del k
    at = torch.arange(score.shape[2], device=DEV)
    n = s["lens"][:, None]
    seen = at < n
    if c["window"]:
        seen = seen & ((at >= n - c["window"]) | (at < c["sinks"]))
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(score - score.amax(2, keepdim=True))
    p = (p / p.sum(2, keepdim=True)).transpose(2, 3).contiguous()
    return torch.matmul(p, whole(s["vc"], s["vs"])).reshape(b, c["hq"], d).to(s["q"].dtype)


def _plain_int4_linear(s):
    c = s["case"]
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(1).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(c["group"], 1)[:, :c["k"]]
    w = (code - zero) * s["scales"].float().repeat_interleave(c["group"], 1)[:, :c["k"]]
    y = torch.matmul(s["x"].float(), w.t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def run(state):
    c = state["case"]
    if own:
        import int8_weight_quantized_amd as ck
        if c["op"] == "qk_norm_rope":
            q, _ = ck.qk_norm_rope(state["q"], state["k"], state["v"], state["positions"], state["table"],
                                   state["qw"], state["kw"], eps=1e-6, interleaved=c["interleaved"],
                                   cache=state["cache"], slots=state["slots"])
        elif c["op"] == "paged_attention":
            return ck.paged_attention(state["q"], state["cache"], state["table"], state["lens"], state["scale"],
                                      window=c["window"], sinks=c["sinks"])
        else:
            return ck.int4_linear(state["x"], state["weight"], state["bias"])
    elif c["op"] == "qk_norm_rope":
        q = _plain_qk_norm_rope(state)
    elif c["op"] == "paged_attention":
        return _plain_paged_attention(state)
    else:
        return _plain_int4_linear(state)
    if state["ks"] is None:
        return dict(q=q, k=state["kc"], v=state["vc"])
    # codes come back as the values that they stand for
    return dict(q=q, k=state["kc"] * state["ks"][..., None], v=state["vc"] * state["vs"][..., None])


# ----------------------------------------------------------------- the floors

def work(case):
    if case["op"] == "int4_linear":
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["group"])
        return dict(bytes=n * k / 2 + n * groups * (3 if case["zeros"] else 2) + 2 * m * (n + k)
                    + (2 * n if case["bias"] else 0), flops=2 * m * n * k)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    row = (d + 4) if case["cache"] == "int8" else 2 * d        # one head's key or value in the cache
    if case["op"] == "qk_norm_rope":
        t = case["tokens"]
        return dict(bytes=t * (2 * (hq + 2 * hk) * d + 2 * hq * d + 2 * hk * row + 4 * case["rot"] + 16),
                    flops=t * (hq + hk) * (4 * d + 3 * case["rot"]))
    # The lengths of a ragged batch go by the seed: their mean is 0.215 of the longest, which one of them has.
    top, b = case["longest"], case["batch"]
    lens = [top] * b if not case["ragged"] else [top] + [max(1, int(top * 0.01 ** ((i + 0.5) / (b - 1))))
                                                        for i in range(b - 1)]
    seen = sum(_visible(case, n) for n in lens)
    return dict(bytes=2 * seen * hk * row + 4 * b * hq * d + 4 * seen // case["page"] + 4 * b,
                flops=4 * seen * hq * d)


# ------------------------------------------------- the definitions in 64 bits

def _exact_heads(x, w, positions, table, rot, interleaved):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
    # a pair of elements is a complex number, turned by its position's unit
    unit = torch.complex(table[:, :rot // 2].double(), table[:, rot // 2:].double())[positions].unsqueeze(1)
    first = torch.arange(rot // 2, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else rot // 2)
    z = torch.complex(y[..., first], y[..., second]) * unit
    out = y.clone()
    out[..., first] = z.real
    out[..., second] = z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int4_linear":
        k, group = case["k"], case["group"]
        w = torch.empty((case["n"], k), dtype=torch.float64, device=DEV)
        w[:, 0::2] = (s["codes"] % 16).double()
        w[:, 1::2] = (s["codes"] // 16).double()
        for j in range(s["scales"].shape[1]):
            cols = slice(j * group, min(k, (j + 1) * group))
            w[:, cols] -= 8 if s["zeros"] is None else s["zeros"][:, j:j + 1].double()
            w[:, cols] *= s["scales"][:, j:j + 1].double()
        y = s["x"].double() @ w.t()
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "qk_norm_rope":
        how = (s["positions"], s["table"], case["rot"], case["interleaved"])
        q, k = _exact_heads(s["q"], s["qw"], *how), _exact_heads(s["k"], s["kw"], *how)
        if case["cache"] == "int8":     # the codes are a choice of the nearest: they have no value in 64 bits
            return dict(q=q, k=None, v=None)
        caches = []
        for x in (k, s["v"].double()):
            flat = torch.zeros((s["kc"].shape[0] * case["page"], case["hk"], case["d"]), dtype=torch.float64,
                               device=DEV)
            flat[s["slots"]] = x
            caches.append(flat.view(-1, case["page"], case["hk"], case["d"]).transpose(1, 2).contiguous())
        return dict(q=q, k=caches[0], v=caches[1])
    out = torch.zeros((case["batch"], case["hq"], case["d"]), dtype=torch.float64, device=DEV)
    g = case["hq"] // case["hk"]
    for i, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device=DEV)
        if case["window"]:
            at = at[(n - at <= case["window"]) | (at < case["sinks"])]
        page, off = s["table"][i][at // case["page"]].long(), at % case["page"]
        for h in range(case["hk"]):
            k, v = s["kc"][page, h, off].double(), s["vc"][page, h, off].double()
            if s["ks"] is not None:
                k = k * s["ks"][page, h, off].double()[:, None]
                v = v * s["vs"][page, h, off].double()[:, None]
            p = torch.softmax(s["q"][i, h * g:(h + 1) * g].double() @ k.t() * s["scale"], -1)
            out[i, h * g:(h + 1) * g] = p @ v
    return out
