"""Plain references of the decode-step operators in 64 bits, and the error
bounds that their fp32 arithmetic allows.  Everything here runs on the CPU."""
import math

import torch

U32 = 2.0 ** -24                     # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def assert_within(got, want, slack, what):
    """|got - want| <= half a step of got's type + slack, everywhere."""
    got64 = got.detach().cpu().double()
    assert got64.shape == want.shape, (what, got64.shape, want.shape)
    assert torch.equal(torch.isfinite(got64), torch.isfinite(want)), f"{what}: not finite where the reference is, or the reverse"
    tol = HALF[got.dtype] * (want.abs() + slack) + TINY[got.dtype] + slack
    off = (got64 - want).abs()
    bad = torch.isfinite(want) & (off > tol)
    if bad.any():
        i = tuple(x.item() for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {got64[i].item()!r}, "
                             f"want {want[i].item()!r}, allowed {tol[i].item():.3g}")


def rope(x, w, cos_sin, positions, rot, interleaved, eps):
    """-> (y, slack): the normed and rotated heads of x [tokens, heads, d],
    and how far fp32 arithmetic may be from them.

    Norm: the sum of d squares is off by at most (d + 1) u relative, the root
    by half of that, and six more roundings (mean, eps, root, reciprocal, two
    products): |dy| <= (d / 2 + 7) u |y|.  Rotation: two products and a sum,
    3 u (|a c| + |b s|) on top of the error of a and b."""
    x = x.detach().cpu().double()
    d = x.shape[-1]
    y, rel = x, 0.0
    if w is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.detach().cpu().double()
        rel = (d / 2 + 7) * U32
    err = y.abs() * rel
    if rot:
        cs = cos_sin.detach().cpu().double()[positions.cpu()][:, None]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        ia = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
        ib = ia + (1 if interleaved else rot // 2)
        a, b = y[..., ia], y[..., ib]
        y, err = y.clone(), err.clone()
        y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
        err[..., ia] = (rel + 3 * U32) * ((a * cos).abs() + (b * sin).abs())
        err[..., ib] = (rel + 3 * U32) * ((b * cos).abs() + (a * sin).abs())
    return y, err


def visible_tokens(n, window, sinks):
    at = torch.arange(n)
    return at[(at >= n - window) | (at < sinks)] if window else at


def attention(q, kc, vc, ks, vs, table, lens, scale, window, sinks):
    """-> (out, slack) of one new token per sequence.  kc, vc: [pages, heads,
    page, d]; ks, vs their scales or None.

    Scores: d products and sums, the scales and the change to base 2 are off
    by at most (d + 6) u times S = scale sum |q_i k_i|; the exponential turns
    that into a relative error of each weight (and of the sum), its own
    rounding adds 4 u.  The weights enter the products in two 16-bit parts:
    2^-16 for bf16, the coarser type.  Sums over n tokens: n u.  All of it is
    relative to sum p |v|, and counts twice (numerator and denominator)."""
    q, kc, vc = (t.detach().cpu() for t in (q, kc, vc))
    ks, vs = (None if t is None else t.detach().cpu().double() for t in (ks, vs))
    table, lens = table.cpu().long(), lens.cpu().tolist()
    b, hq, d = q.shape
    pages, hk, page = kc.shape[:3]
    g = hq // hk
    out, slack = torch.zeros((b, hq, d), dtype=torch.float64), torch.zeros((b, hq, d), dtype=torch.float64)
    for i, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * page))
        at = visible_tokens(n, window, sinks)
        if not len(at):
            continue
        pg = table[i][at // page]
        if ((pg < 0) | (pg >= pages)).any():
            out[i] = math.nan
            continue
        off = at % page
        for h in range(hk):
            k, v = kc[pg, h, off].double(), vc[pg, h, off].double()
            if ks is not None:
                k, v = k * ks[pg, h, off][:, None], v * vs[pg, h, off][:, None]
            qq = q[i, h * g:(h + 1) * g].double()
            p = torch.softmax(qq @ k.t() * scale, -1)
            out[i, h * g:(h + 1) * g] = p @ v
            s = (qq.abs() @ k.abs().t()).amax(-1, keepdim=True) * abs(scale)
            slack[i, h * g:(h + 1) * g] = 2 * ((d + 6) * U32 * s + 2.0 ** -16 + (len(at) + 4) * U32) * (p @ v.abs())
    return out, slack


def unpack_codes(codes):
    c = codes.detach().cpu()
    return torch.stack([c & 15, c >> 4], -1).flatten(1).double()


def int4(x, codes, scales, zeros, bias, group):
    """-> (out, slack).  A group's products, of values up to 31 |x| before the
    zero point is taken off, and the sum of x times it, up to 31 |x|, are each
    summed over the group in fp32; then the groups are: (group + groups + 8)
    roundings of magnitude 62 |x| s."""
    k = 2 * codes.shape[1]
    c = unpack_codes(codes)
    s = scales.detach().cpu().double().repeat_interleave(group, 1)[:, :k]
    z = 8.0 if zeros is None else zeros.detach().cpu().double().repeat_interleave(group, 1)[:, :k]
    x64 = x.detach().cpu().double()
    out = x64 @ ((c - z) * s).t()
    slack = (group + scales.shape[1] + 8) * U32 * 62 * (x64.abs() @ s.abs().t())
    if bias is not None:
        bb = bias.detach().cpu().double()
        slack = slack + U32 * (out.abs() + bb.abs())
        out = out + bb
    return out, slack
