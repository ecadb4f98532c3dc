"""Plain references of the operators of a server's batch in 64 bits, and the
error bounds that their fp32 arithmetic allows.  Everything here runs on the CPU."""
import math

import torch

from tests.decode_ref import HALF, TINY, TYPES, U32, assert_within  # noqa: F401


def shared_prefix(q, cache, prefix_table, prefix_lens, starts, table, lens, scale):
    """-> (out, slack) of one new token per sequence over its prefix's tokens and its own.

    Scores: d products and sums, the scales and the change to base 2 are off by at most (d + 6) u times
    S = scale sum |q_i k_i|; the exponential turns that into a relative error of each weight (and of the sum),
    its own rounding adds 4 u.  The weights enter the value product in 16-bit parts, which leave at most
    2^-17 of each (two parts of bf16, the coarser type: 2^-9 of 2^-9, doubled).  Sums over n tokens: n u.
    All of it is relative to sum p |v|, and counts twice (numerator and denominator)."""
    kc, vc = cache.k.detach().cpu(), cache.v.detach().cpu()
    ks, vs = (None if t is None else t.detach().cpu().double() for t in (cache.k_scale, cache.v_scale))
    q = q.detach().cpu()
    prefix_table, table = prefix_table.cpu().long(), table.cpu().long()
    prefix_lens, starts, lens = prefix_lens.cpu().tolist(), starts.cpu().tolist(), lens.cpu().tolist()
    b, hq, d = q.shape
    pages, hk, page = kc.shape[:3]
    g = hq // hk
    out, slack = torch.zeros((b, hq, d), dtype=torch.float64), torch.zeros((b, hq, d), dtype=torch.float64)
    for i in range(b):
        spans = [(prefix_table[p], prefix_lens[p]) for p in range(len(prefix_lens)) if starts[p] <= i < starts[p + 1]]
        at, pg = [], []
        for tab, n in spans + [(table[i], lens[i])]:
            a = torch.arange(max(0, min(n, tab.shape[0] * page)))
            pg.append(tab[a // page])
            at.append(a % page)
        at, pg = torch.cat(at), torch.cat(pg)
        if not len(at):
            continue
        if ((pg < 0) | (pg >= pages)).any():
            out[i] = math.nan
            continue
        for h in range(hk):
            k, v = kc[pg, h, at].double(), vc[pg, h, at].double()
            if ks is not None:
                k, v = k * ks[pg, h, at][:, None], v * vs[pg, h, at][:, None]
            qq = q[i, h * g:(h + 1) * g].double()
            p = torch.softmax(qq @ k.t() * scale, -1)
            out[i, h * g:(h + 1) * g] = p @ v
            s = (qq.abs() @ k.abs().t()).amax(-1, keepdim=True) * abs(scale)
            slack[i, h * g:(h + 1) * g] = 2 * ((d + 6) * U32 * s + 2.0 ** -17 + (len(at) + 4) * U32) * (p @ v.abs())
    return out, slack


def lora(y, x, a, b, scale, ids):
    """-> (out, slack).  v: k products and sums, off by at most (k + 2) u sum |x a|.  v enters the second product in
    16-bit parts that leave at most 2^-17 of it, and rank products and sums follow: (rank + 4) u, with the scale."""
    y, x, a, b = (t.detach().cpu().double() for t in (y, x, a, b))
    out, slack = y.clone(), torch.zeros_like(y)
    k, rank = a.shape[2], a.shape[1]
    for i, t in enumerate(ids.cpu().tolist()):
        if 0 <= t < a.shape[0]:
            s = 1.0 if scale is None else scale[t].item()
            out[i] += s * ((x[i] @ a[t].t()) @ b[t].t())
            size = abs(s) * ((x[i].abs() @ a[t].abs().t()) @ b[t].abs().t())
            slack[i] = ((k + rank + 8) * U32 + 2.0 ** -17) * size + U32 * (out[i].abs() + size)
    return out, slack


def order(x):
    """Indices of each row in the order of the alternatives: descending, NaN first, of equal ones the lowest index first."""
    v = x.double() + 0.0
    return torch.sort(torch.where(v.isnan(), math.inf, v), dim=1, descending=True, stable=True).indices \
        if not (v.isnan().any() and (v == math.inf).any()) else torch.argsort(-_ranked(v), dim=1, stable=True)


def _ranked(v):
    """Ranks that keep NaN above infinity."""
    keys = torch.where(v.isnan(), math.inf, v)
    _, inv = torch.unique(keys, return_inverse=True)
    return inv.double() + v.isnan().double()


def logprobs(x, tokens, top):
    """-> dict of (value, slack) by name, and ids.

    A term e^t, t = x_j - max <= 0: the difference, its change to base 2 and the exponential are off by at most
    (2 |t| + 3) u of the term; the sum of n terms in partial sums of at most n / 256 + 32 additions by that many u.
    So the log is off by E = u (sum p (2 |t| + 3) + n / 256 + 32), a log probability by E + u (2 |logprob|),
    and the entropy, log S - sum e t / S, by E (1 + sum p |t|) and the terms' own errors."""
    x = x.detach().cpu().double()
    n = x.shape[1]
    high = x.amax(1, keepdim=True)
    t = x - high
    e = torch.exp(t)
    s = e.sum(1, keepdim=True)
    p = e / s
    pt = torch.where(e > 0, p * t, 0.0)
    at = pt.abs().sum(1)
    err = U32 * (2 * at + 3 + n / 256 + 32)
    entropy = s.log()[:, 0] - pt.sum(1)
    out = dict(entropy=(entropy, (err * (1 + at) + U32 * 4 * (at + entropy.abs()) + 2 * U32 * torch.where(e > 0, p * t * t, 0.0).sum(1))))
    if tokens is not None:
        tok = tokens.cpu()
        ok = (tok >= 0) & (tok < n)
        lp = torch.where(ok, (t - s.log()).gather(1, tok.clamp(0, n - 1)[:, None])[:, 0], math.nan)
        out["logprob"] = (lp, err + 2 * U32 * torch.where(lp.isfinite(), lp.abs(), 0.0))
    ids = order(x)[:, :top]
    lt = (t - s.log()).gather(1, ids)          # in this order: the largest logit may be too large to add log S to
    out["top"] = (lt, err[:, None] + 2 * U32 * torch.where(lt.isfinite(), lt.abs(), 0.0))
    return out, ids
