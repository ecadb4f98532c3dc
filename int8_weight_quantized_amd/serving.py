"""Tensor-level entry points of the operators of a server's batch.

What a step of many requests at once needs beside the int8 layers and the
decode-step operators: attention over prefixes that groups of sequences share
(``shared_prefix_attention``), low-rank adapters that differ from row to row
(``LoraWeight``, ``lora_add``), and the log probabilities of what was chosen
(``token_logprobs``).  As for the others these helpers check their arguments,
allocate outputs with torch and pass pointers and the current stream; every
step runs in the library's HIP kernels.  (How the checks are kept short is
told in decode.py.)
"""
from __future__ import annotations

import collections
import functools
import struct

import int8_weight_quantized_amd as _ck
from . import decode as _decode

_PREFIX = struct.Struct("8Q12qfi")
_LORA = struct.Struct("8Q11q2i")
_LOGPROB = struct.Struct("7Q5q2i")
_torch = None
_code = {}                               # ck_out_dtype of a tensor's type


def _load_torch():
    global _torch
    torch = _decode._torch or _decode._load_torch()
    _code.update({torch.bfloat16: _ck.CK_OUT_BF16, torch.float16: _ck.CK_OUT_FP16, torch.float32: _ck.CK_OUT_FP32})
    _torch = torch
    return torch


def _workspace(n, like, what):
    """n bytes on like's device, None for 0."""
    if n < 0:
        raise ValueError(f"sizes that {what} does not take")
    return like.new_empty(n, dtype=(_torch or _load_torch()).uint8) if n else None


def _fine(workspace, device):
    """Whether workspace is None or a tensor as they have to be."""
    return workspace is None or (workspace.dtype is _torch.uint8 and workspace.device == device
                                 and workspace.is_contiguous())


def _need_workspace(workspace, device):
    _ck._need(workspace, (_torch or _load_torch()).uint8, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


# ---------------------------------------------------- shared_prefix_attention

@functools.lru_cache(maxsize=256)
def _prefix_bytes(batch, hq, hk, d, prefixes, prefix_width, width, page_size):
    return _ck.ck_shared_prefix_attention_workspace(batch, hq, hk, d, prefixes, prefix_width, width, page_size)


def shared_prefix_attention_workspace(q, cache, prefix_table, table):
    """A workspace tensor for shared_prefix_attention calls of these shapes
    (or None if they need none): one per stream, kept for any number of calls."""
    n = _prefix_bytes(q.shape[0], q.shape[1], cache.heads, cache.head_dim, prefix_table.shape[0], prefix_table.shape[1],
                      table.shape[1], cache.page_size)
    return _workspace(n, q, "shared_prefix_attention")


def shared_prefix_attention(q, cache, prefix_table, prefix_lens, starts, table, lens, scale=None, out=None,
                            workspace=None):
    """Attention of one new token per sequence over a paged cache, where groups
    of sequences begin with the same tokens: a prefix, whose keys and values
    are in the cache once and are read once for its group.

    q [batch, hq, d] and cache as for paged_attention.  prefix_table int32
    [prefixes, width], the pages of each prefix in order; prefix_lens int32
    [prefixes], its tokens (any number: the last page may be part full).
    starts int32 [prefixes + 1]: sequences starts[p] to starts[p + 1] - 1
    begin with prefix p, those before starts[0] and from starts[-1] on have
    none; the entries must not decrease (every output is NaN where they do).
    table int32 [batch, width] and lens int32 [batch]: each sequence's own
    tokens after the prefix, the new one included.  scale defaults to
    d ** -0.5.  workspace: from shared_prefix_attention_workspace; allocated
    here when None.  -> [batch, hq, d]."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (batch, hq, d), qs, (rows, width) = q.dtype, q.device, q.shape, q.stride(), table.shape
        ts, (prefixes, pwidth), ps = table.stride(), prefix_table.shape, prefix_table.stride()
        i32 = torch.int32
        good = (q.is_cuda and tt in _decode._code16 and qs[2] == 1 and type(cache) is _decode.KVCache
                and cache.device == dev and d == cache.head_dim and rows == batch and table.dtype is i32
                and table.device == dev and (ts[1] == 1 or width <= 1) and lens.dtype is i32 and lens.device == dev
                and lens.shape == (batch,) and lens.is_contiguous() and prefix_table.dtype is i32
                and prefix_table.device == dev and (ps[1] == 1 or pwidth <= 1) and prefix_lens.dtype is i32
                and prefix_lens.device == dev and prefix_lens.shape == (prefixes,) and prefix_lens.is_contiguous()
                and starts.dtype is i32 and starts.device == dev and starts.shape == (prefixes + 1,)
                and starts.is_contiguous() and out is None and _fine(workspace, dev))
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_prefix(q, cache, prefix_table, prefix_lens, starts, table, lens, out, workspace)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = shared_prefix_attention_workspace(q, cache, prefix_table, table)
    wp, wn = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    os = out.stride()
    args = _PREFIX.pack(q.data_ptr(), out.data_ptr(), prefix_table.data_ptr(), prefix_lens.data_ptr(), starts.data_ptr(),
                        table.data_ptr(), lens.data_ptr(), wp, wn, qs[0], qs[1], os[0], os[1], ps[0], ts[0], batch, hq,
                        prefixes, pwidth, width, d ** -0.5 if scale is None else scale, _decode._code16[tt])
    _decode._launch(_ck.ck_shared_prefix_attention, dev.index, args, cache.address)
    return out


def _check_prefix(q, cache, prefix_table, prefix_lens, starts, table, lens, out, workspace):
    """Every check of shared_prefix_attention's arguments, one by one."""
    torch = _torch or _load_torch()
    _decode._check_attention(q, cache, table, lens, 0, 0, out, workspace)
    _ck._need(prefix_table, torch.int32, "prefix_table", q.device)
    if prefix_table.dim() != 2:
        raise ValueError("prefix_table must be [prefixes, pages of a prefix]")
    prefixes = prefix_table.shape[0]
    _ck._need_vector(prefix_lens, torch.int32, "prefix_lens", (prefixes,), q.device)
    _ck._need_vector(starts, torch.int32, "starts", (prefixes + 1,), q.device)


# -------------------------------------------------------------------- lora_add

class LoraWeight(_decode._Fixed):
    """The low-rank adapters of one projection, for lora_add.

    a [adapters, rank, k] and b [adapters, n, rank], bfloat16 or float16, each
    adapter's part contiguous; scale float32 [adapters] or None for 1.  rank
    is a multiple of 8 from 8 to 256 (an adapter of smaller rank is filled up
    with zeros), k a multiple of 8.  The tensors stay the caller's, who may
    write another adapter into a place; the object holds them and their
    addresses, so their storage must stay (no resize_ or set_)."""

    def __init__(self, a, b, scale=None):
        import torch
        dt = _decode._dtype16(a, "a")
        _ck._need(a, a.dtype, "a")
        _ck._need(b, a.dtype, "b", a.device)
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [adapters, rank, k] and b [adapters, n, rank]")
        adapters, rank, k = a.shape
        n = b.shape[1]
        if rank < 8 or rank > 256 or rank % 8 or k % 8:
            raise ValueError("rank must be a multiple of 8 from 8 to 256, k a multiple of 8")
        for name, t in (("a", a), ("b", b)):
            if adapters and not t[0].is_contiguous():
                raise ValueError(f"each adapter's part of {name} must be contiguous")
        if scale is not None:
            _ck._need_vector(scale, torch.float32, "scale", (adapters,), a.device)
        vars(self).update(a=a, b=b, scale=scale, adapters=adapters, rank=rank, k=k, n=n, dtype=a.dtype, device=a.device,
                          code=dt, a_ptr=a.data_ptr(), b_ptr=b.data_ptr(), a_stride=a.stride(0), b_stride=b.stride(0),
                          s_ptr=0 if scale is None else scale.data_ptr())

    def __reduce__(self):
        return type(self), (self.a, self.b, self.scale)


@functools.lru_cache(maxsize=256)
def _lora_bytes(m, n, k, rank):
    return _ck.ck_lora_add_workspace(m, n, k, rank)


def lora_add_workspace(x, weight):
    """A workspace tensor for lora_add calls of these shapes (or None if they
    need none): one per stream, kept for any number of calls."""
    return _workspace(_lora_bytes(x.shape[0], weight.n, weight.k, weight.rank), x, "lora_add")


def lora_add(y, x, weight, ids, out=None, workspace=None):
    """y + scale (x A^T) B^T with the adapter that each row asks for.

    y [m, n], what a shared projection made of x: bf16, fp16 or fp32 (one
    rounding).  x [m, k] of the adapters' type; ids int32 [m], the adapter of
    each row, in any order; -1 (or any number outside the adapters) leaves
    the row as it is.  out: y itself to work in place, but not x, whose rows
    are read while others are written.  workspace: from lora_add_workspace;
    allocated here when None.  -> [m, n]."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (m, n), ys, (rows, k), xs = y.dtype, y.device, y.shape, y.stride(), x.shape, x.stride()
        good = (y.is_cuda and tt in _code and (ys[1] == 1 or n <= 1) and type(weight) is LoraWeight
                and weight.device == dev and x.dtype is weight.dtype and x.device == dev and rows == m and n == weight.n
                and k == weight.k and (xs[1] == 1 or k <= 1) and ids.dtype is torch.int32 and ids.device == dev
                and ids.shape == (m,) and ids.is_contiguous() and (out is None or out is y) and _fine(workspace, dev))
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_lora(y, x, weight, ids, out, workspace)
    if out is None:
        out = torch.empty_like(y, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = lora_add_workspace(x, weight)
    wp, wn = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    xp, op = x.data_ptr(), out.data_ptr()
    if xp == op and m and n and k:
        raise ValueError("out must not be x")
    args = _LORA.pack(xp, weight.a_ptr, weight.b_ptr, weight.s_ptr, ids.data_ptr(), y.data_ptr(),
                      op, wp, wn, xs[0], ys[0], out.stride(0), weight.a_stride, weight.b_stride, m, n, k,
                      weight.rank, weight.adapters, weight.code, _code[tt])
    _decode._launch(_ck.ck_lora_add, dev.index, args)
    return out


def _check_lora(y, x, weight, ids, out, workspace):
    """Every check of lora_add's arguments, one by one."""
    torch = _torch or _load_torch()
    if not isinstance(weight, LoraWeight):
        raise TypeError("weight must be a LoraWeight")
    if not isinstance(y, torch.Tensor) or y.dtype not in _code:
        raise TypeError("y must be a bfloat16, float16 or float32 tensor")
    _ck._need(y, y.dtype, "y", weight.device)
    if y.dim() != 2 or y.shape[1] != weight.n:
        raise ValueError(f"y must be [m, {weight.n}]")
    m = y.shape[0]
    _ck._need_matrix(x, weight.dtype, "x", (m, weight.k), weight.device)
    _ck._need_vector(ids, torch.int32, "ids", (m,), weight.device)
    if out is not None:
        _ck._need_matrix(out, y.dtype, "out", (m, weight.n), weight.device)
    if workspace is not None:
        _need_workspace(workspace, weight.device)


# -------------------------------------------------------------- token_logprobs

TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprob entropy top_ids top_logprobs")


@functools.lru_cache(maxsize=256)
def _logprob_bytes(rows, vocab, top):
    return _ck.ck_token_logprobs_workspace(rows, vocab, top)


def token_logprobs_workspace(logits, top: int = 0):
    """A workspace tensor for token_logprobs calls of these shapes (or None if
    they need none): one per stream, kept for any number of calls."""
    return _workspace(_logprob_bytes(logits.shape[0], logits.shape[1], top), logits, "token_logprobs")


def token_logprobs(logits, tokens=None, top: int = 0, workspace=None):
    """Log probabilities of given tokens, the entropy of each row and its most
    likely tokens, in one pass over the logits.

    logits [rows, vocab] bf16, fp16 or fp32, -inf for what is masked; tokens
    int64 [rows] (a token outside the vocabulary, -1 say, gives NaN) or None;
    top from 0 to 64.  workspace: from token_logprobs_workspace; allocated
    here when None.  -> TokenLogprobs(logprob [rows] or None, entropy [rows],
    top_ids int64 [rows, top], top_logprobs [rows, top]); of equal logits the
    lowest index comes first."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (rows, vocab), ls = logits.dtype, logits.device, logits.shape, logits.stride()
        good = logits.is_cuda and tt in _code and (ls[1] == 1 or vocab <= 1) and _fine(workspace, dev) and top >= 0
        if tokens is not None:
            good = (good and tokens.dtype is torch.int64 and tokens.device == dev and tokens.shape == (rows,)
                    and tokens.is_contiguous())
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_logprobs(logits, tokens, top, workspace)
    if workspace is None:
        workspace = token_logprobs_workspace(logits, top)
    wp, wn = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    f32 = torch.float32
    logprob = None if tokens is None else logits.new_empty(rows, dtype=f32)
    entropy = logits.new_empty(rows, dtype=f32)
    ids = logits.new_empty((rows, top), dtype=torch.int64)
    best = logits.new_empty((rows, top), dtype=f32)
    args = _LOGPROB.pack(logits.data_ptr(), 0 if tokens is None else tokens.data_ptr(),
                         0 if tokens is None else logprob.data_ptr(), entropy.data_ptr(), ids.data_ptr(),
                         best.data_ptr(), wp, wn, ls[0], rows, vocab, top, _code[tt], 0)
    _decode._launch(_ck.ck_token_logprobs, dev.index, args)
    return TokenLogprobs(logprob, entropy, ids, best)


def _check_logprobs(logits, tokens, top, workspace):
    """Every check of token_logprobs' arguments, one by one."""
    torch = _torch or _load_torch()
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _code:
        raise TypeError("logits must be a bfloat16, float16 or float32 tensor")
    _ck._need(logits, logits.dtype, "logits")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be 2-D [rows, vocab]")
    if top < 0 or top > 64 or top > logits.shape[1]:
        raise ValueError("top must be from 0 to 64, and not more than the vocabulary")
    if tokens is not None:
        _ck._need_vector(tokens, torch.int64, "tokens", (logits.shape[0],), logits.device)
    if workspace is not None:
        _need_workspace(workspace, logits.device)
