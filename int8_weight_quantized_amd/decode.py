"""Tensor-level entry points of the decode-step operators.

What a model served with the int8 layers runs between its projections: norm
and rotation of query and key heads with the write into a paged cache
(``qk_norm_rope``), attention of one new token per sequence over that cache
(``paged_attention``), and a projection with 4-bit weights
(``int4_pack``, ``int4_linear``).  As for the int8 layer these helpers check
their arguments, allocate outputs with torch and pass pointers and the
current stream; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import int8_weight_quantized_amd as _ck

# A decode call lasts a few microseconds on the GPU, so these helpers keep the
# host's part short: the checks are one condition over the arguments, and
# only where it does not hold does the second, slower pass go through them one
# by one to raise what is wrong.  The library's argument structures are packed
# as bytes.  (torch is imported on first use, as everywhere in this package.)

_QK = struct.Struct("10Q16qf3i")
_ATTENTION = struct.Struct("5Q11qfi")
_INT4 = struct.Struct("6Q6q2i")
_torch = None
_code16 = {}


def _load_torch():
    global _torch
    import torch
    _code16.update({torch.bfloat16: _ck.CK_DT_BF16, torch.float16: _ck.CK_DT_FP16})
    _torch = torch
    return torch


def _stream(index):
    """The current stream of CUDA device `index`."""
    return _torch._C._cuda_getCurrentRawStream(index)


def _launch(call, index, *args):
    """call(*args, stream) on CUDA device `index` and its current stream (every
    device's default stream is the null stream, which launches on the current
    device).  Host tensors, of no index, have no device to change to."""
    if index is None or index == _torch._C._cuda_getDevice():
        call(*args, _stream(index))
    else:
        with _torch.cuda.device(index):
            call(*args, _stream(index))


def _dtype16(t, name):
    """CK_DT_* of a 16-bit floating tensor."""
    torch = _torch or _load_torch()
    if isinstance(t, torch.Tensor) and t.dtype in _code16:
        return _code16[t.dtype]
    raise TypeError(f"{name} must be a bfloat16 or float16 tensor")


def _strides(t):
    """t's strides, 0 for dimensions of one element (torch leaves any value there)."""
    return tuple(s if n > 1 else 0 for n, s in zip(t.shape, t.stride()))


def _need_heads(t, dtype, name, tokens, heads, d, device):
    """A [tokens, heads, d] view with unit stride in its last dimension."""
    _ck._need(t, dtype, name, device)
    if tuple(t.shape) != (tokens, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, d)}")


class _Fixed:
    """An object that holds tensors and their addresses, made once: its
    attributes do not change, and copies are made from copies of the tensors."""

    def __setattr__(self, name, value):
        raise AttributeError(f"a {type(self).__name__} does not change: make another")

    def __delattr__(self, name):
        self.__setattr__(name, None)


class KVCache(_Fixed):
    """A paged key/value cache of one layer.

    k, v: [pages, heads, page_size, head_dim], bfloat16, float16 or int8; any
    strides with the last dimension contiguous (the same for both), so a view
    of [pages, page_size, heads, head_dim] storage is fine.  An int8 cache has
    fp32 k_scale and v_scale [pages, heads, page_size]: a row is its codes
    times its scale.  The tensors stay the caller's; the object holds them
    and their addresses, so their storage must stay (no resize_ or set_).
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if not isinstance(k, torch.Tensor) or k.dtype not in (torch.bfloat16, torch.float16, torch.int8):
            raise TypeError("k must be a bfloat16, float16 or int8 tensor")
        _ck._need(k, k.dtype, "k")
        _ck._need(v, k.dtype, "v", k.device)
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must both be [pages, heads, page_size, head_dim]")
        if _strides(v) != _strides(k):
            raise ValueError("k and v must have the same strides")
        int8 = k.dtype == torch.int8
        if int8 != (k_scale is not None) or int8 != (v_scale is not None):
            raise ValueError("an int8 cache, and no other, has k_scale and v_scale")
        if int8:
            for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
                if not isinstance(s, torch.Tensor) or s.dtype != torch.float32 or s.device != k.device:
                    raise TypeError(f"{name} must be a float32 tensor on {k.device}")
                if s.shape != k.shape[:3]:
                    raise ValueError(f"{name} has shape {tuple(s.shape)}, expected {tuple(k.shape[:3])}")
            if _strides(k_scale) != _strides(v_scale):
                raise ValueError("k_scale and v_scale must have the same strides")
        pages, heads, page_size, d = k.shape
        if page_size < 1 or page_size & (page_size - 1) or page_size > 32768:
            raise ValueError("page_size must be a power of two up to 32768")
        code = {torch.bfloat16: _ck.CK_DT_BF16, torch.float16: _ck.CK_DT_FP16, torch.int8: _ck.CK_DT_INT8}[k.dtype]
        ss = _strides(k_scale) if int8 else (0, 0, 0)
        struct_ = _ck.CkKvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if int8 else 0,
                                v_scale.data_ptr() if int8 else 0, pages, page_size, heads, d,
                                *_strides(k)[:3], *ss, code, 0)
        vars(self).update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, pages=pages, heads=heads, page_size=page_size,
                          head_dim=d, device=k.device, dtype=k.dtype, struct=struct_, address=ctypes.addressof(struct_))

    def __reduce__(self):
        return type(self), (self.k, self.v, self.k_scale, self.v_scale)

    @classmethod
    def empty(cls, pages, heads, page_size, head_dim, dtype="bf16", device="cuda"):
        """A new cache of dtype "bf16", "fp16" or "int8", zero-filled."""
        import torch
        types = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}
        if dtype not in types:
            raise ValueError(f"dtype must be 'bf16', 'fp16' or 'int8', not {dtype!r}")
        shape = (pages, heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=types[dtype], device=device) for _ in range(2))
        if dtype != "int8":
            return cls(k, v)
        return cls(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


def rope_table(rows: int, rot: int, base: float = 10000.0, device="cuda"):
    """cos and sin of position * base^(-2 i / rot) as qk_norm_rope reads them:
    fp32 [rows, rot], the cosines of the rot / 2 angles, then their sines.
    Made once per model; the angles are formed in 64 bits (an fp32 angle of
    position 131072 is off by up to 2^-8 radians)."""
    import torch
    if rows < 0 or rot < 0 or rot % 2:
        raise ValueError("rows and rot must not be negative, rot even")
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def qk_norm_rope(q, k, v, positions, cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, cache=None, slots=None, q_out=None, k_out=None):
    """RMS norm of every query and key head, the position rotation, and the
    write of keys and values into a paged cache, in one pass.

    q [tokens, hq, d], k and v [tokens, hk, d]: bf16 or fp16, views of a fused
    projection are fine.  positions int64 [tokens]; cos_sin from rope_table
    (its width is the number of elements rotated), None for no rotation.
    q_weight, k_weight fp32 [d]; None skips that norm.  interleaved rotates
    neighbouring elements together, else the halves.  With a cache, keys and
    values go to slots (int64 [tokens], page * page_size + offset, -1 for
    none); keys also go to k_out when it is given or there is no cache.
    q_out = q and k_out = k work in place.
    -> (q_out, k_out or None)."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (tokens, hq, d), qs = q.dtype, q.device, q.shape, q.stride()
        good = q.is_cuda and tt in _code16 and qs[2] == 1
        hk = kp = vp = pp = tp = sp = rot = rows = 0
        ks = vs = (0, 0)
        if k is not None:
            hk, ks, kp = k.shape[1], k.stride(), k.data_ptr()
            good = good and k.dtype is tt and k.device == dev and k.shape == (tokens, hk, d) and ks[2] == 1
        if cos_sin is not None:
            (rows, rot), pp, tp = cos_sin.shape, positions.data_ptr(), cos_sin.data_ptr()
            good = (good and cos_sin.dtype is torch.float32 and cos_sin.device == dev and cos_sin.is_contiguous()
                    and positions.dtype is torch.int64 and positions.device == dev and positions.shape == (tokens,)
                    and positions.is_contiguous())
        if cache is not None:
            vs, vp, sp = v.stride(), v.data_ptr(), slots.data_ptr()
            good = (good and kp and type(cache) is KVCache and cache.device == dev and v.dtype is tt and v.device == dev
                    and v.shape == (tokens, hk, d) and vs[2] == 1 and slots.dtype is torch.int64
                    and slots.device == dev and slots.shape == (tokens,) and slots.is_contiguous())
        qw = kw = 0
        if q_weight is not None:
            qw = q_weight.data_ptr()
            good = (good and q_weight.dtype is torch.float32 and q_weight.device == dev and q_weight.shape == (d,)
                    and q_weight.is_contiguous())
        if k_weight is not None:
            kw = k_weight.data_ptr()
            good = (good and k_weight.dtype is torch.float32 and k_weight.device == dev and k_weight.shape == (d,)
                    and k_weight.is_contiguous())
        good = good and q_out is None and k_out is None and (kp or (v is None and cache is None))
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_qk(q, k, v, positions, cos_sin, q_weight, k_weight, cache, slots, q_out, k_out)
        hk = 0 if k is None else k.shape[1]
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k_out is None and cache is None and k is not None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    os = q_out.stride()
    kop, kos = (0, vs) if k_out is None else (k_out.data_ptr(), k_out.stride())
    args = _QK.pack(q.data_ptr(), kp, vp, pp, tp, qw, kw, q_out.data_ptr(), kop, sp, qs[0], qs[1], ks[0], ks[1],
                    vs[0], vs[1], os[0], os[1], kos[0], kos[1], tokens, hq, hk, d, rot, rows, eps, _code16[tt],
                    1 if interleaved else 0, 0)
    _launch(_ck.ck_qk_norm_rope, dev.index, args, None if cache is None else cache.address)
    return q_out, k_out


def _check_qk(q, k, v, positions, cos_sin, q_weight, k_weight, cache, slots, q_out, k_out):
    """Every check of qk_norm_rope's arguments, one by one."""
    import torch
    _dtype16(q, "q")
    _ck._need(q, q.dtype, "q")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [tokens, heads, head_dim]")
    dev, tt = q.device, q.dtype
    tokens, hq, d = q.shape
    hk = 0
    if k is None:
        if v is not None or cache is not None or k_out is not None:
            raise ValueError("without k there is no v, cache or k_out")
    else:
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("k must be 3-D [tokens, heads, head_dim]")
        hk = k.shape[1]
        _need_heads(k, tt, "k", tokens, hk, d, dev)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _ck._need_vector(w, torch.float32, name, (d,), dev)
    if cos_sin is not None:
        _ck._need(cos_sin, torch.float32, "cos_sin", dev)
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous [rows, rot] tensor")
        _ck._need_vector(positions, torch.int64, "positions", (tokens,), dev)
    if cache is not None:
        if not isinstance(cache, KVCache):
            raise TypeError("cache must be a KVCache")
        if cache.device != dev:
            raise ValueError(f"the cache is on {cache.device}, q on {dev}")
        if v is None or slots is None:
            raise ValueError("a cache needs v and slots")
        _need_heads(v, tt, "v", tokens, hk, d, dev)
        _ck._need_vector(slots, torch.int64, "slots", (tokens,), dev)
    if q_out is not None:
        _need_heads(q_out, tt, "q_out", tokens, hq, d, dev)
    if k_out is not None:
        _need_heads(k_out, tt, "k_out", tokens, hk, d, dev)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(batch, hq, hk, d, width, page_size, window, sinks):
    return _ck.ck_paged_attention_workspace(batch, hq, hk, d, width, page_size, window, sinks)


def paged_attention_workspace(q, cache, table, window: int = 0, sinks: int = 0):
    """A workspace tensor for paged_attention calls of these shapes (or None
    if they need none): one per stream, kept for any number of calls."""
    n = _workspace_bytes(q.shape[0], q.shape[1], cache.heads, cache.head_dim, table.shape[1], cache.page_size,
                         window, sinks)
    if n < 0:
        raise ValueError("sizes that paged_attention does not take")
    return q.new_empty(n, dtype=(_torch or _load_torch()).uint8) if n else None


def paged_attention(q, cache, table, lens, scale=None, window: int = 0, sinks: int = 0, out=None, workspace=None):
    """Attention of one new token per sequence over a paged cache.

    q [batch, hq, d] bf16 or fp16, hq a multiple of the cache's heads; table
    int32 [batch, width], the pages of each sequence in order; lens int32
    [batch], the tokens of each, the new one included (0 gives zeros).  scale
    defaults to d ** -0.5.  With window > 0 only the last `window` and the
    first `sinks` tokens are visible.  workspace: from
    paged_attention_workspace; allocated here when None.  The work is split by
    the table's width: one much wider than the sequences need costs time (64
    sequences of 1000 tokens 48 us, in a table for 131072 580 us).
    -> [batch, hq, d]."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (batch, hq, d), qs, (rows, width) = q.dtype, q.device, q.shape, q.stride(), table.shape
        ts = table.stride()
        good = (q.is_cuda and tt in _code16 and qs[2] == 1 and type(cache) is KVCache and cache.device == dev
                and d == cache.head_dim and rows == batch and table.dtype is torch.int32 and table.device == dev
                and (ts[1] == 1 or width <= 1) and lens.dtype is torch.int32 and lens.device == dev
                and lens.shape == (batch,) and lens.is_contiguous() and out is None and workspace is None
                and window >= 0 and sinks >= 0)
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_attention(q, cache, table, lens, window, sinks, out, workspace)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = paged_attention_workspace(q, cache, table, window, sinks)
    wp, wn = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    os = out.stride()
    args = _ATTENTION.pack(q.data_ptr(), out.data_ptr(), table.data_ptr(), lens.data_ptr(), wp, wn, qs[0], qs[1],
                           os[0], os[1], ts[0], batch, hq, width, window, sinks,
                           d ** -0.5 if scale is None else scale, _code16[tt])
    _launch(_ck.ck_paged_attention, dev.index, args, cache.address)
    return out


def _check_attention(q, cache, table, lens, window, sinks, out, workspace):
    """Every check of paged_attention's arguments, one by one."""
    import torch
    _dtype16(q, "q")
    _ck._need(q, q.dtype, "q")
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    dev = q.device
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [batch, heads, head_dim] with the cache's head_dim")
    if cache.device != dev:
        raise ValueError(f"the cache is on {cache.device}, q on {dev}")
    batch, hq, d = q.shape
    _ck._need(table, torch.int32, "table", dev)
    if table.dim() != 2 or table.shape[0] != batch:
        raise ValueError("table must be [batch, pages of a sequence]")
    _ck._need_vector(lens, torch.int32, "lens", (batch,), dev)
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    if out is not None:
        _need_heads(out, q.dtype, "out", batch, hq, d, dev)
    if workspace is not None:
        _ck._need(workspace, torch.uint8, "workspace", dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")


class Int4Weight(_Fixed):
    """4-bit weights laid out for int4_linear, as int4_pack returns them: w
    uint8 [ceil(n / 16) * ceil(k / 128) * 1024], scales (of `dtype`) and zeros
    (uint8, or None) [ceil(n / 16), ceil(k / group), 16], all contiguous."""

    def __init__(self, w, scales, zeros, n, k, group, dtype):
        import torch
        if n < 0 or k < 0 or k % 8 or group not in (32, 64, 128):
            raise ValueError("n must not be negative, k a multiple of 8, group 32, 64 or 128")
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("dtype must be bfloat16 or float16")
        tiles, chunks, groups = -(-n // 16), -(-k // 128), -(-k // group)
        _ck._need_vector(w, torch.uint8, "w", (tiles * chunks * 1024,))
        for name, t, tt in (("scales", scales, dtype), ("zeros", zeros, torch.uint8)):
            if t is None and name == "zeros":
                continue
            _ck._need(t, tt, name, w.device)
            if tuple(t.shape) != (tiles, groups, 16) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {(tiles, groups, 16)} tensor")
        vars(self).update(w=w, scales=scales, zeros=zeros, n=n, k=k, group=group, dtype=dtype, device=w.device,
                          w_ptr=w.data_ptr(), s_ptr=scales.data_ptr(), z_ptr=0 if zeros is None else zeros.data_ptr())

    def __reduce__(self):
        return type(self), (self.w, self.scales, self.zeros, self.n, self.k, self.group, self.dtype)


def int4_pack(codes, scales, zeros=None, group: int = 128):
    """Lay out 4-bit weights for int4_linear, once, when they are loaded.

    codes uint8 [n, k / 2]: two codes a byte, the even column in the lower
    half.  scales bf16 or fp16 [n, ceil(k / group)] and zeros uint8 of the
    same shape (None: 8 everywhere); a weight is (code - zero) * scale.
    group 32, 64 or 128; k a multiple of 8.  -> Int4Weight."""
    import torch
    _ck._need(codes, torch.uint8, "codes")
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D [n, k / 2]")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    dev = codes.device
    n, k = codes.shape[0], 2 * codes.shape[1]
    if k % 8:
        raise ValueError("k must be a multiple of 8")
    groups = -(-k // group)
    _dtype16(scales, "scales")
    _ck._need_matrix(scales, scales.dtype, "scales", (n, groups), dev)
    if zeros is not None:
        _ck._need_matrix(zeros, torch.uint8, "zeros", (n, groups), dev)
    tiles, chunks = -(-n // 16), -(-k // 128)
    w = torch.empty(tiles * chunks * 1024, dtype=torch.uint8, device=dev)
    s = torch.empty((tiles, groups, 16), dtype=scales.dtype, device=dev)
    z = None if zeros is None else torch.empty((tiles, groups, 16), dtype=torch.uint8, device=dev)
    ldc, lds, ldz = (t.stride(0) if t is not None and n > 1 else row
                     for t, row in ((codes, k // 2), (scales, groups), (zeros, groups)))
    _launch(_ck.ck_int4_pack, dev.index, codes.data_ptr(), ldc, scales.data_ptr(), lds,
            0 if z is None else zeros.data_ptr(), ldz, w.data_ptr(), s.data_ptr(),
            0 if z is None else z.data_ptr(), n, k, group)
    return Int4Weight(w, s, z, n, k, group, scales.dtype)


def int4_linear(x, weight, bias=None, out=None, out_dtype=None):
    """bf16 or fp16 x [m, k] times the 4-bit weight [n, k] (of int4_pack,
    with scales of x's type) -> [m, n] of out_dtype ("bf16", "fp16" or "fp32";
    x's type when None).  bias [n] has the output's type.  x must be finite: a
    row with an infinity gives NaN in every column."""
    torch = _torch or _load_torch()
    try:
        tt, dev, (m, k), xs = x.dtype, x.device, x.shape, x.stride()
        good = (x.is_cuda and type(weight) is Int4Weight and tt is weight.dtype and dev == weight.device
                and k == weight.k and (xs[1] == 1 or k <= 1) and out is None and out_dtype is None)
        n = weight.n
        if bias is not None:
            good = (good and bias.dtype is tt and bias.device == dev and bias.shape == (n,) and bias.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        code, odt = _check_int4(x, weight, bias, out, out_dtype)
    else:
        code, odt = _code16[tt], tt          # the out codes of the two types are the same
    if out is None:
        out = x.new_empty((m, n), dtype=odt)
    args = _INT4.pack(x.data_ptr(), weight.w_ptr, weight.s_ptr, weight.z_ptr, 0 if bias is None else bias.data_ptr(),
                      out.data_ptr(), xs[0], out.stride(0), m, n, k, weight.group, _code16[tt], code)
    _launch(_ck.ck_int4_linear, dev.index, args)
    return out


def _check_int4(x, weight, bias, out, out_dtype):
    """Every check of int4_linear's arguments, one by one; the output type."""
    if not isinstance(weight, Int4Weight):
        raise TypeError("weight must be an Int4Weight (see int4_pack)")
    dt = _dtype16(x, "x")
    _ck._need(x, weight.dtype, "x", weight.device)
    code, tdt = _ck._out_dtype(("bf16", "fp16")[dt] if out_dtype is None else out_dtype)
    if x.dim() != 2 or x.shape[1] != weight.k:
        raise ValueError(f"x must be [m, {weight.k}]")
    if bias is not None:
        _ck._need_vector(bias, tdt, "bias", (weight.n,), x.device)
    if out is not None:
        _ck._need_matrix(out, tdt, "out", (x.shape[0], weight.n), x.device)
    return code, tdt
