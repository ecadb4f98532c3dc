"""The decode-step operators on the host: the C entry points and the binding
refuse bad arguments before any HIP call (no GPU needed)."""
import ctypes
import re

import pytest
import torch

import int8_weight_quantized_amd as ck
from tests.test_abi import HEADER

P = 4096          # a stand-in device address: validation never dereferences it
BAD, UNS, OK, HIP = ck.CK_ERR_INVALID_ARG, ck.CK_ERR_UNSUPPORTED, ck.CK_OK, ck.CK_ERR_HIP


def no_gpu(status):
    if status == HIP and torch.cuda.is_available():
        pytest.skip("needs the no-GPU host")


def cache(**kw):
    a = dict(k=P, v=P, k_scale=0, v_scale=0, pages=10, page_size=16, heads=2, head_dim=128, page_stride=4096,
             head_stride=2048, token_stride=128, dtype=ck.CK_DT_BF16)
    a.update(kw)
    return ck.CkKvCache(**a)


CACHES = [
    (dict(), HIP),
    (dict(dtype=ck.CK_DT_FP16), BAD),                # not q's type
    (dict(dtype=7), BAD),
    (dict(dtype=ck.CK_DT_INT8), BAD),                # no scales
    (dict(dtype=ck.CK_DT_INT8, k_scale=P, v_scale=P), HIP),
    (dict(dtype=ck.CK_DT_INT8, k_scale=P + 2, v_scale=P), UNS),
    (dict(k=0), BAD),
    (dict(v=0), BAD),
    (dict(pages=-1), BAD),
    (dict(pages=1 << 31), UNS),
    (dict(heads=0), BAD),
    (dict(page_size=0), BAD),
    (dict(page_size=24), BAD),
    (dict(page_size=65536), BAD),
    (dict(head_dim=64), BAD),
    (dict(token_stride=120), BAD),
    (dict(page_stride=-4096), BAD),
    (dict(k=P + 8), UNS),
    (dict(token_stride=132), UNS),
    (dict(head_stride=2052), UNS),
    (dict(page_stride=4100), UNS),
]


def qk_args(**kw):
    a = dict(q=P, k=P, v=P, positions=P, cos_sin=P, q_weight=P, k_weight=P, q_out=P, k_out=0, slots=P,
             q_token_stride=1024, q_head_stride=128, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, q_out_token_stride=1024, q_out_head_stride=128, k_out_token_stride=256,
             k_out_head_stride=128, tokens=4, hq=8, hk=2, head_dim=128, rot=128, table_rows=100, eps=1e-6,
             dtype=ck.CK_DT_BF16)
    a.update(kw)
    return ck.CkQkArgs(**a)


def call_qk(a, c):
    return ck.lib().ck_qk_norm_rope(ctypes.byref(a), None if c is None else ctypes.byref(c), 0)


@pytest.mark.parametrize("kw,status", CACHES)
def test_rope_cache_validation(kw, status):
    no_gpu(status)
    assert call_qk(qk_args(), cache(**kw)) == status
    assert status == OK or ck.ck_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP),
    (dict(dtype=2), BAD),
    (dict(tokens=-1), BAD),
    (dict(tokens=0), OK),
    (dict(tokens=0, q=0, q_out=0), OK),
    (dict(q=0), BAD),
    (dict(q_out=0), BAD),
    (dict(k=0), BAD),
    (dict(v=0), BAD),
    (dict(slots=0), BAD),
    (dict(positions=0), BAD),
    (dict(cos_sin=0), BAD),
    (dict(table_rows=0), BAD),
    (dict(rot=0, positions=0, cos_sin=0), HIP),
    (dict(rot=24), UNS),
    (dict(rot=144), BAD),
    (dict(head_dim=132), UNS),
    (dict(head_dim=520), UNS),
    (dict(hk=3), BAD),                       # the cache has two heads
    (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD),
    (dict(q=P + 2), UNS),
    (dict(q_token_stride=1028), UNS),
    (dict(q_out_head_stride=132), UNS),
    (dict(k_head_stride=129), UNS),
    (dict(k_out=P + 4), UNS),
    (dict(v_token_stride=257), UNS),
    (dict(q_weight=P + 4), UNS),
    (dict(positions=P + 4), UNS),
    (dict(q_weight=0, k_weight=0), HIP),
    (dict(tokens=1 << 42), UNS),
    (dict(tokens=1, q_token_stride=3, k_token_stride=3, v_token_stride=3, q_out_token_stride=3), HIP),
])
def test_rope_validation(kw, status):
    no_gpu(status)
    assert call_qk(qk_args(**kw), cache()) == status


def test_rope_without_a_cache():
    assert call_qk(qk_args(v=0, slots=0), None) == BAD                      # no place for the keys
    assert ck.lib().ck_qk_norm_rope(None, None, 0) == BAD
    if not torch.cuda.is_available():
        assert call_qk(qk_args(v=0, slots=0, k_out=P), None) == HIP
        assert call_qk(qk_args(v=0, slots=0, k=0, hk=0), None) == HIP       # queries alone


def attn_args(**kw):
    a = dict(q=P, out=P, table=P, lens=P, workspace=P, workspace_bytes=1 << 40, q_batch_stride=1024, q_head_stride=128,
             out_batch_stride=1024, out_head_stride=128, table_stride=63, batch=3, hq=8, table_width=63, window=0,
             sinks=0, scale=0.1, dtype=ck.CK_DT_BF16)
    a.update(kw)
    return ck.CkAttentionArgs(**a)


@pytest.mark.parametrize("kw,status", CACHES)
def test_attention_cache_validation(kw, status):
    no_gpu(status)
    if "head_dim" in kw:
        pytest.skip("the cache's head_dim is q's here")
    assert ck.lib().ck_paged_attention(ctypes.byref(attn_args()), ctypes.byref(cache(**kw)), 0) == status


@pytest.mark.parametrize("kw,ckw,status", [
    (dict(), dict(), HIP),
    (dict(dtype=2), dict(), BAD),
    (dict(batch=-1), dict(), BAD),
    (dict(batch=0), dict(), OK),
    (dict(hq=0), dict(), OK),
    (dict(hq=7), dict(), BAD),
    (dict(window=-1), dict(), BAD),
    (dict(sinks=-1), dict(), BAD),
    (dict(table_width=-1), dict(), BAD),
    (dict(q=0), dict(), BAD),
    (dict(out=0), dict(), BAD),
    (dict(lens=0), dict(), BAD),
    (dict(table=0), dict(), BAD),
    (dict(table=0, table_width=0), dict(), HIP),
    (dict(table_stride=62), dict(), BAD),
    (dict(table_stride=0, batch=1), dict(), HIP),
    (dict(q=P + 2), dict(), UNS),
    (dict(q_head_stride=129), dict(), UNS),
    (dict(out_batch_stride=1025), dict(), UNS),
    (dict(lens=P + 2), dict(), UNS),
    (dict(scale=float("nan")), dict(), BAD),
    (dict(batch=(1 << 20) + 1), dict(), UNS),
    (dict(table_width=1 << 31, table_stride=1 << 31), dict(), UNS),
    (dict(), dict(head_dim=80, token_stride=80), UNS),
    (dict(), dict(head_dim=512, token_stride=512), UNS),
    (dict(), dict(dtype=ck.CK_DT_INT8, k_scale=P, v_scale=P, k=P + 8), UNS),     # int8 rows 16 bytes apart here
])
def test_attention_validation(kw, ckw, status):
    no_gpu(status)
    assert ck.lib().ck_paged_attention(ctypes.byref(attn_args(**kw)), ctypes.byref(cache(**ckw)), 0) == status


def test_attention_workspace():
    L = ck.lib()
    a, c = attn_args(batch=2, table_width=4096, table_stride=4096), cache()
    need = ck.ck_paged_attention_workspace(2, 8, 2, 128, 4096, 16, 0, 0)
    assert need > 0
    for kw, status in ((dict(workspace=0), BAD), (dict(workspace_bytes=need - 1), BAD), (dict(workspace=P + 16), UNS)):
        b = attn_args(batch=2, table_width=4096, table_stride=4096, **kw)
        assert L.ck_paged_attention(ctypes.byref(b), ctypes.byref(c), 0) == status
    if not torch.cuda.is_available():
        a.workspace_bytes = need
        assert L.ck_paged_attention(ctypes.byref(a), ctypes.byref(c), 0) == HIP
    # never more for a window than for the whole length; refused sizes
    assert 0 <= ck.ck_paged_attention_workspace(2, 8, 2, 128, 4096, 16, 1000, 4) <= need
    for bad in ((-1, 8, 2, 128, 4, 16), (2, 7, 2, 128, 4, 16), (2, 8, 0, 128, 4, 16), (2, 8, 2, 100, 4, 16),
                (2, 8, 2, 128, -4, 16), (2, 8, 2, 128, 4, 12), (2, 8, 2, 128, 4, 16, -1), (2, 8, 2, 128, 4, 16, 1, -1)):
        assert ck.ck_paged_attention_workspace(*bad) == -1


FAR = 1 << 62


@pytest.mark.parametrize("kw,status", [
    # the stride of a dimension with one element is not looked at
    (dict(pages=1, page_stride=FAR), HIP),
    (dict(pages=1, page_stride=-4096), HIP),
    (dict(heads=1, head_stride=-8), HIP),
    (dict(page_size=1, token_stride=-1), HIP),
    (dict(pages=1, page_stride=-8, dtype=ck.CK_DT_INT8, k_scale=P, v_scale=P, scale_page_stride=-1), HIP),
    # others may not leave 64 bits
    (dict(pages=3, page_stride=FAR), UNS),
    (dict(heads=2, head_stride=FAR), UNS),
    (dict(pages=(1 << 31) - 1, page_stride=1 << 40), UNS),
    (dict(dtype=ck.CK_DT_INT8, k_scale=P, v_scale=P, scale_page_stride=FAR), UNS),
    (dict(page_stride=-4096), BAD),
    (dict(head_stride=-2048), BAD),
    (dict(dtype=ck.CK_DT_INT8, k_scale=P, v_scale=P, scale_token_stride=-1), BAD),
])
def test_cache_strides(kw, status):
    no_gpu(status)
    c, hk = cache(**kw), kw.get("heads", 2)
    assert call_qk(qk_args(hk=hk, hq=8), c) == status
    assert ck.lib().ck_paged_attention(ctypes.byref(attn_args()), ctypes.byref(c), 0) == status


def test_cache_of_64_gib():
    """Attention's row offsets are 32 bits of 16-byte units: a cache up to 64 GiB, to the byte."""
    no_gpu(HIP)
    pages = (1 << 36) // (2 * 4096)
    for n, status in ((pages, HIP), (pages + 1, UNS)):
        assert ck.lib().ck_paged_attention(ctypes.byref(attn_args()), ctypes.byref(cache(pages=n)), 0) == status


@pytest.mark.parametrize("batch,hq,hk,width,page", [
    (1 << 20, 65536, 65536, 1 << 25, 32768),     # the workspace's bytes and the blocks pass 64 bits
    (1 << 20, 65536, 1, 1 << 25, 32768),
    (1 << 16, 1024, 1024, 1 << 12, 1024),        # 2^38 blocks
    (1 << 20, 4096, 1, 1, 16),                   # 2^32 rows of the output
])
def test_attention_refuses_what_no_launch_holds(batch, hq, hk, width, page):
    assert ck.ck_paged_attention_workspace(batch, hq, hk, 128, width, page, 0, 0) == -1
    a = attn_args(batch=batch, hq=hq, table_width=width, table_stride=width, workspace=0, workspace_bytes=0)
    c = cache(heads=hk, page_size=page, head_stride=128, token_stride=128, page_stride=128)
    assert ck.lib().ck_paged_attention(ctypes.byref(a), ctypes.byref(c), 0) == UNS


def test_rows_that_are_written_lie_apart():
    """Outputs and caches whose rows overlap (expanded tensors) are refused where they are written;
    heads before tokens is fine, and so is an expanded input, or a cache that is only read."""
    no_gpu(HIP)
    for kw, ckw, status in [
        (dict(q_out_token_stride=128, q_out_head_stride=512), {}, HIP),
        (dict(q_out_token_stride=0), {}, BAD),
        (dict(q_out_head_stride=0), {}, BAD),
        (dict(q_out_head_stride=64), {}, BAD),
        (dict(q_out_token_stride=1016), {}, BAD),
        (dict(tokens=1, q_out_token_stride=0), {}, HIP),
        (dict(k_out=P, k_out_head_stride=0), {}, BAD),
        (dict(k_out=P), {}, HIP),
        (dict(q_token_stride=0, k_head_stride=0, v_head_stride=0), {}, HIP),
        (dict(), dict(head_stride=0), BAD),
        (dict(), dict(page_stride=4088), BAD),
        (dict(), dict(head_stride=128, token_stride=256), HIP),
    ]:
        assert call_qk(qk_args(**kw), cache(**ckw)) == status, (kw, ckw)
    for kw, ckw, status in [
        (dict(out_batch_stride=0), {}, BAD),
        (dict(out_head_stride=120), {}, BAD),
        (dict(out_batch_stride=128, out_head_stride=384), {}, HIP),
        (dict(batch=1, out_batch_stride=0), {}, HIP),
        (dict(q_batch_stride=0, q_head_stride=0), {}, HIP),
        (dict(), dict(head_stride=0), HIP),
    ]:
        assert ck.lib().ck_paged_attention(ctypes.byref(attn_args(**kw)), ctypes.byref(cache(**ckw)), 0) == status, (kw, ckw)


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP),
    (dict(n=0, codes=0, w=0), OK),
    (dict(n=-1), BAD),
    (dict(k=-8), BAD),
    (dict(group=48), UNS),
    (dict(k=132), UNS),
    (dict(codes=0), BAD),
    (dict(scales=0), BAD),
    (dict(w=0), BAD),
    (dict(w_scale=0), BAD),
    (dict(zeros=P), BAD),                    # zeros without w_zero
    (dict(w_zero=P), BAD),
    (dict(zeros=P, ldz=4, w_zero=P), HIP),
    (dict(zeros=P, ldz=3, w_zero=P), BAD),
    (dict(ldc=255), BAD),
    (dict(lds=3), BAD),
    (dict(w=P + 8), UNS),
    (dict(w_scale=P + 8), UNS),
    (dict(scales=P + 1), UNS),
    (dict(n=1 << 31), UNS),
])
def test_int4_pack_validation(kw, status):
    no_gpu(status)
    a = dict(codes=P, ldc=256, scales=P, lds=4, zeros=0, ldz=0, w=P, w_scale=P, w_zero=0, n=64, k=512, group=128)
    a.update(kw)
    assert ck.lib().ck_int4_pack(*a.values(), 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP),
    (dict(m=0, x=0, out=0), OK),
    (dict(n=0, out=0), OK),
    (dict(m=-1), BAD),
    (dict(n=-1), BAD),
    (dict(dtype=2), BAD),
    (dict(out_dtype=3), BAD),
    (dict(group=16), UNS),
    (dict(k=508, ldx=512), UNS),
    (dict(x=0), BAD),
    (dict(w=0), BAD),
    (dict(w_scale=0), BAD),
    (dict(out=0), BAD),
    (dict(ldx=504), BAD),
    (dict(ldx=516), UNS),
    (dict(ldo=63), BAD),
    (dict(x=P + 8), UNS),
    (dict(w=P + 8), UNS),
    (dict(w_zero=P + 4), UNS),
    (dict(out=P + 2, out_dtype=2), UNS),
    (dict(bias=P + 1), UNS),
    (dict(k=0, x=0, w=0, w_scale=0), HIP),   # the bias alone
    (dict(m=1, ldx=3, ldo=1), HIP),          # one row has no stride
])
def test_int4_linear_validation(kw, status):
    no_gpu(status)
    a = dict(x=P, ldx=512, dtype=0, w=P, w_scale=P, w_zero=0, bias=0, out=P, ldo=64, out_dtype=0, m=3, n=64, k=512,
             group=128)
    a.update(kw)
    assert ck.lib().ck_int4_linear(ctypes.byref(ck.CkInt4Args(**a)), 0) == status
    assert ck.lib().ck_int4_linear(None, 0) == BAD


def test_struct_fields_follow_the_header():
    """The binding's structures have the header's fields, in its order."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, cls in (("ck_kv_cache", ck.CkKvCache), ("ck_qk_args", ck.CkQkArgs), ("ck_attention_args", ck.CkAttentionArgs),
                      ("ck_int4_args", ck.CkInt4Args)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        want = []
        for line in body.split(";"):
            if line.strip():
                kind = "ptr" if "*" in line else re.search(r"\b(int64_t|int32_t|float)\b", line).group(1)
                names = re.sub(r"\b(const|void|float|u?int[0-9]+_t)\b|\*", " ", line)
                want += [(n.strip(), kind) for n in names.split(",")]
        kinds = {ctypes.c_void_p: "ptr", ctypes.c_int64: "int64_t", ctypes.c_int32: "int32_t", ctypes.c_float: "float"}
        assert [(n, kinds[t]) for n, t in cls._fields_] == want
    for packed, cls in ((ck.decode._QK, ck.CkQkArgs), (ck.decode._ATTENTION, ck.CkAttentionArgs), (ck.decode._INT4, ck.CkInt4Args)):
        assert packed.size == ctypes.sizeof(cls)


# ------------------------------------------------------------- the binding

@pytest.fixture
def host(monkeypatch):
    class Launched(Exception):
        pass

    def launched(*a, **k):
        raise Launched()

    monkeypatch.setattr(ck, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(ck, "_stream", lambda t: 0)
    monkeypatch.setattr(ck.decode, "_stream", lambda index: 0)
    for f in ("ck_qk_norm_rope", "ck_paged_attention", "ck_int4_pack", "ck_int4_linear"):
        monkeypatch.setattr(ck, f, launched)
    return Launched


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_kv_cache(host):
    c = ck.KVCache.empty(5, 2, 16, 128, "int8", "cpu")
    assert (c.pages, c.heads, c.page_size, c.head_dim) == (5, 2, 16, 128)
    assert c.struct.token_stride == 128 and c.struct.scale_token_stride == 1 and c.struct.dtype == ck.CK_DT_INT8
    nhd = ck.KVCache(bf(5, 16, 2, 128).transpose(1, 2), bf(5, 16, 2, 128).transpose(1, 2))
    assert (nhd.struct.page_stride, nhd.struct.head_stride, nhd.struct.token_stride) == (4096, 128, 256)
    s = torch.zeros(5, 2, 16)
    i8 = torch.zeros((5, 2, 16, 128), dtype=torch.int8)
    for exc, args in [
        (TypeError, (bf(5, 2, 16, 128).float(), bf(5, 2, 16, 128).float())),
        (TypeError, (bf(5, 2, 16, 128), bf(5, 2, 16, 128).half())),
        (ValueError, (bf(5, 2, 16, 128), bf(5, 2, 16, 64))),
        (ValueError, (bf(5, 2, 128), bf(5, 2, 128))),
        (ValueError, (bf(5, 2, 12, 128), bf(5, 2, 12, 128))),
        (ValueError, (bf(5, 2, 128, 16).transpose(2, 3), bf(5, 2, 128, 16).transpose(2, 3))),
        (ValueError, (bf(5, 2, 16, 128), bf(5, 16, 2, 128).transpose(1, 2))),
        (ValueError, (i8, i8)),
        (ValueError, (bf(5, 2, 16, 128), bf(5, 2, 16, 128), s, s)),
        (TypeError, (i8, i8, s.half(), s)),
        (ValueError, (i8, i8, s[:4], s)),
        (ValueError, (i8, i8, s, torch.zeros(5, 16, 2).transpose(1, 2))),
    ]:
        with pytest.raises(exc):
            ck.KVCache(*args)
    with pytest.raises(ValueError):
        ck.KVCache.empty(5, 2, 16, 128, "fp8", "cpu")


def test_binding_rope(host):
    q, k, v = bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128)
    pos, table, w = torch.zeros(4, dtype=torch.int64), ck.rope_table(50, 128, device="cpu"), torch.ones(128)
    c = ck.KVCache.empty(3, 2, 16, 128, "bf16", "cpu")
    good = dict(q=q, k=k, v=v, positions=pos, cos_sin=table, q_weight=w, k_weight=w, cache=c, slots=pos)
    with pytest.raises(host):
        ck.qk_norm_rope(**good)
    with pytest.raises(host):
        ck.qk_norm_rope(q, None, None, pos, table, w)
    with pytest.raises(host):
        ck.qk_norm_rope(q, k, None, None, None, w, w)
    for exc, kw in [
        (TypeError, dict(q=q.float())),
        (ValueError, dict(q=bf(4, 1024))),
        (TypeError, dict(k=k.half())),
        (ValueError, dict(k=bf(3, 2, 128))),
        (ValueError, dict(k=bf(4, 2, 64))),
        (ValueError, dict(v=bf(4, 1, 128))),
        (ValueError, dict(v=None)),
        (ValueError, dict(slots=None)),
        (TypeError, dict(slots=pos.int())),
        (ValueError, dict(slots=pos[:3])),
        (TypeError, dict(positions=pos.int())),
        (TypeError, dict(positions=None)),
        (TypeError, dict(cos_sin=table.double())),
        (ValueError, dict(cos_sin=table.t())),
        (TypeError, dict(q_weight=w.bfloat16())),
        (ValueError, dict(k_weight=w[:64])),
        (TypeError, dict(cache=c.k)),
        (ValueError, dict(q_out=bf(4, 8, 64))),
        (ValueError, dict(k_out=bf(4, 8, 128))),
        (ValueError, dict(k=None)),
        (TypeError, dict(q_weight=torch.ones(128, device="meta"))),
    ]:
        with pytest.raises(exc):
            ck.qk_norm_rope(**{**good, **kw})


def test_binding_attention(host):
    c = ck.KVCache.empty(9, 2, 16, 128, "bf16", "cpu")
    good = dict(q=bf(3, 8, 128), cache=c, table=torch.zeros((3, 4), dtype=torch.int32),
                lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(host):
        ck.paged_attention(**good)
    with pytest.raises(host):
        ck.paged_attention(**good, window=100, sinks=4, scale=1.0, out=bf(3, 8, 128))
    for exc, kw in [
        (TypeError, dict(q=good["q"].float())),
        (ValueError, dict(q=bf(3, 8, 64))),
        (ValueError, dict(q=bf(3, 1024))),
        (TypeError, dict(cache=c.k)),
        (TypeError, dict(table=good["table"].long())),
        (ValueError, dict(table=good["table"][:2])),
        (TypeError, dict(lens=good["lens"].long())),
        (ValueError, dict(lens=good["lens"][:2])),
        (ValueError, dict(window=-1)),
        (ValueError, dict(sinks=-1)),
        (ValueError, dict(q=bf(3, 7, 128))),
        (ValueError, dict(out=bf(3, 8, 64))),
        (TypeError, dict(out=bf(3, 8, 128).half())),
        (TypeError, dict(workspace=torch.zeros(1 << 20))),
    ]:
        with pytest.raises(exc):
            ck.paged_attention(**{**good, **kw})


def test_binding_int4(host):
    codes, scales = torch.zeros((32, 128), dtype=torch.uint8), bf(32, 2)
    with pytest.raises(host):
        ck.int4_pack(codes, scales)
    for exc, kw in [
        (TypeError, dict(codes=codes.to(torch.int8))),
        (ValueError, dict(codes=codes[0])),
        (ValueError, dict(codes=codes[:, :127])),
        (TypeError, dict(scales=scales.float())),
        (ValueError, dict(scales=bf(32, 3))),
        (ValueError, dict(group=64)),
        (ValueError, dict(group=100)),
        (TypeError, dict(zeros=torch.zeros((32, 2)))),
        (ValueError, dict(zeros=torch.zeros((31, 2), dtype=torch.uint8))),
    ]:
        with pytest.raises(exc):
            ck.int4_pack(**{**dict(codes=codes, scales=scales), **kw})
    w = ck.Int4Weight(torch.zeros(4096, dtype=torch.uint8), bf(2, 2, 16), None, 32, 256, 128, torch.bfloat16)
    with pytest.raises(host):
        ck.int4_linear(bf(3, 256), w, bf(32))
    with pytest.raises(host):
        ck.int4_linear(bf(3, 256), w, bf(32).float(), out_dtype="fp32")
    for exc, kw in [
        (TypeError, dict(x=bf(3, 256).float())),
        (TypeError, dict(x=bf(3, 256).half())),
        (ValueError, dict(x=bf(3, 248))),
        (ValueError, dict(x=bf(256))),
        (TypeError, dict(weight=codes)),
        (TypeError, dict(bias=bf(32).float())),
        (ValueError, dict(bias=bf(31))),
        (ValueError, dict(out_dtype="int8")),
        (ValueError, dict(out=bf(3, 31))),
        (TypeError, dict(out=bf(3, 32).half())),
    ]:
        with pytest.raises(exc):
            ck.int4_linear(**{**dict(x=bf(3, 256), weight=w), **kw})


@pytest.mark.parametrize("stride", [0, 1, 64, 127])
def test_binding_int4_pack_passes_the_codes_stride(host, monkeypatch, stride):
    """Rows of codes that overlap (an expanded row among them) reach the library with the stride that
    they have, which it refuses; the stride of a single row is not looked at."""
    seen = []
    monkeypatch.setattr(ck, "ck_int4_pack", lambda codes, ldc, *a: seen.append(ldc))
    codes = torch.zeros(31 * stride + 128, dtype=torch.uint8).as_strided((32, 128), (stride, 1))
    ck.int4_pack(codes, bf(32, 2))
    assert seen == [stride]
    assert ck.lib().ck_int4_pack(P, stride, P, 2, 0, 0, P, P, 0, 32, 256, 128, 0) == BAD
    ck.int4_pack(codes[:1], bf(1, 2))
    assert seen[1] >= 128


def test_weights_and_caches_are_copied_with_their_pointers(host):
    """A copy of a weight or a cache points at its own tensors, however it was made."""
    import copy
    import pickle

    def weight(w):
        return [w.w_ptr, w.s_ptr, w.z_ptr], [t.data_ptr() for t in (w.w, w.scales, w.zeros)]

    def cache_(c):
        s = ctypes.cast(c.address, ctypes.POINTER(ck.CkKvCache)).contents
        return [s.k, s.v, s.k_scale, s.v_scale], [t.data_ptr() for t in (c.k, c.v, c.k_scale, c.v_scale)]

    w = ck.Int4Weight(torch.zeros(4096, dtype=torch.uint8), bf(2, 2, 16), torch.zeros((2, 2, 16), dtype=torch.uint8),
                      32, 256, 128, torch.bfloat16)
    c = ck.KVCache.empty(3, 2, 16, 64, "int8", "cpu")
    for x, pointers in ((w, weight), (c, cache_)):
        had = pointers(x)
        assert had[0] == had[1]
        for copied in (copy.copy(x), copy.deepcopy(x), pickle.loads(pickle.dumps(x))):
            got = pointers(copied)
            assert got[0] == got[1] and type(copied) is type(x)
        assert pointers(x) == had
        assert got[1] != had[1]


def test_weights_and_caches_are_fixed(host):
    """Another tensor in place of one of theirs would not be used: it is an error."""
    w = ck.Int4Weight(torch.zeros(4096, dtype=torch.uint8), bf(2, 2, 16), None, 32, 256, 128, torch.bfloat16)
    c = ck.KVCache.empty(3, 2, 16, 64, "bf16", "cpu")
    for x, names in ((w, ("w", "scales", "zeros", "n", "group")), (c, ("k", "v", "k_scale", "page_size", "struct"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(x, name, getattr(x, name))
            with pytest.raises(AttributeError):
                delattr(x, name)


def test_int4_weight_checks_its_tensors(host):
    """A weight made of tensors that were laid out before (a checkpoint's, say) has their sizes checked:
    the kernels read as much as n, k and group say."""
    good = dict(w=torch.zeros(6144, dtype=torch.uint8), scales=bf(3, 4, 16), zeros=torch.zeros((3, 4, 16), dtype=torch.uint8),
                n=33, k=232, group=64, dtype=torch.bfloat16)
    ck.Int4Weight(**good)
    for exc, kw in [
        (ValueError, dict(w=torch.zeros(6143, dtype=torch.uint8))),
        (ValueError, dict(w=torch.zeros(12288, dtype=torch.uint8)[::2])),
        (TypeError, dict(w=torch.zeros(6144, dtype=torch.int8))),
        (ValueError, dict(scales=bf(3, 3, 16))),
        (ValueError, dict(scales=bf(3, 16, 4).transpose(1, 2))),
        (TypeError, dict(scales=bf(3, 4, 16).half())),
        (ValueError, dict(zeros=torch.zeros((2, 4, 16), dtype=torch.uint8))),
        (TypeError, dict(zeros=bf(3, 4, 16))),
        (ValueError, dict(n=49)),
        (ValueError, dict(n=-1)),
        (ValueError, dict(k=264)),
        (ValueError, dict(k=228)),
        (ValueError, dict(group=48)),
        (ValueError, dict(group=32)),
        (TypeError, dict(dtype=torch.float16)),
        (TypeError, dict(dtype=torch.float32, scales=bf(3, 4, 16).float())),
    ]:
        with pytest.raises(exc):
            ck.Int4Weight(**{**good, **kw})


def test_launches_go_to_the_tensors_device(host, monkeypatch):
    """The default stream of every device is the null stream, which launches on the current device:
    a call on another device's tensors makes that one current for its time."""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.was

    ck.decode._load_torch()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ck.decode, "_stream", lambda index: 100 + index)
    for index in (0, 3):
        ck.decode._launch(lambda *a: seen.append((current[0], a)), index, "args", None)
        assert current[0] == 0
    assert seen == [(0, ("args", None, 100)), (3, ("args", None, 103))]
    calls = []
    monkeypatch.setattr(ck.decode, "_launch", lambda f, index, *a: calls.append(index))
    c = ck.KVCache.empty(9, 2, 16, 128, "bf16", "cpu")
    ck.qk_norm_rope(bf(4, 8, 128), bf(4, 2, 128), None, None, None)
    ck.paged_attention(bf(3, 8, 128), c, torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    w = ck.int4_pack(torch.zeros((32, 128), dtype=torch.uint8), bf(32, 2))
    ck.int4_linear(bf(3, 256), w)
    assert len(calls) == 4


def test_rope_table():
    t = ck.rope_table(1000, 64, 500000.0, device="cpu")
    assert t.shape == (1000, 64) and t.dtype == torch.float32
    angle = 999 * 500000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert (t[999, :32].double() - angle.cos()).abs().max() <= 2.0 ** -25 + 1e-12
    assert (t[999, 32:].double() - angle.sin()).abs().max() <= 2.0 ** -25 + 1e-12
    with pytest.raises(ValueError):
        ck.rope_table(10, 7, device="cpu")
