"""The operators of a server's batch on the host: the C entry points and the
binding refuse bad arguments before any HIP call (no GPU needed)."""
import copy
import ctypes
import pickle
import re

import pytest
import torch

import int8_weight_quantized_amd as ck
from tests.test_abi import HEADER
from tests.test_decode_abi import BAD, CACHES, HIP, OK, P, UNS, bf, cache, no_gpu


def prefix_args(**kw):
    a = dict(q=P, out=P, prefix_table=P, prefix_lens=P, starts=P, table=P, lens=P, workspace=P, workspace_bytes=1 << 40,
             q_batch_stride=1024, q_head_stride=128, out_batch_stride=1024, out_head_stride=128, prefix_table_stride=200,
             table_stride=63, batch=5, hq=8, prefixes=2, prefix_width=200, table_width=63, scale=0.1, dtype=ck.CK_DT_BF16)
    a.update(kw)
    return ck.CkPrefixArgs(**a)


def call_prefix(a, c):
    return ck.lib().ck_shared_prefix_attention(ctypes.byref(a), ctypes.byref(c), 0)


@pytest.mark.parametrize("kw,status", CACHES)
def test_prefix_cache_validation(kw, status):
    no_gpu(status)
    if "head_dim" in kw:
        pytest.skip("the cache's head_dim is q's here")
    assert call_prefix(prefix_args(), cache(**kw)) == status


@pytest.mark.parametrize("kw,ckw,status", [
    (dict(), dict(), HIP),
    (dict(dtype=2), dict(), BAD),
    (dict(batch=-1), dict(), BAD),
    (dict(batch=0), dict(), OK),
    (dict(hq=0), dict(), OK),
    (dict(hq=7), dict(), BAD),
    (dict(prefixes=-1), dict(), BAD),
    (dict(prefix_width=-1), dict(), BAD),
    (dict(table_width=-1), dict(), BAD),
    (dict(q=0), dict(), BAD),
    (dict(out=0), dict(), BAD),
    (dict(lens=0), dict(), BAD),
    (dict(table=0), dict(), BAD),
    (dict(table=0, table_width=0), dict(), HIP),
    (dict(prefix_table=0), dict(), BAD),
    (dict(prefix_table=0, prefix_width=0), dict(), HIP),
    (dict(prefix_lens=0), dict(), BAD),
    (dict(starts=0), dict(), BAD),
    (dict(prefixes=0, prefix_table=0, prefix_lens=0, starts=0, prefix_width=0), dict(), HIP),
    (dict(table_stride=62), dict(), BAD),
    (dict(prefix_table_stride=199), dict(), BAD),
    (dict(prefix_table_stride=0, prefixes=1), dict(), HIP),
    (dict(q=P + 2), dict(), UNS),
    (dict(q_head_stride=129), dict(), UNS),
    (dict(out_batch_stride=1025), dict(), UNS),
    (dict(out_head_stride=64), dict(), BAD),
    (dict(out_batch_stride=512), dict(), BAD),
    (dict(lens=P + 2), dict(), UNS),
    (dict(starts=P + 2), dict(), UNS),
    (dict(prefix_lens=P + 1), dict(), UNS),
    (dict(prefix_table=P + 2), dict(), UNS),
    (dict(scale=float("nan")), dict(), BAD),
    (dict(batch=(1 << 20) + 1), dict(), UNS),
    (dict(prefixes=(1 << 20) + 1), dict(), UNS),
    (dict(table_width=1 << 31, table_stride=1 << 31), dict(), UNS),
    (dict(prefix_width=1 << 40, prefix_table_stride=1 << 40), dict(), UNS),
    (dict(), dict(head_dim=80, token_stride=80), UNS),
    (dict(), dict(pages=1 << 30, page_stride=1 << 20), UNS),
])
def test_prefix_validation(kw, ckw, status):
    no_gpu(status)
    assert call_prefix(prefix_args(**kw), cache(**ckw)) == status


def test_prefix_workspace():
    need = ck.ck_shared_prefix_attention_workspace(5, 8, 2, 128, 2, 200, 63, 16)
    assert need >= 0
    if need:
        for kw, status in ((dict(workspace=0), BAD), (dict(workspace_bytes=need - 1), BAD), (dict(workspace=P + 16), UNS)):
            assert call_prefix(prefix_args(**kw), cache()) == status
    if not torch.cuda.is_available():
        assert call_prefix(prefix_args(workspace_bytes=need), cache()) == HIP
    for bad in ((-1, 8, 2, 128, 2, 200, 63, 16), (5, 7, 2, 128, 2, 200, 63, 16), (5, 8, 0, 128, 2, 200, 63, 16),
                (5, 8, 2, 100, 2, 200, 63, 16), (5, 8, 2, 128, -2, 200, 63, 16), (5, 8, 2, 128, 2, -1, 63, 16),
                (5, 8, 2, 128, 2, 200, -1, 16), (5, 8, 2, 128, 2, 200, 63, 12), (1 << 20, 65536, 1, 256, 1, 1 << 30, 1 << 30, 1),
                (1 << 20, 4096, 4096, 256, 1 << 20, 1 << 25, 1 << 25, 32768)):
        assert ck.ck_shared_prefix_attention_workspace(*bad) == -1, bad
    # a prefix of up to 2^30 tokens
    assert ck.ck_shared_prefix_attention_workspace(5, 8, 2, 128, 2, 1 << 15, 63, 1 << 15) >= 0
    assert ck.ck_shared_prefix_attention_workspace(5, 8, 2, 128, 2, (1 << 15) + 1, 63, 1 << 15) == -1
    # more prefixes than sequences, widths of nothing
    for fine in ((1, 8, 2, 128, 100, 3, 3, 16), (5, 8, 2, 128, 0, 0, 63, 16), (5, 8, 2, 128, 2, 0, 0, 16), (0, 8, 2, 64, 0, 0, 0, 1)):
        assert ck.ck_shared_prefix_attention_workspace(*fine) >= 0, fine


def lora_args(**kw):
    a = dict(x=P, a=P, b=P, scale=P, ids=P, y=P, out=P, workspace=P, workspace_bytes=1 << 40, ldx=256, ldy=100, ldo=100,
             a_stride=16 * 256, b_stride=16 * 100, m=7, n=100, k=256, rank=16, adapters=3, dtype=ck.CK_DT_BF16,
             out_dtype=ck.CK_OUT_BF16)
    a.update(kw)
    return ck.CkLoraArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP),
    (dict(dtype=2), BAD),
    (dict(out_dtype=3), BAD),
    (dict(out_dtype=ck.CK_OUT_FP32), HIP),
    (dict(m=-1), BAD),
    (dict(n=-1), BAD),
    (dict(k=-8), BAD),
    (dict(rank=-8), BAD),
    (dict(adapters=-1), BAD),
    (dict(rank=0), UNS),
    (dict(rank=12), UNS),
    (dict(rank=264, a_stride=264 * 256, b_stride=264 * 100), UNS),
    (dict(k=252), UNS),
    (dict(m=0, x=0, y=0, out=0), OK),
    (dict(n=0), OK),
    (dict(x=0), BAD),
    (dict(a=0), BAD),
    (dict(b=0), BAD),
    (dict(ids=0), BAD),
    (dict(y=0), BAD),
    (dict(out=0), BAD),
    (dict(scale=0), HIP),
    (dict(x=0, a=0, k=0, a_stride=0), HIP),
    (dict(x=0, a=0, b=0, adapters=0), HIP),
    (dict(ldx=248), BAD),
    (dict(ldx=0, ldy=0, ldo=0, m=1), HIP),
    (dict(ldx=260), UNS),
    (dict(ldy=99), BAD),
    (dict(ldo=99), BAD),
    (dict(a_stride=16 * 256 - 8), BAD),
    (dict(b_stride=16 * 100 - 8), BAD),
    (dict(a_stride=0, b_stride=0, adapters=1), HIP),
    (dict(a_stride=16 * 256 + 4), UNS),
    (dict(x=P + 8), UNS),
    (dict(a=P + 2), UNS),
    (dict(b=P + 8), UNS),
    (dict(y=P + 1), UNS),
    (dict(out=P + 2, out_dtype=ck.CK_OUT_FP32), UNS),
    (dict(ids=P + 2), UNS),
    (dict(scale=P + 2), UNS),
    (dict(m=(1 << 24) + 1), UNS),
    (dict(n=(1 << 24) + 8, ldy=1 << 25, ldo=1 << 25, b_stride=1 << 40), UNS),
    (dict(k=(1 << 24) + 8, ldx=1 << 25, a_stride=1 << 40), UNS),
])
def test_lora_validation(kw, status):
    no_gpu(status)
    assert ck.lib().ck_lora_add(ctypes.byref(lora_args(**kw)), 0) == status


def test_lora_workspace():
    assert ck.lib().ck_lora_add(None, 0) == BAD
    for m in (1, 7, 4001):
        need = ck.ck_lora_add_workspace(m, 100, 256, 16)
        assert need >= 0
        if need:
            for kw, status in ((dict(workspace=0), BAD), (dict(workspace_bytes=need - 1), BAD), (dict(workspace=P + 16), UNS)):
                assert ck.lib().ck_lora_add(ctypes.byref(lora_args(m=m, **kw)), 0) == status
    for bad in ((-1, 100, 256, 16), (1, -1, 256, 16), (1, 100, 255, 16), (1, 100, 256, 12), (1, 100, 256, 264), (1, 100, 256, 0)):
        assert ck.ck_lora_add_workspace(*bad) == -1


def logprob_args(**kw):
    a = dict(logits=P, tokens=P, logprob=P, entropy=P, top_ids=P, top_logprobs=P, workspace=P, workspace_bytes=1 << 40, ld=1000,
             rows=4, vocab=1000, top=5, dtype=ck.CK_OUT_BF16)
    a.update(kw)
    return ck.CkLogprobArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP),
    (dict(dtype=3), BAD),
    (dict(dtype=ck.CK_OUT_FP32), HIP),
    (dict(rows=-1), BAD),
    (dict(vocab=0), BAD),
    (dict(top=-1), BAD),
    (dict(top=65), UNS),
    (dict(top=7, vocab=6), BAD),
    (dict(rows=0, logits=0), OK),
    (dict(logits=0), BAD),
    (dict(tokens=0), BAD),
    (dict(logprob=0), BAD),
    (dict(tokens=0, logprob=0), HIP),
    (dict(entropy=0), HIP),
    (dict(top_ids=0), BAD),
    (dict(top_logprobs=0), BAD),
    (dict(top_ids=0, top_logprobs=0, top=0), HIP),
    (dict(ld=999), BAD),
    (dict(ld=0, rows=1), HIP),
    (dict(logits=P + 1), UNS),
    (dict(logits=P + 2, dtype=ck.CK_OUT_FP32), UNS),
    (dict(logits=P + 2), HIP),
    (dict(tokens=P + 4), UNS),
    (dict(top_ids=P + 4), UNS),
    (dict(logprob=P + 2), UNS),
    (dict(entropy=P + 2), UNS),
    (dict(top_logprobs=P + 2), UNS),
    (dict(vocab=1 << 31, ld=1 << 31), UNS),
    (dict(rows=1 << 31), UNS),
])
def test_logprob_validation(kw, status):
    no_gpu(status)
    assert ck.lib().ck_token_logprobs(ctypes.byref(logprob_args(**kw)), 0) == status


def test_logprob_workspace():
    assert ck.lib().ck_token_logprobs(None, 0) == BAD
    for rows, vocab in ((1, 200000), (4, 1000), (3, 100)):
        need = ck.ck_token_logprobs_workspace(rows, vocab, 5)
        assert need >= 0
        if need:
            for kw, status in ((dict(workspace=0), BAD), (dict(workspace_bytes=need - 1), BAD), (dict(workspace=P + 16), UNS)):
                assert ck.lib().ck_token_logprobs(ctypes.byref(logprob_args(rows=rows, vocab=vocab, ld=vocab, **kw)), 0) == status
    for bad in ((-1, 10, 1), (1, 0, 0), (1, 10, 11), (1, 100, 65), (1, 100, -1), (1, 1 << 31, 1)):
        assert ck.ck_token_logprobs_workspace(*bad) == -1


def test_struct_fields_follow_the_header():
    """The binding's structures have the header's fields, in its order."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    kinds = {ctypes.c_void_p: "ptr", ctypes.c_int64: "int64_t", ctypes.c_int32: "int32_t", ctypes.c_float: "float"}
    for name, cls, packed in (("ck_prefix_args", ck.CkPrefixArgs, ck.serving._PREFIX), ("ck_lora_args", ck.CkLoraArgs, ck.serving._LORA),
                              ("ck_logprob_args", ck.CkLogprobArgs, ck.serving._LOGPROB)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        want = []
        for line in body.split(";"):
            if line.strip():
                kind = "ptr" if "*" in line else re.search(r"\b(int64_t|int32_t|float)\b", line).group(1)
                names = re.sub(r"\b(const|void|float|u?int[0-9]+_t)\b|\*", " ", line)
                want += [(n.strip(), kind) for n in names.split(",")]
        assert [(n, kinds[t]) for n, t in cls._fields_] == want
        assert packed.size == ctypes.sizeof(cls)


# ------------------------------------------------------------- the binding

@pytest.fixture
def host(monkeypatch):
    class Launched(Exception):
        pass

    def launched(*a, **k):
        raise Launched()

    monkeypatch.setattr(ck, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(ck.decode, "_stream", lambda index: 0)
    for f in ("ck_shared_prefix_attention", "ck_lora_add", "ck_token_logprobs"):
        monkeypatch.setattr(ck, f, launched)
    return Launched


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_prefix(host):
    c = ck.KVCache.empty(9, 2, 16, 128, "bf16", "cpu")
    good = dict(q=bf(3, 8, 128), cache=c, prefix_table=i32(2, 5), prefix_lens=i32(2), starts=i32(3), table=i32(3, 4), lens=i32(3))
    with pytest.raises(host):
        ck.shared_prefix_attention(**good)
    with pytest.raises(host):
        ck.shared_prefix_attention(**good, scale=1.0, out=bf(3, 8, 128))
    with pytest.raises(host):
        ck.shared_prefix_attention(**{**good, "prefix_table": i32(0, 0), "prefix_lens": i32(0), "starts": i32(1)})
    for exc, kw in [
        (TypeError, dict(q=good["q"].float())),
        (ValueError, dict(q=bf(3, 8, 64))),
        (TypeError, dict(cache=c.k)),
        (TypeError, dict(table=i32(3, 4).long())),
        (ValueError, dict(table=i32(2, 4))),
        (ValueError, dict(lens=i32(2))),
        (TypeError, dict(prefix_table=i32(2, 5).long())),
        (ValueError, dict(prefix_table=i32(5))),
        (ValueError, dict(prefix_table=i32(5, 2).t())),
        (TypeError, dict(prefix_lens=i32(2).long())),
        (ValueError, dict(prefix_lens=i32(3))),
        (ValueError, dict(prefix_lens=i32(4)[::2])),
        (ValueError, dict(starts=i32(2))),
        (TypeError, dict(starts=i32(3).long())),
        (TypeError, dict(starts=None)),
        (TypeError, dict(prefix_table=torch.zeros((2, 5), dtype=torch.int32, device="meta"))),
        (ValueError, dict(q=bf(3, 7, 128))),
        (ValueError, dict(out=bf(3, 8, 64))),
        (TypeError, dict(workspace=torch.zeros(1 << 20))),
    ]:
        with pytest.raises(exc):
            ck.shared_prefix_attention(**{**good, **kw})


def test_binding_lora(host):
    w = ck.LoraWeight(bf(4, 16, 64), bf(4, 50, 16), torch.ones(4))
    assert (w.adapters, w.rank, w.k, w.n) == (4, 16, 64, 50)
    good = dict(y=bf(3, 50), x=bf(3, 64), weight=w, ids=i32(3))
    with pytest.raises(host):
        ck.lora_add(**good)
    with pytest.raises(host):
        ck.lora_add(**{**good, "y": torch.zeros(3, 50)}, out=torch.zeros(3, 60)[:, :50])
    for exc, kw in [
        (TypeError, dict(y=bf(3, 50).double())),
        (ValueError, dict(y=bf(3, 51))),
        (ValueError, dict(y=bf(50))),
        (ValueError, dict(y=bf(50, 3).t())),
        (TypeError, dict(x=bf(3, 64).half())),
        (ValueError, dict(x=bf(4, 64))),
        (ValueError, dict(x=bf(3, 72))),
        (ValueError, dict(x=bf(64, 3).t())),
        (TypeError, dict(weight=w.a)),
        (TypeError, dict(ids=i32(3).long())),
        (ValueError, dict(ids=i32(4))),
        (ValueError, dict(ids=i32(6)[::2])),
        (TypeError, dict(out=bf(3, 50).half())),
        (ValueError, dict(out=bf(3, 49))),
        (TypeError, dict(workspace=torch.zeros(1 << 20))),
    ]:
        with pytest.raises(exc):
            ck.lora_add(**{**good, **kw})
    for exc, args in [
        (TypeError, (bf(4, 16, 64).float(), bf(4, 50, 16).float())),
        (TypeError, (bf(4, 16, 64), bf(4, 50, 16).half())),
        (ValueError, (bf(4, 16, 64), bf(3, 50, 16))),
        (ValueError, (bf(4, 16, 64), bf(4, 50, 8))),
        (ValueError, (bf(4, 64), bf(4, 50, 16))),
        (ValueError, (bf(4, 12, 64), bf(4, 50, 12))),
        (ValueError, (bf(4, 264, 64), bf(4, 50, 264))),
        (ValueError, (bf(4, 16, 60), bf(4, 50, 16))),
        (ValueError, (bf(4, 64, 16).transpose(1, 2), bf(4, 50, 16))),
        (ValueError, (bf(4, 16, 128)[:, :, :64], bf(4, 50, 16))),
        (ValueError, (bf(4, 16, 64), bf(4, 50, 16), torch.ones(3))),
        (TypeError, (bf(4, 16, 64), bf(4, 50, 16), bf(4))),
    ]:
        with pytest.raises(exc):
            ck.LoraWeight(*args)
    had = w.a_ptr
    for copied in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert (copied.a_ptr, copied.b_ptr, copied.s_ptr) == (copied.a.data_ptr(), copied.b.data_ptr(), copied.scale.data_ptr())
    assert copied.a_ptr != had == w.a_ptr
    with pytest.raises(AttributeError):
        w.a = w.a


def test_binding_logprobs(host):
    x, t = bf(3, 100), torch.zeros(3, dtype=torch.int64)
    for args in ((x, t), (x, None, 5), (x.float(), t, 64), (x.half(), t, 100 - 64)):
        with pytest.raises(host):
            ck.token_logprobs(*args)
    for exc, args in [
        (TypeError, (x.double(), t)),
        (ValueError, (x[0], t)),
        (ValueError, (bf(3, 0), t)),
        (ValueError, (bf(100, 3).t(), t)),
        (TypeError, (x, t.int())),
        (ValueError, (x, t[:2])),
        (ValueError, (x, t, -1)),
        (ValueError, (x, t, 65)),
        (ValueError, (bf(3, 6), t, 7)),
        (TypeError, (x, t, 3, torch.zeros(1 << 20))),
    ]:
        with pytest.raises(exc):
            ck.token_logprobs(*args)


def test_launches_go_to_the_tensors_device(host, monkeypatch):
    """Each entry point launches once, on its tensors' device, however it came through its checks."""
    calls = []
    monkeypatch.setattr(ck.decode, "_launch", lambda f, index, *a: calls.append((f, index)))
    c = ck.KVCache.empty(9, 2, 16, 128, "bf16", "cpu")
    q, t, n = torch.zeros((3, 8, 128), dtype=torch.bfloat16), i32(3, 4), i32(3)
    out, big = torch.empty_like(q), torch.empty(1 << 24, dtype=torch.uint8)
    ck.shared_prefix_attention(q, c, i32(2, 4), i32(2), i32(3), t, n)
    ck.shared_prefix_attention(q, c, i32(2, 4), i32(2), i32(3), t, n, out=out, workspace=big)
    w = ck.LoraWeight(torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 30, 8), dtype=torch.bfloat16))
    x, y = torch.zeros((3, 64), dtype=torch.bfloat16), torch.zeros((3, 30))
    ck.lora_add(y, x, w, n)
    ck.lora_add(y, x, w, n, out=torch.empty_like(y), workspace=big)
    ck.token_logprobs(y, None, 3)
    ck.token_logprobs(y, torch.zeros(3, dtype=torch.int64), workspace=big)
    want = [ck.ck_shared_prefix_attention] * 2 + [ck.ck_lora_add] * 2 + [ck.ck_token_logprobs] * 2
    assert calls == [(f, None) for f in want]


def test_lora_out_is_not_x(host):
    """x is read while out is written: the same memory is refused, also where y is x; y itself as out is not."""
    w = ck.LoraWeight(bf(4, 16, 64), bf(4, 64, 16))
    x, y = bf(3, 64), bf(3, 64)
    for args, kw in [((y, x), dict(out=x)), ((x, x), dict(out=x)), ((y, x), dict(out=x.view(3, 64)))]:
        with pytest.raises(ValueError):
            ck.lora_add(*args, w, i32(3), **kw)
    for args, kw in [((y, x), dict(out=y)), ((x, x), dict()), ((x, x), dict(out=y))]:
        with pytest.raises(host):
            ck.lora_add(*args, w, i32(3), **kw)
