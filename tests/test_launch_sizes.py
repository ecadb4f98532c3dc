"""Calls of more blocks than a launch takes (2^32 threads) are refused before anything is launched, and by the
functions that size their workspaces (no GPU needed)."""
import ctypes

import pytest

import int8_weight_quantized_amd as ck
from tests.test_decode_abi import HIP, P, UNS, attn_args, cache, no_gpu, qk_args
from tests.test_serving_abi import logprob_args, prefix_args

MANY = 1 << 20


@pytest.mark.parametrize("rows,status", [((1 << 24) - 1, HIP), (1 << 24, UNS), ((1 << 31) - 1, UNS)])
def test_logprob_rows(rows, status):
    no_gpu(status)
    assert ck.ck_token_logprobs_workspace(rows, 8, 0) == (0 if status == HIP else -1)
    a = logprob_args(rows=rows, vocab=8, ld=8, top=0, workspace=0, workspace_bytes=0)
    assert ck.lib().ck_token_logprobs(ctypes.byref(a), 0) == status


@pytest.mark.parametrize("hq,hk,status", [
    (15, 15, HIP),
    (16, 16, UNS),               # 2^24 blocks of 256 threads
    (48, 1, HIP),
    (64, 1, UNS),                # 2^26 rows, four a block of the join
])
def test_prefix_blocks(hq, hk, status):
    no_gpu(status)
    need = ck.ck_shared_prefix_attention_workspace(MANY, hq, hk, 128, 1, 1, 1, 16)
    assert (need > 0) == (status == HIP) and (need == -1) == (status == UNS)
    a = prefix_args(batch=MANY, hq=hq, prefixes=1, prefix_width=1, prefix_table_stride=1, table_width=1, table_stride=1,
                    q_batch_stride=hq * 128, out_batch_stride=hq * 128, workspace_bytes=1 << 50)
    c = cache(heads=hk, head_stride=2048, page_stride=2048 * hk)
    assert ck.lib().ck_shared_prefix_attention(ctypes.byref(a), ctypes.byref(c), 0) == status


@pytest.mark.parametrize("hk,dtype,width,status", [
    (8, ck.CK_DT_BF16, 1, HIP),
    (15, ck.CK_DT_BF16, 1, HIP),
    (16, ck.CK_DT_BF16, 1, UNS),           # 2^24 blocks of 256 threads
    (7, ck.CK_DT_INT8, 1, HIP),
    (8, ck.CK_DT_INT8, 1, UNS),            # 2^23 blocks of 512
    (1, ck.CK_DT_BF16, 512, HIP),          # chunks of 1024 tokens, 8 a sequence
    (2, ck.CK_DT_BF16, 512, UNS),
])
def test_attention_blocks(hk, dtype, width, status):
    no_gpu(status)
    i8 = dtype == ck.CK_DT_INT8
    a = attn_args(batch=MANY, hq=hk, table_width=width, table_stride=width, q_batch_stride=hk * 128, out_batch_stride=hk * 128,
                  workspace_bytes=1 << 50)
    c = cache(heads=hk, head_stride=2048, page_stride=2048 * hk, dtype=dtype, k_scale=P if i8 else 0, v_scale=P if i8 else 0)
    assert ck.lib().ck_paged_attention(ctypes.byref(a), ctypes.byref(c), 0) == status


def test_attention_workspace_of_what_one_type_of_cache_takes():
    """A size that a 16-bit cache's launch takes and an int8 one's does not: the former's bytes."""
    assert ck.ck_paged_attention_workspace(MANY, 8, 8, 128, 1, 16) == 0
    assert ck.ck_paged_attention_workspace(MANY, 16, 16, 128, 1, 16) == -1
    # rows of the output, one a block of the join
    assert ck.ck_paged_attention_workspace(MANY, 15, 1, 128, 128, 16) > 0
    assert ck.ck_paged_attention_workspace(MANY, 16, 1, 128, 128, 16) == -1


@pytest.mark.parametrize("tokens,status", [(1 << 26, HIP), (1 << 28, UNS)])
def test_rope_blocks(tokens, status):
    no_gpu(status)
    assert ck.lib().ck_qk_norm_rope(ctypes.byref(qk_args(tokens=tokens, hk=0, k=0, v=0, slots=0)), None, 0) == status
