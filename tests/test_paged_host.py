"""Entry points of the paged serving step without a GPU: arguments that are refused before anything
is launched, sizes, and what the binding checks."""

import math

import pytest
import torch

from gqa_attention_split_gb300 import api, build

P = 1 << 20  # a fake device pointer: a refused call never uses it
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (api.GQA_ERR_INVALID_ARG, api.GQA_ERR_UNSUPPORTED,
                                               api.GQA_ERR_MISALIGNED, api.GQA_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _norm(**kw):
    a = dict(q=P, k=P, q_out=P, k_out=P, q_weight=P, k_weight=P, weights_fp32=0, positions=P,
             inv_freq=P, sections=None, axes=1, tokens=10, H_q=8, H_kv=2, d=128, pairs=64,
             interleaved=0, norm=1, eps=1e-6, q_stride_t=1024, q_stride_h=128, k_stride_t=256,
             k_stride_h=128, qo_stride_t=1024, qo_stride_h=128, ko_stride_t=256, ko_stride_h=128,
             stream=None)
    a.update(kw)
    return api.gqa_attn_qk_norm_rope(**a)


def _append(**kw):
    a = dict(k_pages=P, v_pages=P, k_new=P, v_new=P, cu_seqlens=P, starts=P, index=P, block_table=P,
             B=2, H_kv=2, d=128, total=10, total_new=12, num_pages=5, page_size=16, table_width=4,
             k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128,
             k_page_stride=2 * 16 * 128, v_page_stride=2 * 16 * 128, stream=None)
    a.update(kw)
    return api.gqa_attn_paged_append(**a)


def _attend(**kw):
    a = dict(q=P, k_pages=P, v_pages=P, o=P, lse=P, cu_seqlens=P, kv_lens=P, block_table=P, B=2,
             H_q=8, H_kv=2, d=128, total=10, max_tokens=8, max_keys=0, num_pages=5, page_size=16,
             table_width=4, q_stride_t=1024, q_stride_h=128, k_page_stride=2 * 16 * 128,
             v_page_stride=2 * 16 * 128, causal=1, scale=0.1, workspace=P, workspace_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return api.gqa_attn_paged_attention(**a)


def _verify(**kw):
    a = dict(target_probs=P, draft_probs=P, draft_tokens=P, u_accept=P, u_sample=P, cu_seqlens=P,
             accepted=P, next_tokens=P, B=2, total=10, V=1000, target_stride=1000,
             draft_stride=1000, stream=None)
    a.update(kw)
    return api.gqa_attn_verify_drafts(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k_out=None), INVALID), (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID),
    (dict(tokens=-1), INVALID), (dict(H_q=0), INVALID), (dict(H_kv=-1), INVALID),
    (dict(pairs=0), INVALID), (dict(pairs=72), INVALID), (dict(pairs=12), UNSUPPORTED),
    (dict(d=64), INVALID), (dict(d=96), UNSUPPORTED), (dict(axes=0), INVALID),
    (dict(axes=2), INVALID), (dict(axes=5, sections=[8, 8, 16, 16, 16]), UNSUPPORTED),
    (dict(axes=3, sections=[16, 24, 23]), INVALID), (dict(axes=3, sections=[16, 24, 25]), INVALID),
    (dict(axes=3, sections=[-8, 48, 24]), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(q_stride_t=0), INVALID),
    (dict(k_stride_h=-128), INVALID), (dict(q_stride_t=1028), MISALIGNED),
    (dict(qo_stride_h=132), MISALIGNED), (dict(qo_stride_h=64), INVALID),
    (dict(qo_stride_t=512), INVALID), (dict(ko_stride_t=128), INVALID), (dict(q=P + 8), MISALIGNED),
    (dict(k_out=P + 2), MISALIGNED), (dict(positions=P + 2), MISALIGNED),
    (dict(inv_freq=P + 1), MISALIGNED), (dict(q_weight=P + 1), MISALIGNED),
    (dict(weights_fp32=1, k_weight=P + 2), MISALIGNED), (dict(ko_stride_t=1 << 39), INVALID),
])
def test_qk_norm_rope_refuses(kw, code):
    assert _norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k_pages=None), INVALID), (dict(v_new=None), INVALID), (dict(starts=None), INVALID),
    (dict(block_table=None), INVALID), (dict(index=None, total_new=9), INVALID),
    (dict(cu_seqlens=None, total=11), INVALID), (dict(B=-1), INVALID), (dict(B=65536), INVALID),
    (dict(H_kv=0), INVALID), (dict(d=48), UNSUPPORTED), (dict(page_size=0), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=192), UNSUPPORTED), (dict(num_pages=-1), INVALID),
    (dict(table_width=-1), INVALID), (dict(table_width=1 << 27), UNSUPPORTED),
    (dict(k_page_stride=4095), INVALID), (dict(v_page_stride=4100), MISALIGNED),
    (dict(v_page_stride=1 << 39), INVALID), (dict(v_pages=P + 8), MISALIGNED),
    (dict(block_table=P + 2), MISALIGNED), (dict(starts=P + 1), MISALIGNED),
    (dict(k_stride_t=0), INVALID), (dict(k_stride_t=260), MISALIGNED),
])
def test_paged_append_refuses(kw, code):
    assert _append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(k_pages=None), INVALID),
    (dict(v_pages=None), INVALID), (dict(kv_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=P + 16), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE), (dict(B=-1), INVALID), (dict(B=65536), INVALID),
    (dict(H_q=9), INVALID), (dict(H_q=258), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(total=-1), INVALID), (dict(max_tokens=0), INVALID), (dict(max_keys=-1), INVALID),
    (dict(cu_seqlens=None, total=11), INVALID), (dict(cu_seqlens=None, max_tokens=4), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=-16), INVALID), (dict(table_width=1 << 27), UNSUPPORTED),
    (dict(k_page_stride=2048), INVALID), (dict(k_page_stride=4100), MISALIGNED),
    (dict(q_stride_h=0), INVALID), (dict(q_stride_t=1028), MISALIGNED), (dict(q=P + 8), MISALIGNED),
    (dict(k_pages=P + 2), MISALIGNED), (dict(kv_lens=P + 2), MISALIGNED),
    (dict(cu_seqlens=P + 1), MISALIGNED), (dict(lse=P + 2), MISALIGNED),
])
def test_paged_attention_refuses(kw, code):
    assert _attend(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(target_probs=None), INVALID), (dict(draft_tokens=None), INVALID),
    (dict(u_accept=None), INVALID), (dict(u_sample=None), INVALID), (dict(accepted=None), INVALID),
    (dict(next_tokens=None), INVALID), (dict(B=-1), INVALID), (dict(B=65536), INVALID),
    (dict(B=0), INVALID), (dict(total=-1), INVALID), (dict(V=0), INVALID),
    (dict(V=(1 << 30) + 1), UNSUPPORTED), (dict(cu_seqlens=None, total=11), INVALID),
    (dict(target_stride=999), INVALID), (dict(draft_stride=999), INVALID),
    (dict(target_stride=1 << 39), INVALID), (dict(target_probs=P + 2), MISALIGNED),
    (dict(draft_tokens=P + 1), MISALIGNED), (dict(next_tokens=P + 2), MISALIGNED),
])
def test_verify_drafts_refuses(kw, code):
    assert _verify(**kw) == code


def test_empty_calls_launch_nothing():
    assert _norm(tokens=0, q=None, k=None, positions=None) == api.GQA_OK
    assert _append(B=0) == api.GQA_OK and _append(total=0) == api.GQA_OK
    assert _attend(B=0) == api.GQA_OK and _attend(total=0, q=None, o=None) == api.GQA_OK
    assert _verify(B=0, total=0) == api.GQA_OK


def test_strides_of_dimensions_of_size_one_are_ignored():
    odd = dict(q_stride_t=3, k_stride_t=5, qo_stride_t=-7, ko_stride_t=0)
    assert _norm(tokens=0, **odd) == api.GQA_OK
    assert _attend(B=0, total=1, num_pages=1, q_stride_t=3, k_page_stride=5) == api.GQA_OK
    assert _append(B=0, num_pages=1, k_page_stride=5, total_new=1, k_stride_t=3) == api.GQA_OK
    assert _verify(B=0, total=0, target_stride=0) == api.GQA_OK


def test_workspace_size():
    size = api.gqa_attn_paged_attention_workspace_size
    for bad in ((8, 3, 128, 4), (8, 2, 96, 4), (8, 2, 128, 0), (258, 2, 128, 4), (0, 1, 128, 4)):
        assert size(*bad) == 0
    for H_q, H_kv, d, T in ((8, 1, 128, 1), (64, 8, 128, 4096), (128, 1, 64, 128)):
        n = size(H_q, H_kv, d, T)
        assert 0 < n < 1 << 27 and size(H_q, H_kv, d, max(1, T // 2)) <= n
        assert _attend(H_q=H_q, H_kv=H_kv, d=d, max_tokens=max(T, 8), k_page_stride=1 << 20,
                       v_page_stride=1 << 20, workspace_bytes=n - 1) == WORKSPACE


def test_binding_checks_tensors():
    t = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i = torch.tensor([0, 4], dtype=torch.int32)
    f = torch.zeros(64)
    pages = torch.zeros(3, 8, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        api.qk_norm_rope(t, t, i, f)  # not CUDA tensors
    with pytest.raises(TypeError):
        api.paged_append(pages, pages, t, t, i[None], i)
    with pytest.raises(TypeError):
        api.paged_attention(t, pages, pages, i[None], i)
    with pytest.raises(TypeError):
        api.verify_drafts(torch.zeros(2, 9), i, f[:2], f[:1])
