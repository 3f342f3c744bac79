"""Ragged-batch entry points without a GPU: arguments that are refused before anything is launched,
the workspace size, and the plain 64-bit reference of the GPU tests against the oracle."""

import math

import numpy as np
import pytest
import torch

import _ragged as ref
import oracle as orc
from gqa_attention_split_gb300 import api, build

P = 1 << 20  # a fake device pointer: a refused call never uses it


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _packed(**kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, cu_q=P, cu_k=None, B=2, H_q=8, H_kv=2, d=128, total_q=10,
             total_k=10, q_stride_t=1024, q_stride_h=128, k_stride_t=256, k_stride_h=128,
             v_stride_t=256, v_stride_h=128, causal=1, scale=0.1, stream=None)
    a.update(kw)
    return api.gqa_attn_prefill_packed(**a)


def _tree(**kw):
    a = dict(q=P, k_new=P, v_new=P, k_cache=P, v_cache=P, o=P, lse=P, cu_seqlens=P, context_lens=P,
             tree_mask=P, mask_words=1, B=2, H_q=8, H_kv=2, d=128, total=10, max_tokens=8,
             S_max=64, q_stride_t=1024, q_stride_h=128, k_stride_t=256, k_stride_h=128,
             v_stride_t=256, v_stride_h=128, scale=0.1, workspace=P, workspace_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return api.gqa_attn_decode_tree(**a)


def _append(**kw):
    a = dict(k_cache=P, v_cache=P, k_new=P, v_new=P, cu_seqlens=P, starts=P, index=P, B=2, H_kv=2,
             d=128, S_max=64, total=10, total_new=12, k_stride_t=256, k_stride_h=128,
             v_stride_t=256, v_stride_h=128, stream=None)
    a.update(kw)
    return api.gqa_attn_cache_append(**a)


INVALID, UNSUPPORTED, MISALIGNED = (api.GQA_ERR_INVALID_ARG, api.GQA_ERR_UNSUPPORTED,
                                    api.GQA_ERR_MISALIGNED)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(o=None), INVALID), (dict(cu_q=None), INVALID), (dict(B=-1), INVALID),
    (dict(B=65536), INVALID), (dict(H_q=9), INVALID), (dict(H_kv=0), INVALID),
    (dict(total_q=-1), INVALID), (dict(total_k=9), INVALID),
    (dict(cu_k=P, total_k=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(H_q=258, H_kv=2), UNSUPPORTED), (dict(q_stride_t=0), INVALID),
    (dict(k_stride_h=-128), INVALID), (dict(v_stride_t=1 << 39), INVALID),
    (dict(q_stride_t=1028), MISALIGNED), (dict(k_stride_h=132), MISALIGNED), (dict(q=P + 8), MISALIGNED),
    (dict(v=P + 2), MISALIGNED), (dict(o=P + 4), MISALIGNED), (dict(lse=P + 2), MISALIGNED),
    (dict(cu_q=P + 1), MISALIGNED), (dict(cu_k=P + 2), MISALIGNED),
])
def test_prefill_packed_refuses(kw, code):
    assert _packed(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k_new=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(context_lens=None), INVALID), (dict(workspace=None), api.GQA_ERR_WORKSPACE), (dict(S_max=0), INVALID),
    (dict(max_tokens=0), INVALID), (dict(max_tokens=129, mask_words=5), UNSUPPORTED),
    (dict(max_tokens=33), INVALID), (dict(mask_words=0), INVALID), (dict(mask_words=-1), INVALID),
    (dict(cu_seqlens=None, total=11), INVALID), (dict(cu_seqlens=None, total=18), INVALID),
    (dict(H_q=34), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(total=-1), INVALID),
    (dict(B=1 << 15, H_kv=2, S_max=1 << 15), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(q_stride_h=0), INVALID), (dict(v_stride_t=250), MISALIGNED),
    (dict(k_cache=P + 8), MISALIGNED), (dict(tree_mask=P + 2), MISALIGNED),
    (dict(workspace=P + 16), api.GQA_ERR_WORKSPACE), (dict(workspace_bytes=255), api.GQA_ERR_WORKSPACE),
])
def test_decode_tree_refuses(kw, code):
    assert _tree(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k_cache=None), INVALID), (dict(v_new=None), INVALID), (dict(starts=None), INVALID),
    (dict(index=None, total_new=9), INVALID), (dict(cu_seqlens=None, total=11), INVALID),
    (dict(B=-1), INVALID), (dict(S_max=0), INVALID), (dict(total=-1), INVALID),
    (dict(d=48), UNSUPPORTED), (dict(B=1 << 15, S_max=1 << 15), UNSUPPORTED),
    (dict(k_stride_t=0), INVALID), (dict(k_stride_t=260), MISALIGNED),
    (dict(v_cache=P + 8), MISALIGNED), (dict(starts=P + 1), MISALIGNED), (dict(index=P + 2), MISALIGNED),
])
def test_cache_append_refuses(kw, code):
    assert _append(**kw) == code


def test_empty_calls_launch_nothing():
    assert _packed(B=0) == api.GQA_OK and _packed(total_q=0, total_k=0, q=None, o=None) == api.GQA_OK
    assert _tree(B=0) == api.GQA_OK
    assert _tree(total=0, q=None, k_new=None, v_new=None, o=None) == api.GQA_OK
    assert _append(B=0) == api.GQA_OK and _append(total=0) == api.GQA_OK


def test_workspace_size():
    size = api.gqa_attn_decode_tree_workspace_size
    for bad in ((8, 3, 128, 4), (8, 2, 96, 4), (8, 2, 128, 0), (8, 2, 128, 129), (34, 2, 128, 4),
                (0, 1, 128, 4), (8, 0, 128, 4)):
        assert size(*bad) == 0
    for H_q, H_kv, d, T in ((8, 1, 128, 1), (64, 8, 128, 64), (128, 8, 64, 128)):
        n = size(H_q, H_kv, d, T)
        assert 0 < n < 1 << 27 and size(H_q, H_kv, d, max(1, T // 2)) <= n
        assert _tree(H_q=H_q, H_kv=H_kv, d=d, max_tokens=T, mask_words=4,
                     workspace_bytes=n - 1) == api.GQA_ERR_WORKSPACE


def test_binding_checks_tensors():
    t = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        api.prefill_packed(t, t, t, cu)  # not CUDA tensors
    with pytest.raises(TypeError):
        api.decode_tree(t, t, t, t[None], t[None], cu)
    with pytest.raises(TypeError):
        api.cache_append(t[None], t[None], t, t, cu)


def test_reference_agrees_with_the_oracle():
    rng = np.random.RandomState(0)
    q, k, v = (rng.randn(20, h, 64) for h in (6, 2, 2))
    O, L, bO, bL = ref.attend(q, k, v, ref.causal_visible(20, 20), 0.125)
    t = lambda x: torch.from_numpy(x.transpose(1, 0, 2)[None].copy())  # noqa: E731
    O2, L2 = orc.attention(t(q), t(k), t(v), scale=0.125, causal=True)
    assert np.abs(O - O2[0].transpose(1, 0, 2)).max() < 1e-12
    assert np.abs(L - L2[0].T).max() < 1e-12
    assert (bO > 0).all() and (bL > 0).all()


def test_reference_ignores_what_is_not_visible():
    rng = np.random.RandomState(1)
    q, k, v = (rng.randn(3, h, 64) for h in (2, 1, 1))
    vis = np.array([[1, 0, 0], [0, 0, 0], [1, 0, 1]], bool)
    kb, vb = k.copy(), v.copy()
    kb[1], vb[1] = np.nan, np.inf
    O, L, _, _ = ref.attend(q, kb, vb, vis, 0.5)
    assert np.isfinite(O).all() and (O[1] == 0).all() and np.isneginf(L[1]).all()
    assert np.allclose(O[0], np.broadcast_to(v[0], (2, 64)))
    assert np.allclose(L[0], 0.5 * q[0] @ k[0, 0])


def test_strides_of_dimensions_of_size_one_are_ignored():
    odd = dict(q_stride_t=3, k_stride_t=5, v_stride_t=-7)
    assert _packed(B=0, total_q=1, total_k=1, **odd) == api.GQA_OK
    assert _tree(B=0, total=1, **odd) == api.GQA_OK
    odd = dict(k_stride_h=5, v_stride_h=-7)
    assert _packed(B=0, H_q=1, H_kv=1, q_stride_h=3, **odd) == api.GQA_OK
    assert _tree(B=0, H_q=1, H_kv=1, q_stride_h=3, **odd) == api.GQA_OK
    assert _append(B=0, H_kv=1, **odd) == api.GQA_OK
    assert _append(B=0, total_new=1, k_stride_t=5, v_stride_t=-7) == api.GQA_OK
