"""The results of the ragged calls are weighted means of the V rows that the matrix product used: O is
divided by the sum of the rounded weights, as in the uniform prefill. Equal V rows come out as they
are, and V with a mean away from 0 is no less exact than V around 0 (_ragged_convex.py)."""

import math

import numpy as np
import pytest
import torch

import _ragged as ref
import _ragged_convex as convex
from gqa_attention_split_gb300 import api, build

pytestmark = pytest.mark.gpu

HEADS = {"g8": (16, 2, 128), "g1d64": (3, 3, 64), "g7": (14, 2, 128), "g16d64": (16, 1, 64)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


# Equal V rows: O' = v sum w_j / sum w_j. The two sums are of the same values, in fp32, so they differ
# by at most 2^-23 relative a step; up to 2^13 keys that is below 2^-10, and the next bf16 value's
# border is 2^-9 relative away at least: the result rounds to v.


def _rows_equal(o, v, H_q):
    """o [n, H_q, d] holds v [H_kv, d] in every row of its heads."""
    want = v.repeat_interleave(H_q // v.shape[0], 0)
    return (o == want[None]).all().item()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_packed_equal_values_come_out_as_they_are(heads, causal):
    H_q, H_kv, d = HEADS[heads]
    lens = [1, 2, 3, 5, 40, 130, 300]
    n = sum(lens)
    q, k, one = _randn(1, n, H_q, d), _randn(2, n, H_kv, d), _randn(3, 1, H_kv, d)
    o, _ = api.prefill_packed(q, k, one.expand(n, -1, -1).contiguous(), _cu(lens), causal=causal)
    api.check()
    assert _rows_equal(o, one[0], H_q)


# The same where the weights have any mantissa and one key has nearly all of the weight: the scores
# of a query grow by a constant from tile to tile (one key in every tile of 128, the others far below),
# and O is rescaled only every few tiles.


def _growing(n_q, n_k, H_q, H_kv, d):
    """q, k of scores a * j / 64 * sqrt(d) at key 128 j + 17, another a for every query and head."""
    a = 2 + 8 * torch.rand(n_q, H_q, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    q = a.to(torch.bfloat16).expand(-1, -1, d).contiguous()
    k = torch.full((n_k, H_kv, d), -1.0, dtype=torch.bfloat16, device="cuda")
    for j, at in enumerate(range(17, n_k, 128)):
        k[at] = j / 64
    return q, k


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_packed_equal_values_under_growing_scores(heads, causal):
    H_q, H_kv, d = HEADS[heads]
    lens = [1000, 300]
    q, k = (torch.cat(t) for t in zip(*(_growing(n, n, H_q, H_kv, d) for n in lens)))
    one = _randn(3, 1, H_kv, d)
    o, _ = api.prefill_packed(q, k, one.expand(1300, -1, -1).contiguous(), _cu(lens), causal=causal)
    api.check()
    assert _rows_equal(o, one[0], H_q)


# 5 tiles of a row on a cache that is not cut; rows of 9 tiles that are cut into a few parts
@pytest.mark.parametrize("B,T,S_max,ctx", [(2, 3, 512, 500), (2, 128, 512, 500), (40, 3, 1100, 1020),
                                           (30, 128, 1100, 1020)])
@pytest.mark.parametrize("heads", HEADS)
def test_tree_equal_values_under_growing_scores(heads, B, T, S_max, ctx):
    H_q, H_kv, d = HEADS[heads]
    q, k = _growing(B * T, S_max, H_q, H_kv, d)
    kc = k.transpose(0, 1).expand(B, -1, -1, -1).contiguous()
    one = _randn(14, 1, H_kv, 1, d)
    kn = torch.full((B * T, H_kv, d), -1.0, dtype=torch.bfloat16, device="cuda")
    o, _ = api.decode_tree(q, kn, one[:, :, 0].expand(B * T, -1, -1).contiguous(), kc,
                           one.expand(B, -1, S_max, -1).contiguous(),
                           torch.full((B,), ctx, dtype=torch.int32, device="cuda"))
    api.check()
    assert _rows_equal(o, one[0, :, 0], H_q)


# few drafts on a short cache (one part), on a long one (cut), and more drafts than one group of rows
@pytest.mark.parametrize("ctx,drafts,S_max", [([2, 0, 300], [3, 5, 2], 400),
                                              ([3000, 7], [5, 5], 4096),
                                              ([1500, 40], [60, 128], 2048)],
                         ids=["whole", "cut", "wide"])
@pytest.mark.parametrize("heads", HEADS)
def test_tree_equal_values_come_out_as_they_are(heads, ctx, drafts, S_max):
    H_q, H_kv, d = HEADS[heads]
    n, B = sum(drafts), len(ctx)
    q, kn = _randn(11, n, H_q, d), _randn(12, n, H_kv, d)
    kc, one = _randn(13, B, H_kv, S_max, d), _randn(14, 1, H_kv, 1, d)
    vc = one.expand(B, -1, S_max, -1).contiguous()
    vn = one[:, :, 0].expand(n, -1, -1).contiguous()
    o, _ = api.decode_tree(q, kn, vn, kc, vc, torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                           cu_seqlens=_cu(drafts), max_tokens=max(drafts))
    api.check()
    assert _rows_equal(o, one[0, :, 0], H_q)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("mean", [0.0, 1.0, 4.0])
def test_packed_values_with_a_mean(heads, mean):
    H_q, H_kv, d = HEADS[heads]
    lens = [1, 2, 3, 4, 6, 33, 150]
    n = sum(lens)
    q, k = _randn(21, n, H_q, d), _randn(22, n, H_kv, d)
    v = (_randn(23, n, H_kv, d) * 0.25 + mean).contiguous()
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    a = 0
    for m in lens:
        s = slice(a, a + m)
        ref.check(o[s], lse[s], convex.attend(_np(q[s]), _np(k[s]), _np(v[s]),
                                              ref.causal_visible(m, m), 1 / math.sqrt(d)),
                  f"{m} tokens")
        a += m


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("ctx,drafts,S_max", [([0, 3, 90], [4, 2, 9], 256), ([2500, 1], [9, 3], 2600),
                                              ([700, 2], [70, 3], 1024)],
                         ids=["whole", "cut", "wide"])
def test_tree_values_with_a_mean(heads, ctx, drafts, S_max):
    H_q, H_kv, d = HEADS[heads]
    n, B = sum(drafts), len(ctx)
    q, kn = _randn(31, n, H_q, d), _randn(32, n, H_kv, d)
    vn = _randn(33, n, H_kv, d) * 0.25 + 4
    kc, vc = _randn(34, B, H_kv, S_max, d), _randn(35, B, H_kv, S_max, d) * 0.25 + 4
    o, lse = api.decode_tree(q, kn, vn, kc, vc, torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                             cu_seqlens=_cu(drafts), max_tokens=max(drafts))
    api.check()
    a = 0
    for b, (c, m) in enumerate(zip(ctx, drafts)):
        s = slice(a, a + m)
        k = torch.cat([kc[b, :, :c].transpose(0, 1), kn[s]])
        v = torch.cat([vc[b, :, :c].transpose(0, 1), vn[s]])
        vis = np.concatenate([np.ones((m, c), bool), np.tril(np.ones((m, m), bool))], 1)
        ref.check(o[s], lse[s], convex.attend(_np(q[s]), _np(k), _np(v), vis, 1 / math.sqrt(d)),
                  f"row {b}")
        a += m


def test_packed_is_as_exact_as_the_uniform_prefill():
    # the same inputs through either call, held to the same bound
    n, H_q, H_kv, d = 200, 8, 2, 128
    q, k = _randn(41, 2 * n, H_q, d), _randn(42, 2 * n, H_kv, d)
    v = _randn(43, 2 * n, H_kv, d) + 2
    o, lse = api.prefill_packed(q, k, v, _cu([n, n]))
    shape = lambda t: t.view(2, n, -1, d).transpose(1, 2).contiguous()  # noqa: E731
    o2, lse2 = api.prefill(shape(q), shape(k), shape(v))
    api.check()
    for b in range(2):
        s = slice(n * b, n * b + n)
        r = convex.attend(_np(q[s]), _np(k[s]), _np(v[s]), ref.causal_visible(n, n),
                          1 / math.sqrt(d))
        ref.check(o[s], lse[s], r, "packed")
        ref.check(o2[b].transpose(0, 1), lse2[b].t(), r, "uniform")
