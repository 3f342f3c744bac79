"""decode_tree in every way that it cuts its work (_ragged_cut.py): against plain 64-bit attention, the
same bits every time, and on a cache of more than 2^31 elements."""

import math

import numpy as np
import pytest
import torch

import _ragged as ref
import _ragged_convex as convex
from _ragged_cut import cut
from gqa_attention_split_gb300 import api, build

pytestmark = pytest.mark.gpu


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


def _random(seed, B, ctx, T):
    """B rows of 0..ctx context tokens and 0..T drafts, T in one of them."""
    rng = np.random.RandomState(seed)
    drafts = [int(x) for x in rng.randint(0, T + 1, B)]
    drafts[B // 2] = T
    return [int(x) for x in rng.randint(0, ctx + 1, B)], drafts


# name: H_q, H_kv, d, contexts, drafts, S_max, way. With 132 to 152 SMs the ways are the same.
CASES = {
    # teams of 8 CTAs, a row for all of a team's CTAs, one for 7, one whose unit is 2 KV heads
    "line_teams": (32, 2, 64, [4000, 1777, 2500, 900], [128, 100, 7, 77], 4096, "line"),
    # the units of rows with few drafts hold several KV heads
    "line_head_groups": (64, 4, 64, [900, 1500, 700, 1100, 333], [3, 128, 40, 1, 17], 1536, "line"),
    # one CTA to a team, contexts of very different lengths
    "line_ragged": (16, 8, 64, [6007, 4096, 17, 0, 900, 129, 2222], [5, 1, 3, 2, 4, 7, 6], 6100, "line"),
    # more rows than the plan reads at a time, empty ones among them
    "line_70_rows": (16, 4, 64, *_random(1, 70, 1500, 5), 1600, "line"),
    "line_140_rows_wide": (32, 2, 64, *_random(2, 140, 700, 40), 1024, "line"),
    "line_d128": (16, 2, 128, *_random(3, 40, 2500, 9), 2600, "line"),
    "even_many_parts": (16, 2, 128, [6000, 40], [9, 3], 6016, "even"),
    "even_many_parts_wide": (32, 2, 64, [3000], [128], 3200, "even"),
    "even_40_rows": (8, 1, 64, [200] * 40, [2] * 40, 1000, "even"),
    "whole_70_rows": (16, 2, 64, *_random(4, 70, 500, 9), 512, "whole"),
}


def _call(case):
    H_q, H_kv, d, ctx, drafts, S_max, _ = CASES[case]
    n, B = sum(drafts), len(ctx)
    x = (_randn(1, n, H_q, d), _randn(2, n, H_kv, d), _randn(3, n, H_kv, d),
         _randn(4, B, H_kv, S_max, d), _randn(5, B, H_kv, S_max, d),
         torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    return x, lambda **kw: api.decode_tree(*x, cu_seqlens=_cu(drafts), max_tokens=max(drafts), **kw)


def _way(case):
    H_q, H_kv, d, ctx, drafts, S_max, way = CASES[case]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    got, _, parts = cut(ctx, drafts, S_max, H_q, H_kv, max(drafts), sms)
    assert got == way
    return parts


@pytest.mark.parametrize("case", CASES)
def test_every_way_to_cut_the_work(case):
    parts = _way(case)
    if case.startswith("even_many"):
        assert parts > 4  # merged by several warps together
    H_q, H_kv, d, ctx, drafts, _, _ = CASES[case]
    (q, kn, vn, kc, vc, _), run = _call(case)
    o, lse = run()
    api.check()
    a = 0
    for b, (c, T) in enumerate(zip(ctx, drafts)):
        if T == 0:
            continue
        s = slice(a, a + T)
        k = torch.cat([kc[b, :, :c].transpose(0, 1), kn[s]])
        v = torch.cat([vc[b, :, :c].transpose(0, 1), vn[s]])
        seen = np.concatenate([np.ones((T, c), bool), np.tril(np.ones((T, T), bool))], 1)
        ref.check(o[s], lse[s], convex.attend(_np(q[s]), _np(k), _np(v), seen, 1 / math.sqrt(d)),
                  f"row {b}: context {c}, {T} drafts")
        a += T


@pytest.mark.parametrize("case", CASES)
def test_the_same_bits_whatever_the_workspace_holds(case):
    _way(case)
    H_q, H_kv, d, _, drafts, _, _ = CASES[case]
    _, run = _call(case)
    o, lse = run()
    size = api.gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max(drafts))
    for byte in (255, 0):  # fp32 NaN everywhere, then 0
        ws = torch.full((size,), byte, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            o2, lse2 = run(workspace=ws)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    api.check()


def test_a_row_behind_2_to_the_31_elements():
    B, H_kv, S_max, d = 6, 8, 450000, 128
    kc = torch.empty(B, H_kv, S_max, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    assert kc[5].storage_offset() > 2 ** 31
    ctx, drafts = [3, 0, 1, 0, 700, 900], [2, 1, 1, 0, 9, 6]
    n = sum(drafts)
    q, kn, vn = _randn(1, n, 16, d), _randn(2, n, H_kv, d), _randn(3, n, H_kv, d)
    kc[:, :, :1000], vc[:, :, :1000] = _randn(4, B, H_kv, 1000, d), _randn(5, B, H_kv, 1000, d)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                             cu_seqlens=_cu(drafts), max_tokens=9)
    far = torch.tensor([5, 5, 5, 5, S_max - 9, S_max - 6], dtype=torch.int32, device="cuda")
    api.cache_append(kc, vc, kn, vn, far, cu_seqlens=_cu(drafts))
    api.check()
    a = sum(drafts[:5])
    k = torch.cat([kc[5, :, :900].transpose(0, 1), kn[a:]])
    v = torch.cat([vc[5, :, :900].transpose(0, 1), vn[a:]])
    seen = np.concatenate([np.ones((6, 900), bool), np.tril(np.ones((6, 6), bool))], 1)
    ref.check(o[a:], lse[a:], convex.attend(_np(q[a:]), _np(k), _np(v), seen, 1 / math.sqrt(d)))
    assert torch.equal(kc[5, :, S_max - 6:], kn[a:].transpose(0, 1))
    assert torch.equal(vc[5, :, S_max - 6:], vn[a:].transpose(0, 1))
