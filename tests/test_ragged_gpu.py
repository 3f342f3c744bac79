"""Ragged batches on the GPU: attention over packed prompts, attention of drafted token trees over
the cache, appending to the cache, and the three together, each against plain attention in 64 bits
(_ragged.py, which derives the elementwise bounds) or bit for bit."""

import math

import numpy as np
import pytest
import torch

import _ragged as ref
from gqa_attention_split_gb300 import api, build

pytestmark = pytest.mark.gpu

HEADS = {"g8": (8, 1, 128), "g8x2": (16, 2, 128), "g1d64": (3, 3, 64), "g7": (14, 2, 128),
         "g3d64": (6, 2, 64), "g16": (16, 1, 128)}


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


def _packed_inputs(q_lens, k_lens, H_q, H_kv, d, seed=0):
    return (_randn(seed, sum(q_lens), H_q, d), _randn(seed + 1, sum(k_lens), H_kv, d),
            _randn(seed + 2, sum(k_lens), H_kv, d))


def _check_packed(o, lse, q, k, v, q_lens, k_lens, causal, scale, what=""):
    a = c = 0
    for n_q, n_k in zip(q_lens, k_lens):
        vis = ref.causal_visible(n_q, n_k) if causal else np.ones((n_q, n_k), bool)
        ref.check(o[a:a + n_q], lse[a:a + n_q],
                  ref.attend(_np(q[a:a + n_q]), _np(k[c:c + n_k]), _np(v[c:c + n_k]), vis, scale),
                  f"{what} lengths {n_q}/{n_k}")
        a, c = a + n_q, c + n_k


# ------------------------------------------------------------------- packed prompts


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[1], [17, 1, 0, 40, 96], [128, 129, 127, 16, 15], [300, 700]],
                         ids=["one", "short", "edges", "long"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_packed_prompts(heads, lens, causal):
    H_q, H_kv, d = HEADS[heads]
    q, k, v = _packed_inputs(lens, lens, H_q, H_kv, d)
    o, lse = api.prefill_packed(q, k, v, _cu(lens), causal=causal)
    api.check()
    _check_packed(o, lse, q, k, v, lens, lens, causal, 1 / math.sqrt(d))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_packed_keys_of_other_lengths(heads, causal):
    # keys before the queries; fewer keys than queries (the first queries see none); no keys
    H_q, H_kv, d = HEADS[heads]
    q_lens, k_lens = [40, 1, 150, 9, 33, 70], [333, 500, 20, 0, 33, 128]
    q, k, v = _packed_inputs(q_lens, k_lens, H_q, H_kv, d, 5)
    o, lse = api.prefill_packed(q, k, v, _cu(q_lens), _cu(k_lens), causal=causal, scale=0.11)
    api.check()
    _check_packed(o, lse, q, k, v, q_lens, k_lens, causal, 0.11)


def test_packed_no_keys_at_all():
    q, k, v = _packed_inputs([5, 3], [0, 0], 8, 1, 128)
    o, lse = api.prefill_packed(q, k, v, _cu([5, 3]), _cu([0, 0]))
    api.check()
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_packed_many_sequences():
    # more sequences than the schedule keeps in shared memory (1024), most of them short
    rng = np.random.RandomState(3)
    lens = list(rng.randint(0, 6, 1500)) + [130, 0, 257] + list(rng.randint(0, 3, 200))
    q, k, v = _packed_inputs(lens, lens, 4, 2, 64, 9)
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    _check_packed(o, lse, q, k, v, lens, lens, True, 1 / 8)


def test_packed_more_sequences_than_the_schedule_table_holds_twice():
    rng = np.random.RandomState(4)
    lens = list(rng.randint(0, 5, 2100)) + [300, 129] + [0] * 50
    q, k, v = _packed_inputs(lens, lens, 3, 1, 64, 10)
    for causal in (True, False):
        o, lse = api.prefill_packed(q, k, v, _cu(lens), causal=causal)
        api.check()
        _check_packed(o, lse, q, k, v, lens, lens, causal, 1 / 8)


@pytest.mark.parametrize("H_q,H_kv", [(32, 1), (100, 1), (128, 1), (18, 2)])
def test_packed_large_groups_of_heads(H_q, H_kv):
    # 100 heads: one token to a block; 9 heads: 14 tokens, two rows of a block unused
    lens = [7, 1, 150]
    q, k, v = _packed_inputs(lens, lens, H_q, H_kv, 128, 12)
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    _check_packed(o, lse, q, k, v, lens, lens, True, 1 / math.sqrt(128))


def test_packed_persistent_items():
    # several work items per CTA, of very different lengths
    lens = [1500, 3, 260, 900, 31, 1100]
    q, k, v = _packed_inputs(lens, lens, 32, 8, 128, 11)
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    _check_packed(o, lse, q, k, v, lens, lens, True, 1 / math.sqrt(128))


def test_packed_equal_lengths_agree_with_prefill():
    q, k, v = _packed_inputs([200, 200], [200, 200], 8, 2, 128, 21)
    o, lse = api.prefill_packed(q, k, v, _cu([200, 200]))
    shape = lambda t: t.view(2, 200, -1, 128).transpose(1, 2).contiguous()  # noqa: E731
    o2, lse2 = api.prefill(shape(q), shape(k), shape(v))
    api.check()
    # both within the bound of the same exact result
    O = [ref.attend(_np(q[i:i + 200]), _np(k[i:i + 200]), _np(v[i:i + 200]),
                    ref.causal_visible(200, 200), 1 / math.sqrt(128)) for i in (0, 200)]
    for b in range(2):
        ref.check(o[200 * b:200 * b + 200], lse[200 * b:200 * b + 200], O[b])
        ref.check(o2[b].transpose(0, 1), lse2[b].t(), O[b])


@pytest.mark.parametrize("layout", ["fused", "head_major", "padded"])
def test_packed_strides(layout):
    lens, H_q, H_kv, d = [70, 5, 131], 12, 4, 64
    n = sum(lens)
    q, k, v = _packed_inputs(lens, lens, H_q, H_kv, d, 31)
    if layout == "fused":
        qs, ks, vs = torch.cat([q, k, v], 1).split([H_q, H_kv, H_kv], 1)
    elif layout == "head_major":
        qs, ks, vs = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    else:
        def pad(t):
            big = torch.full((n, t.shape[1] + 1, d + 8), float("nan"), dtype=t.dtype,
                             device="cuda")
            big[:, :t.shape[1], :d] = t
            return big[:, :t.shape[1], :d]
        qs, ks, vs = pad(q), pad(k), pad(v)
    o, lse = api.prefill_packed(qs, ks, vs, _cu(lens))
    o2, lse2 = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_packed(o, lse, q, k, v, lens, lens, True, 1 / 8)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads", ["g8", "g1d64", "g7"])
def test_packed_values_of_unseen_keys_do_not_matter(bad, heads):
    # K and V of later tokens of the own sequence, of the next sequence and behind the last one
    H_q, H_kv, d = HEADS[heads]
    lens = [90, 150, 61]
    q, k, v = _packed_inputs(lens, lens, H_q, H_kv, d, 41)
    kb, vb = (torch.cat([t, torch.full_like(t[:40], bad)]) for t in (k, v))
    qb = torch.cat([q, torch.full_like(q[:40], bad)])
    kb[70:90], vb[70:90] = bad, bad            # seen by queries 70..89 of the first sequence
    kb[90 + 149], vb[90 + 149] = bad, bad      # the last token of the second
    o, lse = api.prefill_packed(qb, kb, vb, _cu(lens))
    api.check()
    keep = np.r_[0:70, 90:239, 240:301]
    o2 = o.clone()
    o2[70:90], o2[239] = 0, 0
    assert torch.isfinite(o2[:301].float()).all()
    a = 0
    for n, m in ((90, 70), (150, 149), (61, 61)):
        r = ref.attend(_np(q[a:a + m]), _np(k[a:a + m]), _np(v[a:a + m]),
                       ref.causal_visible(m, m), 1 / math.sqrt(d))
        ref.check(o[a:a + m], lse[a:a + m], r)
        a += n
    assert len(keep) == 70 + 149 + 61


def test_packed_seen_values_that_are_not_finite_come_out():
    # NaN and infinities that a query sees are its result, in their columns only
    lens = [100]
    q, k, v = _packed_inputs(lens, lens, 8, 1, 128, 47)
    vb = v.clone()
    vb[60, 0, 3], vb[70, 0, 5], vb[75, 0, 6], vb[80, 0, 6] = (float(x) for x in
                                                              ("nan", "inf", "inf", "-inf"))
    o, _ = api.prefill_packed(q, k, vb, _cu(lens))
    clean, _ = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    assert torch.isnan(o[60:, :, 3]).all() and torch.isfinite(o[:60].float()).all()
    assert (o[70:, :, 5] == float("inf")).all()
    assert (o[75:80, :, 6] == float("inf")).all() and torch.isnan(o[80:, :, 6]).all()
    other = [c for c in range(128) if c not in (3, 5, 6)]
    assert torch.equal(o[..., other], clean[..., other])


def test_packed_rows_behind_the_last_sequence_are_left():
    lens = [20, 50]
    q, k, v = _packed_inputs([80], [80], 8, 2, 64, 51)
    out = torch.full_like(q, 7.0)
    lse = torch.full((80, 8), 9.0, device="cuda")
    cu = _cu(lens) + 3  # three rows in front belong to nobody either
    api.prefill_packed(q, k, v, cu, out=out, lse=lse)
    api.check()
    for s in (slice(0, 3), slice(73, 80)):
        assert (out[s] == 7).all() and (lse[s] == 9).all()
    _check_packed(out[3:73], lse[3:73], q[3:73], k[3:73], v[3:73], lens, lens, True, 1 / 8)


@pytest.mark.parametrize("cu", [[0, 30, 20, 60], [-5, 10, 20, 60], [0, 10, 20, 99]])
def test_packed_bad_prefix_sums_are_reported(cu):
    q, k, v = _packed_inputs([60], [60], 8, 2, 64, 53)
    api.prefill_packed(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT
    lens = [10, 50]  # the next call is clean
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.check()
    _check_packed(o, lse, q, k, v, lens, lens, True, 1 / 8)


# --------------------------------------------------------------------- draft trees


def _tree_mask(drafts, words, seed, empty=()):
    rng = np.random.RandomState(seed)
    bits, vis = [], []
    for n in drafts:
        m = np.zeros((n, 32 * words), bool)
        for i in range(n):
            if i:
                m[i] = m[rng.randint(max(0, i - 6), i)]
            m[i, i] = True
        for i in empty:
            if i < n:
                m[i] = False
        vis.append(m[:, :n].copy())
        m[:, n:] = rng.rand(n, 32 * words - n) < 0.5  # bits behind the row's tokens are ignored
        bits.append(np.packbits(m, axis=1, bitorder="little").view(np.int32))
    return torch.from_numpy(np.concatenate(bits)).cuda(), vis


def _tree_inputs(ctx, drafts, S_max, H_q, H_kv, d, seed=0):
    n, B = sum(drafts), len(ctx)
    return (_randn(seed, n, H_q, d), _randn(seed + 1, n, H_kv, d), _randn(seed + 2, n, H_kv, d),
            _randn(seed + 3, B, H_kv, S_max, d), _randn(seed + 4, B, H_kv, S_max, d),
            torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, vis, scale, what=""):
    a = 0
    for b, (n, T) in enumerate(zip(ctx, drafts)):
        s = slice(a, a + T)
        k = torch.cat([kc[b, :, :n].transpose(0, 1), kn[s]])
        v = torch.cat([vc[b, :, :n].transpose(0, 1), vn[s]])
        draft = np.tril(np.ones((T, T), bool)) if vis is None else vis[b]
        seen = np.concatenate([np.ones((T, n), bool), draft], 1)
        ref.check(o[s], lse[s], ref.attend(_np(q[s]), _np(k), _np(v), seen, scale),
                  f"{what} row {b}: context {n}, {T} drafts")
        a += T


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("ctx,drafts", [
    ([0], [1]), ([777], [1]), ([333, 0, 128, 127], [7, 16, 1, 8]),
    ([1000, 129, 2000], [33, 64, 0]), ([64, 1500], [128, 77]),
], ids=["first_token", "single", "short", "wide", "widest"])
@pytest.mark.parametrize("tree", [True, False], ids=["tree", "line"])
def test_tree(heads, ctx, drafts, tree):
    H_q, H_kv, d = HEADS[heads]
    S_max, T = max(ctx) + 5, max(drafts)
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, S_max, H_q, H_kv, d)
    mask, vis = _tree_mask(drafts, (T + 31) // 32, 7, (2, 5)) if tree else (None, None)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=T,
                             tree_mask=mask)
    api.check()
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, vis, 1 / math.sqrt(d))


def test_tree_queries_that_see_nothing():
    drafts, ctx = [6, 3], [0, 40]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 64, 8, 2, 64, 3)
    mask = torch.zeros(9, 1, dtype=torch.int32, device="cuda")
    mask[1, 0] = 0b000101
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=6,
                             tree_mask=mask)
    api.check()
    vis = [np.zeros((6, 6), bool), np.zeros((3, 3), bool)]
    vis[0][1, [0, 2]] = True
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, vis, 1 / 8)
    assert torch.isneginf(lse[[0, 2, 3, 4, 5]]).all()


def test_tree_uniform_rows_without_prefix_sums():
    ctx, drafts = [50, 300, 7], [4, 4, 4]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 512, 16, 2, 128, 13)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl)
    o2, lse2 = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=4)
    api.check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, None, 1 / math.sqrt(128))


@pytest.mark.parametrize("seed", range(12))
def test_tree_random_shapes(seed):
    rng = np.random.RandomState(100 + seed)
    H_q, H_kv, d = [(8, 1, 128), (16, 2, 64), (4, 4, 128), (14, 2, 64), (32, 2, 128), (5, 1, 128)][
        seed % 6]
    B = rng.randint(1, 7)
    T = int(rng.choice([1, 2, 5, 13, 40, 100, 128]))
    drafts = [int(x) for x in rng.randint(0, T + 1, B)]
    drafts[rng.randint(B)] = T
    ctx = [int(rng.choice([0, 1, 127, 128, 129, rng.randint(1, 3000)])) for _ in range(B)]
    S_max = max(max(ctx), 1) + int(rng.randint(0, 200))
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, S_max, H_q, H_kv, d, seed)
    mask, vis = _tree_mask(drafts, 4, seed) if seed % 3 else (None, None)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=T,
                             tree_mask=mask, scale=0.1)
    api.check()
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, vis, 0.1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,heads", [(9, "g8"), (60, "g8"), (5, "g1d64")])
def test_tree_values_of_unseen_keys_do_not_matter(bad, T, heads):
    # cache slots behind the context, masked-out drafts, another row's drafts
    H_q, H_kv, d = HEADS[heads]
    ctx, drafts = [200, 13], [T, 3]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 300, H_q, H_kv, d, 17)
    mask, vis = _tree_mask(drafts, (T + 31) // 32, 19)
    for b in range(2):
        kc[b, :, ctx[b]:], vc[b, :, ctx[b]:] = bad, bad
    gone = T - 2  # nobody else descends from it: clear its bit, its own included
    words = mask.cpu().numpy().view(np.uint32)
    words[:T, gone >> 5] &= ~np.uint32(1 << (gone & 31))
    mask = torch.from_numpy(words.view(np.int32)).cuda()
    vis[0][:, gone] = False
    kn2, vn2 = kn.clone(), vn.clone()
    kn2[gone], vn2[gone] = bad, bad
    o, lse = api.decode_tree(q, kn2, vn2, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=T,
                             tree_mask=mask)
    api.check()
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, vis, 1 / math.sqrt(d))


def test_tree_seen_draft_that_is_not_finite_comes_out():
    ctx, drafts = [700], [6]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 1000, 8, 1, 128, 23)
    vb = vn.clone()
    vb[3, 0, 9] = float("nan")
    o, _ = api.decode_tree(q, kn, vb, kc, vc, cl)
    clean, _ = api.decode_tree(q, kn, vn, kc, vc, cl)
    api.check()
    assert torch.isnan(o[3:, :, 9]).all() and torch.equal(o[:3], clean[:3])
    assert torch.equal(o[3:, :, :9], clean[3:, :, :9])


def test_tree_longer_row_than_max_tokens_is_cut_and_reported():
    ctx, drafts = [30, 40], [6, 2]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 64, 8, 2, 64, 29)
    out = torch.full_like(q, 7.0)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=4, out=out)
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT
    assert (o[4:6] == 7).all()
    _check_tree(o[6:], lse[6:], q[6:], kn[6:], vn[6:], kc[1:], vc[1:], ctx[1:], drafts[1:], None,
                1 / 8)


@pytest.mark.parametrize("ctx", [[-3, 40], [30, 99]])
def test_tree_bad_context_is_clamped_and_reported(ctx):
    drafts = [3, 2]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 64, 8, 2, 64, 31)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=3)
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT
    _check_tree(o, lse, q, kn, vn, kc, vc, [min(64, max(0, c)) for c in ctx], drafts, None, 1 / 8)


def test_tree_gives_the_same_bits_every_time():
    ctx, drafts = [1500, 90, 4000], [17, 40, 3]
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 4096, 16, 2, 128, 37)
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=40)
    again, _ = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=40)
    api.check()
    assert torch.equal(o, again)  # the same bits every time
    _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, None, 1 / math.sqrt(128))


def test_tree_offsets_past_32_bits():
    # a cache of more than 2^31 elements: the last row's slab starts behind them
    B, H_kv, S_max, d = 5, 8, 450000, 128
    kc = torch.empty(B, H_kv, S_max, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    ctx, drafts = [3, 0, 1, 0, 700], [2, 1, 1, 0, 9]
    q, kn, vn, ks, vs, cl = _tree_inputs(ctx, drafts, 1000, 16, H_kv, d, 43)
    kc[:, :, :1000], vc[:, :, :1000] = ks, vs
    assert kc.numel() > 2 ** 31 and kc[4].storage_offset() > 2 ** 30
    o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=9)
    far = torch.tensor([S_max - 2, 5, 5, 5, S_max - 9], dtype=torch.int32, device="cuda")
    api.cache_append(kc, vc, kn, vn, far, cu_seqlens=_cu(drafts))
    api.check()
    _check_tree(o, lse, q, kn, vn, ks, vs, ctx, drafts, None, 1 / math.sqrt(d))
    assert torch.equal(kc[4, :, S_max - 9:], kn[4:].transpose(0, 1))
    assert torch.equal(vc[0, :, S_max - 2:], vn[:2].transpose(0, 1))


# -------------------------------------------------------------------- cache append


@pytest.mark.parametrize("d,H_kv", [(128, 8), (64, 3), (128, 1)])
@pytest.mark.parametrize("counts,starts", [([1], [0]), ([3, 0, 200, 1], [10, 5, 0, 255]),
                                           ([1] * 70, list(range(70)))])
@pytest.mark.parametrize("pick", [False, True])
def test_append(d, H_kv, counts, starts, pick):
    B, S_max, n = len(counts), 256, sum(counts)
    kc, vc = _randn(1, B, H_kv, S_max, d), _randn(2, B, H_kv, S_max, d)
    kn, vn = _randn(3, n + 5, H_kv, d), _randn(4, n + 5, H_kv, d)
    rng = np.random.RandomState(5)
    index = rng.randint(0, n + 5, n) if pick else np.arange(n)  # repeated tokens are allowed
    wk, wv = kc.clone(), vc.clone()
    e = 0
    for b in range(B):
        for i in range(counts[b]):
            wk[b, :, starts[b] + i], wv[b, :, starts[b] + i] = kn[index[e]], vn[index[e]]
            e += 1
    api.cache_append(kc, vc, kn if pick else kn[:n], vn if pick else vn[:n],
                     torch.tensor(starts, dtype=torch.int32, device="cuda"), cu_seqlens=_cu(counts),
                     index=torch.from_numpy(index.astype(np.int32)).cuda() if pick else None)
    api.check()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_strides_and_equal_counts():
    kc = torch.zeros(3, 2, 20, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    qkv = _randn(1, 6, 8, 64)
    _, kn, vn = qkv.split([4, 2, 2], 1)
    starts = torch.tensor([0, 18, 7], dtype=torch.int32, device="cuda")
    api.cache_append(kc, vc, kn, vn, starts)
    api.check()
    for b, s in enumerate((0, 18, 7)):
        assert torch.equal(kc[b, :, s:s + 2], kn[2 * b:2 * b + 2].transpose(0, 1))
        assert torch.equal(vc[b, :, s:s + 2], vn[2 * b:2 * b + 2].transpose(0, 1))


@pytest.mark.parametrize("starts,index", [([-1, 3], [0, 1, 2, 3]), ([9, 3], [0, 1, 2, 3]),
                                          ([2 ** 31 - 1, 3], [0, 1, 2, 3]),
                                          ([0, 3], [0, -1, 2, 3]), ([0, 3], [0, 4, 2, 3])])
def test_append_bad_slots_and_tokens_are_left_out_and_reported(starts, index):
    kc = torch.zeros(2, 1, 10, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kn, vn = _randn(1, 4, 1, 64), _randn(2, 4, 1, 64)
    api.cache_append(kc, vc, kn, vn, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                     index=torch.tensor(index, dtype=torch.int32, device="cuda"))
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT
    want = torch.zeros_like(kc)
    for b in range(2):
        for i in range(2):
            s, t = starts[b] + i, index[2 * b + i]
            if 0 <= s < 10 and 0 <= t < 4:
                want[b, :, s] = kn[t]
    assert torch.equal(kc, want)


def test_append_many_rows():
    # more rows than the search looks at in one step, empty ones among them
    rng = np.random.RandomState(6)
    counts = rng.randint(0, 3, 1200)
    n = int(counts.sum())
    kc = torch.zeros(1200, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kn, vn = _randn(1, n + 4, 1, 64), _randn(2, n + 4, 1, 64)
    starts = rng.randint(0, 3, 1200).astype(np.int32)
    cu = _cu(counts) + 2  # two entries in front and two behind belong to nobody
    wk, e = torch.zeros_like(kc), 2
    for b in range(1200):
        for i in range(counts[b]):
            wk[b, :, starts[b] + i] = kn[e]
            e += 1
    api.cache_append(kc, vc, kn, vn, torch.from_numpy(starts).cuda(), cu_seqlens=cu)
    api.check()
    assert torch.equal(kc, wk)


@pytest.mark.parametrize("cu", [[0, 3, 2, 4], [-1, 1, 2, 4], [0, 1, 2, 9]])
def test_append_bad_prefix_sums_are_reported(cu):
    kc = torch.zeros(3, 1, 10, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kn, vn = _randn(1, 4, 1, 64), _randn(2, 4, 1, 64)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    api.cache_append(kc, vc, kn, vn, zero, cu_seqlens=torch.tensor(cu, dtype=torch.int32,
                                                                    device="cuda"))
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT


# ------------------------------------------------------------------ failure reporting


@pytest.mark.parametrize("call", ["packed", "tree", "tree_wide"])
def test_timeout_is_reported_and_the_next_call_is_correct(call):
    # the first block withholds a copy: its waits run out, nothing faults
    ctx, drafts, H_q = [700, 90], ([9, 3] if call != "tree_wide" else [60, 40]), 8
    T = max(drafts)
    q, kn, vn, kc, vc, cl = _tree_inputs(ctx, drafts, 1024, H_q, 1, 128, 97)

    def run():
        if call == "packed":
            return api.prefill_packed(q, kn, vn, _cu(drafts))
        return api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=T)

    api.check()
    assert api.gqa_attn_debug_inject_timeout(1) == api.GQA_OK
    run()
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_TIMEOUT
    o, lse = run()
    api.check()
    if call == "packed":
        _check_packed(o, lse, q, kn, vn, drafts, drafts, True, 1 / math.sqrt(128))
    else:
        _check_tree(o, lse, q, kn, vn, kc, vc, ctx, drafts, None, 1 / math.sqrt(128))


# ----------------------------------------------------------------------- together


def test_serving_steps_agree_with_decode():
    # packed prompts -> cache -> two draft steps, of which a path is accepted -> plain decode
    H_q, H_kv, d, S_max, lens = 16, 2, 128, 512, [200, 1, 77]
    B, scale = 3, 1 / math.sqrt(d)
    q, k, v = _packed_inputs(lens, lens, H_q, H_kv, d, 61)
    kc = torch.full((B, H_kv, S_max, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    o, lse = api.prefill_packed(q, k, v, _cu(lens))
    api.cache_append(kc, vc, k, v, zero, cu_seqlens=_cu(lens))
    _check_packed(o, lse, q, k, v, lens, lens, True, scale)
    # the last query of every prompt, again, as a decode over the cache
    ends = np.cumsum(lens) - 1
    od, ld = api.decode(q[ends].contiguous(), kc, vc, torch.tensor(lens, dtype=torch.int32,
                                                                   device="cuda"))
    a = 0
    for b, n in enumerate(lens):
        r = ref.attend(_np(q[ends[b]])[None], _np(k[a:a + n]), _np(v[a:a + n]),
                       np.ones((1, n), bool), scale)
        ref.check(od[b:b + 1], ld[b:b + 1], r)
        a += n
    ctx = list(lens)
    for step in range(2):
        drafts, accepted = [7, 5, 9], [[0, 2, 5], [0], [0, 1, 3, 8]]
        qd, kn, vn, _, _, _ = _tree_inputs(ctx, drafts, 1, H_q, H_kv, d, 70 + step)
        cl = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        vis, words = [], []
        for n, path in zip(drafts, accepted):  # the accepted path is a branch of the tree
            m = np.eye(n, dtype=bool)
            m[:, 0] = True
            for i, t in enumerate(path):
                m[t, path[:i]] = True
            vis.append(m)
            words.append(np.packbits(np.pad(m, ((0, 0), (0, 32 - n))), axis=1,
                                     bitorder="little").view(np.int32))
        mask = torch.from_numpy(np.concatenate(words)).cuda()
        o, lse = api.decode_tree(qd, kn, vn, kc, vc, cl, cu_seqlens=_cu(drafts), max_tokens=9,
                                 tree_mask=mask)
        _check_tree(o, lse, qd, kn, vn, kc, vc, ctx, drafts, vis, scale, f"step {step}")
        first = np.cumsum([0] + drafts)
        index = np.concatenate([first[b] + np.array(p) for b, p in enumerate(accepted)])
        api.cache_append(kc, vc, kn, vn, cl, cu_seqlens=_cu([len(p) for p in accepted]),
                         index=torch.from_numpy(index.astype(np.int32)).cuda())
        ctx = [n + len(p) for n, p in zip(ctx, accepted)]
        last = [int(first[b]) + p[-1] for b, p in enumerate(accepted)]
        od, ld = api.decode(qd[last].contiguous(), kc, vc,
                            torch.tensor(ctx, dtype=torch.int32, device="cuda"))
        api.check()
        for b in range(B):  # the accepted leaf sees the same tokens through either call
            n = ctx[b]
            r = ref.attend(_np(qd[last[b]])[None], _np(kc[b, :, :n].transpose(0, 1)),
                           _np(vc[b, :, :n].transpose(0, 1)), np.ones((1, n), bool), scale)
            ref.check(od[b:b + 1], ld[b:b + 1], r, "decode")
            ref.check(o[last[b]][None], lse[last[b]][None], r, "tree")


def test_captured_calls_replay_on_new_inputs():
    # two graphs captured on one stream, replayed on two streams at the same time
    H_q, H_kv, d, S_max = 16, 2, 128, 2048
    sets = [_tree_inputs([1500, 90], [9, 4], S_max, H_q, H_kv, d, 80 + 10 * i) for i in range(2)]
    cu = _cu([9, 4])
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for q, kn, vn, kc, vc, cl in sets:
            api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=cu, max_tokens=9)
    torch.cuda.synchronize()
    for q, kn, vn, kc, vc, cl in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            o, lse = api.decode_tree(q, kn, vn, kc, vc, cl, cu_seqlens=cu, max_tokens=9)
            p, pl = api.prefill_packed(q, kn, vn, cu)
            api.cache_append(kc, vc, kn, vn, cl, cu_seqlens=cu)
        graphs.append(g)
        outs.append((o, lse, p, pl))
    for (q, kn, vn, kc, vc, cl), seed in zip(sets, (200, 300)):
        for t, s in zip((q, kn, vn), range(3)):
            t.copy_(_randn(seed + s, *t.shape))
        cl.copy_(torch.tensor([1000 + seed, seed // 2], dtype=torch.int32))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):  # replays write the same slots with the same values
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    api.check()
    for (q, kn, vn, kc, vc, cl), (o, lse, p, pl) in zip(sets, outs):
        ctx = cl.tolist()
        _check_tree(o, lse, q, kn, vn, kc, vc, ctx, [9, 4], None, 1 / math.sqrt(d))
        _check_packed(p, pl, q, kn, vn, [9, 4], [9, 4], True, 1 / math.sqrt(d))
        assert torch.equal(kc[0, :, ctx[0]:ctx[0] + 9], kn[:9].transpose(0, 1))


def test_two_streams_at_once():
    H_q, H_kv, d = 16, 2, 128
    sets = [_tree_inputs([3000, 1, 512], [40, 3, 12], 3100, H_q, H_kv, d, 400 + 10 * i)
            for i in range(2)]
    cu = _cu([40, 3, 12])
    want = [api.decode_tree(*s, cu_seqlens=cu, max_tokens=40) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(api.decode_tree(*sets[i], cu_seqlens=cu, max_tokens=40,
                                          stream=streams[i]))
    torch.cuda.synchronize()
    api.check()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_memory_freed_around_a_call_on_another_stream_is_not_reused():
    # the current stream frees the inputs of a call that waits on a side stream, and writes over
    # whatever memory the allocator hands out next; and the results do not take memory that the
    # current stream still reads
    q, k, v = (_randn(500 + i, 4096, 8, 128) for i in range(3))
    cu = _cu([4096])
    side = torch.cuda.Stream()

    def fill(value):
        return torch.full(q.shape, value, dtype=torch.bfloat16, device="cuda")

    # (every kernel has run once, on either stream: loading one may wait for the device)
    want, want_lse = api.prefill_packed(q, k, v, cu)
    kept = [fill(1.0) for _ in range(8)]
    for t in kept:
        torch.mul(want, 1, out=t)
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            torch.cuda._sleep(1000)
    copies = [t.clone() for t in (q, k, v)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    o, lse = api.prefill_packed(*copies, cu, stream=side)
    del copies
    over = [fill(float("nan")) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)

    x = [fill(1.0) for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for t, u in zip(x, kept):
        torch.mul(t, 1, out=u)
    del x, t
    o, lse = api.prefill_packed(q, k, v, cu, stream=side)
    torch.cuda.synchronize()
    api.check()
    assert torch.equal(o, want) and all((u == 1).all() for u in kept)
    del over


def test_most_rows():
    # the largest batch: one token a row, prompts, drafts and appended tokens
    B, d, S_max = 65535, 64, 8
    kc = torch.zeros(B, 1, S_max, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v = (_randn(510 + i, B, 1, d) for i in range(3))
    ones = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ctx = (ones[:B] % 2).contiguous()
    o, lse = api.prefill_packed(q, k, v, ones)
    assert torch.equal(o, v)  # a token that sees itself alone
    # row b holds b % 2 tokens in the cache, each the row's own
    api.cache_append(kc, vc, k, v, torch.zeros_like(ctx), cu_seqlens=ones)
    o, lse2 = api.decode_tree(q, k, v, kc, vc, ctx, cu_seqlens=ones, max_tokens=1)
    api.check()
    assert torch.equal(kc[:, :, 0], k) and torch.equal(vc[:, :, 0], v)
    assert torch.equal(o, v)  # the same value twice keeps its value
    more = lse2.flatten() - lse.flatten() - ctx * math.log(2)
    assert more.abs().max().item() < 1e-4  # |lse| <= 16: a few steps of 2^-20
