"""The paged serving step on the GPU: norm and rotation, paged append, paged attention and the
verification of drafted tokens, each against plain arithmetic in 64 bits (_ragged.py derives the
elementwise bounds of attention) or bit for bit, and the four together."""

import math

import numpy as np
import pytest
import torch

import _ragged as ref
from gqa_attention_split_gb300 import api, build

pytestmark = pytest.mark.gpu

HEADS = {"g8": (8, 1, 128), "g8x2": (16, 2, 128), "g1d64": (3, 3, 64), "g7": (14, 2, 128),
         "g3d64": (6, 2, 64), "g16": (16, 1, 128)}
BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + [int(x) for x in np.cumsum(lens)])


def _np(t):
    return t.double().cpu().numpy()


def _table(lens, page, seed=0, spare=2, junk=0):
    """Pages of each row, scattered over the pool; entries that no key needs hold junk."""
    need = [-(-n // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(need) + spare)
    t = np.full((len(lens), max(1, max(need)) + 1), junk, dtype=np.int64)
    a = 0
    for b, n in enumerate(need):
        t[b, :n] = order[a:a + n]
        a += n
    return t.astype(np.int32), sum(need) + spare


def _rows(pages, table, b, n):
    """Keys 0 .. n - 1 of row b: [n, H_kv, d] float64."""
    page = pages.shape[2]
    at = torch.as_tensor(table[b][:-(-n // page)], device="cuda").long()
    x = pages[at].permute(0, 2, 1, 3).reshape(-1, pages.shape[1], pages.shape[3])
    return _np(x[:n])


def _check(o, lse, q, kp, vp, table, tokens, lens, causal, scale, what=""):
    a = 0
    for b, (T, n) in enumerate(zip(tokens, lens)):
        if T:
            vis = ref.causal_visible(T, n) if causal else np.ones((T, n), bool)
            ref.check(o[a:a + T], lse[a:a + T],
                      ref.attend(_np(q[a:a + T]), _rows(kp, table, b, n), _rows(vp, table, b, n),
                                 vis, scale), f"{what} row {b}: {T} tokens, {n} keys")
        a += T


def _attend(heads, tokens, lens, page, causal=True, seed=0, **kw):
    H_q, H_kv, d = HEADS[heads] if isinstance(heads, str) else heads
    table, pages = _table(lens, page, seed, junk=BIG)
    q = _randn(seed, sum(tokens), H_q, d)
    kp, vp = _randn(seed + 1, pages, H_kv, page, d), _randn(seed + 2, pages, H_kv, page, d)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), cu_seqlens=_cu(tokens),
                                 max_tokens=max(tokens), causal=causal, **kw)
    api.check()
    _check(o, lse, q, kp, vp, table, tokens, lens, causal, 1 / math.sqrt(d),
           f"{heads} page {page}")
    return o, lse


# ------------------------------------------------------------------- attention


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_single_tokens(heads, page):
    _attend(heads, [1] * 6, [1, 17, 128, 129, 700, 1000], page)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_mixed_step(heads, causal):
    # chunks, drafts, single tokens, rows without tokens, keys or either at once
    _attend(heads, [150, 1, 6, 0, 40, 1, 3, 0, 257], [150, 900, 333, 55, 40, 1, 3, 0, 700], 16,
            causal)


@pytest.mark.parametrize("heads", HEADS)
def test_fewer_keys_than_tokens(heads):
    # the first tokens see nothing; whole blocks that see nothing; no keys at all
    for causal in (True, False):
        _attend(heads, [40, 300, 9, 5], [13, 130, 0, 4], 32, causal)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("tokens", [[1, 1], [5, 2], [70, 33], [300, 1]],
                         ids=["one", "drafts", "chunk", "long"])
def test_long_rows_are_cut(heads, tokens):
    _attend(heads, tokens, [9001, 20011], 64)


def test_one_long_row_over_all_ctas():
    _attend("g8", [1], [70001], 128)
    _attend("g7", [3], [33333], 16)


@pytest.mark.parametrize("B", [40, 333])
def test_many_rows(B):
    rng = np.random.RandomState(B)
    _attend("g3d64", list(rng.randint(0, 3, B)), list(rng.randint(3, 400, B)), 16)
    _attend("g8x2", [1] * B, list(rng.randint(1, 600, B)), 32)


@pytest.mark.parametrize("max_keys", [100, 512, 640, None])
def test_key_bound(max_keys):
    _attend("g8x2", [1, 7, 40], [100, 60, 99], 16, max_keys=max_keys)


@pytest.mark.parametrize("H_q,H_kv", [(32, 1), (100, 1), (128, 1), (18, 2)])
def test_large_groups_of_heads(H_q, H_kv):
    _attend((H_q, H_kv, 128), [7, 1, 150], [300, 1500, 150], 64)


def test_equal_rows_without_prefix_sums():
    q, kp, vp = _randn(3, 12, 8, 128), _randn(4, 40, 2, 16, 128), _randn(5, 40, 2, 16, 128)
    lens = [30, 100, 77]
    table, _ = _table(lens, 16)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), scale=0.2)
    api.check()
    _check(o, lse, q, kp, vp, table, [4, 4, 4], lens, True, 0.2)


def test_shared_prefix_pages_and_strided_pool():
    # K and V of a page side by side in one pool; two rows share their first pages
    H_q, H_kv, d, page = 16, 2, 128, 32
    pool = _randn(7, 30, 2, H_kv, page, d)
    kp, vp = pool[:, 0], pool[:, 1]
    lens, tokens = [300, 290, 64], [1, 20, 2]
    table = np.zeros((3, 12), np.int32)
    table[0, :10] = range(10)
    table[1, :10] = list(range(5)) + list(range(15, 20))
    table[2, :2] = [29, 28]
    q = _randn(8, 23, H_q, d)
    qs = torch.empty(23, 3 * H_q, d, dtype=torch.bfloat16, device="cuda")[:, H_q:2 * H_q]
    qs.copy_(q)
    o, lse = api.paged_attention(qs, kp, vp, _i32(table), _i32(lens), cu_seqlens=_cu(tokens),
                                 max_tokens=32)
    api.check()
    _check(o, lse, q, kp, vp, table, tokens, lens, True, 1 / math.sqrt(d))


@pytest.mark.parametrize("heads", ["g8x2", "g3d64"])
@pytest.mark.parametrize("page", [16, 128])
def test_what_a_token_does_not_see_never_reaches_it(heads, page):
    # NaN and infinities in pages of no row, behind the rows' last keys, and in later tokens' keys
    H_q, H_kv, d = HEADS[heads]
    tokens, lens = [1, 6, 50], [700, 90, 150]
    table, pages = _table(lens, page, 1, spare=3, junk=-5)
    kp, vp = _randn(1, pages, H_kv, page, d), _randn(2, pages, H_kv, page, d)
    clean_k, clean_v = kp.clone(), vp.clone()
    used = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for s in range(n):
            used[table[b, s // page], s % page] = True
    free = torch.from_numpy(~used).cuda()[:, None, :, None]
    kp.masked_fill_(free, float("nan"))
    vp.masked_fill_(free, float("inf"))
    q = _randn(3, sum(tokens), H_q, d)
    args = dict(cu_seqlens=_cu(tokens), max_tokens=50)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), **args)
    api.check()
    _check(o, lse, q, clean_k, clean_v, table, tokens, lens, True, 1 / math.sqrt(d))
    # the last key of every row is not a number: only the last token of a row sees it
    for b, n in enumerate(lens):
        kp[table[b, (n - 1) // page], :, (n - 1) % page] = float("nan")
        vp[table[b, (n - 1) // page], :, (n - 1) % page] = float("-inf")
    o2, lse2 = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), **args)
    api.check()
    last = torch.tensor(np.cumsum(tokens) - 1, device="cuda")
    keep = torch.ones(sum(tokens), dtype=torch.bool, device="cuda")
    keep[last] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert torch.isnan(lse2[last]).all()


def test_infinite_values_that_a_token_sees():
    # an infinite V in the last keys of a cut row: infinite for those that see it, and only there
    H_q, H_kv, d, page = 8, 1, 128, 16
    lens, tokens = [5000], [4]
    table, pages = _table(lens, page, 2)
    kp, vp = _randn(1, pages, H_kv, page, d), _randn(2, pages, H_kv, page, d)
    q = _randn(3, 4, H_q, d)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens))
    vp[table[0, 4998 // page], 0, 4998 % page, 5] = float("inf")
    o2, lse2 = api.paged_attention(q, kp, vp, _i32(table), _i32(lens))
    api.check()
    assert torch.equal(lse, lse2)
    assert torch.isinf(o2[2:, :, 5]).all()
    o2[2:, :, 5] = o[2:, :, 5]
    assert torch.equal(o, o2)


def test_rows_behind_the_last_sequence_are_left():
    lens, tokens = [40, 300], [3, 2]
    table, pages = _table(lens, 16)
    q, kp, vp = _randn(1, 9, 8, 128), _randn(2, pages, 2, 16, 128), _randn(3, pages, 2, 16, 128)
    out = torch.full_like(q, 7.0)
    lse = torch.full((9, 8), 7.0, device="cuda")
    api.paged_attention(q, kp, vp, _i32(table), _i32(lens), cu_seqlens=_cu(tokens), max_tokens=3,
                        out=out, lse=lse)
    api.check()
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    _check(out, lse, q, kp, vp, table, tokens, lens, True, 1 / math.sqrt(128))


def _expect_bad_input():
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT


def test_bad_lengths_and_pages_are_reported():
    lens, tokens = [40, 300, 77], [1, 1, 1]
    table, pages = _table(lens, 16)
    q, kp, vp = _randn(1, 3, 8, 128), _randn(2, pages, 2, 16, 128), _randn(3, pages, 2, 16, 128)

    def run(table, lens, cu=None, **kw):
        return api.paged_attention(q, kp, vp, _i32(table), _i32(lens), cu_seqlens=cu, **kw)

    slots = table.shape[1] * 16
    for bad in (-1, slots + 1, 2 ** 31 - 1):
        run(table, [40, bad, 77])
        _expect_bad_input()
    run(table, lens, max_keys=200)
    _expect_bad_input()
    for cu in ([0, 1, 9, 3], [0, 2, 1, 3], [-1, 1, 2, 3]):
        run(table, lens, _i32(cu), max_tokens=3)
        _expect_bad_input()
    run(table, lens, _i32([0, 3, 3, 3]), max_tokens=2)
    _expect_bad_input()
    for page in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 3] = page
        o, lse = run(t, lens)
        _expect_bad_input()
        _check(o[::2], lse[::2], q[::2], kp, vp, table[::2], [1, 1], lens[::2], True,
               1 / math.sqrt(128))  # the other rows are right
    o, lse = run(table, lens)
    api.check()
    _check(o, lse, q, kp, vp, table, tokens, lens, True, 1 / math.sqrt(128))


def test_bits_repeat_and_streams_graphs_and_workspaces():
    lens, tokens = [3000, 64, 9000, 1], [1, 5, 40, 1]
    H_q, H_kv, d, page = 28, 4, 128, 32
    table, pages = _table([9100] * 4, page)
    q, kp, vp = (_randn(1, 47, H_q, d), _randn(2, pages, H_kv, page, d),
                 _randn(3, pages, H_kv, page, d))
    tab, ln, cu = _i32(table), _i32(lens), _cu(tokens)
    want, want_l = api.paged_attention(q, kp, vp, tab, ln, cu_seqlens=cu, max_tokens=40)
    api.check()
    _check(want, want_l, q, kp, vp, table, tokens, lens, True, 1 / math.sqrt(d))
    for _ in range(5):
        o, lse = api.paged_attention(q, kp, vp, tab, ln, cu_seqlens=cu, max_tokens=40)
        assert torch.equal(o, want) and torch.equal(lse, want_l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = api.paged_attention(q, kp, vp, tab, ln, cu_seqlens=cu, max_tokens=40, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(lse, want_l)
    # a graph goes by the lengths that it finds when it is replayed
    n = api.gqa_attn_paged_attention_workspace_size(H_q, H_kv, d, 40)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, out_l = torch.empty_like(want), torch.empty_like(want_l)

    def call():
        api.paged_attention(q, kp, vp, tab, ln, cu_seqlens=cu, max_tokens=40, out=out, lse=out_l,
                            workspace=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for new in ([3000, 64, 9000, 1], [17, 9100, 40, 5000], [1, 5, 300, 2]):
        ln.copy_(_i32(new))
        g.replay()
        api.check()
        _check(out, out_l, q, kp, vp, table, tokens, new, True, 1 / math.sqrt(d))
    with pytest.raises(api.GqaError) as e:
        api.paged_attention(q, kp, vp, tab, ln, cu_seqlens=cu, max_tokens=40, workspace=ws[:-256])
    assert e.value.code == api.GQA_ERR_WORKSPACE


def test_random_steps():
    rng = np.random.RandomState(11)
    for it in range(25):
        heads = list(HEADS)[rng.randint(len(HEADS))]
        B = rng.randint(1, 20)
        most = [1, 5, 30, 200][rng.randint(4)]
        tokens = [int(x) for x in rng.randint(0, most + 1, B)]
        if not sum(tokens):
            tokens[0] = 1
        lens = [int(t + np.exp(rng.uniform(0, 8.5))) - 1 - (rng.randint(0, 9) if it % 5 == 0 else 0)
                for t in tokens]
        lens = [max(0, n) for n in lens]
        _attend(heads, tokens, lens, [16, 32, 64, 128, 256][rng.randint(5)], bool(rng.randint(5)),
                seed=it)


# ------------------------------------------------------------------- norm and rotation


def _norm_want(x, w, pos, freq, eps, sections, interleaved):
    """64 bits, and the bound: half a bf16 step of the result, 2^-8, and 2^-18 of the magnitudes
    that it is made of. The latter is for 32 bits: a sum of d squares in fp32 (its relative error
    is below 20 * 2^-24 with 8 terms a lane and 4 steps over the lanes, halved by the root),
    rsqrt, the weight's, the sine's and four products' roundings (2^-23 or less each) and the angle
    (2^-26 turns, 2^-23 radians): below 2^-19 together."""
    x = _np(x)
    n, H, d = x.shape
    P = len(freq)
    z = x
    if eps is not None:
        z = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
        if w is not None:
            z = z * w
    pos = np.asarray(pos, np.float64).reshape(-1, n)
    axis = np.repeat(np.arange(len(sections or (P,))), sections or (P,))
    a = pos[axis].T * np.asarray(freq, np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    one = np.arange(P) * 2 if interleaved else np.arange(P)
    two = one + 1 if interleaved else one + P
    y, mag = z.copy(), np.abs(z)
    y[..., one] = z[..., one] * c - z[..., two] * s
    y[..., two] = z[..., two] * c + z[..., one] * s
    mag[..., one] = mag[..., two] = np.abs(z[..., one]) + np.abs(z[..., two])
    return y, np.abs(y) * 2.0 ** -8 + mag * 2.0 ** -18


def _freq(P, base=10000.0):
    return (base ** -(np.arange(P) / P)).astype(np.float32)


def _close(got, want, what=""):
    y, bound = want
    err = np.abs(_np(got) - y)
    assert (err <= bound).all(), f"{what}: worst {(err / np.maximum(bound, 1e-300)).max():.3f}x"


@pytest.mark.parametrize("H_q,H_kv,d", [(8, 1, 128), (64, 8, 128), (3, 3, 64), (28, 4, 128),
                                        (1, 1, 64), (7, 5, 64)])
@pytest.mark.parametrize("n", [1, 5, 100, 700])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
def test_norm_rope(H_q, H_kv, d, n, interleaved):
    q, k = _randn(n, n, H_q, d), _randn(n + 1, n, H_kv, d)
    rng = np.random.RandomState(n)
    for P, sections, far, norm, wide in ((d // 2, None, 200000, True, False),
                                         (d // 4, None, 1 << 20, True, True),
                                         (d // 2, (5, d // 2 - 5), 3000, True, False),
                                         (d // 2, (8, 12, 0, d // 2 - 20), 5000, False, False),
                                         (8, (3, 4, 1), 5000, True, None)):
        f = _freq(P)
        shape = (n,) if sections is None else (len(sections), n)
        pos = rng.randint(-far, far, shape).astype(np.int32)
        w = [None, None]
        if norm and wide is not None:
            dt = torch.float32 if wide else torch.bfloat16
            w = [(1 + 0.2 * _randn(9 + i, d).float()).to(dt) for i in range(2)]
        eps = 1e-5 if norm else None
        qo, ko = api.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(),
                                  q_weight=w[0], k_weight=w[1], eps=eps, sections=sections,
                                  interleaved=interleaved)
        for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
            _close(got, _norm_want(x, None if wt is None else _np(wt), pos, f, eps, sections,
                                   interleaved), f"{P} pairs, sections {sections}")


def test_norm_rope_far_positions():
    # the whole range of int32; frequencies above a turn per token
    n, d = 64, 128
    q, k = _randn(1, n, 4, d), _randn(2, n, 2, d)
    rng = np.random.RandomState(0)
    pos = rng.randint(-2 ** 31, 2 ** 31, n).astype(np.int32)
    pos[:4] = [2 ** 31 - 1, -2 ** 31, 0, 1]
    f = _freq(64)
    qo, _ = api.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda())
    want, bound = _norm_want(q, None, pos, f, 1e-6, None, False)
    # in turns the product of 2^31 positions is off by 2^31 / 6.3 * 2^-51: 2^-22 turns, and numpy's
    # by as much: 2^-18 radians together
    mag = np.abs(want)
    other = np.concatenate([mag[..., 64:], mag[..., :64]], -1)
    assert (np.abs(_np(qo) - want) <= bound + other * 2.0 ** -18).all()
    f = (np.arange(64) + 0.37).astype(np.float32)
    pos = rng.randint(0, 100000, n).astype(np.int32)
    qo, _ = api.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda())
    _close(qo, _norm_want(q, None, pos, f, 1e-6, None, False), "large frequencies")


def test_norm_rope_strides_in_place_and_queries_alone():
    n, H_q, H_kv, d = 77, 16, 2, 128
    qkv = _randn(5, n, H_q + 2 * H_kv, d)
    q, k, v = qkv.split([H_q, H_kv, H_kv], 1)
    pos = _i32(list(range(100, 100 + n)))
    f = torch.from_numpy(_freq(64)).cuda()
    w = 1 + 0.1 * _randn(6, d)
    qo, ko = api.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
    heads_first = torch.empty(H_q, n, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    qt, kt = api.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w, q_out=heads_first)
    assert torch.equal(qt, qo) and torch.equal(kt, ko) and qt is heads_first
    alone, none = api.qk_norm_rope(q, None, pos, f, q_weight=w)
    assert torch.equal(alone, qo) and none is None
    before = v.clone()
    a, b = api.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w, q_out=q, k_out=k)
    assert a is q and torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s, _ = api.qk_norm_rope(qo, ko, pos, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s, api.qk_norm_rope(qo, ko, pos, f)[0])
    for bad in (dict(sections=(32, 32)), dict(eps=None, q_weight=w),
                dict(q_weight=w, k_weight=w.float())):
        with pytest.raises((ValueError, TypeError)):
            api.qk_norm_rope(q, k, pos, f, **bad)


def test_norm_rope_values_at_the_edges():
    # zeros (eps alone), infinities and NaN stay in their head; channels behind the pairs are kept
    n, H, d = 6, 4, 64
    q = _randn(1, n, H, d)
    q[0, 0] = 0
    q[1, 1, 3] = float("nan")
    q[2, 2, 40] = float("inf")
    pos, f = _i32([5] * n), torch.from_numpy(_freq(16)).cuda()
    clean = q.clone()
    clean[1, 1, 3] = clean[2, 2, 40] = 0
    got = api.qk_norm_rope(q, None, pos, f)[0]
    plain = api.qk_norm_rope(clean, None, pos, f)[0]
    assert (got[0, 0] == 0).all()
    keep = torch.ones(n, H, dtype=torch.bool, device="cuda")
    keep[1, 1] = keep[2, 2] = False
    assert torch.equal(got[keep], plain[keep]) and torch.isnan(got[1, 1]).all()
    raw = api.qk_norm_rope(q, None, pos, f, eps=None)[0]
    assert torch.equal(raw[2, 2, 32:], q[2, 2, 32:])  # behind the 16 pairs: as they are
    assert torch.isfinite(raw[2, 2, :32]).all()


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("page", [16, 64, 128, 384])
@pytest.mark.parametrize("H_kv,d", [(8, 128), (1, 64), (3, 64)])
def test_paged_append(page, H_kv, d):
    starts, counts = [0, 517, 33, 700, 5], [130, 1, 0, 77, 400]
    lens = [a + c for a, c in zip(starts, counts)]
    table, pages = _table(lens, page, 3, junk=BIG)
    pool = _randn(1, pages, 2, H_kv, page, d)
    want = pool.clone()
    kn, vn = _randn(2, sum(counts), H_kv, d), _randn(3, sum(counts), 2 * H_kv, d)[:, H_kv:]
    api.paged_append(pool[:, 0], pool[:, 1], kn, vn, _i32(table), _i32(starts),
                     cu_seqlens=_cu(counts))
    api.check()
    e = 0
    for b, (t, c) in enumerate(zip(starts, counts)):
        for i in range(c):
            p, s = int(table[b, (t + i) // page]), (t + i) % page
            want[p, 0, :, s], want[p, 1, :, s] = kn[e], vn[e]
            e += 1
    assert torch.equal(pool, want)


def test_paged_append_by_index_and_bad_entries():
    page, H_kv, d = 16, 2, 128
    table, pages = _table([64, 64], page, 4)
    table[:, -1] = 0
    kp, vp = _randn(1, pages, H_kv, page, d), _randn(2, pages, H_kv, page, d)
    kn, vn = _randn(3, 9, H_kv, d), _randn(4, 9, H_kv, d)
    wk, wv = kp.clone(), vp.clone()
    api.paged_append(kp, vp, kn, vn, _i32(table), _i32([14, 30]), cu_seqlens=_cu([3, 2]),
                     index=_i32([8, 0, 3, 3, 5]))
    api.check()
    for b, s, src in ((0, 14, 8), (0, 15, 0), (0, 16, 3), (1, 30, 3), (1, 31, 5)):
        wk[table[b, s // page], :, s % page] = kn[src]
        wv[table[b, s // page], :, s % page] = vn[src]
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    slots = table.shape[1] * page
    bad = table.copy()
    bad[0, 1] = pages
    bad[1, 1] = -1
    for args in ((table, [-1, slots], [0, 1]), (table, [2 ** 31 - 1, -2 ** 31], [0, 1]),
                 (table, [0, 0], [9, -1]), (bad, [16, 31], [0, 1])):
        api.paged_append(kp, vp, kn, vn, _i32(args[0]), _i32(args[1]), index=_i32(args[2]))
        _expect_bad_input()
        assert torch.equal(kp, wk) and torch.equal(vp, wv)


# ------------------------------------------------------------------- verification


def _dists(seed, rows, V, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.softmax(torch.randn(rows, V, generator=g, device="cuda") * spread, -1)


def _verify_want(p, q, x, ua, us, counts):
    acc, nxt = [], []
    a = 0
    p = p.double().cpu().numpy()
    q = None if q is None else q.double().cpu().numpy()
    x, ua, us = (t.cpu().numpy() for t in (x, ua, us))
    for b, n in enumerate(counts):
        k = 0
        while k < n and float(ua[a + k]) * (1.0 if q is None else q[a + k, x[a + k]]) < \
                p[a + b + k, x[a + k]]:
            k += 1
        w = p[a + b + k].copy()
        if k < n:
            if q is None:
                w[x[a + k]] = 0
            else:
                w = np.maximum(w - q[a + k], 0)
            if not w.sum() > 0:
                w = p[a + b + k].copy()
        c = np.cumsum(w)
        v = int(np.searchsorted(c, float(us[b]) * c[-1], side="right"))
        acc.append(k)
        nxt.append(min(v, int(np.flatnonzero(w).max())))
        a += n
    return acc, nxt


def _verify(counts, V, seed=0, dist=True, pad=0, equal=False):
    n, B = sum(counts), len(counts)
    p = _dists(seed, n + B, V + pad)[:, :V]
    rows = [a + b + i for b, (a, c) in enumerate(zip(np.cumsum([0] + counts), counts))
            for i in range(c)]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = p[rows] * torch.exp(0.5 * torch.randn(n, V, generator=g, device="cuda"))
    q = q / q.sum(-1, keepdim=True) if n else q
    x = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32) if n else _i32([])
    ua, us = torch.rand(n, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    qd = q if dist else None
    acc, nxt = api.verify_drafts(p, x, ua, us, None if equal else _cu(counts), draft_probs=qd)
    api.check()
    want = _verify_want(p, qd, x, ua, us, counts)
    assert acc.tolist() == want[0] and nxt.tolist() == want[1]
    return want


@pytest.mark.parametrize("dist", [True, False], ids=["probs", "certain"])
@pytest.mark.parametrize("V", [1, 2, 31, 128, 1000, 4099, 32000, 128259])
def test_verify(V, dist):
    _verify([3, 0, 7, 1, 5], V, 1, dist)


def test_verify_batches():
    _verify([4] * 6, 50257, 2, equal=True)
    _verify([0] * 5, 20000, 3)
    _verify([5], 151936, 4)
    _verify([2, 3], 1500, 5, pad=37)
    seen = set()
    for seed in range(6):
        for k, n in zip(_verify([i % 6 for i in range(200)], 700, 10 + seed)[0], range(200)):
            seen.add(k)
    assert len(seen) >= 5  # rows of every outcome
    _verify([1 + i % 2 for i in range(700)], 300, 20)


def test_verify_borders():
    # p = q throughout: u q < p always stands but for u q = p; the sum of max(p - q, 0) is 0
    V = 300
    p = _dists(1, 2, V)
    q, x = p[:1].clone(), _i32([7])
    acc, nxt = api.verify_drafts(p, x, torch.ones(1, device="cuda"), _i32([0]).float(),
                                 draft_probs=q)
    api.check()
    assert acc.tolist() == [0] and nxt.tolist() == [0]  # drawn from p instead: u = 0 gives 0
    acc, nxt = api.verify_drafts(p, x, torch.full((1,), 1 - 2.0 ** -24, device="cuda"),
                                 torch.full((1,), 1 - 2.0 ** -24, device="cuda"), draft_probs=q)
    assert acc.tolist() == [1]
    # zeros before, between and behind the values above 0, dyadic so that sums are exact
    w = torch.zeros(1, 1000, device="cuda")
    w[0, 200], w[0, 600], w[0, 601] = 0.25, 0.5, 0.25
    e = _i32([]).float()
    for u, v in ((0.0, 200), (0.2499999, 200), (0.25, 600), (0.7499999, 600), (0.75, 601),
                 (1 - 2.0 ** -24, 601), (1.0, 601)):
        acc, nxt = api.verify_drafts(w, _i32([]), e, torch.tensor([u], device="cuda"))
        assert (acc.item(), nxt.item()) == (0, v), u
    api.check()
    # small differences of large values: p - q is far below a 32-bit step of the sums
    p = torch.full((2, 4096), 2.0 ** -12, device="cuda")
    q = p[:1].clone()
    q[0, :2] -= 2.0 ** -34
    q[0, 4095] -= 2.0 ** -34
    for u, v in ((0.1, 0), (0.34, 1), (0.67, 4095)):
        _, nxt = api.verify_drafts(p, _i32([9]), torch.ones(1, device="cuda"),
                                   torch.tensor([u], device="cuda"), draft_probs=q)
        assert nxt.item() == v
    api.check()


def test_verify_bad_input_is_reported():
    V = 500
    p, us, one = _dists(1, 4, V), torch.tensor([0.4, 0.4], device="cuda"), torch.zeros(2, device="cuda")
    want = api.verify_drafts(p, _i32([3, 4]), one, us)
    api.check()
    assert want[0].tolist() == [1, 1]
    for x in (-1, V, 2 ** 31 - 1):
        acc, nxt = api.verify_drafts(p, _i32([x, 4]), one, us)
        _expect_bad_input()
        assert acc.tolist() == [0, 1] and nxt[1] == want[1][1]
    z = p.clone()
    z[3] = 0
    _, nxt = api.verify_drafts(z, _i32([3, 4]), one, us)
    _expect_bad_input()
    assert nxt[1].item() == -1 and nxt[0] == want[1][0]
    z[3] = p[3]
    z[3, 7] = float("inf")
    _, nxt = api.verify_drafts(z, _i32([3, 4]), one, us)
    _expect_bad_input()
    assert nxt[1].item() == -1
    z[3, 7] = float("nan")  # counts as 0
    _, nxt = api.verify_drafts(z, _i32([3, 4]), one, us)
    api.check()
    c = np.cumsum(np.nan_to_num(_np(z[3])))
    assert nxt[1].item() == int(np.searchsorted(c, 0.4000000059604645 * c[-1], side="right"))
    api.verify_drafts(p, _i32([3, 4]), one, us, _i32([0, 5, 2]))
    _expect_bad_input()


# ------------------------------------------------------------------- the four together


def test_serving_step_with_drafts():
    # a chunk of a prompt, then a step with drafted tokens, as one graph that is replayed
    H_q, H_kv, d, page, V = 16, 2, 128, 16, 5000
    lens, drafts = [100, 37, 260], [3, 5, 4]
    tokens = [n + 1 for n in drafts]  # the last token and the drafts
    cap = [n + t for n, t in zip(lens, tokens)]
    table, pages = _table(cap, page, 9)
    tab = _i32(table)
    kp = torch.full((pages, H_kv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    f, w = torch.from_numpy(_freq(64)).cuda(), 1 + 0.1 * _randn(1, d)

    def step(qkv, pos, starts, kv_lens, cu, most):
        q, k, v = qkv.split([H_q, H_kv, H_kv], 1)
        q, k = api.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
        api.paged_append(kp, vp, k, v, tab, starts, cu_seqlens=cu)
        return q, api.paged_attention(q, kp, vp, tab, kv_lens, cu_seqlens=cu, max_tokens=most)

    def positions(starts, counts):
        return _i32(np.concatenate([np.arange(s, s + c) for s, c in zip(starts, counts)]).tolist())

    zeros = [0, 0, 0]
    x0 = _randn(2, sum(lens), H_q + 2 * H_kv, d)
    q, (o, lse) = step(x0, positions(zeros, lens), _i32(zeros), _i32(lens), _cu(lens), max(lens))
    api.check()
    _check(o, lse, q, kp, vp, table, lens, lens, True, 1 / math.sqrt(d))
    x1 = _randn(3, sum(tokens), H_q + 2 * H_kv, d)
    pos, starts, kv, cu = positions(lens, tokens), _i32(lens), _i32(cap), _cu(tokens)
    step(x1, pos, starts, kv, cu, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, (o, lse) = step(x1, pos, starts, kv, cu, 8)
        proj = o.float().flatten(1).sum(-1, keepdim=True)  # stands in for the model's head
        probs = torch.softmax(torch.cos(proj * torch.arange(1, V + 1, device="cuda") * 1e-3) * 8, -1)
        ua = torch.full((sum(drafts),), 0.3, device="cuda")
        us = torch.full((3,), 0.6, device="cuda")
        x = torch.arange(7, 7 + sum(drafts), dtype=torch.int32, device="cuda")
        acc, nxt = api.verify_drafts(probs, x, ua, us, cu - torch.arange(4, dtype=torch.int32,
                                                                        device="cuda"))
    for seed in (4, 5):
        x1.copy_(_randn(seed, sum(tokens), H_q + 2 * H_kv, d))
        g.replay()
        api.check()
        _check(o, lse, q, kp, vp, table, tokens, cap, True, 1 / math.sqrt(d))
        want = _verify_want(probs, None, x, ua, us, drafts)
        assert (acc.tolist(), nxt.tolist()) == want


# ------------------------------------------------------------------- limits


def test_pages_far_behind_32_bits():
    # a pool of more than 2^32 elements, most of which nobody uses
    H_q, H_kv, d, page, pages = 8, 8, 128, 64, 70000
    kp = torch.empty(pages, H_kv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    starts, counts = [0, 60], [130, 70]
    lens = [130, 130]
    table = np.array([[pages - 1, 5, pages - 2], [pages - 3, 66000, 65999]], np.int32)
    for b in range(2):
        for g in range(3):
            kp[table[b, g]], vp[table[b, g]] = _randn(10 + b, H_kv, page, d), _randn(20 + g, H_kv,
                                                                                    page, d)
    kn, vn = _randn(1, 200, H_kv, d), _randn(2, 200, H_kv, d)
    api.paged_append(kp, vp, kn, vn, _i32(table), _i32(starts), cu_seqlens=_cu(counts))
    q = _randn(3, 70, H_q, d)
    vp[pages - 1, 0, 3, 4] = float("inf")
    args = dict(cu_seqlens=_cu([1, 69]), max_tokens=69)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), **args)
    api.check()
    assert torch.isinf(o[0, 0, 4])
    vp[pages - 1, 0, 3, 4] = 1.0
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), **args)
    api.check()
    _check(o, lse, q, kp, vp, table, [1, 69], lens, True, 1 / math.sqrt(d))
    assert torch.equal(kp[pages - 1, :, 0], kn[0]) and torch.equal(vp[66000, :, 63], vn[197])


@pytest.mark.parametrize("tokens,page", [(1, 16), (6, 128), (40, 32), (40, 128)])
def test_a_withheld_copy_is_reported(tokens, page):
    # (rows so long that the first block has keys to wait for)
    H_q, H_kv, d = 16, 2, 128
    lens = [30000, 500]
    table, pages = _table(lens, page)
    q = _randn(1, 2 * tokens, H_q, d)
    kp, vp = _randn(2, pages, H_kv, page, d), _randn(3, pages, H_kv, page, d)
    api.check()
    assert api.gqa_attn_debug_inject_timeout(1) == api.GQA_OK
    api.paged_attention(q, kp, vp, _i32(table), _i32(lens))
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_TIMEOUT
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens))
    api.check()
    _check(o, lse, q, kp, vp, table, [tokens] * 2, lens, True, 1 / math.sqrt(d))


def test_large_batch():
    # more rows than a scheduling warp keeps in registers, by far; most of them short
    B, page = 20000, 16
    rng = np.random.RandomState(1)
    lens = rng.randint(0, 40, B)
    lens[[7, 15000]] = [3000, 5000]
    table, pages = _table(list(lens), page, 5)
    q = _randn(1, B, 3, 64)
    kp, vp = _randn(2, pages, 1, page, 64), _randn(3, pages, 1, page, 64)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens.tolist()))
    api.check()
    for b in [0, 1, 7, 31, 32, 9999, 15000, B - 1] + list(rng.randint(0, B, 40)):
        _check(o[b:b + 1], lse[b:b + 1], q[b:b + 1], kp, vp, table[b:b + 1], [1], [int(lens[b])],
               True, 1 / 8, f"row {b}")
    assert torch.equal(torch.isneginf(lse).all(1).cpu(), torch.from_numpy(lens == 0))


@pytest.mark.parametrize("rows", [800, 1300])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_many_short_prompts_are_not_cut(causal, rows):
    # a dozen units and more to every CTA; 1300 rows are more than the schedule's table holds
    H_q, H_kv, d, page = 16, 1, 128, 32
    rng = np.random.RandomState(2)
    tokens = [int(t) for t in rng.randint(0, 80, rows)]
    lens = [t + int(rng.randint(0, 30)) for t in tokens]
    table, pages = _table(lens, page, 6, junk=BIG)
    q = _randn(1, sum(tokens), H_q, d)
    kp, vp = _randn(2, pages, H_kv, page, d), _randn(3, pages, H_kv, page, d)
    o, lse = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), cu_seqlens=_cu(tokens),
                                 max_tokens=80, causal=causal)
    api.check()
    first = np.cumsum([0] + tokens)
    for b in [0, 1, 31, 32, 33, rows - 2, rows - 1] + list(rng.randint(0, rows, 60)):
        a, e = first[b], first[b + 1]
        _check(o[a:e], lse[a:e], q[a:e], kp, vp, table[b:b + 1], tokens[b:b + 1], lens[b:b + 1],
               causal, 1 / math.sqrt(d), f"row {b}")
    assert torch.isfinite(o).all()


def test_calls_on_two_streams_at_once():
    # each stream its own rows, workspaces and outputs; the same bits as one call at a time
    H_q, H_kv, d, page = 16, 2, 128, 16
    f = torch.from_numpy(_freq(64)).cuda()
    sets = []
    for s, (tokens, lens) in enumerate([([1] * 20, list(range(50, 4050, 200))),
                                        ([200, 1, 30], [900, 5000, 30])]):
        table, pages = _table(lens, page, s)
        n = sum(tokens)
        sets.append(dict(q=_randn(s, n, H_q, d), kp=_randn(s + 5, pages, H_kv, page, d),
                         vp=_randn(s + 9, pages, H_kv, page, d), table=_i32(table),
                         lens=_i32(lens), cu=_cu(tokens), most=max(tokens),
                         pos=_i32(list(range(n))), p=_dists(s, 8, 3000), u=torch.full(
                             (4,), 0.37 + 0.2 * s, device="cuda")))

    def run(x, stream=None):
        q, _ = api.qk_norm_rope(x["q"], None, x["pos"], f, stream=stream)
        o, lse = api.paged_attention(q, x["kp"], x["vp"], x["table"], x["lens"],
                                     cu_seqlens=x["cu"], max_tokens=x["most"], stream=stream)
        a, t = api.verify_drafts(x["p"], _i32([3, 5, 7, 9]), x["u"], x["u"], stream=stream)
        return o, lse, a, t

    want = [run(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(15):
        for i in range(2):
            got[i].append(run(sets[i], streams[i]))
    torch.cuda.synchronize()
    api.check()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("page", [128, 384, 1024])
@pytest.mark.parametrize("heads", ["g8x2", "g3d64"])
def test_pages_of_several_tiles(page, heads):
    _attend(heads, [1, 1], [3000, 385], page)
    _attend(heads, [1, 150, 7], [2500, 1000, 385], page)
    _attend(heads, [400, 40, 200] * 2, [400, 385, 1030] * 2, page)


@pytest.mark.parametrize("heads", ["g8x2", "g3d64"])
def test_the_page_size_does_not_change_a_bit(heads):
    # long and short prompts, whole and cut rows, single tokens: pages are copied by one warp or
    # two, box by box or tile by tile, and hold the same keys
    H_q, H_kv, d = HEADS[heads]
    for tokens, lens in (([3000, 100, 2500, 40], [3000, 100, 2500, 40]),
                         ([300, 1, 1], [9000, 5000, 77]), ([1] * 5, [9000, 5000, 77, 1, 640])):
        n = sum(lens)
        q, k, v = _randn(1, sum(tokens), H_q, d), _randn(2, n, H_kv, d), _randn(3, n, H_kv, d)
        want = None
        for page in (128, 16, 32, 64, 256):
            table, pages = _table(lens, page, page)
            kp = torch.zeros(pages, H_kv, page, d, dtype=torch.bfloat16, device="cuda")
            vp = torch.zeros_like(kp)
            api.paged_append(kp, vp, k, v, _i32(table), _i32([0] * len(lens)), cu_seqlens=_cu(lens))
            got = api.paged_attention(q, kp, vp, _i32(table), _i32(lens), cu_seqlens=_cu(tokens),
                                      max_tokens=max(tokens), max_keys=max(lens))
            api.check()
            want = want or got
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), page
