"""Measured cases of the ragged-batch operators: attention over packed prompts, attention of
drafted token trees over the KV cache, and appending packed tokens to the cache.

``prefill_packed``  Prompts of different lengths lie one behind the other, [tokens, heads, d].
                    Token t of a sequence with n_q queries and n_k keys sees the keys
                    j <= n_k - n_q + t of its own sequence (causal) or all of them.
``decode_tree``     Every row of a serving batch has a context in the cache and a few drafted
                    tokens that are not in it yet. A drafted token sees the whole context and
                    those drafted tokens of its row that the mask names (its ancestors and
                    itself), or, without a mask, the drafted tokens up to itself.
``cache_append``    Writes packed new tokens, or an indexed choice of them (the accepted path of
                    a draft tree), into the cache slots behind each row's context.

    O = softmax(scale * Q K^T over the visible keys) V        lse = ln sum exp(scale * Q K^T)

A query that sees no key has O = 0 and lse = -inf. K and V head h serves the query heads
h * G .. h * G + G - 1. Tensors are bfloat16, lse is float32.

``own`` chooses between the plain torch form of each operator and the library's calls.
"""

import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------------------- cases


def _packed(name, q_lens, k_lens, H_q, H_kv, d, causal=True, fused=False):
    return {"name": name, "op": "prefill_packed", "q_lens": q_lens, "k_lens": k_lens, "H_q": H_q,
            "H_kv": H_kv, "d": d, "causal": causal, "fused": fused}


def _tree(name, contexts, drafts, S_max, H_q, H_kv, d, mask=True):
    return {"name": name, "op": "decode_tree", "contexts": contexts, "drafts": drafts,
            "S_max": S_max, "H_q": H_q, "H_kv": H_kv, "d": d, "mask": mask}


def _append(name, starts, counts, S_max, H_kv, d, drafts=""):
    return {"name": name, "op": "cache_append", "starts": starts, "counts": counts,
            "S_max": S_max, "H_kv": H_kv, "d": d, "drafts": drafts}


def listed():
    return [
        # A few short turns of a chat, started together: the launch counts. K, Q and V are slices
        # of one fused projection, as they leave a linear layer.
        _packed("packed_short_turns", "17,1,60,9,96,33", "", 64, 8, 128, fused=True),
        # An ordinary prefill step of a server that packs its waiting prompts up to 8K tokens.
        _packed("packed_mixed_8k", "1311,64,905,33,2047,500,128,77,1024,412,731,18,255,686,1,0",
                "", 64, 8, 128),
        # The next chunks of prompts whose first parts are done: the keys reach back further than
        # the queries; head dim 64.
        _packed("packed_chunks_d64", "512,100,301,1,640", "4608,100,2349,1777,6000", 32, 8, 64),
        # Long documents, one of them half of all the tokens.
        _packed("packed_long_32k", "16387,9001,4097,2500,783", "", 64, 8, 128),
        # One speculative step for a single short chat at head dim 64: latency.
        _tree("tree_single_short", "333", "7", 1024, 32, 8, 64),
        # One row with 8K tokens of context and a tree of 26 drafted tokens.
        _tree("tree_8k", "8150", "26", 8192, 64, 8, 128),
        # A batch of ragged contexts, each with its own tree; more queries than one tile holds.
        _tree("tree_batch_32k", "31007,4096,17,12800,22222,129,8191,27003",
              "64,33,64,17,1,48,64,60", 32768, 64, 8, 128),
        # Drafts in a line (no tree), an odd group of heads, four rows.
        _tree("chain_g7", "5003,777,9100,64", "5,5,5,5", 10240, 28, 4, 128, mask=False),
        # A wide tree on 16 query heads to a KV head: the matrix products count.
        _tree("tree_wide_g16", "16000,15999", "128,100", 16384, 128, 8, 128),
        # The K and V of a packed prefill step go into the cache.
        _append("append_prompts", "0,0,512,4096,0,100,2048,0", "2047,1024,905,1311,1,686,731,500",
                8192, 8, 128),
        # One new token for every row of a batch.
        _append("append_step", "100,7,4000,1999,2500,31,0,4095", "1,1,1,1,1,1,1,1", 4096, 8, 128),
        # The accepted tokens of every row's draft tree, picked by index.
        _append("append_accepted",
                "900,17,4000,1999,2500,31,3100,222,1,5,700,800,3999,64,65,1028",
                "4,1,0,5,2,7,3,1,4,4,6,2,1,3,5,8", 4096, 8, 64,
                drafts="32,16,24,32,32,8,32,32,16,32,32,32,20,32,32,32"),
    ]


_HEADS = [(64, 8, 128), (32, 8, 64), (28, 4, 128), (128, 8, 128), (8, 1, 128), (16, 16, 64)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _text(v):
    return ",".join(str(int(x)) for x in v)


def draw(rng):
    op = rng.choice(["prefill_packed", "prefill_packed", "decode_tree", "decode_tree",
                     "cache_append"])
    H_q, H_kv, d = rng.choice(_HEADS)
    if op == "prefill_packed":
        left, q, k = _log(rng, 16, 16384), [], []
        while left > 0 and len(q) < 64:
            n = min(left, _log(rng, 1, 8192))
            q.append(n)
            left -= n
        causal = rng.random() < 0.85
        if rng.random() < 0.4:
            k = [n + (_log(rng, 1, 4096) if rng.random() < 0.7 else 0) for n in q]
        return _packed("", _text(q), _text(k), H_q, H_kv, d, causal, rng.random() < 0.5 and not k)
    B = _log(rng, 1, 16)
    if op == "decode_tree":
        T = _log(rng, 1, 128)
        ctx = [_log(rng, 1, 131072 // B) - 1 for _ in range(B)]
        drafts = [rng.randint(max(1, T // 2), T) for _ in range(B)]
        S_max = max(ctx) + rng.randint(1, 300)
        return _tree("", _text(ctx), _text(drafts), S_max, H_q, H_kv, d, rng.random() < 0.7)
    if rng.random() < 0.5:
        drafts = [rng.randint(1, 64) for _ in range(B)]
        counts = [rng.randint(0, min(8, n)) for n in drafts]
    else:
        drafts, counts = [], [_log(rng, 1, 8192 // B) for _ in range(B)]
    if not sum(counts):
        counts[0] = 1
    starts = [_log(rng, 1, 4096) - 1 for _ in range(B)]
    S_max = max(s + c for s, c in zip(starts, counts)) + rng.randint(0, 300)
    return _append("", _text(starts), _text(counts), S_max, H_kv, d, _text(drafts))


def _lens(text):
    return [int(x) for x in text.split(",")] if text else []


def _cu(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))]).astype(np.int32)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _draft_mask(drafts, seed):
    """Bits of each drafted token's ancestors and itself: int32 [tokens, words]."""
    rng = np.random.RandomState(seed & 0x7FFFFFFF)
    words = (max(drafts) + 31) // 32
    rows = []
    for n in drafts:
        seen = np.zeros((n, 32 * words), dtype=np.uint8)
        for i in range(n):
            if i:  # the parent is one of the tokens just before
                seen[i] = seen[rng.randint(max(0, i - 8), i)]
            seen[i, i] = 1
        rows.append(np.packbits(seen, axis=1, bitorder="little").view(np.int32))
    return torch.from_numpy(np.concatenate(rows)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H_kv, d = case["H_kv"], case["d"]
    s = {"op": case["op"]}
    if case["op"] == "cache_append":
        s["starts"], s["counts"] = _lens(case["starts"]), _lens(case["counts"])
        drafts, B = _lens(case["drafts"]), len(s["starts"])
        n = sum(drafts) if drafts else sum(s["counts"])
        s["k_new"], s["v_new"] = _randn(gen, n, H_kv, d), _randn(gen, n, H_kv, d)
        s["k_cache"] = _randn(gen, B, H_kv, case["S_max"], d)
        s["v_cache"] = _randn(gen, B, H_kv, case["S_max"], d)
        s["index"] = None
        if drafts:  # an increasing path through each row's drafted tokens
            rng = np.random.RandomState(seed & 0x7FFFFFFF)
            pick = [c0 + np.sort(rng.choice(m, c, replace=False))
                    for c0, m, c in zip(_cu(drafts), drafts, s["counts"])]
            s["index"] = torch.from_numpy(np.concatenate(pick).astype(np.int32)).cuda()
        s["starts_dev"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
        s["cu"] = torch.from_numpy(_cu(s["counts"])).cuda()
        return s
    H_q = case["H_q"]
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "prefill_packed":
        s["q_lens"] = _lens(case["q_lens"])
        s["k_lens"] = _lens(case["k_lens"]) or s["q_lens"]
        s["causal"] = case["causal"]
        n_q, n_k = sum(s["q_lens"]), sum(s["k_lens"])
        if case["fused"]:
            qkv = _randn(gen, n_q, H_q + 2 * H_kv, d)
            s["q"], s["k"], s["v"] = qkv.split([H_q, H_kv, H_kv], dim=1)
        else:
            s["q"] = _randn(gen, n_q, H_q, d)
            s["k"], s["v"] = _randn(gen, n_k, H_kv, d), _randn(gen, n_k, H_kv, d)
        s["cu_q"] = torch.from_numpy(_cu(s["q_lens"])).cuda()
        s["cu_k"] = torch.from_numpy(_cu(s["k_lens"])).cuda() if case["k_lens"] else None
        return s
    s["contexts"], s["drafts"] = _lens(case["contexts"]), _lens(case["drafts"])
    n, B = sum(s["drafts"]), len(s["drafts"])
    s["max_tokens"] = max(s["drafts"])
    s["q"] = _randn(gen, n, H_q, d)
    s["k_new"], s["v_new"] = _randn(gen, n, H_kv, d), _randn(gen, n, H_kv, d)
    s["k_cache"] = _randn(gen, B, H_kv, case["S_max"], d)
    s["v_cache"] = _randn(gen, B, H_kv, case["S_max"], d)
    s["context_lens"] = torch.tensor(s["contexts"], dtype=torch.int32, device="cuda")
    s["cu"] = torch.from_numpy(_cu(s["drafts"])).cuda()
    s["mask"] = _draft_mask(s["drafts"], seed) if case["mask"] else None
    return s


# -------------------------------------------------------------------------------- plain forms


def _plain_rows(q, k, v, seen, scale):
    """Attention of q [T, H_q, d] over k, v [H_kv, S, d] in 32 bits; seen: bool [T, S] or None.
    Returns o [T, H_q, d] float32 and lse [T, H_q]."""
    T, H_q, d = q.shape
    H_kv, S = k.shape[0], k.shape[1]
    if S == 0:
        return (torch.zeros(T, H_q, d, device=q.device),
                torch.full((T, H_q), -math.inf, device=q.device))
    qg = q.float().permute(1, 0, 2).reshape(H_kv, (H_q // H_kv) * T, d)
    sc = (qg @ k.float().transpose(1, 2)).mul_(scale).view(H_kv, -1, T, S)
    if seen is not None:
        sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(H_kv, -1, S) @ v.float()).view(H_kv, -1, T, d) / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    return o.reshape(H_q, T, d).permute(1, 0, 2), lse.reshape(H_q, T).t()


def _plain_packed(s):
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    q0 = k0 = 0
    for n_q, n_k in zip(s["q_lens"], s["k_lens"]):
        k, v = (t[k0:k0 + n_k].permute(1, 0, 2) for t in (s["k"], s["v"]))
        block = max(1, (1 << 28) // max(1, n_k * s["q"].shape[1]))
        for a in range(0, n_q, block):
            b = min(n_q, a + block)
            seen = None
            if s["causal"]:
                at = torch.arange(a, b, device="cuda") + (n_k - n_q)
                seen = torch.arange(n_k, device="cuda")[None, :] <= at[:, None]
            oo, ll = _plain_rows(s["q"][q0 + a:q0 + b], k, v, seen, s["scale"])
            o[q0 + a:q0 + b], lse[q0 + a:q0 + b] = oo.to(torch.bfloat16), ll
        q0, k0 = q0 + n_q, k0 + n_k
    return o, lse


def _plain_tree(s):
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    a = 0
    for b, (n, T) in enumerate(zip(s["contexts"], s["drafts"])):
        new = slice(a, a + T)
        k = torch.cat([s["k_cache"][b, :, :n], s["k_new"][new].permute(1, 0, 2)], 1)
        v = torch.cat([s["v_cache"][b, :, :n], s["v_new"][new].permute(1, 0, 2)], 1)
        j = torch.arange(T, device="cuda")
        if s["mask"] is None:
            draft = j[None, :] <= j[:, None]
        else:
            draft = (s["mask"][new][:, j // 32] >> (j % 32)[None, :]) & 1 == 1
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), draft], 1)
        oo, ll = _plain_rows(s["q"][new], k, v, seen, s["scale"])
        o[new], lse[new] = oo.to(torch.bfloat16), ll
        a += T
    return o, lse


def _plain_append(s):
    k, v = s["k_new"], s["v_new"]
    if s["index"] is not None:
        k, v = k[s["index"].long()], v[s["index"].long()]
    a = 0
    for b, (t, n) in enumerate(zip(s["starts"], s["counts"])):
        s["k_cache"][b, :, t:t + n] = k[a:a + n].permute(1, 0, 2)
        s["v_cache"][b, :, t:t + n] = v[a:a + n].permute(1, 0, 2)
        a += n
    return s["k_cache"], s["v_cache"]


def run(state):
    s = state
    if not own:
        return {"prefill_packed": _plain_packed, "decode_tree": _plain_tree,
                "cache_append": _plain_append}[s["op"]](s)
    from gqa_attention_split_gb300 import api

    if s["op"] == "prefill_packed":
        return api.prefill_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                  causal=s["causal"], scale=s["scale"])
    if s["op"] == "decode_tree":
        return api.decode_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                               s["context_lens"], cu_seqlens=s["cu"],
                               max_tokens=s["max_tokens"], tree_mask=s["mask"], scale=s["scale"])
    api.cache_append(s["k_cache"], s["v_cache"], s["k_new"], s["v_new"], s["starts_dev"],
                     cu_seqlens=s["cu"], index=s["index"])
    return s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------------------ work and exact


def work(case):
    H_kv, d = case["H_kv"], case["d"]
    if case["op"] == "cache_append":
        n = sum(_lens(case["counts"]))
        return {"bytes": n * H_kv * d * 8, "flops": 0}
    H_q = case["H_q"]
    if case["op"] == "prefill_packed":
        q = _lens(case["q_lens"])
        k = _lens(case["k_lens"]) or q
        pairs = 0
        for n_q, n_k in zip(q, k):
            if case["causal"]:  # sum over t of max(0, n_k - n_q + t + 1)
                low = max(0, n_k - n_q)
                pairs += n_k * (n_k + 1) // 2 - low * (low + 1) // 2
            else:
                pairs += n_q * n_k
        keys, rows = sum(k), sum(q)
    else:
        ctx, T = _lens(case["contexts"]), _lens(case["drafts"])
        pairs = sum(t * n + (t if case["mask"] else t * (t + 1) // 2) for n, t in zip(ctx, T))
        keys, rows = sum(ctx) + sum(T), sum(T)
    return {"bytes": rows * H_q * (4 * d + 4) + keys * H_kv * d * 4, "flops": 4 * H_q * d * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache_append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        a = 0
        for b, (t, n) in enumerate(zip(s["starts"], s["counts"])):
            for i in range(n):
                src = int(s["index"][a + i]) if s["index"] is not None else a + i
                kc[b, :, t + i] = s["k_new"][src].double()
                vc[b, :, t + i] = s["v_new"][src].double()
            a += n
        return kc, vc
    H_q, G = case["H_q"], case["H_q"] // case["H_kv"]
    n_rows = s["q"].shape[0]
    o = torch.zeros(n_rows, H_q, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(n_rows, H_q, dtype=torch.float64, device="cuda")
    bits = s["mask"].cpu().numpy().view(np.uint32) if case["op"] == "decode_tree" and case["mask"] \
        else None
    a = k0 = 0
    packed = case["op"] == "prefill_packed"
    rows = list(zip(s["q_lens"], s["k_lens"])) if packed else list(zip(s["drafts"], s["contexts"]))
    for b, (n_q, n_k) in enumerate(rows):
        for h in range(case["H_kv"]):
            if packed:
                K, V = s["k"][k0:k0 + n_k, h].double(), s["v"][k0:k0 + n_k, h].double()
                base = n_k - n_q
            else:
                K = torch.cat([s["k_cache"][b, h, :n_k], s["k_new"][a:a + n_q, h]]).double()
                V = torch.cat([s["v_cache"][b, h, :n_k], s["v_new"][a:a + n_q, h]]).double()
                base = n_k
            for r in range(0, n_q, 1024):
                e = min(n_q, r + 1024)
                # keys behind the last one that these rows can see are left out
                end = min(K.shape[0], max(0, base + e)) if not packed or case["causal"] \
                    else K.shape[0]
                if bits is not None:
                    end = K.shape[0]
                if end == 0:
                    lse[a + r:a + e, h * G:(h + 1) * G] = -math.inf
                    continue
                Q = s["q"][a + r:a + e, h * G:(h + 1) * G].double()
                x = torch.einsum("tgc,sc->tgs", Q, K[:end]) * s["scale"]
                if bits is not None:
                    vis = torch.ones(e - r, end, dtype=torch.bool)
                    for t in range(r, e):
                        for j in range(n_q):
                            vis[t - r, n_k + j] = bool((bits[a + t, j >> 5] >> (j & 31)) & 1)
                    x = torch.where(vis.cuda()[:, None, :], x, -math.inf)
                elif not packed or case["causal"]:
                    t = torch.arange(r, e, device="cuda")[:, None, None] + base
                    x = torch.where(torch.arange(end, device="cuda") > t, -math.inf, x)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
                o[a + r:a + e, h * G:(h + 1) * G] = torch.einsum("tgs,sc->tgc", w, V[:end])
                lse[a + r:a + e, h * G:(h + 1) * G] = z
        a, k0 = a + n_q, k0 + n_k
    return o, lse
