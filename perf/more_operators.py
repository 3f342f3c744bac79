"""Measured cases of one serving step over a paged KV cache: the norm and rotation of queries and
keys, appending them to the pages, attention of the step's tokens over the pages, and the
verification of drafted tokens.

``qk_norm_rope``     Every head of q and k [tokens, heads, d] is divided by its root mean square,
                     multiplied by a weight and rotated by the token's position. A position has
                     one axis (text) or several (time, height, width), each of which turns its
                     own section of the pairs of channels.
                         z_c = x_c / sqrt(mean_c x_c^2 + eps) * w_c
                         (y_1, y_2) = (z_1 cos a - z_2 sin a, z_2 cos a + z_1 sin a),
                         a = position * inv_freq of the pair
``paged_append``     The keys and values of packed new tokens go into pages
                     [pages, H_kv, page_size, d]; slot s of row b lies in page
                     block_table[b, s // page_size].
``paged_attention``  The T tokens of a row are its last ones: token t sees the keys
                     j <= n - T + t of the row's n keys in the pages. T is 1 in a decode step, a
                     few with drafted tokens, up to thousands in a chunk of a prompt.
                         O = softmax(scale * Q K^T over the visible keys) V,  lse = ln sum exp
``verify_drafts``    Drafted token x_i stands if u_i q_i(x_i) < p_i(x_i) and all before it stand.
                     The next token is drawn from max(p - q, 0) at the first one that falls (a
                     draft without probabilities has q = 1 at its token), or from the last p: the
                     lowest v whose cumulative sum is above u times the sum.

Tensors are bfloat16, lse and probabilities are float32, counts and tokens are int32.

``own`` chooses between the plain torch form of each operator and the library's calls.
"""

import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------------------- cases


def _norm(name, tokens, H_q, H_kv, d, rotary, axes, norm=True, interleaved=False, far=4096):
    return {"name": name, "op": "qk_norm_rope", "tokens": tokens, "H_q": H_q, "H_kv": H_kv, "d": d,
            "rotary": rotary, "axes": axes, "norm": norm, "interleaved": interleaved, "far": far}


def _append(name, starts, counts, page, H_kv, d):
    return {"name": name, "op": "paged_append", "starts": starts, "counts": counts, "page": page,
            "H_kv": H_kv, "d": d}


def _attend(name, lens, tokens, page, H_q, H_kv, d, causal=True):
    return {"name": name, "op": "paged_attention", "lens": lens, "tokens": tokens, "page": page,
            "H_q": H_q, "H_kv": H_kv, "d": d, "causal": causal}


def _verify(name, drafts, V, agree, dist=True):
    return {"name": name, "op": "verify_drafts", "drafts": drafts, "V": V, "agree": agree,
            "dist": dist}


def listed():
    return [
        # A decode step of eight rows far into their contexts: one launch's latency.
        _norm("norm_rope_step", 8, 64, 8, 128, 128, 1, far=131072),
        # A step of packed prompts; q, k and v are slices of one projection.
        _norm("norm_rope_prompts", 8203, 64, 8, 128, 128, 1),
        # Images and video: time, height and width turn sections of 16, 24 and 24 pairs.
        _norm("norm_rope_video", 5000, 28, 4, 128, 128, 3),
        # One new token for each of 32 rows; some of them begin a page.
        _append("append_step", _text((i * 977) % 8192 for i in range(32)), _text([1] * 32), 64, 8,
                128),
        # Chunks of prompts that begin and end inside pages.
        _append("append_chunks", "0,517,4096,33,1000,8001", "2048,1500,1,777,2048,1003", 16, 8, 128),
        # One short chat at head dim 64: latency.
        _attend("decode_short", "533", "1", 16, 32, 8, 64),
        # A decode step of 32 rows with ragged contexts: bound by the cache's bytes.
        _attend("decode_batch", _text(1000 + (i * i * 31) % 15013 for i in range(32)),
                _text([1] * 32), 64, 64, 8, 128),
        # A chunk of 2048 tokens on 30K tokens of context: the matrix products count.
        _attend("chunk_32k", "32768", "2048", 128, 64, 8, 128),
        # One step that serves chunks of two prompts, drafted tokens and single tokens at once, an
        # odd group of heads.
        _attend("mixed_step", "4100,700,12000,3000,8191,9,1,20011,6000,15", "500,700,6,1,1,6,1,1,3,15",
                32, 28, 4, 128),
        # Five drafted tokens on each of eight rows, 16 query heads to a KV head.
        _attend("drafts_g16", "16000,8000,12345,901,7000,3333,15001,64", "6,6,6,6,6,6,6,6", 16, 128,
                8, 128),
        # One chat with five drafted tokens by a draft model.
        _verify("verify_single", "5", 128256, 0.7),
        # A batch of 48 rows with 2 to 7 drafted tokens each, an odd vocabulary.
        _verify("verify_batch", _text(2 + (i * 5) % 6 for i in range(48)), 128259, 0.8),
    ]


_HEADS = [(64, 8, 128), (32, 8, 64), (28, 4, 128), (128, 8, 128), (8, 1, 128), (16, 16, 64)]
_PAGES = [16, 32, 64, 128, 256]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _text(v):
    return ",".join(str(int(x)) for x in v)


def draw(rng):
    op = rng.choice(["qk_norm_rope", "qk_norm_rope", "paged_append", "paged_attention",
                     "paged_attention", "paged_attention", "verify_drafts"])
    H_q, H_kv, d = rng.choice(_HEADS)
    if op == "qk_norm_rope":
        axes = rng.choice([1, 1, 2, 3])
        rotary = rng.choice([d, d, d // 2])
        return _norm("", _log(rng, 1, 8192), H_q, H_kv, d, rotary, axes, rng.random() < 0.8,
                     rng.random() < 0.3, _log(rng, 16, 1 << 20))
    if op == "verify_drafts":
        B = _log(rng, 1, 32)
        V = _log(rng, 1000, 160000)
        return _verify("", _text(rng.randint(0, 7) for _ in range(B)), V, rng.uniform(0.3, 0.95),
                       rng.random() < 0.7)
    page, B = rng.choice(_PAGES), _log(rng, 1, 32)
    if op == "paged_append":
        counts = [_log(rng, 1, 8192 // B) - (1 if rng.random() < 0.2 else 0) for _ in range(B)]
        if not sum(counts):
            counts[0] = 1
        return _append("", _text(_log(rng, 1, 16384) - 1 for _ in range(B)), _text(counts), page,
                       H_kv, d)
    most = rng.choice([1, 1, 8, 64, 2048])
    tokens = [min(2048 // B + 1, _log(rng, 1, most)) for _ in range(B)]
    lens = [t + _log(rng, 1, max(1, 131072 // B)) - 1 for t in tokens]
    if most == 2048:
        lens = [min(n, 16384) for n in lens]
    return _attend("", _text(lens), _text(tokens), page, H_q, H_kv, d, rng.random() < 0.9)


def _lens(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))]).astype(np.int32)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _pool(gen, rng, lens, page, H_kv, d):
    """K and V pages, some of them of no row, and the block table: the pages of a row lie anywhere
    in the pool."""
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    pages = sum(need) + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.zeros((len(lens), width), dtype=np.int32)
    a = 0
    for b, n in enumerate(need):
        table[b, :n] = order[a:a + n]
        a += n
    return (_randn(gen, pages, H_kv, page, d), _randn(gen, pages, H_kv, page, d),
            torch.from_numpy(table).cuda())


def _sections(case):
    pairs, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return None
    if axes == 2:
        return (pairs // 2, pairs - pairs // 2)
    t = pairs // 4
    return (t, (pairs - t) // 2, pairs - t - (pairs - t) // 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"op": case["op"]}
    if case["op"] == "qk_norm_rope":
        n, H_q, H_kv, d = case["tokens"], case["H_q"], case["H_kv"], case["d"]
        qkv = _randn(gen, n, H_q + 2 * H_kv, d)
        s["q"], s["k"], _ = qkv.split([H_q, H_kv, H_kv], dim=1)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = 1 + 0.1 * _randn(gen, d), 1 + 0.1 * _randn(gen, d)
        s["eps"] = 1e-6 if case["norm"] else None
        pairs = case["rotary"] // 2
        f = 500000.0 ** -(np.arange(pairs) / pairs)
        s["inv_freq"] = torch.from_numpy(f.astype(np.float32)).cuda()
        s["sections"] = _sections(case)
        s["interleaved"] = case["interleaved"]
        shape = (n,) if case["axes"] == 1 else (case["axes"], n)
        s["positions"] = torch.from_numpy(rng.randint(0, case["far"], shape).astype(np.int32)).cuda()
        return s
    if case["op"] == "verify_drafts":
        drafts, V = _lens(case["drafts"]), case["V"]
        B, n = len(drafts), sum(drafts)
        logits = torch.randn(n + B, V, generator=gen, device="cuda")
        logits *= 2.5
        s["target_probs"] = torch.softmax(logits, -1)
        # rows of p that the drafts answer to
        rows = np.concatenate([np.arange(c) + a + b for b, (a, c) in enumerate(zip(_cu(drafts), drafts))]
                              + [np.zeros(0)]).astype(np.int64)
        rows = torch.from_numpy(rows).cuda()
        s["draft_probs"] = None
        # the draft model's distribution is near the target's: E[min(1, p/q)] about `agree`
        near = torch.randn(n, V, generator=gen, device="cuda")
        near *= 2.5 * (1 - case["agree"])
        near += logits[rows]
        q = torch.softmax(near, -1)
        del logits, near
        pick = torch.rand(n, 1, generator=gen, device="cuda", dtype=torch.float64)
        c = torch.cumsum(q, -1, dtype=torch.float64)
        x = torch.searchsorted(c, pick * c[:, -1:]).clamp_(max=V - 1)[:, 0]
        del c
        s["draft_tokens"] = x.to(torch.int32)
        if case["dist"]:
            s["draft_probs"] = q
        else:
            del q
        s["u_accept"] = torch.rand(n, generator=gen, device="cuda")
        s["u_sample"] = torch.rand(B, generator=gen, device="cuda")
        s["cu"] = torch.from_numpy(_cu(drafts)).cuda()
        s["drafts"] = drafts
        return s
    H_kv, d, page = case["H_kv"], case["d"], case["page"]
    s["page"] = page
    if case["op"] == "paged_append":
        s["starts"], s["counts"] = _lens(case["starts"]), _lens(case["counts"])
        lens = [a + c for a, c in zip(s["starts"], s["counts"])]
        s["k_new"] = _randn(gen, sum(s["counts"]), H_kv, d)
        s["v_new"] = _randn(gen, sum(s["counts"]), H_kv, d)
        s["starts_dev"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
        s["cu"] = torch.from_numpy(_cu(s["counts"])).cuda()
    else:
        lens, s["tokens"] = _lens(case["lens"]), _lens(case["tokens"])
        s["lens"], s["causal"] = lens, case["causal"]
        s["q"] = _randn(gen, sum(s["tokens"]), case["H_q"], d)
        s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu"] = torch.from_numpy(_cu(s["tokens"])).cuda()
        s["max_tokens"] = max(s["tokens"])
        s["scale"] = 1.0 / math.sqrt(d)
    s["k_pages"], s["v_pages"], s["table"] = _pool(gen, rng, lens, page, H_kv, d)
    return s


# -------------------------------------------------------------------------------- plain forms


def _plain_norm(s):
    P = s["inv_freq"].numel()
    pos = s["positions"].reshape(-1, s["positions"].shape[-1])
    sec = s["sections"] or (P,)
    axis = torch.repeat_interleave(torch.arange(len(sec)), torch.tensor(sec)).to(pos.device)
    # a far position times a frequency has more digits than 32 bits hold
    a = pos[axis].t().double() * s["inv_freq"].double()
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    outs = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        z = x.float()
        if s["eps"] is not None:
            z = z * (z.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
            if w is not None:
                z = z * w.float()
        if s["interleaved"]:
            z1, z2 = z[..., :2 * P:2], z[..., 1:2 * P:2]
            turned = torch.stack([z1 * cos - z2 * sin, z2 * cos + z1 * sin], -1).flatten(-2)
        else:
            z1, z2 = z[..., :P], z[..., P:2 * P]
            turned = torch.cat([z1 * cos - z2 * sin, z2 * cos + z1 * sin], -1)
        outs.append(torch.cat([turned, z[..., 2 * P:]], -1).to(torch.bfloat16))
    return tuple(outs)


def _plain_append(s):
    a = 0
    for b, (t, n) in enumerate(zip(s["starts"], s["counts"])):
        slot = torch.arange(t, t + n, device="cuda")
        at = s["table"][b].long()[slot // s["page"]]
        s["k_pages"][at, :, slot % s["page"]] = s["k_new"][a:a + n]
        s["v_pages"][at, :, slot % s["page"]] = s["v_new"][a:a + n]
        a += n
    return s["k_pages"], s["v_pages"]


def _plain_attend(s):
    H_q, d = s["q"].shape[1:]
    H_kv = s["k_pages"].shape[1]
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    a = 0
    for b, (T, n) in enumerate(zip(s["tokens"], s["lens"])):
        at = s["table"][b, :-(-n // s["page"])].long()
        k, v = (x[at].permute(1, 0, 2, 3).reshape(H_kv, -1, d)[:, :n].float()
                for x in (s["k_pages"], s["v_pages"]))
        block = max(1, (1 << 28) // (n * H_q))
        for t in range(0, T, block):
            e = min(T, t + block)
            q = s["q"][a + t:a + e].float().permute(1, 0, 2).reshape(H_kv, -1, d)
            x = (q @ k.transpose(1, 2)).mul_(s["scale"]).view(H_kv, -1, e - t, n)
            if s["causal"]:
                last = torch.arange(t, e, device="cuda") + (n - T)
                x.masked_fill_(torch.arange(n, device="cuda") > last[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            p = x.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            oo = (p.view(H_kv, -1, n) @ v).view(H_kv, -1, e - t, d) / l
            o[a + t:a + e] = oo.reshape(H_q, e - t, d).permute(1, 0, 2).to(torch.bfloat16)
            lse[a + t:a + e] = (m + l.log()).reshape(H_q, e - t).t()
        a += T
    return o, lse


def _plain_verify(s):
    n, B = s["draft_tokens"].numel(), len(s["drafts"])
    cu = s["cu"].long()
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), cu.diff(), output_size=n)
    i = torch.arange(n, device="cuda")
    x = s["draft_tokens"].long()
    p = s["target_probs"][i + row, x].double()
    q = s["draft_probs"][i, x].double() if s["draft_probs"] is not None else 1.0
    fell = s["u_accept"].double() * q >= p
    # drafted tokens before the first one that fell
    first = torch.where(fell, i - cu[row], n + 1)
    accepted = cu.diff().scatter_reduce(0, row, first, "amin")
    at = cu[:-1] + accepted
    r = s["target_probs"][at + torch.arange(B, device="cuda")].double()
    some = accepted < cu.diff()
    if n:
        at = at.clamp(max=n - 1)
        if s["draft_probs"] is not None:
            r = torch.where(some[:, None], (r - s["draft_probs"][at].double()).clamp_(min=0), r)
        else:
            hit = (torch.arange(r.shape[1], device="cuda") == x[at][:, None]) & some[:, None]
            r = torch.where(hit, 0.0, r)
    c = r.cumsum(-1)
    above = c > s["u_sample"].double()[:, None] * c[:, -1:]
    return accepted.to(torch.int32), above.byte().argmax(-1).to(torch.int32)


def run(state):
    s = state
    if not own:
        return {"qk_norm_rope": _plain_norm, "paged_append": _plain_append,
                "paged_attention": _plain_attend, "verify_drafts": _plain_verify}[s["op"]](s)
    from gqa_attention_split_gb300 import api

    if s["op"] == "qk_norm_rope":
        return api.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                sections=s["sections"], interleaved=s["interleaved"])
    if s["op"] == "paged_attention":
        return api.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"],
                                   cu_seqlens=s["cu"], max_tokens=s["max_tokens"],
                                   causal=s["causal"], scale=s["scale"])
    if s["op"] == "verify_drafts":
        return api.verify_drafts(s["target_probs"], s["draft_tokens"], s["u_accept"],
                                 s["u_sample"], s["cu"], draft_probs=s["draft_probs"])
    api.paged_append(s["k_pages"], s["v_pages"], s["k_new"], s["v_new"], s["table"],
                     s["starts_dev"], cu_seqlens=s["cu"])
    return s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------------------ work and exact


def work(case):
    if case["op"] == "qk_norm_rope":
        x = case["tokens"] * (case["H_q"] + case["H_kv"]) * case["d"]
        return {"bytes": 4 * x + 4 * case["tokens"] * case["axes"], "flops": 10 * x}
    if case["op"] == "paged_append":
        return {"bytes": 8 * sum(_lens(case["counts"])) * case["H_kv"] * case["d"], "flops": 0}
    if case["op"] == "verify_drafts":
        # a row of p, and one of q in the rows where a drafted token falls
        drafts = _lens(case["drafts"])
        falls = sum(1 - case["agree"] ** n for n in drafts) if case["dist"] else 0.0
        return {"bytes": int(4 * case["V"] * (len(drafts) + falls)) + 16 * sum(drafts),
                "flops": int(2 * case["V"] * (len(drafts) + falls))}
    H_q, H_kv, d = case["H_q"], case["H_kv"], case["d"]
    pairs = rows = keys = 0
    for n, T in zip(_lens(case["lens"]), _lens(case["tokens"])):
        pairs += n * T - (T * (T - 1) // 2 if case["causal"] else 0)
        rows, keys = rows + T, keys + n
    return {"bytes": rows * H_q * (4 * d + 4) + keys * H_kv * d * 4, "flops": 4 * H_q * d * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_norm_rope":
        d, P = case["d"], case["rotary"] // 2
        pos = s["positions"].double().reshape(case["axes"], -1)
        sec = s["sections"] or (P,)
        # y = z times a matrix of each token: the rotation of its pairs, 1 elsewhere
        R = torch.zeros(case["tokens"], d, 2, dtype=torch.float64, device="cuda")
        R[:, :, 0] = 1
        other = torch.arange(d, device="cuda")
        at = 0
        for axis, n in enumerate(sec):
            for i in range(at, at + n):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + P)
                w = pos[axis] * float(s["inv_freq"][i])
                R[:, a, 0] = R[:, b, 0] = torch.cos(w)
                R[:, a, 1], R[:, b, 1] = -torch.sin(w), torch.sin(w)
                other[a], other[b] = b, a
            at += n
        outs = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            z = x.double()
            if case["norm"]:
                z = z / torch.sqrt((z * z).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            outs.append(z * R[:, None, :, 0] + z[..., other] * R[:, None, :, 1])
        return tuple(outs)
    if case["op"] == "verify_drafts":
        counts, tokens = [], []
        a = 0
        for b, n in enumerate(_lens(case["drafts"])):
            k = 0
            while k < n:
                x = int(s["draft_tokens"][a + k])
                q = float(s["draft_probs"][a + k, x]) if case["dist"] else 1.0
                if not float(s["u_accept"][a + k]) * q < float(s["target_probs"][a + b + k, x]):
                    break
                k += 1
            r = s["target_probs"][a + b + k].cpu().numpy().astype(np.float64)
            if k < n and case["dist"]:
                r = np.maximum(r - s["draft_probs"][a + k].cpu().numpy().astype(np.float64), 0)
            elif k < n:
                r[int(s["draft_tokens"][a + k])] = 0
            c = np.cumsum(r)
            counts.append(k)
            tokens.append(int(np.searchsorted(c, float(s["u_sample"][b]) * c[-1], side="right")))
            a += n
        return (torch.tensor(counts, dtype=torch.int32, device="cuda"),
                torch.tensor(tokens, dtype=torch.int32, device="cuda"))
    if case["op"] == "paged_append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        table = s["table"].cpu().numpy()
        a = 0
        for b, (t, n) in enumerate(zip(s["starts"], s["counts"])):
            for g in range(t // case["page"], -(-(t + n) // case["page"]) if n else 0):
                lo, hi = max(t, g * case["page"]), min(t + n, (g + 1) * case["page"])
                to = slice(lo - g * case["page"], hi - g * case["page"])
                src = slice(a + lo - t, a + hi - t)
                k[int(table[b, g]), :, to] = s["k_new"][src].double().transpose(0, 1)
                v[int(table[b, g]), :, to] = s["v_new"][src].double().transpose(0, 1)
            a += n
        return k, v
    if work(case)["flops"] > 4e12:
        return None
    H_q, H_kv, d = case["H_q"], case["H_kv"], case["d"]
    G = H_q // H_kv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    a = 0
    for b, (T, n) in enumerate(zip(s["tokens"], s["lens"])):
        slot = torch.arange(n, device="cuda")
        page, at = s["table"][b].long()[slot // case["page"]], slot % case["page"]
        for h in range(H_kv):
            K, V = s["k_pages"][page, h, at].double(), s["v_pages"][page, h, at].double()
            for t in range(0, T, 512):
                e = min(T, t + 512)
                Q = s["q"][a + t:a + e, h * G:(h + 1) * G].double()
                x = torch.einsum("tgc,sc->tgs", Q, K) * s["scale"]
                if case["causal"]:
                    limit = torch.arange(t, e, device="cuda")[:, None, None] + (n - T)
                    x = torch.where(slot > limit, -math.inf, x)
                z = torch.logsumexp(x, -1)
                o[a + t:a + e, h * G:(h + 1) * G] = torch.einsum("tgs,sc->tgc",
                                                                 torch.exp(x - z[..., None]), V)
                lse[a + t:a + e, h * G:(h + 1) * G] = z
        a += T
    return o, lse
