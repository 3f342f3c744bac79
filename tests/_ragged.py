"""Plain 64-bit attention over explicit visibility, with the error bound of a bf16 kernel.

For each query: O = sum_j p_j v_j over the visible keys, lse = ln sum exp(scale q.k_j). A kernel
that rounds the weights to bf16 before the product with V, normalises by the sum of the unrounded
weights and rounds O to bf16 is off by at most (u = 2^-8, half a bf16 step)
    |dO_c| <= u sum_j p_j |v_jc| + 2 e sum_j p_j |v_jc - O_c| + u (|O_c| + those) + 2^-18 max|v|
since its O' = sum p_j (1 + d_j) v_j / sum p_j with |d_j| <= u, and relative errors e_j of the
weights themselves move O by sum p_j e_j (v_j - O) / sum p_j (1 + e_j), where e bounds the fp32
error of a scaled score: d products summed in fp32, each step off by at most 2^-23 of the sum of
magnitudes (the tensor core may truncate), plus the exponential's and the exponent's own
roundings, 2^-20 of the largest score and of 1. lse is off by at most e plus fp32 roundings.
"""

import numpy as np

U = 2.0 ** -8


def attend(q, k, v, visible, scale):
    """q [T,H_q,d], k/v [S,H_kv,d] float64 arrays, visible bool [T,S]. Invisible keys may hold
    anything. Returns O [T,H_q,d], lse [T,H_q], and the bounds dO, dlse of the same shapes."""
    T, H_q, d = q.shape
    S, H_kv = k.shape[:2]
    O = np.zeros((T, H_q, d))
    L = np.full((T, H_q), -np.inf)
    bO, bL = np.zeros((T, H_q, d)), np.zeros((T, H_q))
    if S == 0:
        return O, L, bO, bL
    used = visible.any(0)  # rows of K and V that some query sees
    k = np.where(used[:, None, None], k, 0.0)
    v = np.where(used[:, None, None], v, 0.0)
    G = H_q // H_kv
    for h in range(H_q):
        K, V = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ K.T) * scale
        mag = np.where(visible, (np.abs(q[:, h]) @ np.abs(K).T) * scale, 0.0).max(1)
        s = np.where(visible, s, -np.inf)
        m = s.max(1, keepdims=True)
        some = np.isfinite(m[:, 0])
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        l = p.sum(1, keepdims=True)
        p = p / np.where(l == 0, 1.0, l)
        O[:, h] = p @ V
        L[some, h] = m[some, 0] + np.log(l[some, 0])
        e = d * 2.0 ** -23 * mag + 2.0 ** -20 * (mag + 1.0)
        spread = np.zeros((T, d))
        for t0 in range(0, T, 64):  # sum_j p_j |v_j - O|, blockwise to bound the memory
            blk = slice(t0, min(T, t0 + 64))
            for s0 in range(0, S, 256):
                kb = slice(s0, s0 + 256)
                spread[blk] += np.einsum("ts,tsc->tc", p[blk, kb],
                                         np.abs(V[None, kb] - O[blk, None, h]))
        bO[:, h] = ((U * (p @ np.abs(V)) + 2 * e[:, None] * spread) * (1 + U) + U * np.abs(O[:, h])
                    + 2.0 ** -18 * np.abs(V).max())
        bL[:, h] = e + 2.0 ** -20 * (np.abs(np.where(some, L[:, h], 0.0)) + 1.0)
    return O, L, bO, bL


def check(o, lse, ref, what=""):
    """Every element of a kernel's o, lse (torch tensors) against attend()'s result."""
    O, L, bO, bL = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isneginf(L)
    assert (np.isneginf(lse) == none).all(), f"{what}: empty rows differ"
    assert (o[none] == 0).all(), f"{what}: a row that sees no key is not 0"
    err = np.abs(o - O)
    assert np.isfinite(o).all(), f"{what}: not finite"
    over = (err > bO).sum()
    assert over == 0, f"{what}: {over} elements over the bound, worst {(err / (bO + 1e-30)).max():.2f}x"
    dl = np.abs(np.where(none, 0.0, lse) - np.where(none, 0.0, L))
    assert (dl <= bL).all(), f"{what}: lse off by {dl.max():.2e}"


def causal_visible(n_q, n_k):
    return np.arange(n_k)[None, :] <= np.arange(n_q)[:, None] + (n_k - n_q)
