"""Error bound of attention whose result is a weighted mean of the V rows that it rounds.

A kernel that rounds its weights to bf16 before the product with V, divides by the sum of the same
rounded weights and rounds O to bf16 computes O' = sum w_j v_j / sum w_j, w_j = p_j (1 + d_j). With
|d_j| <= D,
    O' - O = sum p_j d_j (v_j - O) / sum p_j (1 + d_j),   |O'_c - O_c| <= D / (1 - D) sum p_j |v_jc - O_c|
whatever the mean of V is: a common error of all weights drops out. D = (1 + u)(1 + 2 e) - 1, u = 2^-8
(half a bf16 step) and e the fp32 error of a scaled score, of which exp(e) - 1 <= 2 e is the relative
error of a weight (e < 1): d products summed in fp32, each step off by at most 2^-23 of the sum of
magnitudes, and the exponent's and the exponential's own roundings, 2^-20 of the largest score and
of 1. The products with V and the sums are in fp32: 2^-18 max|v|. Last, O' is rounded:
u (|O| + all of that).
"""

import numpy as np

import _ragged as ref

U = 2.0 ** -8


def attend(q, k, v, visible, scale):
    """ref.attend() with the bound above in place of its own."""
    O, L, _, bL = ref.attend(q, k, v, visible, scale)
    T, H_q, d = q.shape
    G = H_q // k.shape[1]
    bO = np.zeros_like(O)
    for h in range(H_q):
        K, V = k[:, h // G], v[:, h // G]
        s = np.where(visible, (q[:, h] @ K.T) * scale, -np.inf)
        p = np.exp(s - np.where(np.isfinite(L[:, h]), L[:, h], 0.0)[:, None])
        mag = np.where(visible, (np.abs(q[:, h]) @ np.abs(K).T) * scale, 0.0).max(1)
        e = d * 2.0 ** -23 * mag + 2.0 ** -20 * (mag + 1.0)
        D = ((1 + U) * (1 + 2 * e) - 1)[:, None]
        spread = np.stack([p[t] @ np.abs(V - O[t, h]) for t in range(T)])
        b = D / (1 - D) * spread + 2.0 ** -18 * np.abs(V).max()
        bO[:, h] = b + U * (np.abs(O[:, h]) + b)
    return O, L, bO, bL
