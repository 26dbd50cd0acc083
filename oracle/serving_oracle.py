"""The operators around the paged latent cache, in plain fp64 NumPy.

Norms with the rotation, gathered attention weights and eviction, one token,
query and sequence at a time, from their definitions.  Test infrastructure:
nothing here is imported by the product path.
"""

from __future__ import annotations

import numpy as np

from .mla_oracle import rope

F64 = np.float64


def rms_norm(x, w, eps):
    """x / sqrt(mean(x^2) + eps) * w over the last axis; x itself where w is None."""
    x = np.asarray(x, F64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(w, F64)


def norm_rope(y, H, d_nope, d_rope, d_latent, w_q, w_c, w_kr, eps, pos, base=10000.0):
    """Rows [q_1 .. q_H | c | k_rope] normed vector by vector and rotated by pos.

    Returns (q [T, H, d_nope + d_rope], ckr [T, d_latent + d_rope])."""
    y = np.asarray(y, F64)
    T, dqk = y.shape[0], d_nope + d_rope
    pos = np.asarray(pos, F64)
    q = rms_norm(y[:, :H * dqk].reshape(T, H, dqk), w_q, eps).copy()
    q[..., d_nope:] = rope(q[..., d_nope:], pos[:, None], base)
    c = rms_norm(y[:, H * dqk:H * dqk + d_latent], w_c, eps)
    kr = rope(rms_norm(y[:, H * dqk + d_latent:H * dqk + d_latent + d_rope], w_kr, eps), pos, base)
    return q, np.concatenate([c, kr], 1)


def attention_weights(q_abs, rows, lse, scale):
    """What the tokens of one sequence receive from its last S_q queries:
    w[t] = sum over the queries j and heads i that see t of exp(scale q_ji . row_t - lse_ji).

    q_abs [S_q, H, D], rows [L, D], lse [S_q, H]; query j sees t <= L - S_q + j."""
    q_abs, rows, lse = (np.asarray(a, F64) for a in (q_abs, rows, lse))
    L, S_q = rows.shape[0], q_abs.shape[0]
    w = np.zeros(L)
    for j in range(S_q):
        vis = L - S_q + j + 1
        for i in range(q_abs.shape[1]):
            if np.isneginf(lse[j, i]):
                continue
            w[:vis] += np.exp(scale * (rows[:vis] @ q_abs[j, i]) - lse[j, i])
    return w


def evict(weights, positions, budget, n_sink, n_recent):
    """One sequence's eviction: (pairs [(to, from)], new length).

    The free slots (position not among the first n_sink nor the last n_recent) with the smallest
    (weight, slot) leave until `budget` slots remain; the k-th survivor behind the new end moves
    to the k-th slot vacated before it.  NaN sorts behind +inf, -0 equals 0."""
    w = [float(x) + 0.0 for x in weights]
    L = len(w)
    end = max(positions, default=-1) + 1
    free = [t for t in range(L) if n_sink <= positions[t] < end - n_recent]
    n_out = min(max(L - max(budget, 0), 0), len(free))
    free.sort(key=lambda t: (w[t] != w[t], 0.0 if w[t] != w[t] else w[t], t))
    gone = set(free[:n_out])
    new = L - n_out
    to = [t for t in range(new) if t in gone]
    frm = [t for t in range(new, L) if t not in gone]
    assert len(to) == len(frm)
    return list(zip(to, frm)), new
